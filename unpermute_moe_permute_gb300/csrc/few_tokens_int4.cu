// The layer for a few tokens over 4-bit weights (apart from the others, so that
// the kernels are compiled beside each other).
#include "few_tokens.cuh"

using namespace moe;
using namespace moe::tc;

extern "C" int moe_layer_few_tokens_int4(const void* tokens, const int32_t* expert_ids,
                                         const float* probs, int T, int H, int K, int I, int E,
                                         int num_special, const uint8_t* active_mask, int mask_dims,
                                         int group, int down_group, const uint8_t* W_gate_q,
                                         const void* gate_scale, const uint8_t* W_up_q,
                                         const void* up_scale, const uint8_t* W_down_q,
                                         const void* down_scale, const void* shared_x, void* out,
                                         void* workspace, size_t workspace_bytes,
                                         int32_t* dev_status, cudaStream_t stream) {
  return few_tokens<4>(tokens, expert_ids, probs, T, H, K, I, E, num_special, active_mask, mask_dims, group,
                    down_group, FewWeights{W_gate_q, W_up_q, W_down_q, gate_scale, up_scale, down_scale}, shared_x,
                    out, workspace, workspace_bytes, dev_status, stream);
}
