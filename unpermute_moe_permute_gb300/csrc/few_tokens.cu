// The layer for a few tokens over bf16 and 8-bit weights.
#include "few_tokens.cuh"

using namespace moe;
using namespace moe::tc;

extern "C" size_t moe_layer_few_tokens_workspace_size(int T, int K, int H, int I, int E) {
  if (T <= 0 || K <= 0 || H <= 0 || I <= 0 || E <= 0 || T > MOE_FEW_TOKENS || K > kMaxK) return 0;
  if (H > MOE_FEW_MAX_SIZE || I > MOE_FEW_MAX_SIZE) return 0;
  return few_layout(T, K, H, I, E).total;
}

extern "C" int moe_layer_few_tokens(const void* tokens, const int32_t* expert_ids,
                                    const float* probs, int T, int H, int K, int I, int E,
                                    int num_special, const uint8_t* active_mask, int mask_dims,
                                    int weight_dtype, const void* W_gate, const void* W_up,
                                    const void* W_down, const float* gate_scale,
                                    const float* up_scale, const float* down_scale,
                                    const void* shared_x, void* out, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_status,
                                    cudaStream_t stream) {
  if (weight_dtype != MOE_BF16 && weight_dtype != MOE_INT8) return MOE_ERR_INVALID_ARG;
  const FewWeights w{W_gate, W_up, W_down, gate_scale, up_scale, down_scale};
  return (weight_dtype == MOE_INT8 ? few_tokens<8> : few_tokens<16>)(
      tokens, expert_ids, probs, T, H, K, I, E, num_special, active_mask, mask_dims, 0, 0, w, shared_x, out,
      workspace, workspace_bytes, dev_status, stream);
}
