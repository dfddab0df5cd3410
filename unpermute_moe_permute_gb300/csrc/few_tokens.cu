// The whole expert layer for a few tokens.
//
// Two kernels: a warp per (slot, intermediate column) for silu(g) * u, and a
// warp per (token, output column) for the weighted sum of the K down rows.
#include <math.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;

// Expert of slot (t, k), or -1 for a slot that adds nothing (inactive,
// special, out of range or repeated).
__device__ __forceinline__ int slot_expert(const int32_t* ids, const uint8_t* mask, int mask_dims,
                                           int t, int k, int K, int E, int E_all, int32_t* status) {
  const int e = ids[t * K + k];
  bool bad = e < 0 || e >= E_all;
  for (int j = 0; j < k; ++j) bad |= ids[t * K + j] == e;
  if (bad) {
    set_status(status, MOE_ERR_BAD_ID);
    return -1;
  }
  if (mask != nullptr && mask[mask_dims == 1 ? t : t * K + k] == 0) return -1;
  return e < E ? e : -1;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// 8 weights as floats
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  VecTraits<__nv_bfloat16>::unpack(ld_v4(p), f);
}
__device__ __forceinline__ void load8(const int8_t* p, float (&f)[8]) {
  const int2 v = *reinterpret_cast<const int2*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = (float)(int8_t)(v.x >> (8 * i));
    f[4 + i] = (float)(int8_t)(v.y >> (8 * i));
  }
}

template <typename A, typename W>
__device__ __forceinline__ float dot_row(const A* a, const W* w, int n, int lane) {
  float s = 0.f;
  for (int c = lane * 8; c < n; c += 256) {
    float x[8], y[8];
    load8(a + c, x);
    load8(w + c, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
  }
  return warp_sum(s);
}

template <typename W>
__global__ void __launch_bounds__(kWarps * 32)
few_gate_up_kernel(const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ ids,
                   const uint8_t* __restrict__ mask, int mask_dims, int H, int K, int I, int E,
                   int E_all, const W* __restrict__ Wg, const W* __restrict__ Wu,
                   const float* __restrict__ gs, const float* __restrict__ us,
                   __nv_bfloat16* __restrict__ act, int32_t* status) {
  const int lane = threadIdx.x & 31, i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int f = blockIdx.y, t = f / K;
  const int e = slot_expert(ids, mask, mask_dims, t, f % K, K, E, E_all, status);
  if (i >= I || e < 0) return;
  const size_t r = (size_t)e * I + i;
  float g = dot_row(x + (size_t)t * H, Wg + r * H, H, lane);
  float u = dot_row(x + (size_t)t * H, Wu + r * H, H, lane);
  if (gs != nullptr) g *= gs[r], u *= us[r];
  if (lane == 0) act[(size_t)f * I + i] = __float2bfloat16_rn(g / (1.f + expf(-g)) * u);
}

template <typename W>
__global__ void __launch_bounds__(kWarps * 32)
few_down_kernel(const __nv_bfloat16* __restrict__ act, const int32_t* __restrict__ ids,
                const uint8_t* __restrict__ mask, int mask_dims, const float* __restrict__ probs,
                int H, int K, int I, int E, int E_all, const W* __restrict__ Wd,
                const float* __restrict__ ds, const __nv_bfloat16* __restrict__ shared_x,
                __nv_bfloat16* __restrict__ out, int32_t* status) {
  const int lane = threadIdx.x & 31, h = blockIdx.x * kWarps + (threadIdx.x >> 5), t = blockIdx.y;
  if (h >= H) return;
  float y = 0.f;
  for (int k = 0; k < K; ++k) {
    const int e = slot_expert(ids, mask, mask_dims, t, k, K, E, E_all, status);
    if (e < 0) continue;
    const size_t r = (size_t)e * H + h;
    float d = dot_row(act + (size_t)(t * K + k) * I, Wd + r * I, I, lane);
    if (ds != nullptr) d *= ds[r];
    y = fmaf(probs[t * K + k], d, y);
  }
  if (shared_x != nullptr) y += __bfloat162float(shared_x[(size_t)t * H + h]);
  if (lane == 0) out[(size_t)t * H + h] = __float2bfloat16_rn(y);
}

template <typename W>
int launch_few(const __nv_bfloat16* x, const int32_t* ids, const float* probs, int T, int H, int K,
               int I, int E, int E_all, const uint8_t* mask, int mask_dims, const void* Wg,
               const void* Wu, const void* Wd, const float* gs, const float* us, const float* ds,
               const __nv_bfloat16* shared_x, __nv_bfloat16* out, __nv_bfloat16* act,
               int32_t* status, cudaStream_t s) {
  few_gate_up_kernel<W><<<dim3((I + kWarps - 1) / kWarps, T * K), kWarps * 32, 0, s>>>(
      x, ids, mask, mask_dims, H, K, I, E, E_all, static_cast<const W*>(Wg),
      static_cast<const W*>(Wu), gs, us, act, status);
  few_down_kernel<W><<<dim3((H + kWarps - 1) / kWarps, T), kWarps * 32, 0, s>>>(
      act, ids, mask, mask_dims, probs, H, K, I, E, E_all, static_cast<const W*>(Wd), ds, shared_x,
      out, status);
  MOE_LAUNCH_CHECK();
  count_launches(2);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_layer_few_tokens_workspace_size(int T, int K, int H, int I, int E) {
  if (T <= 0 || K <= 0 || H <= 0 || I <= 0 || E <= 0) return 0;
  return (size_t)T * K * I * 2;
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
  if (T < 0 || H <= 0 || K <= 0 || I <= 0 || E <= 0 || num_special < 0) return MOE_ERR_INVALID_ARG;
  if (weight_dtype != MOE_BF16 && weight_dtype != MOE_INT8) return MOE_ERR_INVALID_ARG;
  if (active_mask != nullptr && mask_dims != 1 && mask_dims != 2) return MOE_ERR_INVALID_ARG;
  if (T > MOE_FEW_TOKENS || K > kMaxK || E > kMaxExperts) return MOE_ERR_SHAPE;
  if ((long long)E + num_special > 0x7fffffffLL || (long long)K > (long long)E + num_special)
    return MOE_ERR_SHAPE;
  if (H % 64 || I % 64) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!tokens || !expert_ids || !probs || !W_gate || !W_up || !W_down || !out || !workspace)
    return MOE_ERR_INVALID_ARG;
  const bool i8 = weight_dtype == MOE_INT8;
  if (i8 != (gate_scale != nullptr) || i8 != (up_scale != nullptr) || i8 != (down_scale != nullptr))
    return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {tokens, W_gate, W_up, W_down, shared_x, out, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_layer_few_tokens_workspace_size(T, K, H, I, E))
    return MOE_ERR_INVALID_ARG;
  auto go = [&](auto w) {
    return launch_few<decltype(w)>(
        static_cast<const __nv_bfloat16*>(tokens), expert_ids, probs, T, H, K, I, E, E + num_special,
        active_mask, mask_dims, W_gate, W_up, W_down, gate_scale, up_scale, down_scale,
        static_cast<const __nv_bfloat16*>(shared_x), static_cast<__nv_bfloat16*>(out),
        static_cast<__nv_bfloat16*>(workspace), dev_status, stream);
  };
  return i8 ? go(int8_t{}) : go(__nv_bfloat16{});
}
