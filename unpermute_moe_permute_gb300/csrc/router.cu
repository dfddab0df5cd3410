// Router: the K largest logits of each token and their weights, and the
// gradient of the logits.
//
// One warp per token; lane i holds the logits i, i + 32, ... of the row in
// registers (E <= 1024: at most 32 each).  Selection compares 32-bit keys
// whose unsigned order is the order of the floats: K rounds of a warp-wide
// maximum (redux), the lowest index among equals, and the winner taken out.
// Both scores grow with the logit, so no rounded score enters the selection.
#include <math.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

// A logit as the definition takes it: NaN as -inf (flagged), +inf as the
// largest finite float, -0 as +0 (they compare equal).
__device__ __forceinline__ float clean_logit(float v, bool& nan) {
  if (v != v) {
    nan = true;
    return -INFINITY;
  }
  return v == 0.f ? 0.f : fminf(v, 3.402823466e+38f);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Unsigned keys in the order of the floats; every float's key is above 0.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// sigmoid(l) / sigmoid(l0) for l <= l0, without overflow:
// sigmoid(l) = e^min(l, 0) / (1 + e^-|l|).
__device__ __forceinline__ float sigmoid_ratio(float l, float l0) {
  return expf(fminf(l, 0.f) - fminf(l0, 0.f)) * (1.f + expf(-fabsf(l0))) / (1.f + expf(-fabsf(l)));
}

// Weights q_k (before the scale) of the selected logits: lane k < K holds
// sel, the k-th largest logit, and s1 = its sum of e^(l - m) over the row.
// -inf gives 0; sel of lane 0 is the row's maximum m.
__device__ __forceinline__ float selected_weight(float sel, int lane, int K, int scoring,
                                                 bool renormalize, float row_sum) {
  const float m = __shfl_sync(kAll, sel, 0);
  const bool on = lane < K && sel > -INFINITY;
  float w = 0.f;
  if (scoring == MOE_SCORE_SOFTMAX) {
    if (on) w = expf(sel - m);
    const float s = renormalize ? warp_sum(w) : row_sum;
    return on ? w / s : 0.f;
  }
  if (!renormalize) return on ? 1.f / (1.f + expf(-sel)) : 0.f;
  if (on) w = sigmoid_ratio(sel, m);
  const float s = warp_sum(w);
  return on ? w / s : 0.f;
}

template <int NPL, typename T>
__global__ void __launch_bounds__(kWarps * 32)
router_topk_kernel(const T* __restrict__ logits, int n_tok, int E, int K, int scoring,
                   int renormalize, float scale, int32_t* __restrict__ expert_ids,
                   float* __restrict__ probs, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= n_tok) return;
  const T* row = logits + (size_t)t * E;
  uint32_t key[NPL];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int j = lane + 32 * i;
    key[i] = j < E ? key_of(clean_logit(to_f32(row[j]), nan)) : 0u;
  }
  if (nan) set_status(status, MOE_ERR_INVALID_ARG);
  float row_sum = 0.f;
  if (scoring == MOE_SCORE_SOFTMAX && !renormalize) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) top = max(top, key[i]);
    const float m = value_of(__reduce_max_sync(kAll, top));
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const float v = value_of(key[i]);
      if (key[i] != 0u && v > -INFINITY) row_sum += expf(v - m);
    }
    row_sum = warp_sum(row_sum);
  }
  float sel = -INFINITY;
  int sel_id = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) top = max(top, key[i]);
    const uint32_t best = __reduce_max_sync(kAll, top);
    uint32_t at = 0xffffffffu;  // lowest index of this lane that holds it
#pragma unroll
    for (int i = NPL - 1; i >= 0; --i)
      if (key[i] == best) at = lane + 32 * i;
    const uint32_t id = __reduce_min_sync(kAll, at);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (id == (uint32_t)(lane + 32 * i)) key[i] = 0u;
    if (lane == k) {
      sel = value_of(best);
      sel_id = (int)id;
    }
  }
  const float q = selected_weight(sel, lane, K, scoring, renormalize != 0, row_sum);
  if (lane < K) {
    expert_ids[(size_t)t * K + lane] = sel_id;
    probs[(size_t)t * K + lane] = scale * q;
  }
}

template <int NPL, typename T>
__global__ void __launch_bounds__(kWarps * 32)
router_grad_kernel(const float* __restrict__ grad_probs, const T* __restrict__ logits,
                   const int32_t* __restrict__ expert_ids, int n_tok, int E, int K, int scoring,
                   int renormalize, float scale, T* __restrict__ grad_logits, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= n_tok) return;
  const T* row = logits + (size_t)t * E;
  T* drow = grad_logits + (size_t)t * E;
  bool nan = false;
  int id = -1;
  float g = 0.f, sel = -INFINITY;
  if (lane < K) {
    id = expert_ids[(size_t)t * K + lane];
    if (id < 0 || id >= E) {
      set_status(status, MOE_ERR_BAD_ID);
      id = -1;
    } else {
      g = scale * grad_probs[(size_t)t * K + lane];
      sel = clean_logit(to_f32(row[id]), nan);
    }
  }
  // the largest selected logit, whatever the order of the ids
  const float m_sel = value_of(__reduce_max_sync(kAll, key_of(sel)));
  float d = 0.f;
  if (scoring == MOE_SCORE_SOFTMAX && !renormalize) {
    float v[NPL], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int j = lane + 32 * i;
      v[i] = j < E ? clean_logit(to_f32(row[j]), nan) : -INFINITY;
      m = fmaxf(m, v[i]);
    }
    m = value_of(__reduce_max_sync(kAll, key_of(m)));
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      v[i] = v[i] > -INFINITY ? expf(v[i] - m) : 0.f;
      s += v[i];
    }
    s = warp_sum(s);
    const float inv = s > 0.f ? 1.f / s : 0.f;
    const float q = sel > -INFINITY ? expf(sel - m) * inv : 0.f;
    const float D = warp_sum(q > 0.f ? g * q : 0.f);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int j = lane + 32 * i;
      if (j < E) put(drow + j, v[i] > 0.f ? -(v[i] * inv) * D : 0.f);
    }
    float gs = 0.f;  // an id named twice collects both gradients
    for (int k = 0; k < K; ++k) {
      const int ik = __shfl_sync(kAll, id, k);
      const float gk = __shfl_sync(kAll, g, k);
      if (ik == id) gs += gk;
    }
    d = q > 0.f ? q * (gs - D) : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int j = lane + 32 * i;
      if (j < E) put(drow + j, 0.f);
    }
    const bool on = sel > -INFINITY;
    float q = 0.f, mine;
    if (scoring == MOE_SCORE_SOFTMAX) {
      q = on ? expf(sel - m_sel) : 0.f;
    } else if (renormalize) {
      q = on ? sigmoid_ratio(sel, m_sel) : 0.f;
    }
    if (renormalize) {
      const float s = warp_sum(q);
      q = on ? q / s : 0.f;
      const float D = warp_sum(on ? g * q : 0.f);
      mine = on ? q * (g - D) : 0.f;
    } else {
      mine = on ? g / (1.f + expf(-sel)) : 0.f;
    }
    // 1 - sigmoid(l) = 1 / (1 + e^l)
    if (scoring == MOE_SCORE_SIGMOID && on) mine *= 1.f / (1.f + expf(sel));
    for (int k = 0; k < K; ++k) {
      const int ik = __shfl_sync(kAll, id, k);
      const float mk = __shfl_sync(kAll, mine, k);
      if (ik == id) d += mk;
    }
  }
  if (nan) set_status(status, MOE_ERR_INVALID_ARG);
  __syncwarp();  // the row's values are in place before the selected ones replace theirs
  if (lane < K && id >= 0) put(drow + id, d);
}

int check_router(const void* logits, int dtype, int T, int E, int K, int scoring) {
  if (T < 0 || E <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (K > kMaxK || K > E || E > kMaxExperts) return MOE_ERR_SHAPE;
  if ((long long)T * K > 0x7fffffffLL) return MOE_ERR_SHAPE;
  if (T > 0 && (!logits || !aligned16(logits))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

template <typename T, typename F>
void by_width(int E, F&& f) {
  if (E <= 32) f(std::integral_constant<int, 1>{});
  else if (E <= 64) f(std::integral_constant<int, 2>{});
  else if (E <= 128) f(std::integral_constant<int, 4>{});
  else if (E <= 256) f(std::integral_constant<int, 8>{});
  else if (E <= 512) f(std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 32>{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_router_topk(const void* logits, int dtype, int T, int E, int K, int scoring,
                               int renormalize, float scale, int32_t* expert_ids, float* probs,
                               int32_t* dev_status, cudaStream_t stream) {
  if (int rc = check_router(logits, dtype, T, E, K, scoring)) return rc;
  if (T == 0) return MOE_OK;
  if (!expert_ids || !probs || !aligned16(expert_ids) || !aligned16(probs))
    return MOE_ERR_INVALID_ARG;
  const int grid = (T + kWarps - 1) / kWarps;
  auto go = [&](auto* x) {
    using D = std::remove_pointer_t<decltype(x)>;
    by_width<D>(E, [&](auto n) {
      router_topk_kernel<decltype(n)::value, std::remove_const_t<D>><<<grid, kWarps * 32, 0, stream>>>(
          x, T, E, K, scoring, renormalize, scale, expert_ids, probs, dev_status);
    });
  };
  if (dtype == MOE_F32) go(static_cast<const float*>(logits));
  else go(static_cast<const __nv_bfloat16*>(logits));
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}

extern "C" int moe_router_topk_grad(const float* grad_probs, const void* logits, int dtype,
                                    const int32_t* expert_ids, int T, int E, int K, int scoring,
                                    int renormalize, float scale, void* grad_logits,
                                    int32_t* dev_status, cudaStream_t stream) {
  if (int rc = check_router(logits, dtype, T, E, K, scoring)) return rc;
  if (T == 0) return MOE_OK;
  if (!grad_probs || !expert_ids || !grad_logits || !aligned16(grad_probs) ||
      !aligned16(expert_ids) || !aligned16(grad_logits))
    return MOE_ERR_INVALID_ARG;
  const int grid = (T + kWarps - 1) / kWarps;
  auto go = [&](auto* x, auto* d) {
    using D = std::remove_pointer_t<decltype(d)>;
    by_width<D>(E, [&](auto n) {
      router_grad_kernel<decltype(n)::value, D><<<grid, kWarps * 32, 0, stream>>>(
          grad_probs, x, expert_ids, T, E, K, scoring, renormalize, scale, d, dev_status);
    });
  };
  if (dtype == MOE_F32) go(static_cast<const float*>(logits), static_cast<float*>(grad_logits));
  else go(static_cast<const __nv_bfloat16*>(logits), static_cast<__nv_bfloat16*>(grad_logits));
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}
