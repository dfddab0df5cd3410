// Router: the K largest logits of each token and their weights, and the
// gradient of the logits.
//
// One warp per token, the row in registers (E <= 1024: at most 32 logits a
// lane).  Both scores grow with the logit, so no rounded score enters the
// selection.  Memory asks for 5.2 us at 16384 x 256 fp32 forward and backward
// together; what bounds the kernels is the instructions of the selection and
// of the row's exponentials (issue slots 65-70 % busy; 14.8 us and 12.3 us):
//   * a logit is packed into 32 bits as the upper bits of a key that orders
//     like the float, and its index (5 to 10 bits) counted down: one warp-wide
//     maximum (redux) gives the largest and, among equals, the lowest index.
//     bf16 logits fit the 22 bits that are left at least;
//   * each lane puts the largest 4 of its packed logits (8 for K > 8) in order
//     (networks of min / max pairs) and gives up its head when it wins.  In
//     order as a whole (8 of 8) the same kernel took 16.4 us;
//   * rows where a lane has given up all of those, and for fp32 logits rows
//     where two of the first K + 1 share their upper bits without being equal,
//     are done again with full keys (two reductions and a scan a round).  Of
//     rows of normal logits at E = 256 K = 8: 0.13 % for the first reason, 0.2 %
//     for the second.  The first is commonest where few lanes hold a row (bf16,
//     E = 136 in 17 lanes: 1 %), the second in long rows (E = 1024: 1.2 % at
//     K = 8, 4 % at K = 16).
#include <math.h>

#include <type_traits>

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

// e^x, x <= 0, with what is below 2^-126 flushed to 0: a term of a sum that is
// at least 1, or of a gradient.  (__expf keeps subnormals, at three more
// instructions each.)
__device__ __forceinline__ float exp_flush(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
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

// The launch overlaps the end of the kernel before, and the next one's may
// overlap the end of this.
__device__ __forceinline__ void begin_dependent() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

// Element i of a lane: 16-byte vectors when kVec (16-byte rows, and a lane
// holds whole vectors), else every 32nd.
template <typename T, int NPL, bool kVec>
__device__ __forceinline__ int index_of(int i, int lane) {
  constexpr int V = VecTraits<T>::kElems;
  return kVec ? (i / V) * 32 * V + lane * V + i % V : lane + 32 * i;
}

// The row's logits as the definition takes them, -inf past its end; nan: one
// of them was a NaN.  Lanes whose logits are all finite, as nearly always, skip
// the clamps: 0 v summed is NaN as soon as one is not (two multiply-adds an
// element, on the pipe that the selection leaves idle).
template <typename T, int NPL, bool kVec>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, float (&v)[NPL], bool& nan) {
  constexpr int V = VecTraits<T>::kElems;
  float check = 0.f;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      const int j = index_of<T, NPL, kVec>(i, lane);
      if (j < E) {
        VecTraits<T>::unpack(ld_v4(row + j), v + i);
#pragma unroll
        for (int k = 0; k < V; ++k) check = fmaf(v[i + k], 0.f, check);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) v[i + k] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const bool in = lane + 32 * i < E;
      v[i] = in ? to_f32(row[lane + 32 * i]) : -INFINITY;
      check = fmaf(in ? v[i] : 0.f, 0.f, check);
    }
  }
  if (check != check) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      nan |= v[i] != v[i];
      v[i] = fminf(fmaxf(v[i], -INFINITY), 3.402823466e+38f);  // NaN: -inf
    }
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) v[i] += 0.f;  // -0: +0
}

template <int N>
__device__ __forceinline__ void order(uint32_t (&a)[N], int i, int j) {
  const uint32_t x = a[i], y = a[j];
  a[i] = max(x, y);
  a[j] = min(x, y);
}

// a[0..D) in descending order becomes the D largest of a, D a power of two:
// each D elements by a merging network (Batcher's odd-even merge sort), then
// group by group the larger of a[i] and b[D-1-i], a bitonic sequence of the D
// largest of both, put in order.
template <int D, int N>
__device__ __forceinline__ void top_desc(uint32_t (&a)[N]) {
#pragma unroll
  for (int g = 0; g < N; g += D) {
#pragma unroll
    for (int p = 1; p < D; p <<= 1)
#pragma unroll
      for (int k = p; k >= 1; k >>= 1)
#pragma unroll
        for (int j = k % p; j + k < D; j += 2 * k)
#pragma unroll
          for (int i = 0; i < k; ++i)
            if (i + j + k < D && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(a, g + i + j, g + i + j + k);
  }
#pragma unroll
  for (int w = D; w < N; w <<= 1)
#pragma unroll
    for (int g = 0; g < N; g += 2 * w) {
#pragma unroll
      for (int i = 0; i < D; ++i) a[g + i] = max(a[g + i], a[g + w + D - 1 - i]);
#pragma unroll
      for (int k = D / 2; k >= 1; k >>= 1)
#pragma unroll
        for (int i = 0; i < D; ++i)
          if (!(i & k)) order(a, g + i, g + i + k);
    }
}

// The selection by full keys; lane k < K gets the k-th id.
template <int NPL, typename T>
__device__ __noinline__ int select_exact(const T* row, int E, int K, int lane) {
  uint32_t key[NPL];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int j = lane + 32 * i;
    key[i] = j < E ? key_of(clean_logit(to_f32(row[j]), nan)) : 0u;
  }
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
    if (lane == k) sel_id = (int)id;
  }
  return sel_id;
}

// D: how many of its logits a lane keeps in order.  A lane whose D all win (4
// of the first 9: one row in 800 at E = 256 when the order is random) does the
// row again with full keys.
template <int NPL, int D, bool kVec, typename T>
__global__ void __launch_bounds__(kWarps * 32)
router_topk_kernel(const T* __restrict__ logits, int n_tok, int E, int K, int scoring,
                   int renormalize, float scale, int32_t* __restrict__ expert_ids,
                   float* __restrict__ probs, int32_t* status) {
  constexpr uint32_t kIndex = 32 * NPL - 1;  // the bits of an index
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  begin_dependent();
  if (t >= n_tok) return;
  const T* row = logits + (size_t)t * E;
  float v[NPL];
  bool nan = false;
  load_row<T, NPL, kVec>(row, E, lane, v, nan);
  if (nan) set_status(status, MOE_ERR_INVALID_ARG);
  uint32_t pk[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int j = index_of<T, NPL, kVec>(i, lane);
    pk[i] = j < E ? (key_of(v[i]) & ~kIndex) | (kIndex - j) : 0u;
  }
  top_desc<D>(pk);
  const bool more = D < NPL && pk[D - 1] != 0u;  // the lane may hold others
  const int rounds = min(K + 1, E);
  uint32_t mine = 0u;  // lane k: the k-th of the packed logits
#pragma unroll 3
  for (int k = 0; k < rounds; ++k) {
    const uint32_t best = __reduce_max_sync(kAll, pk[0]);
    const bool won = pk[0] == best;
#pragma unroll
    for (int i = 0; i + 1 < D; ++i) pk[i] = won ? pk[i + 1] : pk[i];
    if (won) pk[D - 1] = 0u;
    if (lane == k) mine = best;
  }
  int sel_id = (int)(kIndex - (mine & kIndex));
  const bool on = lane < rounds;
  float sel = on ? to_f32(row[sel_id]) : 0.f;
  sel = fminf(fmaxf(sel, -INFINITY), 3.402823466e+38f) + 0.f;
  bool again = more && pk[0] == 0u;
  if constexpr (sizeof(T) == 4) {
    // equal leading bits of different logits, or at the edge of the selection
    // (where further logits may share them)
    const uint32_t next = __shfl_down_sync(kAll, mine, 1);
    const float next_sel = __shfl_down_sync(kAll, sel, 1);
    again |= lane + 1 < rounds && ((mine ^ next) & ~kIndex) == 0u && (sel != next_sel || lane == K - 1);
  }
  if (__any_sync(kAll, again)) {
    sel_id = select_exact<NPL>(row, E, K, lane);
    sel = lane < K ? to_f32(row[sel_id]) : 0.f;
    sel = fminf(fmaxf(sel, -INFINITY), 3.402823466e+38f) + 0.f;
  }
  float row_sum = 0.f;
  if (scoring == MOE_SCORE_SOFTMAX && !renormalize) {
    const float m = __shfl_sync(kAll, sel, 0);  // the row's largest
    if (m > -INFINITY) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) row_sum += exp_flush(v[i] - m);
      row_sum = warp_sum(row_sum);
    }
  }
  const float q = selected_weight(sel, lane, K, scoring, renormalize != 0, row_sum);
  if (lane < K) {
    expert_ids[(size_t)t * K + lane] = sel_id;
    probs[(size_t)t * K + lane] = scale * q;
  }
}

// The dense part of a gradient row: -c v[i], or zeros.
template <typename T, int NPL, bool kVec>
__device__ __forceinline__ void store_row(T* row, int E, int lane, const float (&v)[NPL]) {
  constexpr int V = VecTraits<T>::kElems;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      const int j = index_of<T, NPL, kVec>(i, lane);
      if (j < E) st_v4(row + j, VecTraits<T>::pack(v + i));
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane + 32 * i < E) put(row + lane + 32 * i, v[i]);
  }
}

template <int NPL, bool kVec, typename T>
__global__ void __launch_bounds__(kWarps * 32)
router_grad_kernel(const float* __restrict__ grad_probs, const T* __restrict__ logits,
                   const int32_t* __restrict__ expert_ids, int n_tok, int E, int K, int scoring,
                   int renormalize, float scale, T* __restrict__ grad_logits, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  begin_dependent();
  if (t >= n_tok) return;
  const T* row = logits + (size_t)t * E;
  T* drow = grad_logits + (size_t)t * E;
  bool nan = false;
  int id = -1;
  float g = 0.f, sel = -INFINITY;
  if (lane < K) {
    id = expert_ids[(size_t)t * K + lane];
    g = scale * grad_probs[(size_t)t * K + lane];
  }
  const bool full_row = scoring == MOE_SCORE_SOFTMAX && !renormalize;
  float v[NPL];
  if (full_row) load_row<T, NPL, kVec>(row, E, lane, v, nan);
  if (lane < K) {
    if (id < 0 || id >= E) {
      set_status(status, MOE_ERR_BAD_ID);
      id = -1;
      g = 0.f;
    } else {
      sel = clean_logit(to_f32(row[id]), nan);
    }
  }
  // an id named twice collects both gradients
  bool same = false;
  for (int d = 1; 2 * d <= K; ++d) {
    const int other = lane + d < K ? lane + d : lane + d - K;  // lanes < K: the d-th next, in a ring
    const int ik = __shfl_sync(kAll, id, other & 31);
    same |= lane < K && id >= 0 && ik == id;
  }
  const bool twice = __any_sync(kAll, same);
  auto collect = [&](float x) {
    if (!twice) return x;
    float s = 0.f;
    for (int k = 0; k < K; ++k) {
      const int ik = __shfl_sync(kAll, id, k);
      const float xk = __shfl_sync(kAll, x, k);
      if (ik == id) s += xk;
    }
    return s;
  };
  const bool on = sel > -INFINITY;
  float d = 0.f;
  if (full_row) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) m = fmaxf(m, v[i]);
    // (a row of -inf alone: every term and the sum are 0)
    m = fmaxf(value_of(__reduce_max_sync(kAll, key_of(m))), -3.402823466e+38f);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      v[i] = exp_flush(v[i] - m);
      s += v[i];
    }
    s = warp_sum(s);
    const float inv = s > 0.f ? 1.f / s : 0.f;
    const float q = on ? exp_flush(sel - m) * inv : 0.f;
    const float D = warp_sum(on ? g * q : 0.f), c = inv * D;
    if (fabsf(c) <= 3.402823466e+38f) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) v[i] = fmaf(-v[i], c, 0.f);
    } else {  // an infinite or NaN gradient leaves the masked logits' at 0
#pragma unroll
      for (int i = 0; i < NPL; ++i) v[i] = v[i] > 0.f ? -v[i] * c : 0.f;
    }
    const float both = collect(g);
    d = on ? q * (both - D) : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = 0.f;
    // the largest selected logit, whatever the order of the ids
    const float m_sel = value_of(__reduce_max_sync(kAll, key_of(sel)));
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
    d = collect(mine);
  }
  store_row<T, NPL, kVec>(drow, E, lane, v);
  if (nan) set_status(status, MOE_ERR_INVALID_ARG);
  __syncwarp();  // the row's values are in place before the selected ones replace theirs
  if (lane < K && id >= 0) put(drow + id, d);
}

template <typename F, typename... A>
void launch_pdl(F* kernel, int grid, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  (void)cudaLaunchKernelEx(&cfg, kernel, args...);
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

// f(logits per lane, 16-byte vectors) for rows of E logits.  Vectors need rows
// of whole vectors and a lane that holds whole ones.
template <typename T, typename F>
void by_width(int E, F&& f) {
  constexpr int V = VecTraits<T>::kElems;
  const bool vec = E % V == 0;
  auto go = [&](auto n) {
    if constexpr (decltype(n)::value >= V) {
      if (vec) return f(n, std::true_type{});
    }
    f(n, std::false_type{});
  };
  if (E <= 32) go(std::integral_constant<int, 1>{});
  else if (E <= 64) go(std::integral_constant<int, 2>{});
  else if (E <= 128) go(std::integral_constant<int, 4>{});
  else if (E <= 256) go(std::integral_constant<int, 8>{});
  else if (E <= 512) go(std::integral_constant<int, 16>{});
  else go(std::integral_constant<int, 32>{});
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
  const int grid = (T - 1) / kWarps + 1;  // (T + kWarps - 1 may pass 31 bits)
  auto go = [&](auto* x) {
    using D = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    by_width<D>(E, [&](auto n, auto vec) {
      constexpr int N = decltype(n)::value;
      auto* kernel = K <= 8 ? router_topk_kernel<N, N < 4 ? N : 4, decltype(vec)::value, D>
                            : router_topk_kernel<N, N < 8 ? N : 8, decltype(vec)::value, D>;
      launch_pdl(kernel, grid, stream, x, T, E, K, scoring, renormalize, scale, expert_ids, probs, dev_status);
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
  const int grid = (T - 1) / kWarps + 1;  // (T + kWarps - 1 may pass 31 bits)
  auto go = [&](auto* x, auto* d) {
    using D = std::remove_pointer_t<decltype(d)>;
    by_width<D>(E, [&](auto n, auto vec) {
      launch_pdl(router_grad_kernel<decltype(n)::value, decltype(vec)::value, D>, grid, stream, grad_probs, x,
                 expert_ids, T, E, K, scoring, renormalize, scale, d, dev_status);
    });
  };
  if (dtype == MOE_F32) go(static_cast<const float*>(logits), static_cast<float*>(grad_logits));
  else go(static_cast<const __nv_bfloat16*>(logits), static_cast<__nv_bfloat16*>(grad_logits));
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}
