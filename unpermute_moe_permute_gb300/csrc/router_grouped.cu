// Router with a bias for each expert and groups of experts.
//
//   s_j = sigmoid(l_j) or softmax(l)_j,   c_j = s_j + bias_j
//   v_g = the sum of the `each` largest c_j of group g (1 or 2)
//   the top_groups largest v_g, then the K largest c_j of those groups;
//   weights from the s_j alone
//
// One warp per token; a group belongs to 32 / P neighbouring lanes (P: the
// number of groups, rounded up to a power of two), so its two largest are a
// few shuffles, and a lane's group is kept or dropped as a whole.
//
// The selection is that of exact scores.  c is computed in fp32 and carried as
// a 32-bit key whose lowest bits (3 for 8 scores a lane) say which of the lane's
// scores it is; one warp-wide maximum a round finds the next.  What lies closer
// together than fp32's error and the missing bits, at the border between kept
// and dropped groups or anywhere among the first K + 1, is decided again in 64
// bits (select_exact).  Of normal logits at E = 256 in 8 groups K = 8 that is
// one row in 200.  Where no score is needed (no bias, and no sum of two) the
// logits themselves are compared and their keys hold the whole index, as in the
// plain router.
#include <type_traits>

#include "router.cuh"

namespace moe {
namespace {

struct GroupParams {
  const float* bias;
  int n_tok, E, K, G, size, top, each;  // size: experts of a group
  int lg;                               // log2 of the lanes of a group
  int scoring, renormalize;
  float scale;
};

// Element i of a lane inside its group.
template <typename T, bool kVec>
__device__ __forceinline__ int place(int i, int r, int lg) {
  constexpr int V = VecTraits<T>::kElems;
  return kVec ? (((i / V) << lg) + r) * V + i % V : (i << lg) + r;
}

// A bias as the definition takes it: what is not below +inf takes the expert
// out, as -inf does, and is flagged.
__device__ __forceinline__ float clean_bias(float b, bool& bad) {
  if (b < INFINITY) return b;
  bad = true;
  return -INFINITY;
}

// The selection in 64 bits; lane k < K gets the k-th id.  by_logit: c is the
// logit.  Groups with fewer experts above -inf (of `each`) come last; when the
// kept groups have fewer than K of those, their others follow in order.
template <int NPL, typename T>
__device__ __noinline__ int select_exact(const T* row, const GroupParams& p, bool by_logit, int lane) {
  const int g = lane >> p.lg, r = lane & ((1 << p.lg) - 1);
  double c[NPL];
  bool flag = false;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int o = place<T, false>(i, r, p.lg);
    const float l = g < p.G && o < p.size ? clean_logit(to_f32(row[g * p.size + o]), flag) : -INFINITY;
    c[i] = l;
    m = fmaxf(m, l);
  }
  if (!by_logit) {
    double inv = 0.0;
    if (p.scoring == MOE_SCORE_SOFTMAX) {
      m = fmaxf(value_of(__reduce_max_sync(kAll, key_of(m))), -3.402823466e+38f);
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) s += c[i] = exp(c[i] - m);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kAll, s, d);
      inv = s;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int o = place<T, false>(i, r, p.lg);
      const bool in = g < p.G && o < p.size;
      const float l = in ? clean_logit(to_f32(row[g * p.size + o]), flag) : -INFINITY;
      const float b = in && p.bias ? clean_bias(p.bias[g * p.size + o], flag) : 0.f;
      double s;
      if (p.scoring == MOE_SCORE_SOFTMAX) {
        s = c[i] / inv;
      } else {
        const double e = exp(-fabs(c[i]));
        s = (c[i] < 0.0 ? e : 1.0) / (1.0 + e);
      }
      c[i] = l > -INFINITY ? s + b : -INFINITY;
    }
  }
  // the two largest of the group
  double a1 = -INFINITY, a2 = -INFINITY;
  unsigned long long open = 0;  // elements that may be chosen yet
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if (g < p.G && place<T, false>(i, r, p.lg) < p.size) open |= 1ull << i;
    a2 = fmax(a2, fmin(a1, c[i]));
    a1 = fmax(a1, c[i]);
  }
  for (int d = 1; d < 1 << p.lg; d <<= 1) {
    const double b1 = __shfl_xor_sync(kAll, a1, d), b2 = __shfl_xor_sync(kAll, a2, d);
    a2 = fmax(fmin(a1, b1), fmax(a2, b2));
    a1 = fmax(a1, b1);
  }
  const int live = (a1 > -INFINITY) + (p.each > 1 && a2 > -INFINITY);
  const double v = live > 1 ? a1 + a2 : a1;
  int rank = 0;
  for (int h = 0; h < p.G; ++h) {
    const double vh = __shfl_sync(kAll, v, h << p.lg);
    const int lh = __shfl_sync(kAll, live, h << p.lg);
    rank += lh > live || (lh == live && (vh > v || (vh == v && h < g)));
  }
  if (rank >= p.top) open = 0;
  int sel_id = 0;
  for (int k = 0; k < p.K; ++k) {
    double best = -INFINITY;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {  // (in ascending order of the index)
      if (((open >> i) & 1) && (at == 0x7fffffff || c[i] > best)) {
        best = c[i];
        at = g * p.size + place<T, false>(i, r, p.lg);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double ob = __shfl_xor_sync(kAll, best, d);
      const int oa = __shfl_xor_sync(kAll, at, d);
      if (oa != 0x7fffffff && (at == 0x7fffffff || ob > best || (ob == best && oa < at))) best = ob, at = oa;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (g * p.size + place<T, false>(i, r, p.lg) == at) open &= ~(1ull << i);
    if (lane == k) sel_id = at;
  }
  return sel_id;
}

// NPL: scores of a lane, D: how many of them it keeps in order.
template <int NPL, int D, bool kVec, bool kByLogit, typename T>
__global__ void __launch_bounds__(kWarps * 32)
router_grouped_kernel(const T* __restrict__ logits, const __grid_constant__ GroupParams p,
                      int32_t* __restrict__ expert_ids, float* __restrict__ probs, int32_t* status) {
  constexpr int V = VecTraits<T>::kElems;
  constexpr uint32_t kLow = kByLogit ? kMaxExperts - 1 : NPL - 1;  // bits of a key that name its element
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int g = lane >> p.lg, r = lane & ((1 << p.lg) - 1);
  begin_dependent();
  if (t >= p.n_tok) return;
  const T* row = logits + (size_t)t * p.E;
  float c[NPL];
  bool flag = false;
  // the logits as the definition takes them, -inf past the group's end
  float check = 0.f;
#pragma unroll
  for (int i = 0; i < NPL; i += kVec ? V : 1) {
    const int o = place<T, kVec>(i, r, p.lg);
    const bool in = g < p.G && o < p.size;
    if constexpr (kVec) {
      if (in) VecTraits<T>::unpack(ld_v4(row + g * p.size + o), c + i);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (!in) c[i + k] = -INFINITY;
        else check = fmaf(c[i + k], 0.f, check);
      }
    } else {
      c[i] = in ? to_f32(row[g * p.size + o]) : -INFINITY;
      check = fmaf(in ? c[i] : 0.f, 0.f, check);
    }
  }
  if (check != check) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      flag |= c[i] != c[i];
      c[i] = fminf(fmaxf(c[i], -INFINITY), 3.402823466e+38f);  // NaN: -inf
    }
  }
  // softmax: the row's largest logit and its sum, for the scores or for weights
  // that are not renormalised
  float m = 0.f, row_sum = 1.f;
  const bool soft = p.scoring == MOE_SCORE_SOFTMAX;
  if (soft && (!kByLogit || !p.renormalize)) {
    m = c[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) m = fmaxf(m, c[i]);
    m = fmaxf(value_of(__reduce_max_sync(kAll, key_of(m))), -3.402823466e+38f);
    row_sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) row_sum += exp_flush(c[i] - m);
    row_sum = fmaxf(warp_sum(row_sum), 1e-30f);  // (a row of -inf alone: every term is 0)
  }
  // Error of a difference of two c: the approximate exponential and reciprocal
  // are off by 2^-22 each, s (1 - s) |l| < 0.23 takes the rounding of the
  // exponential's argument, so s is off by less than 2^-22; for softmax also the
  // sum's rounding, 37 additions at most: p 2^-18.
  float eps = 0.f;
  if constexpr (!kByLogit) {
    const float inv = 1.f / row_sum;
    eps = soft ? inv * 0x1p-17f : 0x1p-20f;
    float bcheck = 0.f, b[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) b[i] = 0.f;
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < NPL; i += kVec ? V : 1) {
        const int o = place<T, kVec>(i, r, p.lg);
        if (g < p.G && o < p.size) {
          if constexpr (kVec) {
#pragma unroll
            for (int k = 0; k < V; k += 4) VecTraits<float>::unpack(ld_v4(p.bias + g * p.size + o + k), b + i + k);
          } else {
            b[i] = p.bias[g * p.size + o];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) bcheck = fmaf(b[i], 0.f, bcheck);
      if (bcheck != bcheck) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) b[i] = clean_bias(b[i], flag);
      }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      float s;
      if (soft) {
        s = exp_flush(c[i] - m) * inv;
      } else {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(c[i] * -1.4426950408889634f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + s));
      }
      c[i] = c[i] > -INFINITY ? s + b[i] : -INFINITY;
    }
  }
  if (flag) set_status(status, MOE_ERR_INVALID_ARG);
  bool again = false, keep = g < p.G;
  if (p.top < p.G) {
    float a1 = c[0], a2 = -INFINITY;
#pragma unroll
    for (int i = 1; i < NPL; ++i) {
      a2 = fmaxf(a2, fminf(a1, c[i]));
      a1 = fmaxf(a1, c[i]);
    }
    for (int d = 1; d < 1 << p.lg; d <<= 1) {
      const float b1 = __shfl_xor_sync(kAll, a1, d), b2 = __shfl_xor_sync(kAll, a2, d);
      a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
      a1 = fmaxf(a1, b1);
    }
    // (a group with one expert of two ranks between those with two and none)
    again = keep && p.each > 1 && a1 > -INFINITY && a2 == -INFINITY;
    const float v = p.each > 1 ? a1 + a2 : a1;
    int rank = 0;
    for (int h = 0; h < p.G; ++h) {
      const float vh = __shfl_sync(kAll, v, h << p.lg);
      rank += vh > v || (vh == v && h < g);
    }
    keep = keep && rank < p.top;
    if constexpr (!kByLogit) {  // the border between kept and dropped groups
      const float lo = value_of(__reduce_min_sync(kAll, keep ? key_of(v) : 0xffffffffu));
      const float hi = value_of(__reduce_max_sync(kAll, !keep && g < p.G ? key_of(v) : 0u));
      again |= lo - hi <= 2.f * eps + 0x1p-21f * (fabsf(lo) + fabsf(hi));
    }
  }
  uint32_t pk[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const uint32_t low = kByLogit ? kLow - (g * p.size + place<T, kVec>(i, r, p.lg)) : kLow - i;
    pk[i] = keep && c[i] > -INFINITY ? (key_of(c[i] + 0.f) & ~kLow) | low : 0u;
  }
  top_desc<D>(pk);
  const bool more = D < NPL && pk[D - 1] != 0u;  // the lane may hold others
  uint32_t mine = 0u;  // lane k: the k-th key, and its lane
  int from = 0;
#pragma unroll 3
  for (int k = 0; k <= p.K; ++k) {
    const uint32_t best = __reduce_max_sync(kAll, pk[0]);
    const int src = __ffs(__ballot_sync(kAll, pk[0] == best)) - 1;
    const bool won = lane == src;
#pragma unroll
    for (int i = 0; i + 1 < D; ++i) pk[i] = won ? pk[i + 1] : pk[i];
    if (won) pk[D - 1] = 0u;
    if (lane == k) mine = best, from = src;
  }
  int sel_id;
  if constexpr (kByLogit) {
    sel_id = (int)(kLow - (mine & kLow));
  } else {
    sel_id = (from >> p.lg) * p.size + place<T, kVec>((int)(kLow - (mine & kLow)), from & ((1 << p.lg) - 1), p.lg);
  }
  float sel = lane < p.K && mine != 0u ? to_f32(row[sel_id]) : -INFINITY;
  sel = fminf(sel, 3.402823466e+38f) + 0.f;
  again |= (more && pk[0] == 0u) || (lane < p.K && mine == 0u);
  const uint32_t next = __shfl_down_sync(kAll, mine, 1);
  if constexpr (!kByLogit) {
    const float x = value_of(mine & ~kLow), y = value_of(next & ~kLow);
    again |= lane < p.K && next != 0u && x - y <= eps + (0x1p-23f * NPL + 0x1p-22f) * (fabsf(x) + fabsf(y));
  } else if constexpr (sizeof(T) == 4) {
    // equal leading bits of different logits, or at the edge of the selection
    // (where further logits may share them)
    const float next_sel = __shfl_down_sync(kAll, sel, 1);
    again |= lane < p.K && next != 0u && ((mine ^ next) & ~kLow) == 0u && (sel != next_sel || lane == p.K - 1);
  }
  if (__any_sync(kAll, again)) {
    sel_id = select_exact<NPL>(row, p, kByLogit, lane);
    sel = lane < p.K ? to_f32(row[sel_id]) : -INFINITY;
    sel = fminf(fmaxf(sel, -INFINITY), 3.402823466e+38f) + 0.f;
  }
  const bool on = lane < p.K && sel > -INFINITY;
  float q = 0.f;
  if (soft || p.renormalize) {
    const float top = soft && !p.renormalize
                          ? m
                          : fmaxf(value_of(__reduce_max_sync(kAll, key_of(on ? sel : -INFINITY))), -3.402823466e+38f);
    if (on) q = soft ? expf(sel - top) : sigmoid_ratio(sel, top);
    const float s = p.renormalize ? warp_sum(q) : row_sum;
    q = on ? q / s : 0.f;
  } else if (on) {
    q = 1.f / (1.f + expf(-sel));
  }
  if (lane < p.K) {
    expert_ids[(size_t)t * p.K + lane] = sel_id;
    probs[(size_t)t * p.K + lane] = p.scale * q;
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_router_topk_grouped(const void* logits, int dtype, const float* bias, int T, int E,
                                       int K, int num_groups, int top_groups, int group_top,
                                       int scoring, int renormalize, float scale, int32_t* expert_ids,
                                       float* probs, int32_t* dev_status, cudaStream_t stream) {
  if (T < 0 || E <= 0 || K <= 0 || num_groups <= 0 || top_groups <= 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (group_top != 1 && group_top != 2) return MOE_ERR_INVALID_ARG;
  if (K > kMaxK || E > kMaxExperts || num_groups > 32 || top_groups > num_groups) return MOE_ERR_SHAPE;
  if (E % num_groups || group_top > E / num_groups) return MOE_ERR_SHAPE;
  if (K > top_groups * (E / num_groups)) return MOE_ERR_SHAPE;
  if ((long long)T * K > 0x7fffffffLL) return MOE_ERR_SHAPE;
  GroupParams p{bias, T, E, K, num_groups, E / num_groups, top_groups, group_top, 5, scoring, renormalize, scale};
  for (int n = 1; n < num_groups; n *= 2) --p.lg;
  const int each = ((p.size - 1) >> p.lg) + 1;  // scores of a lane
  if (each > 32) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!logits || !expert_ids || !probs) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(expert_ids) || !aligned16(probs))
    return MOE_ERR_INVALID_ARG;
  const int grid = (T - 1) / kWarps + 1;  // (T + kWarps - 1 may pass 31 bits)
  const bool by_logit = bias == nullptr && (group_top == 1 || top_groups == num_groups);
  auto go = [&](auto* x) {
    using D = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    constexpr int V = VecTraits<D>::kElems;
    auto launch = [&](auto n, auto vec, auto by) {
      constexpr int N = decltype(n)::value;
      // Eight in order: four of 16 lanes' scores (4 groups of 8 kept) run out in 3 % of the rows.
      launch_pdl(router_grouped_kernel<N, N < 8 ? N : 8, decltype(vec)::value, decltype(by)::value, D>, grid, stream,
                 x, p, expert_ids, probs, dev_status);
    };
    auto width = [&](auto n) {
      constexpr bool can = decltype(n)::value >= V;
      const bool vec = p.size % V == 0;
      if constexpr (can) {
        if (vec) return by_logit ? launch(n, std::true_type{}, std::true_type{})
                                 : launch(n, std::true_type{}, std::false_type{});
      }
      return by_logit ? launch(n, std::false_type{}, std::true_type{}) : launch(n, std::false_type{}, std::false_type{});
    };
    if (each <= 1) width(std::integral_constant<int, 1>{});
    else if (each <= 2) width(std::integral_constant<int, 2>{});
    else if (each <= 4) width(std::integral_constant<int, 4>{});
    else if (each <= 8) width(std::integral_constant<int, 8>{});
    else if (each <= 16) width(std::integral_constant<int, 16>{});
    else width(std::integral_constant<int, 32>{});
  };
  if (dtype == MOE_F32) go(static_cast<const float*>(logits));
  else go(static_cast<const __nv_bfloat16*>(logits));
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}
