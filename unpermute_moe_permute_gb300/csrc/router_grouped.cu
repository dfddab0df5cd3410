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
// together than fp32's error, at the border between kept and dropped groups or
// anywhere among the first K + 1, is decided again in 64 bits, a lane for each
// score in question (exact_groups, exact_among); rows that those cannot take
// (more than 32 scores in question, groups or rows with too few experts left) by
// the whole row in 64 bits (select_exact).  Of normal logits at E = 256 in 8 groups
// K = 8 two rows in a thousand need it.  The whole row takes a warp 7 us of the slow
// 64-bit pipe, which at first was half of the launch, its tail (16384 rows 38 us,
// now 21; softmax, whose sum takes the row's exponentials in 64 bits, 38 and 26).
// Rows of one logit, as padding gives them, need neither: with one bias (or none) they
// are in the order of the index (16384 of them 23 us, by the whole row 413), and where
// balancing has moved the biases, in multiples of its step, so that many scores tie,
// in the order of the biases (select_by_bias: 55 us; before, one step of 1e-3 from
// zeros took 424, a hundred steps 45 with sigmoid scores and 187 with softmax).
// Where no score is needed (no bias, and no sum of two) the logits themselves are
// compared and their keys hold the whole index, as in the plain router.
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
  double even;                          // 1 / E: the softmax score in a row of one logit
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

// Error of c in fp32 for sigmoid, and of a difference of two: z = -l log2(e) is
// off by 1.5 |z| 2^-24 and its exponential by 2^-22, of which s (1 - s) <= 1/4
// (times |l|: 0.224) reaches s; 1 + e^-l rounds, the reciprocal is off by 2^-23:
// together under 2^-21.9.  For softmax 2^-22 and the sum's rounding, 37 additions
// at most: under p 2^-18.
__device__ __forceinline__ float margin_of(float x, float y, float eps) {
  return eps + 0x1p-23f * (fabsf(x) + fabsf(y));  // (the sums with the biases round)
}
constexpr float kSigmoidEps = 0x1p-20f;

__device__ __forceinline__ float sigmoid_fast(float l) {
  float s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(l * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + s));
  return s;
}

__device__ __forceinline__ double sigmoid_exact(double l) {
  const double e = exp(-fabs(l));
  return (l < 0.0 ? e : 1.0) / (1.0 + e);
}

// Unsigned keys in the order of the doubles (compared as integers: the 64-bit
// float pipe is slow).
__device__ __forceinline__ unsigned long long key64(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return (unsigned long long)(b < 0 ? ~b : b ^ (long long)0x8000000000000000ull);
}
__device__ __forceinline__ double value64(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

// How a row's scores come from its logits: in fp32, and in 64 bits.
struct Scores {
  bool soft;
  float m, inv, eps;  // softmax: the largest logit, 1 / the sum; the error (margin_of)
  __device__ __forceinline__ float fast(float l) const { return soft ? exp_flush(l - m) * inv : sigmoid_fast(l); }
  __device__ __forceinline__ double exact(double l, double sum) const {
    return soft ? exp(l - m) / sum : sigmoid_exact(l);
  }
};

// The sum of e^(l - m) over the row, in every lane.
template <int NPL, typename T>
__device__ __forceinline__ double exact_sum(const T* row, const GroupParams& p, float m, int lane) {
  const int g = lane >> p.lg, r = lane & ((1 << p.lg) - 1);
  bool flag = false;
  double s = 0.0;
#pragma unroll 1
  for (int i = 0; i < NPL; ++i) {
    const int o = place<T, false>(i, r, p.lg);
    if (g < p.G && o < p.size) s += exp((double)clean_logit(to_f32(row[g * p.size + o]), flag) - m);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kAll, s, d);
  return s;
}

// Whether all of the row's experts have one logit (padding rows of zeros), which
// leaves the order to the biases; and one bias, which leaves it to the index.
enum Row { kNotKnown, kDiffers, kOneLogit, kAllTheSame };
template <typename T>
__device__ __noinline__ Row row_of(const T* row, const GroupParams& p, int lane) {
  const float l = to_f32(row[0]), b = p.bias ? p.bias[0] : 0.f;
  bool one = l > -INFINITY, same = b > -INFINITY && b < INFINITY;
  for (int j = lane; one && j < p.E; j += 32) {
    one = to_f32(row[j]) == l;
    same = same && (!p.bias || p.bias[j] == b);
  }
  if (!__all_sync(kAll, one)) return kDiffers;
  return __all_sync(kAll, same) ? kAllTheSame : kOneLogit;
}

// Whether the group of this lane is kept, by the exact sums of its
// `each` largest; fail where it is not those that fp32 names without doubt.
// list: 32 words of the warp's own.
template <int NPL, typename T>
__device__ __noinline__ bool exact_groups(const T* row, const GroupParams& p, const Scores& f, int lane, int* list, bool& fail) {
  const int g = lane >> p.lg, r = lane & ((1 << p.lg) - 1);
  float c[NPL], a1 = -INFINITY, a2 = -INFINITY;
  bool flag = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int o = place<T, false>(i, r, p.lg), j = g * p.size + o;
    const bool in = g < p.G && o < p.size;
    const float l = in ? clean_logit(to_f32(row[j]), flag) : -INFINITY;
    const float b = in && p.bias ? clean_bias(p.bias[j], flag) : 0.f;
    c[i] = l > -INFINITY ? f.fast(l) + b : -INFINITY;
    a2 = fmaxf(a2, fminf(a1, c[i]));
    a1 = fmaxf(a1, c[i]);
  }
  for (int d = 1; d < 1 << p.lg; d <<= 1) {
    const float b1 = __shfl_xor_sync(kAll, a1, d), b2 = __shfl_xor_sync(kAll, a2, d);
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
  }
  const float last = p.each > 1 ? a2 : a1, cut = last - margin_of(last, last, f.eps);
  const unsigned mine = (p.lg == 5 ? kAll : (1u << (1 << p.lg)) - 1u) << (g << p.lg);  // the group's lanes
  int n = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const bool on = c[i] > -INFINITY && c[i] >= cut;
    const unsigned m = __ballot_sync(kAll, on) & mine;
    const int at = n + __popc(m & lanemask_lt());
    if (on && at < p.each) list[g * p.each + at] = g * p.size + place<T, false>(i, r, p.lg);
    n += __popc(m);
  }
  fail = !__all_sync(kAll, g >= p.G || n == p.each);
  if (fail) return false;
  __syncwarp();
  const double sum = f.soft ? exact_sum<NPL>(row, p, f.m, lane) : 0.0;
  double v = 0.0;
  if (lane < p.G * p.each) {
    const int j = list[lane];
    v = f.exact(clean_logit(to_f32(row[j]), flag), sum) + (p.bias ? (double)p.bias[j] : 0.0);
  }
  if (p.each > 1) v += __shfl_xor_sync(kAll, v, 1);
  const unsigned long long key = __shfl_sync(kAll, key64(v), (g * p.each) & 31);
  int rank = 0;
  for (int h = 0; h < p.G; ++h) {
    const unsigned long long other = __shfl_sync(kAll, key, h << p.lg);
    rank += other > key || (other == key && h < g);
  }
  __syncwarp();
  return g < p.G && rank < p.top;
}

// The selection among the scores (by_logit: logits) of kept groups that are at
// least cut; lane k < K gets the k-th id.  fail: more than 32 of them.
template <int NPL, typename T>
__device__ __noinline__ int exact_among(const T* row, const GroupParams& p, const Scores& f, bool by_logit, bool keep,
                                        float cut, int lane, int* list, bool& fail) {
  const int g = lane >> p.lg, r = lane & ((1 << p.lg) - 1);
  bool flag = false;
  int n = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int o = place<T, false>(i, r, p.lg), j = g * p.size + o;
    const bool in = keep && o < p.size;
    float c = in ? clean_logit(to_f32(row[j]), flag) : -INFINITY;
    if (!by_logit && c > -INFINITY) c = f.fast(c) + (p.bias ? clean_bias(p.bias[j], flag) : 0.f);
    const bool on = c > -INFINITY && c >= cut;
    const unsigned m = __ballot_sync(kAll, on);
    const int at = n + __popc(m & lanemask_lt());
    if (on && at < 32) list[at] = j;
    n += __popc(m);
  }
  fail = n > 32 || n < p.K;
  if (fail) return 0;
  __syncwarp();
  const double sum = f.soft && !by_logit ? exact_sum<NPL>(row, p, f.m, lane) : 0.0;
  int id = 0;
  unsigned long long key = 0;
  if (lane < n) {
    id = list[lane];
    const double l = clean_logit(to_f32(row[id]), flag);
    key = key64(by_logit ? l : f.exact(l, sum) + (p.bias ? (double)p.bias[id] : 0.0));
  }
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const unsigned long long other = __shfl_sync(kAll, key, i);
    const int oid = __shfl_sync(kAll, id, i);
    rank += other > key || (other == key && oid < id);
  }
  if (lane < n && rank < p.K) list[rank] = id;
  __syncwarp();
  return lane < p.K ? list[lane] : 0;
}

// The score of every expert in a row of one logit.  (The 64-bit pipe is slow, and
// padding's logits are zeros.)
__device__ __forceinline__ double score_of_all(float l, const GroupParams& p) {
  return p.scoring == MOE_SCORE_SOFTMAX ? p.even : l == 0.f ? 0.5 : sigmoid_exact(l);
}

// The selection in a row of one logit with the score s; lane k < K gets the k-th
// id.  s + b is in the order of b, and no two biases share a sum, where all are
// multiples of 2^-50 (all from 2^-27 up are): two of them are 2^-50 apart then, at
// least, and a sum under 2 rounds by 2^-53 (larger biases are further apart).  fail:
// one is not, or the kept groups have fewer than K experts left.
template <int NPL>
__device__ __noinline__ int select_by_bias(const GroupParams& p, double s, int lane, bool& fail) {
  const int g = lane >> p.lg, r = lane & ((1 << p.lg) - 1);
  uint32_t key[NPL], a1 = 0u, a2 = 0u;  // 0: out
  bool small = false, flag = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int o = place<float, false>(i, r, p.lg);
    const float b = g < p.G && o < p.size ? clean_bias(p.bias[g * p.size + o], flag) + 0.f : -INFINITY;
    small |= fabsf(b) < 0x1p-27f && b * 0x1p50f != rintf(b * 0x1p50f);
    key[i] = b > -INFINITY ? key_of(b) : 0u;
    a2 = max(a2, min(a1, key[i]));
    a1 = max(a1, key[i]);
  }
  bool keep = g < p.G;
  if (p.top < p.G) {
    for (int d = 1; d < 1 << p.lg; d <<= 1) {
      const uint32_t b1 = __shfl_xor_sync(kAll, a1, d), b2 = __shfl_xor_sync(kAll, a2, d);
      a2 = max(min(a1, b1), max(a2, b2));
      a1 = max(a1, b1);
    }
    const int live = (a1 != 0u) + (p.each > 1 && a2 != 0u);
    unsigned long long v = a1;
    if (p.each > 1) {
      const unsigned long long sum = key64((s + value_of(a1)) + (s + value_of(a2)));
      if (live > 1) v = sum;
    }
    int rank = 0;
    for (int h = 0; h < p.G; ++h) {
      const unsigned long long vh = __shfl_sync(kAll, v, h << p.lg);
      const int lh = __shfl_sync(kAll, live, h << p.lg);
      rank += lh > live || (lh == live && (vh > v || (vh == v && h < g)));
    }
    keep = keep && rank < p.top;
  }
  int left = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if (!keep) key[i] = 0u;
    left += key[i] != 0u;
  }
  fail = __any_sync(kAll, small) || (int)__reduce_add_sync(kAll, (unsigned)left) < p.K;
  if (fail) return 0;
  int sel_id = 0;
  for (int k = 0; k < p.K; ++k) {
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < NPL; ++i) top = max(top, key[i]);
    const uint32_t best = __reduce_max_sync(kAll, top);
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = NPL - 1; i >= 0; --i)
      if (key[i] == best) at = g * p.size + place<float, false>(i, r, p.lg);
    const uint32_t id = __reduce_min_sync(kAll, at);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (at == id && id == (uint32_t)(g * p.size + place<float, false>(i, r, p.lg))) key[i] = 0u;
    if (lane == k) sel_id = (int)id;
  }
  return sel_id;
}

// The selection in 64 bits; lane k < K gets the k-th id.  by_logit: c is the
// logit; one_logit: all of them are the same, one score to compute.  Groups with
// fewer experts above -inf (of `each`) come last; when the kept groups have fewer
// than K of those, their others follow in order.
template <int NPL, typename T>
__device__ __noinline__ int select_exact(const T* row, const GroupParams& p, bool by_logit, bool one_logit, int lane) {
  const int g = lane >> p.lg, r = lane & ((1 << p.lg) - 1);
  const bool soft = p.scoring == MOE_SCORE_SOFTMAX;
  double c[NPL];
  bool flag = false;
  if (one_logit && !by_logit) {
    const double s = score_of_all(clean_logit(to_f32(row[0]), flag), p);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int o = place<T, false>(i, r, p.lg);
      c[i] = g < p.G && o < p.size ? s + (p.bias ? clean_bias(p.bias[g * p.size + o], flag) : 0.f) : -INFINITY;
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int o = place<T, false>(i, r, p.lg);
      const float l = g < p.G && o < p.size ? clean_logit(to_f32(row[g * p.size + o]), flag) : -INFINITY;
      c[i] = l;
      m = fmaxf(m, l);
    }
    if (!by_logit) {
      double sum = 0.0;
      if (soft) {
        m = fmaxf(value_of(__reduce_max_sync(kAll, key_of(m))), -3.402823466e+38f);
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += c[i] = exp(c[i] - m);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int o = place<T, false>(i, r, p.lg);
        const bool in = g < p.G && o < p.size;
        const float l = in ? clean_logit(to_f32(row[g * p.size + o]), flag) : -INFINITY;
        const float b = in && p.bias ? clean_bias(p.bias[g * p.size + o], flag) : 0.f;
        const double s = soft ? c[i] / sum : sigmoid_exact(c[i]);
        c[i] = l > -INFINITY ? s + b : -INFINITY;
      }
    }
  }
  // keys, 0 for -inf, and the two largest of the group
  unsigned long long key[NPL], a1 = 0, a2 = 0;
  unsigned long long open = 0;  // elements that may be chosen yet
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if (g < p.G && place<T, false>(i, r, p.lg) < p.size) open |= 1ull << i;
    key[i] = __double_as_longlong(c[i]) == (long long)0xfff0000000000000ull ? 0ull : key64(c[i]);
    a2 = max(a2, min(a1, key[i]));
    a1 = max(a1, key[i]);
  }
  for (int d = 1; d < 1 << p.lg; d <<= 1) {
    const unsigned long long b1 = __shfl_xor_sync(kAll, a1, d), b2 = __shfl_xor_sync(kAll, a2, d);
    a2 = max(min(a1, b1), max(a2, b2));
    a1 = max(a1, b1);
  }
  const int live = (a1 != 0) + (p.each > 1 && a2 != 0);
  const unsigned long long v = live > 1 ? key64(value64(a1) + value64(a2)) : a1;
  int rank = 0;
  for (int h = 0; h < p.G; ++h) {
    const unsigned long long vh = __shfl_sync(kAll, v, h << p.lg);
    const int lh = __shfl_sync(kAll, live, h << p.lg);
    rank += lh > live || (lh == live && (vh > v || (vh == v && h < g)));
  }
  if (rank >= p.top) open = 0;
  int sel_id = 0;
  for (int k = 0; k < p.K; ++k) {
    unsigned long long best = 0;
    uint32_t at = 0x7fffffffu;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {  // (in ascending order of the index)
      if (((open >> i) & 1) && (at == 0x7fffffffu || key[i] > best)) {
        best = key[i];
        at = g * p.size + place<T, false>(i, r, p.lg);
      }
    }
    // the largest of the upper halves, of the lower ones among those, the lowest index
    const uint32_t upper = __reduce_max_sync(kAll, (uint32_t)(best >> 32));
    const bool first = (uint32_t)(best >> 32) == upper;
    const uint32_t lower = __reduce_max_sync(kAll, first ? (uint32_t)best : 0u);
    const uint32_t id = __reduce_min_sync(kAll, first && (uint32_t)best == lower ? at : 0x7fffffffu);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (at == id && (uint32_t)(g * p.size + place<T, false>(i, r, p.lg)) == id) open &= ~(1ull << i);
    if (lane == k) sel_id = (int)id;
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
  const float inv = 1.f / row_sum;
  const Scores f{soft, m, inv, soft ? 0x1p-20f + inv * 0x1p-17f : kSigmoidEps};
  if constexpr (!kByLogit) {
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
      c[i] = c[i] > -INFINITY ? f.fast(c[i]) + b[i] : -INFINITY;
    }
  }
  if (flag) set_status(status, MOE_ERR_INVALID_ARG);
  bool again = false, keep = g < p.G;  // again: by the whole row
  Row kind = kNotKnown;
  __shared__ int lists[kWarps][32];
  int* list = lists[threadIdx.x >> 5];
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
    // (a sum past fp32's range is still a sum, and more than none)
    constexpr float kMost = 3.402823466e+38f;
    float v = a1;
    if (p.each > 1) v = a2 > -INFINITY ? fminf(fmaxf(a1 + a2, -kMost), kMost) : -INFINITY;
    int rank = 0;
    for (int h = 0; h < p.G; ++h) {
      const float vh = __shfl_sync(kAll, v, h << p.lg);
      rank += vh > v || (vh == v && h < g);
    }
    keep = keep && rank < p.top;
    if constexpr (!kByLogit) {  // the border between kept and dropped groups
      // A sum's error is that of its scores, the half steps of both with their
      // biases (which may cancel in the sum) and its own: 3 2^-24 of the two.
      const float err = f.eps + 0x1p-22f * fabsf(a1) + (p.each > 1 ? 0x1p-22f * fabsf(a2) : 0.f);
      const float lo = value_of(__reduce_min_sync(kAll, keep ? key_of(v - err) : 0xffffffffu));
      const float hi = value_of(__reduce_max_sync(kAll, !keep && v > -INFINITY && g < p.G ? key_of(v + err) : 0u));
      // (dropped groups without experts are no question, nor are kept ones)
      if (hi > -INFINITY && lo > -INFINITY && lo <= hi) {
        kind = row_of(row, p, lane);
        bool fail = kind != kDiffers || __any_sync(kAll, again) || p.G * p.each > 32;
        if (!fail) keep = exact_groups<NPL>(row, p, f, lane, list, fail);
        again |= fail;
      }
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
  float sel = lane <= p.K && mine != 0u ? to_f32(row[sel_id]) : -INFINITY;
  sel = fminf(sel, 3.402823466e+38f) + 0.f;
  again |= (more && pk[0] == 0u) || (lane < p.K && mine == 0u);
  // Two neighbours of the first K + 1 that are too close.  Below the last of the K
  // may be any score with the upper bits of the next key.
  const uint32_t next = __shfl_down_sync(kAll, mine, 1);
  const bool pair = lane < p.K && next != 0u, edge = lane == p.K - 1;
  bool close = false;
  if constexpr (!kByLogit) {
    const float bias = p.bias && lane <= p.K && mine != 0u ? p.bias[sel_id] : 0.f;
    const float own = f.fast(sel) + bias;
    float below = __shfl_down_sync(kAll, own, 1);
    if (edge) below = value_of(next | kLow);
    close = pair && own - below <= margin_of(own, below, f.eps);
  } else if constexpr (sizeof(T) == 4) {
    const float below = __shfl_down_sync(kAll, sel, 1);
    close = pair && ((mine ^ next) & ~kLow) == 0u && (sel != below || edge);
  }
  if (__any_sync(kAll, again || close)) {
    bool whole = __any_sync(kAll, again);
    if (kind == kNotKnown) kind = row_of(row, p, lane);
    if (kind == kAllTheSame) {
      sel_id = lane;
      whole = false;
    } else if (kind == kOneLogit) {
      sel_id = select_by_bias<NPL>(p, score_of_all(clean_logit(to_f32(row[0]), flag), p), lane, whole);
    } else if (!whole) {
      // none of the K is below this, and none of the exact K below it less the margin
      const float low = value_of(__shfl_sync(kAll, mine, p.K - 1) & ~kLow);
      const float cut = kByLogit ? low : low - margin_of(low, low, f.eps);
      sel_id = exact_among<NPL>(row, p, f, kByLogit, keep, cut, lane, list, whole);
    }
    if (whole) sel_id = select_exact<NPL>(row, p, kByLogit, kind == kOneLogit, lane);
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
  GroupParams p{bias, T, E, K, num_groups, E / num_groups, top_groups, group_top, 5, scoring, renormalize, scale,
                1.0 / E};
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
