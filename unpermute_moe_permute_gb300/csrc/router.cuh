// What the two routers share: logits as the definition takes them, ordered
// keys, sorting networks, the weights of the selected, launches.
#pragma once

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

template <typename F, typename... A>
inline void launch_pdl(F* kernel, int grid, cudaStream_t stream, A... args) {
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

}  // namespace
}  // namespace moe
