// Rows in 8-bit integers with a scale each, written to one row or, with a
// row map, to the K expert-major rows of the token (each token is read and
// rounded once).
//
// Bound by memory: TPR threads (32 to 256) hold a row in registers, 16
// elements a chunk, find its largest magnitude (the bits of |x| order like
// |x|, and a NaN's are the largest of all, so an integer maximum finds both)
// and round it without reading it again.
//
// q = rint(127 x / top), the division rounded to fp32.  For bf16 rows the
// rounding decision is that of exact arithmetic (127 x / top is a quotient of
// a 15-bit and an 8-bit integer: a tie exactly, or further from one than the
// division's error), so x * (127 / top) decides all but the elements within
// 2^-15 of a tie, and for those the exact residual 127 x - q top (one fma)
// does.  fp32 rows divide: their quotients can lie closer to a tie.
#include <math.h>

#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Chunk {  // 16 elements as loaded
  static constexpr int n = 16 / VecTraits<T>::kElems;
  uint4 v[n];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = ld_nc_v4(p + i * VecTraits<T>::kElems);
  }
  __device__ __forceinline__ void get(float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < n; ++i) VecTraits<T>::unpack(v[i], f + i * VecTraits<T>::kElems);
  }
};

// Round to nearest even by the addition of 1.5 * 2^23: the low byte of the
// sum's bits is the integer's low byte.
constexpr float kMagic = 12582912.f;

struct Rounding {
  float mul, div, k;  // q = rint(x * mul / div), k = mul / div
};

// 16 elements in 8 bits.
template <typename T>
__device__ __forceinline__ uint4 round16(const Chunk<T>& c, const Rounding& r) {
  float f[16];
  c.get(f);
  uint32_t b[16];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] = __float_as_uint(__fdiv_rn(f[i] * r.mul, r.div) + kMagic);
  } else {
    // x k is within 128 * 2^-23 < 2^-15 of the quotient: only nearer to a tie
    // than that can its rounding differ
    bool near = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = f[i] * r.k, z = y + kMagic;
      near |= fabsf(y - (z - kMagic)) > 0.5f - 0x1p-15f;
      b[i] = __float_as_uint(z);
    }
    if (near) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float q = __uint_as_float(b[i]) - kMagic, e = fmaf(-q, r.div, f[i] * r.mul);  // exact
        const float two = 2.f * fabsf(e);
        if (two > r.div || (two == r.div && (b[i] & 1u))) b[i] += e > 0.f ? 1u : 0xffffffffu;
      }
    }
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                       __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// TPR threads per row, NV chunks each in registers; NV = 0: rows of any
// length, read twice.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(kThreads)
quantize_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ row_map, int n_tok,
                     int H, int K, int N, int8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t part[kThreads / 32];
  const int t = blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  const int i = threadIdx.x % TPR, lane = threadIdx.x & 31;
  const bool live = t < n_tok;
  const T* row = x + (size_t)t * H;
  // largest magnitude: of fp32 the bits' maximum; of bf16 two at a time (the
  // maximum that keeps a NaN)
  uint32_t top = 0;
  auto widen = [&](const Chunk<T>& c) {
#pragma unroll
    for (int j = 0; j < Chunk<T>::n; ++j) {
      const uint32_t w[4] = {c.v[j].x, c.v[j].y, c.v[j].z, c.v[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 4) {
          top = max(top, w[q] & 0x7fffffffu);
        } else {
          const uint32_t a = w[q] & 0x7fff7fffu;
          const __nv_bfloat162 h = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                               *reinterpret_cast<const __nv_bfloat162*>(&top));
          top = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
    }
  };
  Chunk<T> c[NV > 0 ? NV : 1];
  if constexpr (NV > 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int h = (v * TPR + i) * 16;
      if (live && h < H) c[v].load(row + h);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (live && (v * TPR + i) * 16 < H) widen(c[v]);
  } else {
    for (int h = i * 16; live && h < H; h += TPR * 16) {
      c[0].load(row + h);
      widen(c[0]);
    }
  }
  // rows that the K slots of this token go to: lane k holds the k-th
  int dest = -1;
  if (live && lane < K) {
    dest = row_map != nullptr ? row_map[(size_t)t * K + lane] : t;
    if (dest >= N) dest = -1;
  }
  if constexpr (sizeof(T) == 2) top = max(top & 0xffff0000u, top << 16);  // as fp32
  top = __reduce_max_sync(0xffffffffu, top);
  if constexpr (TPR > 32) {
    if (lane == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) top = max(top, part[threadIdx.x / TPR * (TPR / 32) + w]);
  }
  const bool finite = top < 0x7f800000u;
  const float m = __uint_as_float(top);
  const bool zero = !finite || top == 0u;
  // 127 x would pass the range of fp32 from 2^121 on, and 127 / top below
  // 2^-119: such rows are scaled by a power of two, which changes no quotient
  const float by = m >= 0x1p119f ? 0x1p-10f : m < 0x1p-100f ? 0x1p60f : 1.f;
  Rounding r;
  r.mul = zero ? 0.f : 127.f * by;
  r.div = zero ? 1.f : m * by;
  r.k = r.mul / r.div;
  if (i < K && live && dest >= 0) scale[dest] = finite ? m / 127.f : __int_as_float(0x7fffffff);
  auto put = [&](const Chunk<T>& ch, int h) {
    const uint4 w = zero ? make_uint4(0u, 0u, 0u, 0u) : round16(ch, r);
    for (int k = 0; k < K; ++k) {
      const int d = __shfl_sync(0xffffffffu, dest, k);
      if (d >= 0 && h < H) st_v4(q + (size_t)d * H + h, w);
    }
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) put(c[v], (v * TPR + i) * 16);
  } else {
    for (int h0 = 0; h0 < H; h0 += TPR * 16) {
      const int h = h0 + i * 16;
      if (live && h < H) c[0].load(row + h);
      put(c[0], h);
    }
  }
}

template <typename T>
void launch_quantize(const T* x, const int32_t* row_map, int n_tok, int H, int K, int N, int8_t* q,
                     float* scale, cudaStream_t s) {
  auto go = [&](auto tpr, auto nv) {
    constexpr int R = kThreads / decltype(tpr)::value;
    quantize_rows_kernel<T, decltype(tpr)::value, decltype(nv)::value>
        <<<(n_tok + R - 1) / R, kThreads, 0, s>>>(x, row_map, n_tok, H, K, N, q, scale);
  };
  using std::integral_constant;
  // at most four chunks (32 or 64 registers) a thread
  if (H <= 512) go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (H <= 1024) go(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  else if (H <= 2048) go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  else if (H <= 4096) go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (H <= 8192) go(integral_constant<int, 128>{}, integral_constant<int, 4>{});
  else if (H <= 16384) go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else go(integral_constant<int, 256>{}, integral_constant<int, 0>{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_quantize_rows(const void* x, int dtype, const int32_t* row_map, int T, int H,
                                 int K, int N, int8_t* q, float* scale, cudaStream_t stream) {
  if (T < 0 || H <= 0 || K <= 0 || N < 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (H % 16 || K > kMaxK || (long long)T * K > 0x7fffffffLL) return MOE_ERR_SHAPE;
  if (row_map == nullptr && (K != 1 || N < T)) return MOE_ERR_SHAPE;
  if (T == 0 || N == 0) return MOE_OK;
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_F32)
    launch_quantize(static_cast<const float*>(x), row_map, T, H, K, N, q, scale, stream);
  else
    launch_quantize(static_cast<const __nv_bfloat16*>(x), row_map, T, H, K, N, q, scale, stream);
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}
