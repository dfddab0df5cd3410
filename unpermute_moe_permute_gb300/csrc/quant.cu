// Rows in 8-bit integers with a scale each, written to one row or, with a
// row map, to the K expert-major rows of the token.
//
// One block of 128 threads per row, 16 elements per thread and step: the
// row's largest magnitude (the bits of |x| order like |x| and a NaN's are the
// largest of all, so an integer maximum finds both), then the rounding.
// q = rint(127 x / top) is one exact product (127 x has 15 significant bits
// for bf16 x) and one IEEE division, so for bf16 rows the rounding decision
// is the one of exact arithmetic: 127 x / top is a quotient of a 15-bit and
// an 8-bit integer, and either a tie exactly or further from one than the
// division's rounding error.
#include <math.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&f)[16]) {
  constexpr int n = VecTraits<T>::kElems;
#pragma unroll
  for (int i = 0; i < 16 / n; ++i) VecTraits<T>::unpack(ld_v4(p + i * n), f + i * n);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
quantize_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ row_map, int n_tok,
                     int H, int K, int N, int8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t part[kThreads / 32];
  const int t = blockIdx.x;
  const T* row = x + (size_t)t * H;
  uint32_t top = 0;
  for (int c = threadIdx.x * 16; c < H; c += kThreads * 16) {
    float f[16];
    load16(row + c, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) top = max(top, part[i]);
  const bool finite = top < 0x7f800000u;
  const float m = __uint_as_float(top);
  const float s = finite ? m / 127.f : __int_as_float(0x7fffffff);
  const bool zero = !finite || top == 0u;
  // 127 x would pass the range of fp32 from 2^121 on: such rows are scaled by
  // a power of two, which changes no quotient
  const float by = m >= 0x1p119f ? 0x1p-10f : 1.f;
  const float mul = 127.f * by, div = m * by;
  for (int c = threadIdx.x * 16; c < H; c += kThreads * 16) {
    float f[16];
    load16(row + c, f);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = zero ? 0 : __float2int_rn(__fdiv_rn(f[4 * i + j] * mul, div));
        w[i] |= (uint32_t)(v & 0xff) << (8 * j);
      }
    }
    const uint4 out = make_uint4(w[0], w[1], w[2], w[3]);
    for (int k = 0; k < K; ++k) {
      const int r = row_map != nullptr ? row_map[(size_t)t * K + k] : t;
      if (r >= 0 && r < N) st_v4(q + (size_t)r * H + c, out);
    }
  }
  if (threadIdx.x < K) {
    const int r = row_map != nullptr ? row_map[(size_t)t * K + threadIdx.x] : t;
    if (r >= 0 && r < N) scale[r] = s;
  }
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
    quantize_rows_kernel<<<T, kThreads, 0, stream>>>(static_cast<const float*>(x), row_map, T, H, K,
                                                     N, q, scale);
  else
    quantize_rows_kernel<<<T, kThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(x), row_map,
                                                     T, H, K, N, q, scale);
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}
