// Weights in 4 bits with a scale for each group of inputs, and back to bf16.
//
//   scale = max |w| / 7 over the group, to five significant bits
//   q     = round(w / scale), ties to even
//
// Five bits of scale times three of q fit bf16's eight, so the weight q * scale
// that the products multiply with is exact in bf16.  max / scale stays under
// 7.25, so the largest q is 7.
//
// Both are passes over memory.  A CTA takes 32 rows x 256 inputs: a warp four of
// the rows, a lane eight inputs of each (16 or 32 bytes in, one word out, four
// rows in flight); the scales, which lie along the other axis, are turned
// through shared memory into runs of 64 bytes.
#include <math.h>

#include "common.cuh"
#include "int4.cuh"

namespace moe {
namespace {

constexpr int kRows = 32, kCols = 256, kQuantThreads = 256;
constexpr int kPerWarp = kRows / (kQuantThreads / 32);

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const uint4 a = ld_nc_v4(p), b = ld_nc_v4(p + 4);
  VecTraits<float>::unpack(a, f);
  VecTraits<float>::unpack(b, f + 4);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  VecTraits<__nv_bfloat16>::unpack(ld_nc_v4(p), f);
}

// top / 7 to five significant bits, ties to even (below 2^-126 to a multiple of
// 2^-130): a bf16 value.
__device__ __forceinline__ float scale_of(float top) {
  uint32_t b = __float_as_uint(top * (1.f / 7.f));
  b = (b + 0x3ffffu + ((b >> 19) & 1u)) & ~0x7ffffu;
  return __uint_as_float(b);
}

// Grid: column tiles x row tiles, experts.  L: log2 of the lanes of a group.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
quantize_int4_kernel(const T* __restrict__ w, int rows, int cols, int lanes, uint32_t* __restrict__ q,
                     uint16_t* __restrict__ scale) {
  __shared__ uint16_t tile[kCols / 32][kRows + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (cols + kCols - 1) / kCols;
  const int r0 = (int)(blockIdx.x / tiles) * kRows, c0 = (int)(blockIdx.x % tiles) * kCols;
  const int groups = cols / (8 * lanes), c = c0 + 8 * lane;
  const size_t e = blockIdx.y;
  float f[kPerWarp][8];
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    const int r = r0 + warp * kPerWarp + i;
    if (r < rows && c < cols) {
      load8(w + (e * rows + r) * cols + c, f[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    const int r = r0 + warp * kPerWarp + i;
    // the group's largest magnitude; NaN and infinity order above every float
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[i][j]) & 0x7fffffffu);
    for (int d = 1; d < lanes; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const bool bad = top >= 0x7f800000u;
    const float s = bad ? 0.f : scale_of(__uint_as_float(top));
    uint32_t word = 0;
    if (top - 0x0d800000u < 0x65000000u) {  // 2^-100 <= top < 2^102
      // w / s rounded as a division rounds it, from the reciprocal rounded to
      // nearest and one residual (Markstein), then to the nearest integer in the
      // lowest bits of 1.5 2^23 + q.
      const float inv = __frcp_rn(s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = f[i][j] * inv;
        const float y = __fadd_rn(fmaf(fmaf(-x, s, f[i][j]), inv, x), 12582912.f);
        word |= (__float_as_uint(y) & 15u) << (4 * (j >> 1) + 16 * (j & 1));
      }
    } else if (s > 0.f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = fminf(fmaxf(rintf(__fdiv_rn(f[i][j], s)), -8.f), 7.f);
        word |= ((uint32_t)(int)x & 15u) << (4 * (j >> 1) + 16 * (j & 1));
      }
    }
    if (r < rows && c < cols) q[((e * rows + r) * cols + c) >> 3] = word;
    if ((lane & (lanes - 1)) == 0)
      tile[lane / lanes][warp * kPerWarp + i] = bad ? 0x7fc0u : (uint16_t)(__float_as_uint(s) >> 16);
  }
  __syncthreads();
  const int g0 = c0 / (8 * lanes), n = min(32 / lanes, groups - g0);
  for (int i = threadIdx.x; i < n * kRows; i += kQuantThreads) {
    const int gi = i / kRows, r = r0 + i % kRows;
    if (r < rows) scale[(e * groups + g0 + gi) * rows + r] = tile[gi][i % kRows];
  }
}

__global__ void __launch_bounds__(kQuantThreads)
dequantize_int4_kernel(const uint32_t* __restrict__ q, const uint16_t* __restrict__ scale, int rows,
                       int cols, int lanes, __nv_bfloat16* __restrict__ w) {
  __shared__ uint16_t tile[kCols / 32][kRows + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (cols + kCols - 1) / kCols;
  const int r0 = (int)(blockIdx.x / tiles) * kRows, c0 = (int)(blockIdx.x % tiles) * kCols;
  const int groups = cols / (8 * lanes), c = c0 + 8 * lane;
  const size_t e = blockIdx.y;
  const int g0 = c0 / (8 * lanes), n = min(32 / lanes, groups - g0);
  const uint32_t mask = int4_mask();
  uint32_t v[kPerWarp];
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    const int r = r0 + warp * kPerWarp + i;
    v[i] = r < rows && c < cols ? __ldg(q + (((e * rows + r) * cols + c) >> 3)) : 0u;
  }
  for (int i = threadIdx.x; i < n * kRows; i += kQuantThreads) {
    const int gi = i / kRows, r = r0 + i % kRows;
    tile[gi][i % kRows] = r < rows ? scale[(e * groups + g0 + gi) * rows + r] : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    const int r = r0 + warp * kPerWarp + i;
    if (r < rows && c < cols) {
      const uint32_t s = tile[lane / lanes][warp * kPerWarp + i] * 0x10001u;
      uint32_t x[4];
      expand_int4(v[i], s, mask, x);
      st_cs_v4(w + (e * rows + r) * cols + c, make_uint4(x[0], x[1], x[2], x[3]));
    }
  }
}

int check_int4(const void* a, const void* b, const void* c, int E, int rows, int cols, int group) {
  if (E < 0 || rows < 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  if (cols % 64 || cols % group || cols > MOE_INT4_MAX_SIZE || rows > MOE_INT4_MAX_SIZE || E > 65535)
    return MOE_ERR_SHAPE;
  const long long blocks = (long long)((rows + kRows - 1) / kRows) * ((cols + kCols - 1) / kCols);
  if (blocks > 0x7fffffffLL) return MOE_ERR_SHAPE;
  if (E == 0 || rows == 0) return MOE_OK;
  if (!a || !b || !c || !aligned16(a) || !aligned16(b) || !aligned16(c)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

dim3 int4_grid(int E, int rows, int cols) {
  return dim3(((rows + kRows - 1) / kRows) * ((cols + kCols - 1) / kCols), E);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_quantize_weights_int4(const void* W, int dtype, int E, int rows, int cols, int group,
                                         uint8_t* W_q, void* scale, cudaStream_t stream) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (int rc = check_int4(W, W_q, scale, E, rows, cols, group)) return rc;
  if (E == 0 || rows == 0) return MOE_OK;
  uint32_t* q = reinterpret_cast<uint32_t*>(W_q);
  uint16_t* s = static_cast<uint16_t*>(scale);
  const dim3 grid = int4_grid(E, rows, cols);
  if (dtype == MOE_F32)
    quantize_int4_kernel<<<grid, kQuantThreads, 0, stream>>>(static_cast<const float*>(W), rows, cols, group / 8, q, s);
  else
    quantize_int4_kernel<<<grid, kQuantThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(W), rows, cols,
                                                             group / 8, q, s);
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}

extern "C" int moe_dequantize_weights_int4(const uint8_t* W_q, const void* scale, int E, int rows, int cols,
                                           int group, void* W, cudaStream_t stream) {
  if (int rc = check_int4(W_q, scale, W, E, rows, cols, group)) return rc;
  if (E == 0 || rows == 0) return MOE_OK;
  dequantize_int4_kernel<<<int4_grid(E, rows, cols), kQuantThreads, 0, stream>>>(
      reinterpret_cast<const uint32_t*>(W_q), static_cast<const uint16_t*>(scale), rows, cols, group / 8,
      static_cast<__nv_bfloat16*>(W));
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}
