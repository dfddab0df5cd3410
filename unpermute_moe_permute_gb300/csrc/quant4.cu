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

#include <type_traits>

#include "common.cuh"
#include "int4.cuh"

namespace moe {
namespace {

constexpr int kRows = 32, kCols = 256, kQuantThreads = 256;
constexpr int kPerWarp = kRows / (kQuantThreads / 32);

// Eight inputs as they are in memory.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) { a = ld_nc_v4(p), b = ld_nc_v4(p + 4); }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    VecTraits<float>::unpack(a, f);
    VecTraits<float>::unpack(b, f + 4);
  }
  // the bits of the largest magnitude; NaN and infinity order above every number
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fffffffu;
    return max(max(max(a.x & m, a.y & m), max(a.z & m, a.w & m)), max(max(b.x & m, b.y & m), max(b.z & m, b.w & m)));
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = ld_nc_v4(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const { VecTraits<__nv_bfloat16>::unpack(a, f); }
  __device__ __forceinline__ static uint32_t max2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = max2(max2(a.x & m, a.y & m), max2(a.z & m, a.w & m));
    return max(t << 16, t & 0xffff0000u);
  }
};

// top / 7 to five significant bits, ties to even (below 2^-126 to a multiple of
// 2^-130): a bf16 value.
__device__ __forceinline__ float scale_of(float top) {
  uint32_t b = __float_as_uint(top * (1.f / 7.f));
  b = (b + 0x3ffffu + ((b >> 19) & 1u)) & ~0x7ffffu;
  return __uint_as_float(b);
}

// 1 / s rounded to nearest for a scale of five significant bits, of which there
// are sixteen but for the power of two: the approximate reciprocal and one
// Newton step (Markstein), checked for all of them.
__device__ __forceinline__ float reciprocal_of(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(fmaf(-s, r, 1.f), r, r);
}

// Two quotients a / s and b / s as divisions round them, from the rounded
// reciprocal and one residual (Markstein), and then to the nearest integer, which
// is left in the lowest bits of 1.5 2^23 + q.
__device__ __forceinline__ void round2(float a, float b, float s, float inv, uint32_t& qa, uint32_t& qb) {
  asm("{\n\t.reg .b64 f, n, i, m, x, r;\n\tmov.b64 f, {%2, %3};\n\tmov.b64 n, {%4, %4};\n\tmov.b64 i, {%5, %5};\n\t"
      "mov.b64 m, {%6, %6};\n\tmul.rn.f32x2 x, f, i;\n\tfma.rn.f32x2 r, x, n, f;\n\tfma.rn.f32x2 x, r, i, x;\n\t"
      "add.rn.f32x2 x, x, m;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=r"(qa), "=r"(qb)
      : "f"(a), "f"(b), "f"(-s), "f"(inv), "f"(12582912.f));
}

// Eight integers, each in the lowest byte of its word, as the format's word.
__device__ __forceinline__ uint32_t pack_int4(const uint32_t (&y)[8]) {
  const uint32_t a = __byte_perm(__byte_perm(y[0], y[4], 0x0040), __byte_perm(y[1], y[5], 0x0040), 0x5410);
  const uint32_t b = __byte_perm(__byte_perm(y[2], y[6], 0x0040), __byte_perm(y[3], y[7], 0x0040), 0x5410);
  return (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
}

// Grid: column tiles, row tiles, experts.  kLanes: those of a group.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kQuantThreads)
quantize_int4_kernel(const T* __restrict__ w, int rows, int cols, uint32_t* __restrict__ q,
                     uint16_t* __restrict__ scale) {
  __shared__ uint16_t tile[32 / kLanes][kRows + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = (int)blockIdx.y * kRows, c0 = (int)blockIdx.x * kCols;
  const int groups = cols / (8 * kLanes), c = c0 + 8 * lane, row = r0 + warp * kPerWarp;
  const size_t e = blockIdx.z, at = (e * rows + row) * cols + c;
  const int n_rows = c < cols ? min(kPerWarp, rows - row) : 0;  // this lane's
  const T* src = w + at;
  uint32_t* dst = q + (at >> 3);
  Eight<T> v[kPerWarp];
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    if (i < n_rows) v[i].load(src + (size_t)i * cols);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    uint32_t top = v[i].top();  // the group's largest magnitude
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const bool bad = top >= 0x7f800000u;
    const float s = bad ? 0.f : scale_of(__uint_as_float(top));
    float f[8];
    v[i].get(f);
    uint32_t word = 0;
    if (top - 0x0d800000u < 0x65000000u) {  // 2^-100 <= top < 2^102
      const float inv = reciprocal_of(s);
      uint32_t y[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) round2(f[j], f[j + 1], s, inv, y[j], y[j + 1]);
      word = pack_int4(y);
    } else if (s > 0.f) {
      uint32_t y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(f[j], s)), -8.f), 7.f);
      word = pack_int4(y);
    }
    if (i < n_rows) dst[(size_t)i * (cols >> 3)] = word;
    if (lane % kLanes == 0)
      tile[lane / kLanes][warp * kPerWarp + i] = bad ? 0x7fc0u : (uint16_t)(__float_as_uint(s) >> 16);
  }
  __syncthreads();
  const int g0 = c0 / (8 * kLanes), n = min(32 / kLanes, groups - g0);
  for (int i = threadIdx.x; i < n * kRows; i += kQuantThreads) {
    const int gi = i / kRows, r = r0 + i % kRows;
    if (r < rows) scale[(e * groups + g0 + gi) * rows + r] = tile[gi][i % kRows];
  }
}

template <int kLanes>
__global__ void __launch_bounds__(kQuantThreads)
dequantize_int4_kernel(const uint32_t* __restrict__ q, const uint16_t* __restrict__ scale, int rows,
                       int cols, __nv_bfloat16* __restrict__ w) {
  __shared__ uint16_t tile[32 / kLanes][kRows + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = (int)blockIdx.y * kRows, c0 = (int)blockIdx.x * kCols;
  const int groups = cols / (8 * kLanes), c = c0 + 8 * lane, row = r0 + warp * kPerWarp;
  const size_t e = blockIdx.z, at = (e * rows + row) * cols + c;
  const int n_rows = c < cols ? min(kPerWarp, rows - row) : 0;  // this lane's
  const uint32_t* src = q + (at >> 3);
  __nv_bfloat16* dst = w + at;
  const uint32_t mask = int4_mask();
  uint32_t v[kPerWarp];
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) v[i] = i < n_rows ? __ldg(src + (size_t)i * (cols >> 3)) : 0u;
  const int g0 = c0 / (8 * kLanes), n = min(32 / kLanes, groups - g0);
  for (int i = threadIdx.x; i < n * kRows; i += kQuantThreads) {
    const int gi = i / kRows, r = r0 + i % kRows;
    tile[gi][i % kRows] = r < rows ? scale[(e * groups + g0 + gi) * rows + r] : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    if (i < n_rows) {
      const uint32_t s = tile[lane / kLanes][warp * kPerWarp + i] * 0x10001u;
      uint32_t x[4];
      expand_int4(v[i], s, mask, x);
      st_cs_v4(dst + (size_t)i * cols, make_uint4(x[0], x[1], x[2], x[3]));
    }
  }
}

int check_int4(const void* a, const void* b, const void* c, int E, int rows, int cols, int group) {
  if (E < 0 || rows < 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  if (cols % 64 || cols % group || cols > MOE_INT4_MAX_SIZE || rows > MOE_INT4_MAX_SIZE || E > 65535)
    return MOE_ERR_SHAPE;
  if (E == 0 || rows == 0) return MOE_OK;
  if (!a || !b || !c || !aligned16(a) || !aligned16(b) || !aligned16(c)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

dim3 int4_grid(int E, int rows, int cols) {
  return dim3((cols + kCols - 1) / kCols, (rows + kRows - 1) / kRows, E);
}

// f(lanes of a group)
template <typename F>
void by_group(int group, F&& f) {
  if (group == 32) f(std::integral_constant<int, 4>{});
  else if (group == 64) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
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
  by_group(group, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    if (dtype == MOE_F32)
      quantize_int4_kernel<float, L><<<grid, kQuantThreads, 0, stream>>>(static_cast<const float*>(W), rows, cols, q, s);
    else
      quantize_int4_kernel<__nv_bfloat16, L>
          <<<grid, kQuantThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(W), rows, cols, q, s);
  });
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}

extern "C" int moe_dequantize_weights_int4(const uint8_t* W_q, const void* scale, int E, int rows, int cols,
                                           int group, void* W, cudaStream_t stream) {
  if (int rc = check_int4(W_q, scale, W, E, rows, cols, group)) return rc;
  if (E == 0 || rows == 0) return MOE_OK;
  by_group(group, [&](auto lanes) {
    dequantize_int4_kernel<decltype(lanes)::value><<<int4_grid(E, rows, cols), kQuantThreads, 0, stream>>>(
        reinterpret_cast<const uint32_t*>(W_q), static_cast<const uint16_t*>(scale), rows, cols,
        static_cast<__nv_bfloat16*>(W));
  });
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}
