// Rows in 8-bit integers with a scale each, written to one row or, with a
// row map, to the K expert-major rows of the token (each token is read and
// rounded once).
//
// Memory bounds it if the instructions are few: TPR threads (32 to 256) hold a
// row in registers, 8 elements a chunk, find its largest magnitude (a NaN
// stays one) and round it without reading it again.  32768 x 768 18 us (75 MB:
// 11 us at the copy rate), 8192 x 4096 20.6 us (100 MB: 15), 4096 x 2048 to 8
// rows each 19.4 us (84 MB: 12, the stores).  Deciding near ties by a second
// product and a division took 24.6 us at 8192 x 4096: x = top / 2 is a tie and
// so common a value that a third of the warps' chunks divided.
//
// q = rint(127 x / top), the division rounded to fp32.
//
// bf16: a quotient 127 x / top = 127 m / (M 2^j), m and M of 8 bits, is a tie or
// at least 2^-16 of itself away from one.  So with k above 127 / top by 2^-20 of
// itself at most, x k rounds as the quotient does, and a tie upwards.
// The ties are 127 / 2 (x = top / 2, a common value: to 64, upwards), and any
// n + 1/2 when 127 divides M, M = 254: there k is a power of two and exact.
//
// fp32: x k (1 + 2^-20) and x k (1 - 2^-20) enclose the quotient whatever the
// roundings of k (2^-22), 127 x and the division (2^-24 each); the chunks where
// they round to different integers (one in 60 of a warp) divide.
#include <math.h>

#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Chunk {  // 8 elements as loaded
  static constexpr int n = 8 / VecTraits<T>::kElems;
  uint4 v[n];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = ld_nc_v4(p + i * VecTraits<T>::kElems);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < n; ++i) VecTraits<T>::unpack(v[i], f + i * VecTraits<T>::kElems);
  }
};

// Round to nearest even by the addition of 1.5 * 2^23: the low byte of the
// sum's bits is the integer's low byte.
constexpr float kMagic = 12582912.f;

// Two fused multiply-adds at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// The larger magnitudes of two pairs of bf16, a NaN if one is; the signs are of no meaning.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

struct Rounding {
  float mul, div;      // q = rint(x * mul / div)
  float above, below;  // mul / div, a little more and a little less
  bool divide;         // that is out of range: every element is divided
};

// Low bytes of 8 words.
__device__ __forceinline__ uint2 low_bytes(const uint32_t (&b)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                       __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
  return make_uint2(w[0], w[1]);
}

template <typename T>
__device__ __noinline__ uint2 round8_divide(Chunk<T> c, float mul, float div) {
  float f[8];
  c.get(f);
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(__fdiv_rn(f[i] * mul, div) + kMagic);
  return low_bytes(b);
}

// 8 elements in 8 bits.
template <typename T>
__device__ __forceinline__ uint2 round8(const Chunk<T>& c, const Rounding& r) {
  float f[8];
  c.get(f);
  uint32_t b[8], differ = 0u;
  const float2 magic = make_float2(kMagic, kMagic);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 x = make_float2(f[i], f[i + 1]);
    const float2 z = fma2(x, make_float2(r.above, r.above), magic);
    b[i] = __float_as_uint(z.x), b[i + 1] = __float_as_uint(z.y);
    if constexpr (sizeof(T) == 4) {
      const float2 y = fma2(x, make_float2(r.below, r.below), magic);
      differ |= b[i] ^ __float_as_uint(y.x);
      differ |= b[i + 1] ^ __float_as_uint(y.y);
    }
  }
  if (differ || r.divide) return round8_divide<T>(c, r.mul, r.div);
  return low_bytes(b);
}

// TPR threads per row, NV chunks each in registers; NV = 0: rows of any
// length, read twice.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(kThreads)
quantize_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ row_map, int n_tok,
                     int H, int K, int N, int8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t part[kThreads / 32];
  // The launch overlaps the end of the kernel before, and the next kernel's CTAs
  // may be set up once all of this grid's have come here (one that asks for it
  // waits for this one's end before it reads).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
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
        if constexpr (sizeof(T) == 4) top = max(top, w[q] & 0x7fffffffu);
        else top = max_abs_bf16x2(top, w[q]);
      }
    }
  };
  Chunk<T> c[NV > 0 ? NV : 1];
  if constexpr (NV > 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int h = (v * TPR + i) * 8;
      if (live && h < H) c[v].load(row + h);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (live && (v * TPR + i) * 8 < H) widen(c[v]);
  } else {
    for (int h = i * 8; live && h < H; h += TPR * 8) {
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
  if constexpr (sizeof(T) == 2) top = max(top & 0x7fff0000u, (top & 0x7fffu) << 16);  // as fp32
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
  r.divide = !zero && by != 1.f;
  const float k = __fdividef(r.mul, r.div);
  if constexpr (sizeof(T) == 4) {
    r.above = k * (1.f + 0x1p-20f), r.below = k * (1.f - 0x1p-20f);
  } else {
    r.above = k * (1.f + 0x1p-21f);
    if ((top & 0x7f0000u) == 0x7e0000u) r.above = __fdiv_rn(r.mul, r.div);  // M = 254
  }
  if (i < K && live && dest >= 0) scale[dest] = finite ? m / 127.f : __int_as_float(0x7fffffff);
  // the rows of the K slots in turn, a row's chunks together
  constexpr int kW = NV > 0 ? NV : 1;
  uint2 w[kW];
  auto put = [&](int h0) {
    for (int k = 0; k < K; ++k) {
      const int d = __shfl_sync(0xffffffffu, dest, k);
      if (d < 0) continue;
      int8_t* to = q + (size_t)d * H;
#pragma unroll
      for (int v = 0; v < kW; ++v) {
        const int h = h0 + (v * TPR + i) * 8;
        if (h < H) *reinterpret_cast<uint2*>(to + h) = w[v];
      }
    }
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) w[v] = zero ? make_uint2(0u, 0u) : round8(c[v], r);
    put(0);
  } else {
    for (int h0 = 0; h0 < H; h0 += TPR * 8) {
      const int h = h0 + i * 8;
      if (live && h < H) c[0].load(row + h);
      w[0] = zero ? make_uint2(0u, 0u) : round8(c[0], r);
      put(h0);
    }
  }
}

template <typename T>
void launch_quantize(const T* x, const int32_t* row_map, int n_tok, int H, int K, int N, int8_t* q,
                     float* scale, cudaStream_t s) {
  auto go = [&](auto tpr, auto nv) {
    constexpr int R = kThreads / decltype(tpr)::value;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((n_tok - 1) / R + 1);  // (n_tok + R - 1 may pass 31 bits)
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    (void)cudaLaunchKernelEx(&cfg, quantize_rows_kernel<T, decltype(tpr)::value, decltype(nv)::value>, x,
                             row_map, n_tok, H, K, N, q, scale);
  };
  using std::integral_constant;
  // at most four chunks a thread up to 8192 elements: eight in half as many
  // threads took 22.6 us against 20.9 at 16384 x 2048 (8192 x 4096: 21.2 and
  // 21.4), two in twice as many 24.5 (and 23.0)
  if (H <= 256) go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (H <= 512) go(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  else if (H <= 768) go(integral_constant<int, 32>{}, integral_constant<int, 3>{});
  else if (H <= 1024) go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  else if (H <= 1536) go(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  else if (H <= 2048) go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (H <= 4096) go(integral_constant<int, 128>{}, integral_constant<int, 4>{});
  else if (H <= 8192) go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else if (H <= 16384) go(integral_constant<int, 256>{}, integral_constant<int, 8>{});
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
  if (H > MOE_QUANTIZE_MAX_LENGTH) return MOE_ERR_SHAPE;  // (a step past a row's end stays within 31 bits)
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
