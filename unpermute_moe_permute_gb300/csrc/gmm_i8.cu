// Grouped products of 8-bit rows and 8-bit expert weights with a scale for
// each row and each channel, on the 4-way integer dot product (exact int32
// sums).  Tiles of 64 x 64 outputs, 256 threads, 4 x 4 outputs per thread, a
// 64-deep k slice staged in shared memory as 16 words.
#include <math.h>

#include "common.cuh"
#include "sched.cuh"

namespace moe {
namespace {

constexpr int BM = 64, BN = 64, BKW = 16, kThreads = 256;

template <bool kSwiglu, typename O>
__global__ void __launch_bounds__(kThreads)
gmm_i8_kernel(const int8_t* __restrict__ A, const float* __restrict__ rs,
              const int8_t* __restrict__ B0, const float* __restrict__ s0,
              const int8_t* __restrict__ B1, const float* __restrict__ s1,
              const int32_t* __restrict__ off, int N, int Kd, int Nout, int E,
              O* __restrict__ out) {
  __shared__ int32_t prefix[kMaxExperts + 1];
  __shared__ int32_t offs[kMaxExperts + 1];
  __shared__ int32_t scratch[32];
  __shared__ int As[BKW][BM + 1];
  __shared__ int Bs0[BKW][BN + 1];
  __shared__ int Bs1[kSwiglu ? BKW : 1][BN + 1];
  stage_offsets(off, E, N, offs, scratch);
  build_tile_prefix(offs, E, N, BM, prefix, scratch);
  const int tile = blockIdx.x;
  if (tile >= prefix[E]) return;  // uniform across the CTA
  const int e = find_expert(prefix, E, tile);
  const ExpertRows rows = expert_rows(offs, e, N);
  const int row0 = rows.lo + (tile - prefix[e]) * BM;
  const int n0 = blockIdx.y * BN;
  const int8_t* b0 = B0 + (size_t)e * Nout * Kd;
  const int8_t* b1 = kSwiglu ? B1 + (size_t)e * Nout * Kd : nullptr;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  int acc0[4][4] = {}, acc1[4][4] = {};
  const int lr = tid >> 2, lw = (tid & 3) * 4;
  for (int k0 = 0; k0 < Kd; k0 += BKW * 4) {
    const int c = k0 + lw * 4;
    const int r = row0 + lr, n = n0 + lr;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const uint4 a = (r < rows.hi && c < Kd) ? ld_v4(A + (size_t)r * Kd + c) : z;
    const uint4 w = (n < Nout && c < Kd) ? ld_v4(b0 + (size_t)n * Kd + c) : z;
    As[lw][lr] = a.x, As[lw + 1][lr] = a.y, As[lw + 2][lr] = a.z, As[lw + 3][lr] = a.w;
    Bs0[lw][lr] = w.x, Bs0[lw + 1][lr] = w.y, Bs0[lw + 2][lr] = w.z, Bs0[lw + 3][lr] = w.w;
    if constexpr (kSwiglu) {
      const uint4 v = (n < Nout && c < Kd) ? ld_v4(b1 + (size_t)n * Kd + c) : z;
      Bs1[lw][lr] = v.x, Bs1[lw + 1][lr] = v.y, Bs1[lw + 2][lr] = v.z, Bs1[lw + 3][lr] = v.w;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BKW; ++kk) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int av = As[kk][ty * 4 + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc0[i][j] = __dp4a(av, Bs0[kk][tx * 4 + j], acc0[i][j]);
          if constexpr (kSwiglu) acc1[i][j] = __dp4a(av, Bs1[kk][tx * 4 + j], acc1[i][j]);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + ty * 4 + i;
    if (r >= rows.hi) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= Nout) continue;
      float y = (float)acc0[i][j] * rs[r] * s0[(size_t)e * Nout + n];
      if constexpr (kSwiglu) {
        const float u = (float)acc1[i][j] * rs[r] * s1[(size_t)e * Nout + n];
        y = y / (1.f + expf(-y)) * u;
      }
      out[(size_t)r * Nout + n] = (O)y;
    }
  }
}

int check_i8(const void* A, const float* rs, const int32_t* off, int N, int H, int I, int E) {
  if (N < 0 || H <= 0 || I <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts) return MOE_ERR_SHAPE;
  if (off == nullptr && E != 1) return MOE_ERR_INVALID_ARG;
  if (H % 16 || I % 16 || H > 131072 || I > 131072) return MOE_ERR_SHAPE;
  if (N > 0 && (!A || !rs || !aligned16(A))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

template <bool kSwiglu, typename O>
int launch_i8(const int8_t* A, const float* rs, const int8_t* B0, const float* s0, const int8_t* B1,
              const float* s1, const int32_t* off, int N, int Kd, int Nout, int E, O* out,
              cudaStream_t s) {
  const long long tiles = (long long)(N + BM - 1) / BM + (E < N ? E : N);  // at most
  const dim3 grid((unsigned)tiles, (Nout + BN - 1) / BN);
  gmm_i8_kernel<kSwiglu, O><<<grid, kThreads, 0, s>>>(A, rs, B0, s0, B1, s1, off, N, Kd, Nout, E, out);
  MOE_LAUNCH_CHECK();
  count_launches(1);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_gate_up_swiglu_int8(const int8_t* permuted_q, const float* row_scale,
                                       const int32_t* expert_offsets, int N, int H, int I, int E,
                                       const int8_t* W_gate_q, const float* gate_scale,
                                       const int8_t* W_up_q, const float* up_scale, void* act,
                                       int32_t* dev_status, cudaStream_t stream) {
  if (int rc = check_i8(permuted_q, row_scale, expert_offsets, N, H, I, E)) return rc;
  if (N == 0) return MOE_OK;
  if (!W_gate_q || !W_up_q || !gate_scale || !up_scale || !act) return MOE_ERR_INVALID_ARG;
  if (!aligned16(W_gate_q) || !aligned16(W_up_q) || !aligned16(act)) return MOE_ERR_INVALID_ARG;
  (void)dev_status;
  return launch_i8<true>(permuted_q, row_scale, W_gate_q, gate_scale, W_up_q, up_scale,
                         expert_offsets, N, H, I, E, static_cast<__nv_bfloat16*>(act), stream);
}

extern "C" int moe_down_proj_int8(const int8_t* act_q, const float* row_scale,
                                  const int32_t* expert_offsets, int N, int H, int I, int E,
                                  const int8_t* W_down_q, const float* down_scale, void* expanded,
                                  int out_dtype, int32_t* dev_status, cudaStream_t stream) {
  if (int rc = check_i8(act_q, row_scale, expert_offsets, N, H, I, E)) return rc;
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (N == 0) return MOE_OK;
  if (!W_down_q || !down_scale || !expanded) return MOE_ERR_INVALID_ARG;
  if (!aligned16(W_down_q) || !aligned16(expanded)) return MOE_ERR_INVALID_ARG;
  (void)dev_status;
  if (out_dtype == MOE_F32)
    return launch_i8<false>(act_q, row_scale, W_down_q, down_scale, nullptr, nullptr, expert_offsets,
                            N, I, H, E, static_cast<float*>(expanded), stream);
  return launch_i8<false>(act_q, row_scale, W_down_q, down_scale, nullptr, nullptr, expert_offsets, N,
                          I, H, E, static_cast<__nv_bfloat16*>(expanded), stream);
}
