// Grouped products of 8-bit rows and 8-bit expert weights with a scale for
// each row and each channel, on tcgen05 tensor cores (sm_103a).
//
//   y[i, n] = rs[i] cs[e, n] sum_k q[i, k] w[e, n, k]
//
// sm_103a has no 8-bit integer MMA with tensor-memory accumulators, so both
// operands are expanded on chip to fp16, which holds every byte exactly, and
// multiplied by kind::f16 with fp32 sums (exact while they stay under 2^24).
// DRAM and L2 see bytes only.  What bounds it is the tensor pipe at its fp16
// rate when experts have rows enough, else the stream of weights; next to
// either stands shared memory, which the expansion crosses twice, so:
//
//   * the weights are the A operand (M = channels): they go from the 8-bit
//     tile through registers into tensor memory, never back to shared memory;
//   * the rows are the B operand (N = rows), so a tile takes as many rows as
//     an expert has, in steps of 32 up to 320 (two accumulators of 160): 25
//     rows cost 32 columns, not 128 rows, and the weights of an expert of up
//     to 320 rows are loaded and expanded once;
//   * CTA pairs (cta_group::2): 256 channels per MMA, each CTA expands its
//     own 128 channels and half of the rows.
//
// Shared memory moves, per 128-deep stage and CTA, 32 KB for the weights (in and
// out) and 768 bytes for each of its N / 2 rows (in, out, expanded in, read by
// the MMA) in the MMA's 4 N cycles: 121 of its 128 bytes a cycle at N = 320, all
// of them at N = 256.  So 8192 x 4096 x 4096 runs at 1.72 PFLOP/s (160 us, tensor pipe 82 %
// busy).  With 256 rows an expert the two accumulators fill tensor memory, and
// the part of the epilogue that no MMA overlaps is 20 % of gate/up (H=2048
// I=768 E=128: 161 us) and 30 % of down (104 us), whose tiles are 6 stages.
//
// Warps: 1 TMA producer, 1 MMA issuer (in the leading CTA), epilogue warps (one
// or two per tensor-memory lane quarter), groups that expand A and B of the
// 128-deep stages in turn, 32 operand rows a warp (I8Cfg).
//
// The expanding warps of both CTAs arrive on the leader's barrier with the
// default (CTA-scope) release: what they wrote, tensor memory and shared
// memory of their own SM, is read by that SM's tensor core alone, and is
// ordered by tcgen05.wait::st and the async-proxy fence before the arrival.
// A cluster-scope release there, by one forwarding thread, cost 1100 cycles a
// step (8192 x 4096 x 4096: 399 us against 262 us, the rest being as it was).
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "per_device.h"
#include "sched.cuh"
#include "tc_warp.cuh"
#include "tma_host.cuh"

namespace moe {
namespace tc {
namespace {

// kSub: B rows (N) of one accumulator, at most; a tile has up to two.
// kGroups: expanding groups, which take the 128-deep stages in turn, with an
// expanded buffer each.  kEpi: epilogue warps.  kStages: 8-bit stages.
template <int SUB, int GROUPS, int EPI, int STAGES>
struct I8Cfg {
  static constexpr int kSub = SUB, kGroups = GROUPS, kEpi = EPI, kStages = STAGES;
  static constexpr int kRowTile = 2 * kSub;             // B rows of a tile
  static constexpr uint32_t kA8 = 128 * 128;            // 8-bit A bytes of a stage
  static constexpr uint32_t kB8 = kRowTile / 2 * 128;   // 8-bit B bytes of a stage
  static constexpr uint32_t kB16 = kRowTile / 2 * 256;  // fp16 B bytes, two 64-deep halves
  static constexpr uint32_t kACol = 2 * kSub;           // tensor memory: accumulators, A buffers
  static constexpr int kBGroup = (kRowTile + 63) / 64;  // warps that expand B, per group
  static constexpr int kAWarp = 2 + kEpi, kBWarp = kAWarp + 4 * kGroups;
  static constexpr int kThreads = (kBWarp + kGroups * kBGroup) * 32;
  // A group handles every kGroups-th stage, so it would meet a slot's "loaded"
  // barrier only at every second use (3 slots, 2 groups), where the phase
  // parity of the use it waits for and of the one two before are the same: a
  // late load in between would let it through early.  So each (slot, group)
  // has a barrier of its own: stage i signals number i mod lcm(slots, groups).
  static constexpr int lcm(int a, int b) {
    int m = a;
    while (m % b) m += a;
    return m;
  }
  static constexpr int kFulls = lcm(kStages, kGroups);
  static constexpr int kBars = kFulls + kStages + 2 * kGroups + 4 + 1;
  static constexpr uint32_t kStageWarp = 2048 + 128;  // epilogue staging of a warp: rows, row scales
  static constexpr uint32_t kStage = kStages * (kA8 + kB8) + kGroups * kB16;
  static constexpr uint32_t kCtrl = kStage + kEpi * kStageWarp;
  static constexpr uint32_t kHolder = kCtrl + 8 * kBars;
  static constexpr uint32_t kTable = kHolder + 8;  // prefix, offsets, scan scratch
  static constexpr uint32_t kSmem = kTable + 2 * (kMaxExperts + 1) * 4 + 32 * 4 + 1024;
  static_assert(kSmem <= 232448, "more shared memory than one CTA may use");
  static_assert(kACol + kGroups * 64 <= 512, "more tensor memory than there is");
  static_assert(kGroups <= kStages && kSub % 32 == 0 && kFulls % kGroups == 0, "geometry");
};

// Experts with rows: two accumulators of 160 columns.  Experts with few rows
// each: the stream of weights bounds it, so the room goes to a deeper ring and
// to more warps that expand weights.
using I8Many = I8Cfg<160, 2, 8, 3>;
using I8Few = I8Cfg<32, 4, 4, 8>;
constexpr int kTmaWarp = 0, kMmaWarp = 1, kEpiWarp = 2;

struct I8Params {
  const int32_t* off;
  const float *rs, *s0, *s1;
  void* out;
  int32_t* status;
  int N, E, Kd, Nout;
  int ch_tiles;  // channel tiles per expert: of 256 (128 for gate/up)
};

struct I8Tile {
  int e, row0, hi;  // expert, first row, end of the tile's rows
  int subs;         // accumulators the rows take: 1 or 2
  int n, n1;        // MMA N of the first and of the second: multiples of 32
  int ch0;          // first channel of this CTA
  __device__ __forceinline__ int b_rows() const { return (n + n1) / 2; }  // of this CTA
};

// Tile t is channel tile (t mod ch_tiles) of row tile t / ch_tiles; the rows
// of an expert are split evenly over its ceil(rows / (2 kSub)) row tiles, the rows
// of a row tile over its accumulators in steps of 32.
template <bool kSwiglu, int kSub>
__device__ __forceinline__ I8Tile i8_tile(int t, const I8Params& p, const int32_t* prefix,
                                          const int32_t* offs, int rank) {
  I8Tile x;
  const int g = t / p.ch_tiles;
  x.e = find_expert(prefix, p.E, g);
  const ExpertRows r = expert_rows(offs, x.e, p.N);
  const int parts = prefix[x.e + 1] - prefix[x.e], i = g - prefix[x.e];
  const int per = (r.hi - r.lo + parts - 1) / parts;
  x.row0 = r.lo + i * per;
  x.hi = min(r.hi, x.row0 + per);
  x.subs = per > kSub ? 2 : 1;
  const int steps = (per + 31) >> 5;  // (pairs take N in steps of 32)
  x.n = x.subs == 2 ? ((steps + 1) >> 1) * 32 : steps * 32;
  x.n1 = steps * 32 - x.n;
  x.ch0 = (t - g * p.ch_tiles) * (kSwiglu ? 128 : 256) + rank * (kSwiglu ? 64 : 128);
  return x;
}

// Four signed bytes as fp16: 0x64uu is 1024 + u with u = byte + 128, less
// 1152.  The pairs are bytes (0, 2) and (1, 3): both operands are expanded
// alike, so the sum over k only changes its order.
__device__ __forceinline__ void expand4(uint32_t w, uint32_t& even, uint32_t& odd) {
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = (w & 0x00ff00ffu) ^ 0x64806480u, b = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
  __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
  __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  even = *reinterpret_cast<uint32_t*>(&x);
  odd = *reinterpret_cast<uint32_t*>(&y);
}

__device__ __forceinline__ void expand16(uint4 v, uint32_t* r) {
  expand4(v.x, r[0], r[1]);
  expand4(v.y, r[2], r[3]);
  expand4(v.z, r[4], r[5]);
  expand4(v.w, r[6], r[7]);
}

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Two products at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(uint32_t x, uint32_t y, float s, float t) {
  return mul2(make_float2(__uint_as_float(x), __uint_as_float(y)), make_float2(s, t));
}

// x / (1 + e^-x): the approximate exponential and reciprocal in the forms that
// flush what is below 2^-126 (half the instructions of those that keep it).
__device__ __forceinline__ float silu(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return x * r;
}

template <typename C, bool kSwiglu, typename O>
__global__ void __launch_bounds__(C::kThreads, 1)
gmm_i8_kernel(const __grid_constant__ CUtensorMap mapW0, const __grid_constant__ CUtensorMap mapW1,
              const __grid_constant__ CUtensorMap mapX32, const __grid_constant__ CUtensorMap mapX16,
              const I8Params p) {
  constexpr int kSub = C::kSub, kGroups = C::kGroups, kStages = C::kStages, kBGroup = C::kBGroup;
  constexpr int kAWarp = C::kAWarp, kBWarp = C::kBWarp, kEpi = C::kEpi, kFulls = C::kFulls;
  constexpr uint32_t kA8 = C::kA8, kB8 = C::kB8, kB16 = C::kB16, kACol = C::kACol;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* g = smem_raw + (base - raw);
  const uint32_t sA8 = base, sB8 = base + kStages * kA8, sB16 = sB8 + kStages * kB8;
  const uint32_t bars = base + C::kCtrl;
  auto q_full = [&](int i) { return bars + 8u * i; };  // i: stage mod kFulls
  auto q_empty = [&](int s) { return bars + 8u * (kFulls + s); };
  const uint32_t bars2 = bars + 8u * (kFulls + kStages);
  auto c_full = [&](int b) { return bars2 + 8u * b; };
  auto c_empty = [&](int b) { return bars2 + 8u * (kGroups + b); };
  auto t_full = [&](int a) { return bars2 + 8u * (2 * kGroups + a); };
  auto t_empty = [&](int a) { return bars2 + 8u * (2 * kGroups + 2 + a); };
  const uint32_t drain = bars2 + 8u * (2 * kGroups + 4);
  uint32_t* holder = reinterpret_cast<uint32_t*>(g + C::kHolder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(g + C::kHolder + 4);
  int32_t* prefix = reinterpret_cast<int32_t*>(g + C::kTable);
  int32_t* offs = prefix + (kMaxExperts + 1);
  int32_t* scratch = offs + (kMaxExperts + 1);
  const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kFulls; ++i) mbar_init(q_full(i), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(q_empty(s), 4 + kBGroup);  // an expanding group
    }
    for (int b = 0; b < kGroups; ++b) {
      mbar_init(c_full(b), 2 * (4 + kBGroup));  // the leader's: a group of both CTAs
      mbar_init(c_empty(b), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(t_full(a), 1);
      mbar_init(t_empty(a), 2 * kEpi);  // the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&mapW0);
    if constexpr (kSwiglu) tma_prefetch_desc(&mapW1);
    tma_prefetch_desc(&mapX32);
    tma_prefetch_desc(&mapX16);
  }
  // Both CTAs are present and their barriers initialised before either uses
  // the other's (the pair's tensor-memory allocation included).
  cluster_sync_all();
  if (warp == kMmaWarp) {
    tmem_alloc_pair(smem_u32(holder), 512);
    tmem_relinquish_pair();
  }
  // From here on what earlier kernels of the stream wrote is read: the part
  // above may overlap the end of the one before (as the rows' rounding lets it).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  stage_offsets(p.off, p.E, p.N, offs, scratch);
  build_tile_prefix(offs, p.E, p.N, C::kRowTile, prefix, scratch);  // ends with __syncthreads
  const int total = prefix[p.E] * p.ch_tiles;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const int rank = (int)cluster_ctarank();
  const int t0 = (int)cluster_id_x(), dt = (int)cluster_count_x();
  const int stages = (p.Kd + 127) / 128;

  if (warp == kTmaWarp) {  // the whole warp, one lane elected for each copy
    const uint32_t ub = uniform(base);
    int s = 0, f = 0, n = 0;  // slot, its barrier, stages so far
    uint32_t ph = 0;
    bool run = true;
    for (int t = t0; run && t < total; t += dt) {
      const I8Tile x = i8_tile<kSwiglu, kSub>(t, p, prefix, offs, rank);
      const int nh0 = (int)uniform(x.n) / 2, nh1 = (int)uniform(x.n1) / 2, e = (int)uniform(x.e);
      const int ch0 = (int)uniform(x.ch0), r0 = (int)uniform(x.row0);
      const uint32_t tx = kA8 + (uint32_t)(nh0 + nh1) * 128u;
      for (int k = 0; k < stages; ++k) {
        run = mbar_wait_warp(q_empty(s), ph ^ 1u, abort_flag, p.status);
        if (!run) break;
        mbar_arrive_expect_tx_warp(q_full(f), tx);
        const uint32_t a = ub + s * kA8;
        uint32_t b = ub + kStages * kA8 + s * kB8;
        tma_load_3d_warp(a, &mapW0, q_full(f), k * 128, ch0, e);
        if constexpr (kSwiglu) tma_load_3d_warp(a + kA8 / 2, &mapW1, q_full(f), k * 128, ch0, e);
        // this CTA's half of each accumulator's rows, one after the other
        for (int j = 0; j < 2; ++j) {
          const int nh = j ? nh1 : nh0, rj = r0 + (j ? 2 * nh0 : 0) + rank * nh;
          int r = 0;
          for (; r + 32 <= nh; r += 32, b += 4096)
            tma_load_2d_warp(b, &mapX32, q_full(f), k * 128, rj + r);
          if (r < nh) {
            tma_load_2d_warp(b, &mapX16, q_full(f), k * 128, rj + r);
            b += 2048;
          }
        }
        ++n;
        if (++s == kStages) s = 0, ph ^= 1u;
        if (++f == kFulls) f = 0;
      }
    }
    // every copy has landed before the CTA may exit
    for (int i = max(0, n - kStages); i < n; ++i)
      mbar_wait_warp(q_full(i % kFulls), (uint32_t)(i / kFulls) & 1u, abort_flag, p.status, false);
  } else if (warp == kMmaWarp) {
    if (rank == 0) {  // the whole warp, one lane elected for each MMA
      const uint64_t bdesc0 = desc_sw128(uniform(sB16), 16, 1024);
      const uint32_t tm = uniform(tmem);
      int b = 0, it = 0;
      uint32_t ph = 0;
      bool run = true;
      for (int t = t0; run && t < total; t += dt) {
        const I8Tile x = i8_tile<kSwiglu, kSub>(t, p, prefix, offs, rank);
        const int n = (int)uniform(x.n), subs = (int)uniform(x.subs);
        const uint32_t idesc = idesc_f16_f32(256, n), idesc1 = idesc_f16_f32(256, (int)uniform(x.n1));
        // accumulators it, it + 1 (mod 2), as they become free
        for (int j = 0; run && j < subs; ++j)
          run = __all_sync(0xffffffffu, mbar_wait<true>(t_empty((it + j) & 1), (((it + j) >> 1) & 1) ^ 1u,
                                                        abort_flag, p.status));
        if (!run) break;
        tc_fence_after();
        const uint32_t d0 = tm + (it & 1) * kSub, d1 = tm + ((it + 1) & 1) * kSub;
        const uint32_t sub1 = (uint32_t)n * 64u >> 4;  // the second's rows in shared memory
        uint32_t accum = 0u;
        for (int k = 0; k < stages; ++k) {
          run = mbar_wait_warp(c_full(b), ph, abort_flag, p.status);
          if (!run) break;
          tc_fence_after();
          const uint64_t bd = bdesc0 + (uint64_t)b * (kB16 >> 4);
          const uint32_t a = tm + kACol + b * 64;
          // (past the end of Kd both operands are zeros)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t bh = bd + h * (kB16 >> 5);
            umma_f16_ta_k64_warp<true>(d0, a + h * 32, bh, idesc, accum);
            if (subs > 1) umma_f16_ta_k64_warp<true>(d1, a + h * 32, bh + sub1, idesc1, accum);
            accum = 1u;
          }
          umma_commit_pair_warp(c_empty(b), 3);
          if (++b == kGroups) b = 0, ph ^= 1u;
        }
        if (!run) break;
        for (int j = 0; j < subs; ++j) umma_commit_pair_warp(t_full((it + j) & 1), 3);
        it += subs;
      }
      umma_commit_pair_warp(drain, 3);  // the last signal to either CTA
      mbar_wait_warp(drain, 0, abort_flag, p.status, false);
    }
  } else if (warp >= kAWarp) {
    // ---- expand: a lane takes one 128-byte row of the stage ----
    const bool is_a = warp < kBWarp;
    const int grp = is_a ? (warp - kAWarp) >> 2 : (warp - kBWarp) / kBGroup;
    const int quarter = warp & 3;                              // A: tensor-memory lanes
    const int rg = is_a ? 0 : (warp - kBWarp) - kBGroup * grp;  // B: rows 32 rg + lane
    // A row of this lane: gate/up stages hold 64 gate rows, then 64 up rows; a
    // warp takes 16 of each, so that gate and up of a channel meet in lanes i
    // and i + 16 of one epilogue warp.
    const int row = is_a ? (kSwiglu ? (lane < 16 ? quarter * 16 + lane : 48 + quarter * 16 + lane)
                                    : quarter * 32 + lane)
                         : rg * 32 + lane;
    // Chunk c of row r sits at chunk c ^ (r & 7) (128-byte swizzle), in the
    // 8-bit rows and in the fp16 rows, where it has become chunks 2c, 2c + 1
    // of two 64-deep halves.
    const uint32_t src0 = (is_a ? sA8 : sB8) + row * 128 + ((row & 7) << 4);
    const uint32_t a_dst = tmem + kACol + grp * 64 + ((uint32_t)(quarter * 32) << 16);
    const uint32_t b_dst = sB16 + grp * kB16 + row * 128 + ((row & 7) << 4);
    const uint32_t step = is_a ? kA8 : kB8;
    const uint32_t full_of_leader = mapa_shared(c_full(grp), 0);
    int s = grp, f = grp, n0 = 0;  // slot, its barrier; stages before this tile (mod kGroups)
    uint32_t ph = 0, bph = 0;
    bool run = true;
    for (int t = t0; run && t < total; t += dt) {
      // B rows past the tile's own are not expanded (the MMA does not read them)
      const bool any = is_a || rg * 32 < i8_tile<kSwiglu, kSub>(t, p, prefix, offs, rank).b_rows();
      for (int k = (grp - n0 + kGroups) % kGroups; k < stages; k += kGroups) {
        run = mbar_wait_warp(q_full(f), ph, abort_flag, p.status);
        if (!run) break;
        uint4 v[4];
        uint32_t r[32];
        const uint32_t src = src0 + s * step;
        if (any) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = ld_shared_v4(src ^ (j << 4));
#pragma unroll
          for (int j = 0; j < 4; ++j) expand16(v[j], r + 8 * j);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = ld_shared_v4(src ^ ((j + 4) << 4));
        }
        // All of the rows are read: the fence orders these reads before the
        // copy that refills the slot (the arrival alone does not wait for the
        // loads' data).  1 % of 8192 x 4096 x 4096.
        fence_proxy_async_smem();
        mbar_arrive_warp(q_empty(s));
        run = mbar_wait_warp(c_empty(grp), bph ^ 1u, abort_flag, p.status);
        if (!run) break;
        if (is_a) {
          tc_fence_after();
          tmem_st_32x32b_x32(a_dst, r);
#pragma unroll
          for (int j = 0; j < 4; ++j) expand16(v[j], r + 8 * j);
          tmem_st_32x32b_x32(a_dst + 32, r);
          tmem_st_wait();
          tc_fence_before();
        } else if (any) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared_v4(b_dst ^ (j << 4), r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) expand16(v[j], r + 8 * j);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared_v4((b_dst ^ (j << 4)) + kB16 / 2, r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
          fence_proxy_async_smem();
        }
        mbar_arrive_cluster_warp(full_of_leader);
        bph ^= 1u;
        s += kGroups;
        if (s >= kStages) s -= kStages;
        f += kGroups;
        if (f >= kFulls) f -= kFulls, ph ^= 1u;
      }
      n0 = (n0 + stages) % kGroups;
    }
    // the last of the leader's signals to this CTA's barriers has arrived
    if (run) mbar_wait_warp(c_empty(grp), bph ^ 1u, abort_flag, p.status);
  } else {
    // ---- epilogue: lanes are channels, accumulator columns are rows ----
    // The warps of a quarter take pieces of 32 columns in turn.  A piece
    // is scaled, turned through the warp's staging rows and written in 16-byte
    // chunks of 8 channels.
    const int quarter = warp & 3, part = (warp - kEpiWarp) >> 2;
    constexpr int kCh = kSwiglu ? 16 : 32;  // channels per warp
    O* out = static_cast<O*>(p.out);
    const uint32_t stage_u = base + C::kStage + (uint32_t)(warp - kEpiWarp) * C::kStageWarp;
    float* scale = reinterpret_cast<float*>(g + C::kStage + (warp - kEpiWarp) * C::kStageWarp + 2048);
    const int ch_l = kSwiglu ? quarter * 16 + (lane & 15) : quarter * 32 + lane;
    int it = 0;
    bool run = true;
    for (int t = t0; run && t < total; t += dt) {
     const I8Tile x = i8_tile<kSwiglu, kSub>(t, p, prefix, offs, rank);
     const int ch = x.ch0 + ch_l;
     const float cs = ch >= p.Nout ? 0.f
                                   : ((kSwiglu && lane >= 16) ? p.s1 : p.s0)[(size_t)x.e * p.Nout + ch];
     // row scales of the first pieces (the second accumulator's ahead of its
     // wait, which is short)
     const int r_first = x.row0 + part * 32 + lane, r_second = r_first + x.n;
     const float rs_first = part * 32 + lane < min(x.hi - x.row0, x.n) ? p.rs[r_first] : 0.f;
     const float rs_second = x.subs > 1 && r_second < x.hi ? p.rs[r_second] : 0.f;
     for (int sub = 0; sub < x.subs; ++sub, ++it) {
      const int acc = it & 1, row0 = x.row0 + sub * x.n;
      const int rows = min(x.hi - row0, sub ? x.n1 : x.n);
      float rs = sub ? rs_second : rs_first;
      run = mbar_wait_warp(t_full(acc), (it >> 1) & 1, abort_flag, p.status);
      if (!run) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * kSub + ((uint32_t)(quarter * 32) << 16);
      auto give_back = [&]() {
        tc_fence_before();
        mbar_arrive_cluster_warp(mapa_shared(t_empty(acc), 0));
      };
      for (int c0 = part * 32; c0 < rows; c0 += 8 * kEpi) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(d + c0, v);
        scale[lane] = rs;
        rs = c0 + 8 * kEpi + lane < rows ? p.rs[row0 + c0 + 8 * kEpi + lane] : 0.f;
        __syncwarp();
        tmem_ld_wait();
        if (c0 + 8 * kEpi >= rows) give_back();  // the warp's last piece is in registers
        if constexpr (sizeof(O) == 4) {
          // fp32: staging rows of 32 channels, 16 columns at a time
#pragma unroll
          for (int p0 = 0; p0 < 32; p0 += 16) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              st_shared_u32(stage_u + lane * 4 + j * 128,
                            __float_as_uint(__uint_as_float(v[p0 + j]) * cs * scale[p0 + j]));
            __syncwarp();
            const int wr = lane >> 3, wch = x.ch0 + quarter * kCh + (lane & 7) * 4;
            if (wch < p.Nout) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = c0 + p0 + wr + i * 4;
                if (r < rows)
                  st_v4(out + (size_t)(row0 + r) * p.Nout + wch, ld_shared_v4(stage_u + lane * 16 + i * 512));
              }
            }
            __syncwarp();
          }
        } else {
          // bf16: words of two rows of a channel; [pair][channel]
          uint32_t w[kSwiglu ? 8 : 16];
          if constexpr (kSwiglu) {
            // lanes 0-15 hold gate, 16-31 up of the same channels: the lower
            // half takes the even rows, the upper half the odd ones
            const bool up = lane >= 16;
            float y[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 f = mul2(mul2(v[j], v[j + 1], cs, cs), *reinterpret_cast<const float2*>(scale + j));
              const float got = __shfl_xor_sync(0xffffffffu, up ? f.x : f.y, 16);
              const float gate = up ? got : f.x, u = up ? f.y : got;
              y[j / 2] = silu(gate) * u;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = VecTraits<__nv_bfloat16>::pack2(y[2 * j], y[2 * j + 1]);
            // word row 2j + up: rows 4j + up and 4j + up + 2
            const uint32_t st = stage_u + (lane & 15) * 4 + (up ? 64 : 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) st_shared_u32(st + j * 128, w[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 f =
                  mul2(mul2(v[2 * j], v[2 * j + 1], cs, cs), *reinterpret_cast<const float2*>(scale + 2 * j));
              w[j] = VecTraits<__nv_bfloat16>::pack2(f.x, f.y);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) st_shared_u32(stage_u + lane * 4 + j * 128, w[j]);
          }
          __syncwarp();
          // a lane takes 8 channels of a pair of rows: 32 bytes of words (the
          // halves in an order that keeps 8 lanes on distinct banks)
          constexpr int G = kCh / 8, kWordRow = kCh * 4;
#pragma unroll
          for (int i = 0; i < 16 * G / 32; ++i) {
            const int pr = (lane + 32 * i) / G, gch = (lane + 32 * i) % G;
            const uint32_t src = stage_u + pr * kWordRow + gch * 32;
            const uint32_t first = kSwiglu ? ((pr >> 1) & 1) * 16 : (pr & 1) * 16;
            const uint4 m0 = ld_shared_v4(src + first), m1 = ld_shared_v4(src + (first ^ 16));
            const uint4 a = first ? m1 : m0, b = first ? m0 : m1;
            const uint4 lo = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                        __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
            const uint4 hi = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                        __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
            const int r = c0 + (kSwiglu ? (pr >> 1) * 4 + (pr & 1) : 2 * pr);
            constexpr int dr = kSwiglu ? 2 : 1;
            const int wch = x.ch0 + quarter * kCh + gch * 8;
            if (wch < p.Nout) {
              O* dst = out + (size_t)(row0 + r) * p.Nout + wch;
              if (r < rows) st_v4(dst, lo);
              if (r + dr < rows) st_v4(dst + (size_t)dr * p.Nout, hi);
            }
          }
          __syncwarp();
        }
      }
      if (part * 32 >= rows) give_back();  // (it had none)
     }
    }
    // the peer too ends after the leader's last signal, when a wait ran out as well
    if (rank != 0 && warp == kEpiWarp) mbar_wait_warp(drain, 0, abort_flag, p.status, false);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still signal its barriers
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

int check_i8(const void* A, const float* rs, const int32_t* off, int N, int H, int I, int E) {
  if (N < 0 || H <= 0 || I <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts) return MOE_ERR_SHAPE;
  if (off == nullptr && E != 1) return MOE_ERR_INVALID_ARG;
  if (H % 16 || I % 16 || H > 131072 || I > 131072) return MOE_ERR_SHAPE;
  if (N > MOE_INT8_MAX_ROWS) return MOE_ERR_SHAPE;  // (rows and row tiles added up stay within 31 bits)
  if (N > 0 && (!A || !rs || !aligned16(A))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

template <typename C, bool kSwiglu, typename O>
int launch_cfg(const CUtensorMap& w0, const CUtensorMap& w1, const CUtensorMap& x32,
               const CUtensorMap& x16, const I8Params& p, cudaStream_t s) {
  static PerDevice smem_allowed, resident_pairs;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const int allowed = smem_allowed.get(dev, [] {
    return cudaFuncSetAttribute(gmm_i8_kernel<C, kSwiglu, O>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::kSmem) == cudaSuccess;
  });
  if (!allowed) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  // one persistent CTA per SM, as many whole pairs as can be resident
  cfg.gridDim = dim3(sm_count() / 2 * 2, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const int pairs = resident_pairs.get(dev, [&] {
    int n = 0;
    const bool known = cudaOccupancyMaxActiveClusters(&n, gmm_i8_kernel<C, kSwiglu, O>, &cfg) == cudaSuccess;
    (void)cudaGetLastError();
    return known && n > 0 ? n : INT_MAX;
  });
  if (pairs < (int)cfg.gridDim.x / 2) cfg.gridDim.x = 2 * pairs;
  if (cudaLaunchKernelEx(&cfg, gmm_i8_kernel<C, kSwiglu, O>, w0, w1, x32, x16, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  count_launches(1);
  return MOE_OK;
}

// Rows per expert, on average, up to which the few-rows form runs (the routing
// itself is not known on the host; where it is skewed, an expert of many rows
// reads its weights once for every 64 of them, which was not measured).  GB300,
// E=64 H=2048, as many rows for every expert, us, few / many:
//   rows  I=512 gate/up    down        I=768 gate/up    down
//     25  42.0 / 49.4   28.7 / 33.0    53.9 / 66.3   33.8 / 41.0
//     48  43.4 / 50.1   32.3 / 33.7    57.3 / 67.6   36.9 / 41.0
//     64  45.1 / 53.5   37.1 / 35.6    67.6 / 69.9   45.1 / 43.0
//     80  57.3 / 53.5   45.6 / 36.9    75.8 / 71.7   51.2 / 43.7
constexpr long long few_rows(bool swiglu) { return swiglu ? 64 : 48; }

template <bool kSwiglu, typename O>
int launch_i8(const int8_t* A, const float* rs, const int8_t* B0, const float* s0, const int8_t* B1,
              const float* s1, const int32_t* off, int N, int Kd, int Nout, int E, O* out,
              int32_t* status, cudaStream_t s) {
  if (int rc = device_ok()) return rc;
  CUtensorMap w0, w1, x32, x16;
  const uint64_t dw[3] = {(uint64_t)Kd, (uint64_t)Nout, (uint64_t)E};
  const uint32_t bw[3] = {128, kSwiglu ? 64u : 128u, 1};
  const uint64_t dx[2] = {(uint64_t)Kd, (uint64_t)N};
  const uint32_t b32[2] = {128, 32}, b16[2] = {128, 16};
  if (!make_map_sw128(&w0, B0, 1, 3, dw, bw) || (kSwiglu && !make_map_sw128(&w1, B1, 1, 3, dw, bw)) ||
      !make_map_sw128(&x32, A, 1, 2, dx, b32) || !make_map_sw128(&x16, A, 1, 2, dx, b16))
    return MOE_ERR_CUDA;
  if (!kSwiglu) w1 = w0;
  const int per = kSwiglu ? 128 : 256;
  const I8Params p{off, rs, s0, s1, out, status, N, E, Kd, Nout, (Nout + per - 1) / per};
  return (long long)N <= few_rows(kSwiglu) * E
             ? launch_cfg<I8Few, kSwiglu, O>(w0, w1, x32, x16, p, s)
             : launch_cfg<I8Many, kSwiglu, O>(w0, w1, x32, x16, p, s);
}

}  // namespace
}  // namespace tc
}  // namespace moe

using namespace moe;
using namespace moe::tc;

extern "C" int moe_gate_up_swiglu_int8(const int8_t* permuted_q, const float* row_scale,
                                       const int32_t* expert_offsets, int N, int H, int I, int E,
                                       const int8_t* W_gate_q, const float* gate_scale,
                                       const int8_t* W_up_q, const float* up_scale, void* act,
                                       int32_t* dev_status, cudaStream_t stream) {
  if (int rc = check_i8(permuted_q, row_scale, expert_offsets, N, H, I, E)) return rc;
  if (N == 0) return MOE_OK;
  if (!W_gate_q || !W_up_q || !gate_scale || !up_scale || !act) return MOE_ERR_INVALID_ARG;
  if (!aligned16(W_gate_q) || !aligned16(W_up_q) || !aligned16(act)) return MOE_ERR_INVALID_ARG;
  return launch_i8<true>(permuted_q, row_scale, W_gate_q, gate_scale, W_up_q, up_scale,
                         expert_offsets, N, H, I, E, static_cast<__nv_bfloat16*>(act), dev_status,
                         stream);
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
  if (out_dtype == MOE_F32)
    return launch_i8<false>(act_q, row_scale, W_down_q, down_scale, nullptr, nullptr, expert_offsets,
                            N, I, H, E, static_cast<float*>(expanded), dev_status, stream);
  return launch_i8<false>(act_q, row_scale, W_down_q, down_scale, nullptr, nullptr, expert_offsets, N,
                          I, H, E, static_cast<__nv_bfloat16*>(expanded), dev_status, stream);
}
