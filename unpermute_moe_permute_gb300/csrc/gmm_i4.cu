// Grouped products of bf16 rows and 4-bit expert weights with a scale for each
// group of inputs, on tcgen05 tensor cores (sm_103a).
//
//   y[i, n] = sum_k x[i, k] bf16(q[e, n, k] s[e, k / group, n])
//
// The weights are expanded to bf16 on chip (exact for scales of five
// significant bits) and multiplied by kind::f16 with fp32 sums.  DRAM and L2 see
// half a byte a weight.  What bounds it is the tensor pipe when experts have rows
// enough, else the stream of weights and the integer pipe that expands them:
//
//   * the weights are the A operand (M = channels): 64 bytes of a row, 128 of
//     its inputs, go through registers into tensor memory at a time;
//   * the rows are the B operand (N = rows), as they come by TMA: up to 320 of an
//     expert in two accumulators of 160, so the weights of an expert of up to 320
//     rows are loaded and expanded once (fewer rows: one accumulator of 128 or 160,
//     the other is the next tile's);
//   * CTA pairs (cta_group::2): 256 channels per MMA, each CTA expands its own
//     128 channels and holds half of the rows;
//   * the scales come by TMA beside the weights they belong to, a column of 128
//     channels for each group (zeros past the ends, as the weights).
//
// Where there are too few tiles for the SMs (a dense layer of a few rows), the
// pairs of a cluster share a tile's inputs: pair s of S takes the s-th part of k,
// and pair 0 adds the others' sums, which they write into its shared memory, to
// its own, in their order.
//
// Warps: 1 TMA producer, 1 MMA issuer (in the leading CTA), epilogue warps, and
// groups of four warps that expand 128 of k in turn.  A stage has two barriers: the
// expanding groups wait for its weights and scales, each CTA's on its own; the MMA
// issuer for its rows, both CTAs' on the leader's.  Its instructions read the peer's
// shared memory, and the copies into it signal the leader themselves: an arrival of
// the peer's warps after they have seen a copy land says so only with release and
// acquire at cluster scope (gate/up of 256 rows an expert 176 us, not 132).  The issuer
// tries both barriers of a part at once (one after the other: few rows 62 -> 66 us).
//
// Few rows: stages are 256 deep, because the copies' 128-byte rows take the TMA unit
// half the time of 64-byte ones.  (With 128-deep stages 203 tokens of 64 experts,
// H=2048 I=512, took 29.5 us, now 26.9.)
#include <limits.h>

#include "common.cuh"
#include "int4.cuh"
#include "pair_tile.cuh"
#include "per_device.h"
#include "tma_host.cuh"

namespace moe {
namespace tc {
namespace {

// DEEP: k of a stage.  SUBS: accumulators of a tile.  SPLIT: pairs that share a tile.
template <int SUB, int GROUPS, int EPI, int DEEP, int STAGES, int SUBS = 2, int SPLIT = 1>
struct I4Cfg {
  static constexpr int kSub = SUB, kGroups = GROUPS, kEpi = EPI, kDeep = DEEP, kStages = STAGES, kSplit = SPLIT;
  // The parts of 128 k of a stage go to the groups of a team, the stages to the
  // teams in turn.
  static constexpr int kPer = DEEP / 128, kTeams = GROUPS / kPer;
  // The first accumulator's products go ahead of the second's: two parts (128 k) at
  // a tile's beginning, while the second's last sums are still being read, three at
  // its end, so that the first's can be.  (256 rows of each of 128 experts, H=2048
  // I=768: gate/up 143 -> 133 us, down 90 -> 82; with two and two 135 and 80, three
  // and two 135 and 85.  The forms for few rows take 3 to 20 % longer with that loop.)
  static constexpr bool kAhead = SUBS == 2 && kPer == 1;
  static constexpr int kHead = 2, kTail = 3;
  static constexpr int kRowTile = SUBS * kSub;          // B rows of a tile
  static constexpr uint32_t kB = kRowTile / 2 * DEEP * 2;  // B bytes of a stage: 64-deep pieces
  static constexpr uint32_t kA = 128 * DEEP / 2;        // 4-bit A bytes of a stage
  static constexpr uint32_t kS = DEEP / 32 * 128 * 2;   // scales of a stage, at most
  static constexpr uint32_t kACol = 2 * kSub;           // tensor memory: two accumulators, A buffers
  static constexpr int kAWarp = 2 + kEpi;
  static constexpr int kThreads = (kAWarp + 4 * kGroups) * 32;
  // (A barrier for each slot and team, so that a team meets every phase of its
  // barriers: with 3 teams and 4 slots it would else see every third.)
  static constexpr int lcm(int a, int b) {
    int m = a;
    while (m % b) m += a;
    return m;
  }
  static constexpr int kFulls = lcm(kStages, kTeams);
  static constexpr int kBars = kFulls + 2 * kStages + 2 * kGroups + 4 + 1 + 2 + 1;
  static constexpr uint32_t kStageWarp = 2048;  // epilogue staging of a warp
  static constexpr uint32_t kPart = kRowTile * 128 * 4;  // sums of another pair: [row][channel]
  static constexpr uint32_t kParts = kStages * (kB + kA + kS);
  static constexpr uint32_t kStage = kParts + (kSplit - 1) * kPart;
  static constexpr uint32_t kCtrl = kStage + kEpi * kStageWarp;
  static constexpr uint32_t kHolder = kCtrl + 8 * kBars;
  static constexpr uint32_t kTable = kHolder + 16;  // prefix, offsets, scan scratch
  static constexpr uint32_t kSmem = kTable + 2 * (kMaxExperts + 1) * 4 + 32 * 4 + 1024;
  static_assert(kSmem <= 232448, "more shared memory than one CTA may use");
  static_assert(kACol + kGroups * 64 <= 512, "more tensor memory than there is");
  static_assert(!kAhead || (kHead <= kGroups && kTail <= kGroups && kGroups <= kStages), "parts ahead");
  static_assert(kTeams <= kStages && kSub % 32 == 0 && kGroups % kPer == 0, "geometry");
};

using I4Many = I4Cfg<160, 3, 8, 128, 4>;
using I4Few = I4Cfg<32, 4, 4, 256, 6>;
using I4Split2 = I4Cfg<32, 4, 4, 256, 5, 2, 2>;
using I4To80 = I4Cfg<128, 4, 4, 256, 4, 1>;
using I4To128 = I4Cfg<160, 3, 8, 128, 6, 1>;

struct I4Params {
  const int32_t* off;
  void* out;
  int32_t* status;
  int N, E, Kd, Nout;
  int ch_tiles;    // channel tiles per expert: of 256 (128 for gate/up)
  int group;       // inputs of a scale
};

// The pairs of a cluster that share a tile: what pair 0 needs to add the others'
// sums, and they to hand theirs over.
template <typename C>
struct SplitTile {
  uint32_t parts, full, empty;  // shared memory: sums; pair 0's barrier, the others' barrier
  int pair, rank, lane, quarter;
  volatile int* abort_flag;
  int32_t* status;
  uint32_t tile = 0;  // tiles so far
  __device__ __forceinline__ uint32_t at(int s, int c) const {
    return parts + s * C::kPart + (uint32_t)c * 512u + (uint32_t)(quarter * 32 + lane) * 4u;
  }
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_wait<true>(bar, parity, abort_flag, status));
  }
  // the last tile's sums have been read
  __device__ __forceinline__ bool begin() { return pair == 0 || wait(empty, (tile & 1u) ^ 1u); }
  __device__ __forceinline__ bool piece(uint32_t (&v)[32], int c) {
    if (pair != 0) {
      const uint32_t dst = mapa_shared(at(pair - 1, c), rank);
#pragma unroll
      for (int j = 0; j < 32; ++j)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + j * 512), "r"(v[j]) : "memory");
      return false;
    }
    if (!wait(full, tile & 1u)) return false;
#pragma unroll
    for (int s = 0; s < C::kSplit - 1; ++s)
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float f;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(at(s, c + j)));
        v[j] = __float_as_uint(__uint_as_float(v[j]) + f);
      }
    return true;
  }
  __device__ __forceinline__ void end() {
    if (pair != 0) {
      mbar_arrive_release_cluster_warp(mapa_shared(full, rank));
    } else {
#pragma unroll
      for (int s = 1; s < C::kSplit; ++s) mbar_arrive_release_cluster_warp(mapa_shared(empty, 2 * s + rank));
    }
    ++tile;
  }
};

template <typename C, bool kSwiglu, typename O>
__global__ void __launch_bounds__(C::kThreads, 1)
gmm_i4_kernel(const __grid_constant__ CUtensorMap mapW0, const __grid_constant__ CUtensorMap mapW1,
              const __grid_constant__ CUtensorMap mapS0, const __grid_constant__ CUtensorMap mapS1,
              const __grid_constant__ CUtensorMap mapX32, const __grid_constant__ CUtensorMap mapX16,
              const I4Params p) {
  constexpr int kSub = C::kSub, kGroups = C::kGroups, kStages = C::kStages, kEpi = C::kEpi;
  constexpr int kAWarp = C::kAWarp, kFulls = C::kFulls, kDeep = C::kDeep, kPer = C::kPer, kTeams = C::kTeams;
  constexpr uint32_t kA = C::kA, kB = C::kB, kS = C::kS, kACol = C::kACol;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* g = smem_raw + (base - raw);
  const uint32_t sB = base, sA = sB + kStages * kB, sS = sA + kStages * kA;
  const uint32_t bars = base + C::kCtrl;
  auto q_full = [&](int i) { return bars + 8u * i; };  // i: stage mod kFulls
  auto q_empty = [&](int s) { return bars + 8u * (kFulls + s); };
  const uint32_t bars2 = bars + 8u * (kFulls + kStages);
  auto c_full = [&](int b) { return bars2 + 8u * b; };
  auto c_empty = [&](int b) { return bars2 + 8u * (kGroups + b); };
  auto t_full = [&](int a) { return bars2 + 8u * (2 * kGroups + a); };
  auto t_empty = [&](int a) { return bars2 + 8u * (2 * kGroups + 2 + a); };
  const uint32_t drain = bars2 + 8u * (2 * kGroups + 4), part_full = drain + 8u, part_empty = drain + 16u;
  const uint32_t counted = drain + 24u;
  auto rows_full = [&](int s) { return drain + 32u + 8u * s; };
  uint32_t* holder = reinterpret_cast<uint32_t*>(g + C::kHolder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(g + C::kHolder + 4);
  volatile int* peer_stages = reinterpret_cast<volatile int*>(g + C::kHolder + 8);
  int32_t* prefix = reinterpret_cast<int32_t*>(g + C::kTable);
  int32_t* offs = prefix + (kMaxExperts + 1);
  int32_t* scratch = offs + (kMaxExperts + 1);
  const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kFulls; ++i) mbar_init(q_full(i), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(q_empty(s), 4 * kPer + 1);  // a team, the MMAs
      mbar_init(rows_full(s), 2);           // the leader's: both CTAs' copies
    }
    for (int b = 0; b < kGroups; ++b) {
      mbar_init(c_full(b), 2 * 4);  // the leader's: a group of both CTAs
      mbar_init(c_empty(b), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(t_full(a), 1);
      mbar_init(t_empty(a), 2 * kEpi);  // the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    mbar_init(counted, 1);
    mbar_init(part_full, C::kSplit > 1 ? (C::kSplit - 1) * kEpi : 1);
    mbar_init(part_empty, kEpi);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&mapW0);
    tma_prefetch_desc(&mapS0);
    if constexpr (kSwiglu) {
      tma_prefetch_desc(&mapW1);
      tma_prefetch_desc(&mapS1);
    }
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
  // above may overlap the end of the one before.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  stage_offsets(p.off, p.E, p.N, offs, scratch);
  build_tile_prefix(offs, p.E, p.N, C::kRowTile, prefix, scratch);  // ends with __syncthreads
  const int total = prefix[p.E] * p.ch_tiles;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  // the CTA in its pair, the pair in its cluster and the part of k that it takes
  const int crank = (int)cluster_ctarank(), rank = crank & 1, leader = crank & ~1, pair = crank >> 1;
  const uint16_t both = (uint16_t)(3 << leader);
  const int t0 = (int)cluster_id_x(), dt = (int)cluster_count_x();
  const int all = (p.Kd + kDeep - 1) / kDeep, k_lo = all * pair / C::kSplit;
  const int stages = all * (pair + 1) / C::kSplit - k_lo;

  if (warp == kTmaWarp) {  // the whole warp, one lane elected for each copy
    const uint32_t ub = uniform(base);
    const int per = kDeep / (int)uniform(p.group);
    const uint32_t rows_of_leader = uniform(mapa_shared(rows_full(0), leader));
    int s = 0, f = 0, n = 0;  // slot, its barrier, stages so far
    uint32_t ph = 0;
    bool run = true;
    for (int t = t0; run && t < total; t += dt) {
      const PairTile x = pair_tile<kSwiglu, kSub>(t, p, prefix, offs, rank);
      const int nh0 = (int)uniform(x.n) / 2, nh1 = (int)uniform(x.n1) / 2, e = (int)uniform(x.e);
      const int ch0 = (int)uniform(x.ch0), r0 = (int)uniform(x.row0);
      const uint32_t tx = kA + (uint32_t)per * 256u, tx_rows = (uint32_t)(nh0 + nh1) * (2u * kDeep);
      for (int k = 0; k < stages; ++k) {
        run = mbar_wait_warp(q_empty(s), ph ^ 1u, abort_flag, p.status);
        if (!run) break;
        mbar_arrive_expect_tx_warp(q_full(f), tx);
        const uint32_t a = ub + kStages * kB + s * kA, sc = ub + kStages * (kB + kA) + s * kS;
        tma_load_3d_warp(a, &mapW0, q_full(f), (k_lo + k) * (kDeep / 2), ch0, e);
        tma_load_3d_warp(sc, &mapS0, q_full(f), ch0, (k_lo + k) * per, e);
        if constexpr (kSwiglu) {
          tma_load_3d_warp(a + kA / 2, &mapW1, q_full(f), (k_lo + k) * (kDeep / 2), ch0, e);
          tma_load_3d_warp(sc + per * 128, &mapS1, q_full(f), ch0, (k_lo + k) * per, e);
        }
        // this CTA's half of each accumulator's rows, one after the other
        const uint32_t rows = rows_of_leader + 8u * s;
        mbar_arrive_expect_tx_cluster_warp(rows, tx_rows);
#pragma unroll
        for (int h = 0; h < kDeep / 64; ++h) {
          uint32_t b = ub + s * kB + h * (kB / (kDeep / 64));
          for (int j = 0; j < 2; ++j) {
            const int nh = j ? nh1 : nh0, rj = r0 + (j ? 2 * nh0 : 0) + rank * nh;
            int r = 0;
            for (; r + 32 <= nh; r += 32, b += 4096)
              tma_load_2d_pair_warp(b, &mapX32, rows, (k_lo + k) * kDeep + h * 64, rj + r);
            if (r < nh) {
              tma_load_2d_pair_warp(b, &mapX16, rows, (k_lo + k) * kDeep + h * 64, rj + r);
              b += 2048;
            }
          }
        }
        ++n;
        if (++s == kStages) s = 0, ph ^= 1u;
        if (++f == kFulls) f = 0;
      }
    }
    // Every copy has landed, and the leader's signals to the slots have come,
    // before the CTA may exit.  The leader waits for both CTAs' rows (the peer stays
    // until the closing cluster barrier).  When its wait ran out the two may have
    // stopped at different stages: it arrives for the one that did not come so far
    // (kStages apart at most: the slots are freed in both together).
    if (rank != 0) {
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(holder) + 8u, leader)), "r"(n) : "memory");
      mbar_arrive_release_cluster_warp(mapa_shared(counted, leader));
    } else {
      int m = n;  // the peer's stages
      if (!run && __all_sync(0xffffffffu, mbar_wait<true>(counted, 0, abort_flag, p.status, false)))
        m = (int)uniform(*peer_stages);
      const int most = max(n, m);
      for (int i = min(n, m); i < most; ++i) mbar_arrive_warp(rows_full(i % kStages));
      for (int i = max(0, most - kStages); i < most; ++i)
        mbar_wait_warp(rows_full(i % kStages), (uint32_t)(i / kStages) & 1u, abort_flag, p.status, false);
    }
    for (int i = max(0, n - kStages); i < n; ++i) {
      mbar_wait_warp(q_full(i % kFulls), (uint32_t)(i / kFulls) & 1u, abort_flag, p.status, false);
      if (run) run = mbar_wait_warp(q_empty(i % kStages), (uint32_t)(i / kStages) & 1u, abort_flag, p.status);
    }
  } else if (warp == kMmaWarp) {
    if (rank == 0) {  // the whole warp, one lane elected for each MMA
      const uint64_t bdesc0 = desc_sw128(uniform(sB), 16, 1024);
      const uint32_t tm = uniform(tmem);
      constexpr uint64_t kPiece = kB / (kDeep / 64) >> 4;  // 64 of k of a stage's rows
      int b = 0, s = 0, it = 0;
      uint32_t ph = 0, sph = 0;
      bool run = true;
      for (int t = t0; run && t < total; t += dt) {
        const PairTile x = pair_tile<kSwiglu, kSub>(t, p, prefix, offs, rank);
        const int n = (int)uniform(x.n), subs = (int)uniform(x.subs);
        const uint32_t idesc = idesc_bf16_f32(256, n, false, false);
        const uint32_t idesc1 = idesc_bf16_f32(256, (int)uniform(x.n1), false, false);
        // accumulator it + j (mod 2) is free
        auto acc_wait = [&](int j) {
          run = __all_sync(0xffffffffu, mbar_wait<true>(t_empty((it + j) & 1), (((it + j) >> 1) & 1) ^ 1u,
                                                        abort_flag, p.status));
          tc_fence_after();
          return run;
        };
        if (!acc_wait(0)) break;
        const uint32_t d0 = tm + (it & 1) * kSub, d1 = tm + ((it + 1) & 1) * kSub;
        const uint32_t sub1 = (uint32_t)n * 64u >> 4;  // the second's rows in shared memory
        if constexpr (C::kAhead) {
          for (int k = 0; k < stages;) {
            const int left = stages - k;
            const int ahead = subs == 1 ? 1 : k == 0 ? min(C::kHead, left) : left <= C::kTail ? left : 1;
            int b1 = b, s1 = s;
            for (int i = 0; i < ahead; ++i) {
              run = mbar_wait2_warp(rows_full(s1), s1 < s ? sph ^ 1u : sph, c_full(b1), b1 < b ? ph ^ 1u : ph, abort_flag,
                                    p.status);
              if (!run) break;
              tc_fence_after();
#pragma unroll
              for (int h = 0; h < 2; ++h)
                umma_f16_ta_k64_warp<true>(d0, tm + kACol + b1 * 64 + h * 32, bdesc0 + (uint64_t)s1 * (kB >> 4) + h * kPiece,
                                           idesc, (uint32_t)(k + i + h > 0));
              if (++b1 == kGroups) b1 = 0;
              if (++s1 == kStages) s1 = 0;
            }
            if (!run) break;
            if (subs > 1) {
              if (k == 0 && !acc_wait(1)) break;
              if (ahead == left) umma_commit_pair_warp(t_full(it & 1), both);
            }
            for (int i = 0; i < ahead; ++i, ++k) {
              if (subs > 1) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  umma_f16_ta_k64_warp<true>(d1, tm + kACol + b * 64 + h * 32,
                                             bdesc0 + (uint64_t)s * (kB >> 4) + h * kPiece + sub1, idesc1,
                                             (uint32_t)(k + h > 0));
              }
              umma_commit_pair_warp(c_empty(b), both);
              if (++b == kGroups) b = 0, ph ^= 1u;
              umma_commit_pair_warp(q_empty(s), both);
              if (++s == kStages) s = 0, sph ^= 1u;
            }
          }
          if (!run) break;
        } else {
          if (subs > 1 && !acc_wait(1)) break;
          uint32_t accum = 0u;
          for (int k = 0; k < stages; ++k) {
            const uint64_t bd = bdesc0 + (uint64_t)s * (kB >> 4);
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
              run = q == 0 ? mbar_wait2_warp(rows_full(s), sph, c_full(b), ph, abort_flag, p.status)
                           : mbar_wait_warp(c_full(b), ph, abort_flag, p.status);
              if (!run) break;
              tc_fence_after();
              const uint32_t a = tm + kACol + b * 64;
              // (past the end of Kd both operands are zeros)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint64_t bh = bd + (uint64_t)(2 * q + h) * kPiece;
                umma_f16_ta_k64_warp<true>(d0, a + h * 32, bh, idesc, accum);
                if (subs > 1) umma_f16_ta_k64_warp<true>(d1, a + h * 32, bh + sub1, idesc1, accum);
                accum = 1u;
              }
              umma_commit_pair_warp(c_empty(b), both);
              if (++b == kGroups) b = 0, ph ^= 1u;
            }
            if (!run) break;
            umma_commit_pair_warp(q_empty(s), both);
            if (++s == kStages) s = 0, sph ^= 1u;
          }
          if (!run) break;
          if (subs > 1) umma_commit_pair_warp(t_full(it & 1), both);
        }
        umma_commit_pair_warp(t_full((it + subs - 1) & 1), both);
        it += subs;
      }
      umma_commit_pair_warp(drain, both);  // the last signal to either CTA
      mbar_wait_warp(drain, 0, abort_flag, p.status, false);
    }
  } else if (warp >= kAWarp) {
    // ---- expand: a lane takes 64 bytes of a row of the stage ----
    const int grp = (warp - kAWarp) >> 2, quarter = warp & 3;  // quarter: tensor-memory lanes
    const int team = grp / kPer, part = grp % kPer;
    // Row of this lane: gate/up stages hold 64 gate rows, then 64 up rows; a warp
    // takes 16 of each, so that gate and up of a channel meet in lanes i and
    // i + 16 of one epilogue warp.
    const int row = kSwiglu ? (lane < 16 ? quarter * 16 + lane : 48 + quarter * 16 + lane) : quarter * 32 + lane;
    // Chunk c of row r sits at chunk c ^ (r / 2 & 3) (64-byte swizzle) or c ^ (r & 7).
    const uint32_t src0 = sA + row * (kDeep / 2) +
                          (kDeep == 128 ? ((row >> 1) & 3) << 4 : ((row & 7) ^ (4 * part)) << 4);
    // its scales: 64 (128) channels of the first group, of the second, ...
    const int up = kSwiglu && row >= 64;
    constexpr uint32_t kScaleRow = kSwiglu ? 128 : 256;
    const int shift = p.group == 32 ? 0 : p.group == 64 ? 1 : 2;  // chunks of 32 inputs to groups
    const uint32_t sc0 = sS + (up ? kDeep / p.group * 128 : 0) + (row - (up ? 64 : 0)) * 2;
    const uint32_t dst = tmem + kACol + grp * 64 + ((uint32_t)(quarter * 32) << 16);
    const uint32_t full_of_leader = mapa_shared(c_full(grp), leader);
    const uint32_t mask = int4_mask();
    int s = team, f = team, n0 = 0;  // slot, its barrier; stages before this tile (mod kTeams)
    uint32_t ph = 0, bph = 0;
    bool run = true;
    for (int t = t0; run && t < total; t += dt) {
      for (int k = (team - n0 + kTeams) % kTeams; k < stages; k += kTeams) {
        run = mbar_wait_warp(q_full(f), ph, abort_flag, p.status);
        if (!run) break;
        uint4 v[4];
        uint32_t sc[4], r[32];
        const uint32_t src = src0 + s * kA, scs = sc0 + s * kS;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = ld_shared_v4(src ^ (j << 4));
          sc[j] = ld_shared_u16(scs + ((4 * part + j) >> shift) * kScaleRow);
        }
        expand_int4_row(v[0], sc[0], mask, r);
        expand_int4_row(v[1], sc[1], mask, r + 16);
        // The row and its scales are read: the fence orders these reads before
        // the copy that refills the slot.
        fence_proxy_async_smem();
        mbar_arrive_warp(q_empty(s));
        run = mbar_wait_warp(c_empty(grp), bph ^ 1u, abort_flag, p.status);
        if (!run) break;
        tc_fence_after();
        tmem_st_32x32b_x32(dst, r);
        expand_int4_row(v[2], sc[2], mask, r);
        expand_int4_row(v[3], sc[3], mask, r + 16);
        tmem_st_32x32b_x32(dst + 32, r);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_cluster_warp(full_of_leader);
        bph ^= 1u;
        s += kTeams;
        if (s >= kStages) s -= kStages;
        f += kTeams;
        if (f >= kFulls) f -= kFulls, ph ^= 1u;
      }
      n0 = (n0 + stages) % kTeams;
    }
    // the last of the leader's signals to this CTA's barriers has arrived
    if (run) mbar_wait_warp(c_empty(grp), bph ^ 1u, abort_flag, p.status);
  } else {
    auto go = [&](auto&& split) {
      pair_epilogue<C, kSwiglu, false, O>(p, base, g, tmem, warp, lane, rank, leader, t0, dt, total, t_full(0),
                                          t_empty(0), abort_flag, prefix, offs, split);
    };
    if constexpr (C::kSplit > 1)
      go(SplitTile<C>{base + C::kParts, part_full, part_empty, pair, rank, lane, warp & 3, abort_flag, p.status});
    else
      go(WholeTile());
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

constexpr int kNoRoom = -1;  // more tiles than clusters that can be resident

template <typename C, bool kSwiglu, typename O>
int launch_cfg(const CUtensorMap (&m)[6], const I4Params& p, long long tiles, cudaStream_t s) {
  static PerDevice smem_allowed, resident;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const int allowed = smem_allowed.get(dev, [] {
    return cudaFuncSetAttribute(gmm_i4_kernel<C, kSwiglu, O>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::kSmem) == cudaSuccess;
  });
  if (!allowed) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2 * C::kSplit;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  // one persistent CTA per SM, as many whole clusters as can be resident
  constexpr int kCluster = 2 * C::kSplit;
  cfg.gridDim = dim3(sm_count() / kCluster * kCluster, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const int clusters = resident.get(dev, [&] {
    int n = 0;
    const bool known = cudaOccupancyMaxActiveClusters(&n, gmm_i4_kernel<C, kSwiglu, O>, &cfg) == cudaSuccess;
    (void)cudaGetLastError();
    return known && n > 0 ? n : INT_MAX;
  });
  if (clusters < (int)cfg.gridDim.x / kCluster) cfg.gridDim.x = kCluster * clusters;
  // tiles: at most that many, or not known
  if (C::kSplit > 1 && tiles > (int)cfg.gridDim.x / kCluster) return kNoRoom;
  if (cudaLaunchKernelEx(&cfg, gmm_i4_kernel<C, kSwiglu, O>, m[0], m[1], m[2], m[3], m[4], m[5], p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  count_launches(1);
  return MOE_OK;
}

// Rows per expert, on average, up to which a form runs (the routing itself is not
// known on the host).  Tiles of one accumulator hold few enough rows that a slot
// has room for more or longer stages, and the epilogue overlaps the next tile;
// experts of more rows than it takes have their weights expanded again for each
// tile.  GB300, random routing, gate/up and down, us, I4Few, I4To80, I4To128, I4Many:
//   rows  E=128 H=2048 I=768                    E=128 H=4096 I=1536
//     24  63+41  --     71+41   85+51          209+113  --       242+131  301+159
//     40  69+45  71+45  77+45   89+53          223+125  242+132  264+140  311+164
//     64  --     75+47  81+48   93+56            --     251+137  277+145  323+169
//     96  --     81+49  85+50   97+60            --     269+146  291+154  339+176
//    128  --    108+66  92+53  102+62            --     387+216  312+171  351+185
//    160  --     --    118+70  110+68            --      --      455+241  391+212
// and with experts' shares as 1 / sqrt(rank), E=128 H=2048 I=768:
//     48  77+51  --     79+46   92+55      (40: 73+48  72+45  77+45  91+54)
//     64  --     77+49  82+49   95+57
//     96  --     91+57  92+55  101+61
//    128  --    104+64 103+60  109+67
//    160  --     --    112+68  111+73
// Rows on few of the experts are the most that choosing by the average costs, and
// take less than the same rows spread evenly: E=128 H=2048 I=768, all rows on 4 of
// them, the form chosen and I4Many: 16 rows an expert 24+18 17+12, 40 rows 47+31
// 32+18, 64 rows 46+28 44+23, 100 rows 61+37 58+33.
constexpr long long kFewRows = 40, kRowsTo80 = 80, kRowsTo128 = 128;

struct I4Call {
  const void *x, *W0, *s0, *W1, *s1;
  int group;
};

template <typename C, bool kSwiglu, typename O>
int launch_maps(const I4Call& c, I4Params p, long long tiles, cudaStream_t s) {
  CUtensorMap m[6];
  const uint32_t ch = kSwiglu ? 64 : 128;
  const uint64_t dw[3] = {(uint64_t)p.Kd / 2, (uint64_t)p.Nout, (uint64_t)p.E};
  const uint32_t bw[3] = {C::kDeep / 2, ch, 1};
  const uint64_t ds[3] = {(uint64_t)p.Nout, (uint64_t)(p.Kd / c.group), (uint64_t)p.E};
  const uint32_t bs[3] = {ch, (uint32_t)(C::kDeep / c.group), 1};
  const uint64_t dx[2] = {(uint64_t)p.Kd, (uint64_t)p.N};
  const uint32_t b32[2] = {64, 32}, b16[2] = {64, 16};
  const CUtensorMapSwizzle swizzle = C::kDeep == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!make_map(&m[0], c.W0, 1, 3, dw, bw, swizzle) ||
      !make_map(&m[1], kSwiglu ? c.W1 : c.W0, 1, 3, dw, bw, swizzle) ||
      !make_map(&m[2], c.s0, 2, 3, ds, bs, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map(&m[3], kSwiglu ? c.s1 : c.s0, 2, 3, ds, bs, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map_sw128(&m[4], c.x, 2, 2, dx, b32) || !make_map_sw128(&m[5], c.x, 2, 2, dx, b16))
    return MOE_ERR_CUDA;
  return launch_cfg<C, kSwiglu, O>(m, p, tiles, s);
}

template <bool kSwiglu, typename O>
int launch_i4(const void* x, const uint8_t* W0, const void* s0, const uint8_t* W1, const void* s1,
              const int32_t* off, int N, int Kd, int Nout, int E, int group, O* out, int32_t* status,
              cudaStream_t s) {
  if (int rc = device_ok()) return rc;
  const int chs = kSwiglu ? 128 : 256;
  const I4Params p{off, out, status, N, E, Kd, Nout, (Nout + chs - 1) / chs, group};
  const I4Call c{x, W0, s0, W1, s1, group};
  // The tiles of 64 rows that there can be: one for every 64 rows, and one more for
  // every expert with rows.
  const long long tiles = (E == 1 ? (N - 1) / 64 + 1 : (long long)(N < E ? N : E) + N / 64) * p.ch_tiles;
  // The few-rows form too where each of its tiles has a pair of its own: smaller
  // tiles are more SMs then (256 rows, 2048 inputs, 4096 channels 16.2 -> 11.7 us).
  if (N > kFewRows * E && tiles > sm_count() / 2) {
    if (N > kRowsTo128 * E) return launch_maps<I4Many, kSwiglu, O>(c, p, 0, s);
    if (N > kRowsTo80 * E) return launch_maps<I4To128, kSwiglu, O>(c, p, 0, s);
    return launch_maps<I4To80, kSwiglu, O>(c, p, 0, s);
  }
  // Two pairs share a tile where all of them have a cluster of their own: 19 rows,
  // 4096 channels, with 4096 inputs 14.4 -> 11.7 us, 2048 10.2 -> 9.6, 1024 8.2 -> 8.6.
  // (Four pairs: 10.5 us for 1024 channels, 11.6 with two; of their clusters fewer than 16
  // can be resident.)
  int rc = kNoRoom;
  if (Kd >= 2048 && tiles <= sm_count() / 4) rc = launch_maps<I4Split2, kSwiglu, O>(c, p, tiles, s);
  return rc == kNoRoom ? launch_maps<I4Few, kSwiglu, O>(c, p, tiles, s) : rc;
}

int check_i4(const void* x, const int32_t* off, int N, int H, int I, int E, int Kd, int group) {
  if (N < 0 || H <= 0 || I <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts) return MOE_ERR_SHAPE;
  if (off == nullptr && E != 1) return MOE_ERR_INVALID_ARG;
  if (H % 64 || I % 64 || Kd % group || H > MOE_INT4_MAX_SIZE || I > MOE_INT4_MAX_SIZE) return MOE_ERR_SHAPE;
  if (N > MOE_INT8_MAX_ROWS) return MOE_ERR_SHAPE;  // (rows and row tiles added up stay within 31 bits)
  if (N > 0 && (!x || !aligned16(x))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace
}  // namespace tc
}  // namespace moe

using namespace moe;
using namespace moe::tc;

extern "C" int moe_gate_up_swiglu_int4(const void* permuted, const int32_t* expert_offsets, int N, int H,
                                       int I, int E, int group, const uint8_t* W_gate_q,
                                       const void* gate_scale, const uint8_t* W_up_q,
                                       const void* up_scale, void* act, int32_t* dev_status,
                                       cudaStream_t stream) {
  if (int rc = check_i4(permuted, expert_offsets, N, H, I, E, H, group)) return rc;
  if (N == 0) return MOE_OK;
  const void* ptrs[] = {W_gate_q, gate_scale, W_up_q, up_scale, act};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  return launch_i4<true>(permuted, W_gate_q, gate_scale, W_up_q, up_scale, expert_offsets, N, H, I, E, group,
                         static_cast<__nv_bfloat16*>(act), dev_status, stream);
}

extern "C" int moe_down_proj_int4(const void* act, const int32_t* expert_offsets, int N, int H, int I,
                                  int E, int group, const uint8_t* W_down_q, const void* down_scale,
                                  void* expanded, int out_dtype, int32_t* dev_status,
                                  cudaStream_t stream) {
  if (int rc = check_i4(act, expert_offsets, N, H, I, E, I, group)) return rc;
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (N == 0) return MOE_OK;
  const void* ptrs[] = {W_down_q, down_scale, expanded};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (out_dtype == MOE_F32)
    return launch_i4<false>(act, W_down_q, down_scale, nullptr, nullptr, expert_offsets, N, I, H, E, group,
                            static_cast<float*>(expanded), dev_status, stream);
  return launch_i4<false>(act, W_down_q, down_scale, nullptr, nullptr, expert_offsets, N, I, H, E, group,
                          static_cast<__nv_bfloat16*>(expanded), dev_status, stream);
}
