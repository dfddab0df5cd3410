// The whole expert layer for T <= 64 tokens, in one kernel (16-, 8- and 4-bit
// weights).
//
//   act[a, t, :] = silu(Wg[e_a] x_t) * (Wu[e_a] x_t)      (phase 1)
//   out[t]       = shared[t] + sum_a p(t, a) Wd[e_a] act[a, t, :]   (phase 2)
//
// over the experts e_a that some token chose.  The floor is one read of those
// experts' weights, so the kernel is a stream of weights that does not pause:
//
//   * one CTA per SM, and each phase's weights cut into equal runs of 32 KB
//     units (128 bytes of k of 128 gate and 128 up rows, or of 256 down rows):
//     CTA c takes units [U c / G, U (c + 1) / G), whatever tiles they fall in,
//     so all SMs read the same amount.  A tile that several CTAs share is
//     summed from their fp32 partials in the order of the CTAs: in phase 1 by
//     the one that finishes last, in phase 2 each of them sums a share of the
//     tile when all have finished;
//   * the weights are the A operand (M = 128 of their rows), the tokens the B
//     operand (N = 16, 32 or 64): every active expert is multiplied with all
//     tokens, which the tensor cores have time for (at N = 64 they are busy 16 %
//     of the time with bf16 weights, 24 % with 8-bit ones), and a (token,
//     expert) pair that was not chosen is left out when the result is read;
//   * one warp streams weights through a ring of 3 to 5 stages (TMA) without
//     ever waiting for results: at the turn from phase 1 to phase 2 it fills
//     the ring with down weights while the last activations are still being
//     made.  Another warp loads the tokens' and activations' tiles and alone
//     waits for an expert's activations to be complete.  For up to 16 tokens and
//     16- or 4-bit weights phase 1 may take narrow tiles: 64 gate and 64 up rows
//     in each of two k blocks;
//   * 8-bit weights go from the ring through registers to tensor memory as
//     bf16 (exact) and are the A operand there; the scale of a channel is a
//     lane's own factor in the epilogue;
//   * 4-bit weights go the same way, 256 of k in a unit of the same bytes, each
//     multiplied by its group's scale as it is expanded (exact for scales of five
//     significant bits).  The scales come by TMA beside their weights.  The tokens'
//     tiles have a ring of their own, 128 of k in a slot, so that a stage is free as
//     soon as it is expanded.
//
// CTAs wait for one another, so the launch is cooperative (all of it
// resident); every wait is bounded.  The counters are zeroed by the kernel
// itself: each CTA clears its share and then sets its flag to a tag made from
// the workspace's epoch word; a CTA counts only after it has seen all flags.
// The last CTA to have seen them zeroes the flags and opens the next epoch, so
// a call leaves no tag behind: whatever else uses the workspace's memory
// between two calls, and whichever words of it that changes, the next call
// finds flags that match its tag only when its own CTAs set them.  Nothing has
// to be cleared, neither before the first call nor between the replays of a
// graph.  (Flags left in place would match as soon as something wrote the epoch
// word back, a small tensor in the same memory for one.  Counters that carried
// the tag themselves, changed by compare-and-swap, need no flags, but 152 CTAs
// retrying on one word cost 75 us.)
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "int4.cuh"
#include "per_device.h"
#include "tc_warp.cuh"
#include "tma_host.cuh"

namespace moe {
namespace tc {
namespace {

constexpr int kMaxCtas = 160;
constexpr int kMaxSlots = MOE_FEW_TOKENS * kMaxK;
constexpr uint32_t kBox16 = 128 * 128;  // bytes of a weight box: 128 rows of 128 bytes

struct FewParams {
  const int32_t* ids;
  const float* probs;
  const uint8_t* mask;
  const float *gs, *us, *ds;
  const __nv_bfloat16* shared_x;
  __nv_bfloat16* out;
  __nv_bfloat16* act;          // [A, T, I]; 4-bit weights: [A, 2, T, I]
  float *part1, *part2;        // [CTA][2][T][2][128], [CTA][2][T][256]
  unsigned long long* epoch;   // epoch, flag of each CTA
  uint32_t* count;             // ready[A], tiles of phase 1, tiles of phase 2, seen
  int32_t* status;
  int mask_dims, T, H, K, I, E, E_all, A_max;
  int per1, per2;  // 4-bit weights: scale groups of a unit in each phase, 8, 4, 2
};

template <int NP, int BITS>
struct FewTraits {
  static constexpr int k = 1024 / BITS;                  // k of a unit
  static constexpr uint32_t b_box = NP * 128;            // 64 k of the tokens
  static constexpr bool can_narrow = NP == 16 && BITS != 8;  // (see narrow below)
  static constexpr int b_boxes = (can_narrow ? 2 : 1) * k / 64;
  // A stage: a unit's weights, and the tokens' rows or (4-bit) two tiles' scales.
  static constexpr uint32_t scales = 2 * kBox16;
  static constexpr uint32_t stage = scales + (BITS == 4 ? 2 * 8 * 256 : b_boxes * b_box);
  // 4-bit weights, the tokens' ring: a slot holds the rows for 128 of expanded k, two
  // boxes, each twice (a narrow tile's two k blocks, the activations' two halves).
  static constexpr uint32_t slot = 4 * b_box;
  static constexpr int slots = BITS != 4 ? 0 : NP == 64 ? 3 : NP == 32 ? 4 : 5;
  static constexpr int stages = (int)((212992 - slots * slot) / stage);  // 5; 4 for N = 64 with 8-bit weights; 4, 4, 3 with 4-bit
  // Warps that expand, and the buffers of 128 expanded k (128 columns of tensor
  // memory) that they fill in turn.  4-bit weights: twice the warps where registers
  // have room, a third buffer where tensor memory has it (17 to 32 tokens give it to
  // the halves side by side: 32 tokens 85 us, one after the other 87).
  static constexpr int expand = BITS == 4 && NP <= 32 ? 16 : 8;
  static constexpr int bufs = BITS == 4 && NP <= 16 ? 3 : 2;
  static constexpr int threads = (12 + (BITS == 16 ? 0 : expand)) * 32;
  // Warps that issue MMAs: with 4-bit weights one for each of a unit's two boxes.
  static constexpr int issuers = BITS == 4 ? 2 : 1;
  // The activations' two halves as one B operand, their sums in columns of their own.
  static constexpr bool side = BITS == 4 && NP <= 32;
  static constexpr int dn = side ? 2 * NP : NP;            // columns of a box's sums
  static constexpr int bars = 2 * stages + 4 + 2 * bufs + 2 + 2 * slots;
  static constexpr uint32_t ring2 = stages * stage;       // 4-bit: the tokens' slots
  static constexpr uint32_t ctrl = ring2 + slots * slot;
  static constexpr uint32_t holder = ctrl + 8 * bars;     // tensor memory, abort, flag, A
  static constexpr uint32_t bitmap = holder + 16;          // 32 words
  static constexpr uint32_t issued = bitmap + 128;        // stages filled by warps 0 and 10
  static constexpr uint32_t list = issued + 16;            // active experts
  static constexpr uint32_t expert = list + 2 * kMaxSlots;  // of each (token, slot)
  static constexpr uint32_t prob = expert + 2 * kMaxSlots;
  static constexpr uint32_t cross = prob + 4 * kMaxSlots;  // up values of a narrow tile [16][64]
  static constexpr uint32_t smem = cross + (can_narrow ? 4096 : 0) + 1024;
  static_assert(smem <= 232448, "more shared memory than one CTA may use");
};

// The U units of a phase are shared by G = min(CTAs, U) CTAs, so that each of
// those has one at least.  First unit of CTA c:
__device__ __forceinline__ int first_unit(int U, int c, int G) { return (int)((long long)U * c / G); }

// CTA whose run holds unit u.
__device__ __forceinline__ int cta_of(int U, int u, int G) {
  int c = (int)((long long)u * G / U);
  while (c + 1 < G && first_unit(U, c + 1, G) <= u) ++c;
  while (first_unit(U, c, G) > u) --c;
  return c;
}

// Tile segments of a run [lo, hi) in the order they are taken: the first and
// the last, which other CTAs may share, before the whole tiles between them,
// so that shared tiles are put together while there is other work.
struct Segments {
  int lo, hi, KB, first, count;
  __device__ __forceinline__ Segments(int lo_, int hi_, int KB_)
      : lo(lo_), hi(hi_), KB(KB_), first(hi_ > lo_ ? lo_ / KB_ : 0),
        count(hi_ > lo_ ? (hi_ - 1) / KB_ - lo_ / KB_ + 1 : 0) {}
  __device__ __forceinline__ void get(int i, int& tile, int& u, int& len) const {
    tile = first + (i == 0 ? 0 : i == 1 ? count - 1 : i - 1);
    u = max(lo, tile * KB);
    len = min(hi, (tile + 1) * KB) - u;
  }
};

// Tag that CTA c sets in an epoch: a multiple of 2^64 / golden ratio, which
// spreads neighbouring numbers over all 64 bits, made odd.  Zeros are no tag,
// every CTA has another, and memory that holds something else (one byte
// repeated, small integers, minus ones) holds none.
__device__ __forceinline__ unsigned long long tag_of(unsigned long long e, int c) {
  return (e + (unsigned long long)c + 1) * 0x9e3779b97f4a7c15ull | 1ull;
}

// Wait by a whole warp until ok() holds in every lane; false when the limit
// ran out or the CTA is giving up.
template <typename F>
__device__ __forceinline__ bool poll_warp(F&& ok, volatile int* abort_flag, int32_t* status) {
  unsigned long long t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xffffffffu, ok())) {
      __threadfence();
      return true;
    }
    if ((i & 31u) == 31u) {
      const unsigned long long now = globaltimer();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, *abort_flag || now - t0 > kWaitTimeoutNs)) {
        *abort_flag = 1;
        set_status(status, MOE_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// Relaxed loads for polling (an acquire load waits for the one before it); a
// fence follows the poll.
__device__ __forceinline__ unsigned long long ld_relaxed(const unsigned long long* p) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_relaxed(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Release of what this thread has seen, acquire of what earlier adders released.
__device__ __forceinline__ uint32_t add_acq_rel(uint32_t* p) {
  uint32_t v;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The epilogue warps' common decision to go on: a warp whose wait ran out
// must not leave the others in a barrier.
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\tbar.red.and.pred p, 1, 256, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// Two signed bytes of w (selected by sel) as bf16, exactly: 0x43bb is 128 + m
// or 256 + 2m for a byte of sign s and low bits m; clearing the sign bit
// leaves 128 + m, and keeping only it leaves 128 or 256.
__device__ __forceinline__ uint32_t bytes_to_bf16(uint32_t w, uint32_t sel) {
  const uint32_t t = __byte_perm(w, 0x43434343u, sel);
  const uint32_t lo = t & 0xff7fff7fu, hi = t & 0xff80ff80u;
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo),
                             *reinterpret_cast<const __nv_bfloat162*>(&hi));
  return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ void expand16_bf16(uint4 v, uint32_t* r) {
  r[0] = bytes_to_bf16(v.x, 0x4140), r[1] = bytes_to_bf16(v.x, 0x4342);
  r[2] = bytes_to_bf16(v.y, 0x4140), r[3] = bytes_to_bf16(v.y, 0x4342);
  r[4] = bytes_to_bf16(v.z, 0x4140), r[5] = bytes_to_bf16(v.z, 0x4342);
  r[6] = bytes_to_bf16(v.w, 0x4140), r[7] = bytes_to_bf16(v.w, 0x4342);
}

// act in fp32.  16- and 8-bit weights: rounded to bf16 once where it is stored, as
// the layer's other path rounds it; the second product's tensor instruction takes
// both operands in one 16-bit type, and its weights are bf16 (8-bit ones are exact
// in it).  fp16 would be finer, but act has the range of a product of two sums and
// bf16 weights are not exact in fp16.  It is the only rounding to fewer than 32 bits
// before the output's own: it moves the output by 0.0026 of its norm (T=64 H=2048
// E=128 K=8 I=768; the output's own rounding is 0.0017), and from the same formula
// with that rounding the kernel is 0.0005 off, the roundings that fall the other way.
// 4-bit weights: two bf16, the nearest and the nearest to what it leaves, 16 bits of
// it, and the expanded weights are multiplied with both: side by side in one
// instruction where tensor memory has the columns (up to 32 tokens), else one after
// the other.  The output is then as near to the formula's as its own rounding allows
// for any number of tokens (the same case 0.0017, with one bf16 0.0023), and costs 2
// to 4 % from 9 tokens on (16 tokens H=7168 146 us against 141, 45 tokens 109 against
// 107).  The exponential and the quotient are the approximate ones, off by
// 2 + 1.16 |g| units of the 24th bit: under 2^-17 of act for |g| < 88.
__device__ __forceinline__ float swiglu(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

template <int NP, int BITS>
__global__ void __launch_bounds__(FewTraits<NP, BITS>::threads, 1)
few_tokens_kernel(const __grid_constant__ CUtensorMap mapG, const __grid_constant__ CUtensorMap mapU,
                  const __grid_constant__ CUtensorMap mapG64, const __grid_constant__ CUtensorMap mapU64,
                  const __grid_constant__ CUtensorMap mapD, const __grid_constant__ CUtensorMap mapX,
                  const __grid_constant__ CUtensorMap mapAct, const __grid_constant__ CUtensorMap mapGS,
                  const __grid_constant__ CUtensorMap mapUS, const __grid_constant__ CUtensorMap mapGS64,
                  const __grid_constant__ CUtensorMap mapUS64, const __grid_constant__ CUtensorMap mapDS,
                  const FewParams p) {
  using TR = FewTraits<NP, BITS>;
  constexpr bool I8 = BITS == 8, I4 = BITS == 4;
  constexpr int S = TR::stages;
  constexpr int kWide = BITS == 16 ? 64 : 128;  // a unit's width in the weights' maps: 128 bytes
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = uniform((raw + 1023u) & ~1023u);
  uint8_t* g = smem_raw + (base - raw);
  const uint32_t bars = base + TR::ctrl;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S + s); };
  auto t_full = [&](int a) { return bars + 8u * (2 * S + a); };
  auto t_empty = [&](int a) { return bars + 8u * (2 * S + 2 + a); };
  auto c_full = [&](int b) { return bars + 8u * (2 * S + 4 + b); };
  auto c_empty = [&](int b) { return bars + 8u * (2 * S + 4 + TR::bufs + b); };
  const uint32_t drain = bars + 8u * (2 * S + 4 + 2 * TR::bufs), clear = drain + 8u;
  auto b_full = [&](int b) { return clear + 8u + 8u * b; };
  auto b_empty = [&](int b) { return clear + 8u + 8u * (TR::slots + b); };
  uint32_t* holder = reinterpret_cast<uint32_t*>(g + TR::holder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(holder + 1);
  volatile int* flag = reinterpret_cast<volatile int*>(holder + 2);
  uint32_t* bitmap = reinterpret_cast<uint32_t*>(g + TR::bitmap);
  int16_t* list = reinterpret_cast<int16_t*>(g + TR::list);
  int16_t* slot = reinterpret_cast<int16_t*>(g + TR::expert);
  float* prob = reinterpret_cast<float*>(g + TR::prob);
  float* cross = reinterpret_cast<float*>(g + TR::cross);
  int* issued = reinterpret_cast<int*>(g + TR::issued);
  const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int TK = p.T * p.K, G = (int)gridDim.x, cta = (int)blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), I4 ? 1 : 2);      // weights, tokens
      mbar_init(empty(s), (I4 ? 0 : 1) + (BITS == 16 ? 0 : TR::expand));  // MMAs, expanding warps
    }
    for (int b = 0; b < TR::slots; ++b) {
      mbar_init(b_full(b), 1);
      mbar_init(b_empty(b), TR::issuers);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(t_full(a), TR::issuers);
      mbar_init(t_empty(a), 8);  // the epilogue warps
    }
    for (int b = 0; b < TR::bufs; ++b) {
      mbar_init(c_full(b), TR::expand);
      mbar_init(c_empty(b), TR::issuers);
    }
    mbar_init(drain, TR::issuers);
    mbar_init(clear, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&mapG);
    tma_prefetch_desc(&mapU);
    if (TR::can_narrow) {
      tma_prefetch_desc(&mapG64);
      tma_prefetch_desc(&mapU64);
    }
    tma_prefetch_desc(&mapD);
    tma_prefetch_desc(&mapX);
    tma_prefetch_desc(&mapAct);
    if (I4) {
      tma_prefetch_desc(&mapGS);
      tma_prefetch_desc(&mapUS);
      tma_prefetch_desc(&mapDS);
      if (TR::can_narrow) {
        tma_prefetch_desc(&mapGS64);
        tma_prefetch_desc(&mapUS64);
      }
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(holder), 512);
    tmem_relinquish();
  }
  // this CTA's share of the counters, then its flag
  const unsigned long long epoch = *p.epoch;
  const int n_count = p.A_max + p.A_max * ((p.I + 127) / 128) + (p.H + 255) / 256 + 1;
  for (int i = cta * TR::threads + threadIdx.x; i < n_count; i += G * TR::threads) p.count[i] = 0u;
  // the slots' experts, and the experts that some slot chose, in order
  if (threadIdx.x < 32) bitmap[threadIdx.x] = 0u;
  __syncthreads();
  int32_t* ids = reinterpret_cast<int32_t*>(g);  // (in the ring, which is not in use yet)
  for (int f = threadIdx.x; f < TK; f += TR::threads) {
    ids[f] = p.ids[f];
    prob[f] = p.probs[f];
    slot[f] = p.mask == nullptr ? 1 : p.mask[p.mask_dims == 1 ? f / p.K : f];
  }
  __syncthreads();
  for (int f = threadIdx.x; f < TK; f += TR::threads) {
    // -1: a slot that adds nothing (inactive, special, out of range or repeated)
    const int k = f % p.K;
    int e = ids[f];
    bool bad = e < 0 || e >= p.E_all;
    for (int j = 1; j <= k; ++j) bad |= ids[f - j] == e;
    if (bad && cta == 0) set_status(p.status, MOE_ERR_BAD_ID);
    if (bad || slot[f] == 0 || e >= p.E) e = -1;
    slot[f] = (int16_t)e;
    if (e >= 0) atomicOr(&bitmap[e >> 5], 1u << (e & 31));
  }
  fence_proxy_async_smem();  // (before TMA writes where the ids were)
  __syncthreads();
  if (threadIdx.x == 32)
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p.epoch + 1 + cta), "l"(tag_of(epoch, cta))
                 : "memory");
  if (warp == 0) {
    const int n = __popc(bitmap[lane]);
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    int a = incl - n;
    for (uint32_t w = bitmap[lane]; w != 0u; w &= w - 1) list[a++] = (int16_t)(lane * 32 + __ffs(w) - 1);
    if (lane == 31) holder[3] = (uint32_t)incl;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(holder[0]);
  const int A = (int)uniform(holder[3]);
  // Phase 1, when a CTA has at most one tile: whole tiles, one CTA each, need no
  // partial sums (8 us of stores, counts and loads at the end of the phase),
  // but only as many CTAs stream as there are tiles, each at up to 60 GB/s
  // against 6.7 TB/s for all.  For N = 16 also in tiles of 64 columns (gate and
  // up rows together one A operand of 128).  T=1 H=2048 E=128 K=8 I=768: 96
  // whole narrow tiles 32.8 us, 48 tiles in 152 equal runs 35.8 us (from cold).
  const int wide1 = (p.I + 127) / 128, bytes1 = 32 * p.H * BITS;  // of a wide tile
  // (4-bit weights: 30 GB/s of a CTA and 4.1 TB/s of all, the rate of their expansion)
  constexpr int r_all = I4 ? 4100 : 6550, r_one = I4 ? 30000 : 60000;
  const int t_split = A * wide1 * (bytes1 / 1024) / r_all + 8;             // us
  const int t_whole = A * wide1 <= G ? bytes1 / r_one : t_split + 1;
  const int t_narrow = TR::can_narrow && A * (p.I / 64) <= G ? bytes1 / (2 * r_one) : t_split + 1;
  const bool narrow = t_narrow <= t_split && t_narrow < t_whole;
  const int rows1 = narrow ? 64 : 128;
  const int nt1 = (p.I + rows1 - 1) / rows1, nt2 = (p.H + 255) / 256;
  const int k1 = narrow ? 2 * TR::k : TR::k;  // k of a unit of phase 1
  const int KB1 = (p.H + k1 - 1) / k1, KB2 = (p.I + TR::k - 1) / TR::k;
  const int U1 = A * nt1 * KB1, U2 = nt2 * A * KB2;
  const int G1 = narrow || t_whole <= t_split ? A * nt1 : min(G, U1), G2 = min(G, U2);
  const int lo1 = cta < G1 ? first_unit(U1, cta, G1) : 0, hi1 = cta < G1 ? first_unit(U1, cta + 1, G1) : 0;
  const int lo2 = cta < G2 ? first_unit(U2, cta, G2) : 0, hi2 = cta < G2 ? first_unit(U2, cta + 1, G2) : 0;
  const Segments seg1(lo1, hi1, KB1);
  uint32_t* ready = p.count;
  uint32_t* cnt1 = ready + p.A_max;
  uint32_t* cnt2 = cnt1 + (size_t)p.A_max * wide1;
  uint32_t* seen = p.count + n_count - 1;
  unsigned long long* flags = p.epoch + 1;

  // One warp waits until every CTA's counters are clear (and every CTA has read
  // the epoch), while the first weights are under way.  Then it counts itself
  // among those that need the flags no more.
  if (warp == 11) {
    const bool ok = poll_warp([&]() {
      unsigned long long w[(kMaxCtas + 31) / 32];
#pragma unroll
      for (int i = 0; i < (kMaxCtas + 31) / 32; ++i)
        w[i] = lane + 32 * i < G ? ld_relaxed(flags + lane + 32 * i) : 0ull;
      bool all = true;
#pragma unroll
      for (int i = 0; i < (kMaxCtas + 31) / 32; ++i)
        all &= lane + 32 * i >= G || w[i] == tag_of(epoch, lane + 32 * i);
      return all;
    }, abort_flag, p.status);
    if (ok) {
      mbar_arrive_warp(clear);
      const uint32_t before = uniform(lane == 0 ? add_acq_rel(seen) : 0u);
      if (before == (uint32_t)G - 1) {
        for (int i = lane; i < G; i += 32) flags[i] = 0ull;
        if (lane == 0) *p.epoch = epoch + 1;
      }
    } else if (lane == 0) {  // (flags of a call that ran out stay, under an epoch that is over)
      *p.epoch = epoch + 1;
    }
  }

  if (A == 0) {
    for (int i = cta * TR::threads + threadIdx.x; i < p.T * p.H; i += G * TR::threads)
      p.out[i] = p.shared_x ? p.shared_x[i] : __float2bfloat16_rn(0.f);
  }

  // The end of the two loading warps (w: 0 weights, 1 tokens; n stages filled):
  // every copy has landed before the CTA may exit.  When a wait ran out they
  // may have stopped at different stages; each arrives for those that only the
  // other filled, so that their barriers complete.
  auto drain_ring = [&](int w, int n) {
    if constexpr (I4) {  // (each has a ring of its own)
      const int size = w == 0 ? S : TR::slots;
      for (int i = max(0, n - size); i < n; ++i)
        mbar_wait_warp(w == 0 ? full(i % size) : b_full(i % size), (uint32_t)(i / size) & 1u, abort_flag, p.status, false);
      return;
    }
    if (lane == 0) issued[w] = n;
    asm volatile("bar.sync 2, 64;" ::: "memory");
    const int other = issued[w ^ 1], all = max(n, other);
    for (int i = n; i < other; ++i) mbar_arrive_warp(full(i % S));
    for (int i = max(0, all - S); i < all; ++i)
      mbar_wait_warp(full(i % S), (uint32_t)(i / S) & 1u, abort_flag, p.status, false);
  };

  if (warp == 0) {
    // ---------------- weights: the whole warp, one lane elected for each copy ----------------
    int s = 0, n = 0;
    uint32_t ph = 0;
    bool run = true;
    auto next = [&]() {
      ++n;
      if (++s == S) s = 0, ph ^= 1u;
    };
    for (int i = 0; run && i < seg1.count; ++i) {
      int tile, u, len;
      seg1.get(i, tile, u, len);
      const int kb = u - tile * KB1, e = (int)uniform(list[tile / nt1]);
      const int i0 = (tile % nt1) * rows1;
      for (int k = kb; k < kb + len; ++k) {
        run = mbar_wait_warp(empty(s), ph ^ 1u, abort_flag, p.status);
        if (!run) break;
        const uint32_t a = base + s * TR::stage;
        mbar_arrive_expect_tx_warp(full(s), 2 * kBox16 + (I4 ? 512u * p.per1 : 0u));
        if (I4 && narrow) {  // of each k block: 64 gate channels, 64 up channels
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sc = a + TR::scales + 256 * p.per1 * h;
            tma_load_3d_warp(sc, &mapGS64, full(s), i0, (2 * k + h) * p.per1, e);
            tma_load_3d_warp(sc + 128 * p.per1, &mapUS64, full(s), i0, (2 * k + h) * p.per1, e);
          }
        } else if (I4) {
          tma_load_3d_warp(a + TR::scales, &mapGS, full(s), i0, k * p.per1, e);
          tma_load_3d_warp(a + TR::scales + 256 * p.per1, &mapUS, full(s), i0, k * p.per1, e);
        }
        if (narrow) {  // 64 rows of each, two k blocks
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tma_load_3d_warp(a + h * kBox16, &mapG64, full(s), (2 * k + h) * kWide, i0, e);
            tma_load_3d_warp(a + h * kBox16 + kBox16 / 2, &mapU64, full(s), (2 * k + h) * kWide, i0, e);
          }
        } else {
          tma_load_3d_warp(a, &mapG, full(s), k * kWide, i0, e);
          tma_load_3d_warp(a + kBox16, &mapU, full(s), k * kWide, i0, e);
        }
        next();
      }
    }
    for (int u = lo2; run && u < hi2;) {
      const int ta = u / KB2, kb = u - ta * KB2, len = min(KB2 - kb, hi2 - u);
      const int e = (int)uniform(list[ta % A]), h0 = (ta / A) * 256;
      for (int k = kb; k < kb + len; ++k) {
        run = mbar_wait_warp(empty(s), ph ^ 1u, abort_flag, p.status);
        if (!run) break;
        const uint32_t a = base + s * TR::stage;
        mbar_arrive_expect_tx_warp(full(s), 2 * kBox16 + (I4 ? 512u * p.per2 : 0u));
        if constexpr (I4) {
          tma_load_3d_warp(a + TR::scales, &mapDS, full(s), h0, k * p.per2, e);
          tma_load_3d_warp(a + TR::scales + 256 * p.per2, &mapDS, full(s), h0 + 128, k * p.per2, e);
        }
        tma_load_3d_warp(a, &mapD, full(s), k * kWide, h0, e);
        tma_load_3d_warp(a + kBox16, &mapD, full(s), k * kWide, h0 + 128, e);
        next();
      }
      u += len;
    }
    drain_ring(0, n);
  } else if (warp == 10) {
    // ---------------- tokens, activations ----------------
    int s = 0, n = 0;
    uint32_t ph = 0;
    bool run = true;
    auto next = [&]() {
      ++n;
      if (++s == (I4 ? TR::slots : S)) s = 0, ph ^= 1u;
    };
    for (int i = 0; run && i < seg1.count; ++i) {
     int tile, u, len;
     seg1.get(i, tile, u, len);
     for (int k = u - tile * KB1; len > 0; ++k, --len) {
      if constexpr (I4) {  // (of a narrow tile's k blocks the same 128 k in turn)
        const int k0 = k * k1, boxes = narrow ? 2 : 1;
#pragma unroll
        for (int q = 0; q < 2 && run; ++q) {
          if (!(run = mbar_wait_warp(b_empty(s), ph ^ 1u, abort_flag, p.status))) break;
          const uint32_t b = base + TR::ring2 + s * TR::slot;
          mbar_arrive_expect_tx_warp(b_full(s), 2 * boxes * TR::b_box);
          for (int h = 0; h < 2 * boxes; ++h)
            tma_load_2d_warp(b + (2 * (h & 1) + (h >> 1)) * TR::b_box, &mapX, b_full(s),
                             k0 + (h >> 1) * TR::k + q * 128 + (h & 1) * 64, 0);
          next();
        }
        if (!run) break;
        continue;
      }
      if (!(run = mbar_wait_warp(empty(s), ph ^ 1u, abort_flag, p.status))) break;
      const uint32_t b = base + s * TR::stage + 2 * kBox16;
      const int boxes = k1 / 64;
      mbar_arrive_expect_tx_warp(full(s), boxes * TR::b_box);
      for (int q = 0; q < boxes; ++q) tma_load_2d_warp(b + q * TR::b_box, &mapX, full(s), k * k1 + q * 64, 0);
      next();
     }
    }
    if (run) run = mbar_wait_warp(clear, 0, abort_flag, p.status);
    int seen = -1, checked = 0;  // last expert; experts known to be complete
    for (int u = lo2; run && u < hi2; ++u) {
      const int ta = u / KB2, k = u - ta * KB2, a = ta % A;
      if (a != seen && checked < A) {  // (the experts come round in order)
        run = poll_warp([&]() { return ld_relaxed(ready + a) == (uint32_t)nt1; }, abort_flag, p.status);
        if (!run) break;
        asm volatile("fence.proxy.async.global;" ::: "memory");  // (before the copies read them)
        seen = a;
        ++checked;
      }
      if constexpr (I4) {  // 128 k of either half
#pragma unroll
        for (int q = 0; q < 2 && run; ++q) {
          if (!(run = mbar_wait_warp(b_empty(s), ph ^ 1u, abort_flag, p.status))) break;
          const uint32_t b = base + TR::ring2 + s * TR::slot;
          mbar_arrive_expect_tx_warp(b_full(s), 4 * TR::b_box);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_3d_warp(b + 2 * h * TR::b_box, &mapAct, b_full(s), k * TR::k + q * 128 + h * 64, 0, 2 * a);
          next();
        }
        if (!run) break;
        continue;
      }
      if (!(run = mbar_wait_warp(empty(s), ph ^ 1u, abort_flag, p.status))) break;
      const uint32_t b = base + s * TR::stage + 2 * kBox16;
      mbar_arrive_expect_tx_warp(full(s), TR::k / 64 * TR::b_box);
#pragma unroll
      for (int q = 0; q < TR::k / 64; ++q)
        tma_load_3d_warp(b + q * TR::b_box, &mapAct, full(s), k * TR::k + q * 64, 0, a);
      next();
    }
    drain_ring(1, n);
  } else if (warp == 1 || (I4 && warp == 11)) {
    // ---------------- MMA: the whole warp, one lane elected for each ----------------
    // (4-bit: the unit's first box, or its second)
    const uint32_t box = warp == 1 ? 0u : 1u;
    constexpr uint32_t idesc = idesc_bf16_f32(128, NP, false, false), idesc2 = idesc_bf16_f32(128, TR::dn, false, false);
    const uint64_t d0 = desc_sw128(base, 16, 1024);
    int s = 0, c = 0, it = 0;
    uint32_t ph = 0, cph = 0;
    bool run = true;
    // one segment: len units of one tile (phase 1) or one tile and expert (phase 2)
    // (two: boxes of different rows; the first product's narrow tiles have k blocks;
    // halves: of the activations, multiplied with the same expanded weights)
    auto segment = [&](int len, bool two, bool halves) {
      const int acc = it & 1;
      run = mbar_wait_warp(t_empty(acc), ((it >> 1) & 1) ^ 1u, abort_flag, p.status);
      if (!run) return;
      tc_fence_after();
      const uint32_t d = tmem + acc * 2 * TR::dn;
      uint32_t accum = 0u;
      if constexpr (I4) {
        for (int k = 0; k < 2 * len; ++k) {  // expanded 128 of k at a time
          run = mbar_wait_warp(b_full(s), ph, abort_flag, p.status) &&
                mbar_wait_warp(c_full(c), cph, abort_flag, p.status);
          if (!run) return;
          tc_fence_after();
          const uint32_t a = tmem + 512 - 128 * TR::bufs + c * 128 + box * 64;
          // (a narrow tile's boxes are two k blocks, summed in an accumulator each)
          const uint64_t b = d0 + (TR::ring2 >> 4) + (uint64_t)s * (TR::slot >> 4) + (two ? 0u : box) * (TR::b_box >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t bh = b + 2 * h * (TR::b_box >> 4);
            umma_f16_ta_k64_warp<false>(d + box * TR::dn, a + h * 32, bh, TR::side && halves ? idesc2 : idesc, accum);
            if (!TR::side && halves)
              umma_f16_ta_k64_warp<false>(d + box * TR::dn, a + h * 32, bh + (TR::b_box >> 4), idesc, 1u);
            accum = 1u;
          }
          umma_commit_warp(c_empty(c));
          if (++c == TR::bufs) c = 0, cph ^= 1u;
          umma_commit_warp(b_empty(s));
          if (++s == TR::slots) s = 0, ph ^= 1u;
        }
        umma_commit_warp(t_full(acc));
        ++it;
        return;
      }
      for (int k = 0; k < len; ++k) {
        run = mbar_wait_warp(full(s), ph, abort_flag, p.status);
        if (!run) return;
        tc_fence_after();
        const uint64_t ad = d0 + (uint64_t)s * (TR::stage >> 4);
        const uint64_t bd = ad + (2 * kBox16 >> 4);
        if constexpr (I8) {
          run = mbar_wait_warp(c_full(c), cph, abort_flag, p.status);
          if (!run) return;
          tc_fence_after();
          const uint32_t a = tmem + 512 - 128 * TR::bufs + c * 128;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t b = bd + h * (TR::b_box >> 4);
            umma_f16_ta_k64_warp<false>(d, a + h * 32, b, idesc, accum);
            umma_f16_ta_k64_warp<false>(d + NP, a + 64 + h * 32, b, idesc, accum);
            accum = 1u;
          }
          umma_commit_warp(c_empty(c));
          if (++c == TR::bufs) c = 0, cph ^= 1u;
        } else {
          umma_f16_k64_warp(d, ad, bd, idesc, accum);
          if (two) umma_f16_k64_warp(d + NP, ad + (kBox16 >> 4), bd, idesc, accum);
          else umma_f16_k64_warp(d, ad + (kBox16 >> 4), bd + (TR::b_box >> 4), idesc, 1u);
          accum = 1u;
        }
        umma_commit_warp(empty(s));
        if (++s == S) s = 0, ph ^= 1u;
      }
      umma_commit_warp(t_full(acc));
      ++it;
    };
    for (int i = 0; run && i < seg1.count; ++i) {
      int tile, u, len;
      seg1.get(i, tile, u, len);
      segment(len, !narrow, false);
    }
    for (int u = lo2; run && u < hi2;) {
      const int len = min(KB2 - u % KB2, hi2 - u);
      segment(len, true, true);
      u += len;
    }
    umma_commit_warp(drain);
    mbar_wait_warp(drain, 0, abort_flag, p.status, false);
  } else if (warp < 10) {
    // ---------------- epilogue: lanes are weight rows, columns are tokens ----------------
    // Two warps of a lane quarter, half of the columns each.
    constexpr int NC = NP / 2;           // columns of this warp
    constexpr int CH = NC < 16 ? NC : 16;  // read at a time
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const int col0 = ((warp - 2) >> 2) * NC;
    const int T = min(p.T - col0, NC);   // tokens of this warp (none: <= 0)
    const bool lead = threadIdx.x == 64;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16) + col0;
    int it = 0;
    bool run = true;
    // Counts this CTA's part of a tile; whether it was the last one.  The
    // barrier orders every thread's partials before the one release.
    run = epi_all(mbar_wait_warp(clear, 0, abort_flag, p.status));
    auto arrive_last = [&](uint32_t* w, int pieces) {
      epi_sync();
      if (lead) *flag = add_acq_rel(w) == (uint32_t)pieces - 1;
      epi_sync();
      return *flag != 0;
    };
    for (; run && it < seg1.count; ++it) {
      int tile, u, len;
      seg1.get(it, tile, u, len);
      const int a = tile / nt1, e = list[a], i = (tile % nt1) * rows1 + (r & (rows1 - 1));
      const bool in = i < p.I;
      const int acc = it & 1;
      float gsc = 1.f, usc = 1.f;
      if (I8 && in) gsc = p.gs[(size_t)e * p.I + i], usc = p.us[(size_t)e * p.I + i];
      run = epi_all(mbar_wait_warp(t_full(acc), (it >> 1) & 1, abort_flag, p.status));
      if (!run) break;
      tc_fence_after();
      const uint32_t d = tq + acc * 2 * TR::dn;
      const bool whole = len == KB1;
      __nv_bfloat16* act = p.act + ((size_t)a * (I4 ? 2 : 1) * p.T + col0) * p.I + i;
      // act of tokens t and t + 1 (if there is one), by whole warps.  4-bit weights: a
      // bf16 and, T rows on, the bf16 of what that leaves.  Neighbouring lanes turn two
      // tokens of a channel into two channels of a token, which halves the stores
      // (45 tokens: they would add 10 us).
      auto put_act = [&](int t, float v, float w) {
        if constexpr (I4) {
          auto halves = [](float x) {
            const __nv_bfloat16 hi = __float2bfloat16_rn(x);
            const float h = __bfloat162float(hi);  // (infinite and NaN values leave nothing)
            return VecTraits<__nv_bfloat16>::pack2(h, fabsf(h) <= 3.402823466e+38f ? x - h : 0.f);
          };
          const uint32_t a = halves(v), b = halves(w);
          const bool odd = lane & 1;
          const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
          const uint32_t x = odd ? got : a, y = odd ? b : got;
          if (odd && t + 1 >= T) return;
          uint32_t* dst = reinterpret_cast<uint32_t*>(act + (size_t)(t + odd) * p.I - odd);
          dst[0] = __byte_perm(x, y, 0x5410);
          dst[(size_t)p.T * p.I / 2] = __byte_perm(x, y, 0x7632);
        } else {
          act[(size_t)t * p.I] = __float2bfloat16_rn(v);
          if (t + 1 < T) act[(size_t)(t + 1) * p.I] = __float2bfloat16_rn(w);
        }
      };
      const size_t pstride = (size_t)p.T * 256;  // floats of a partial
      float* part = p.part1 + (size_t)col0 * 256 + r;
      float* mine = part + ((size_t)cta * 2 + (u == lo1 ? 0 : 1)) * pstride;
      if constexpr (TR::can_narrow) {
        if (narrow) {  // lanes 0-63 hold gate, 64-127 up: up crosses through shared memory
          uint32_t v[8];
          tmem_ld_32x32b_x8(d, v);
          if constexpr (I4) {  // the other k block's sums
            uint32_t w[8];
            tmem_ld_32x32b_x8(d + TR::dn, w);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
          }
          tmem_ld_wait();
          float* x = cross + (size_t)col0 * 64 + (r & 63);
          if (r >= 64)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j * 64] = __uint_as_float(v[j]);
          epi_sync();
          if (r < 64)
#pragma unroll
            for (int j = 0; j < 8; j += 2)
              if (j < T)
                put_act(j, swiglu(__uint_as_float(v[j]), x[j * 64]), swiglu(__uint_as_float(v[j + 1]), x[j * 64 + 64]));
        }
      }
#pragma unroll
      for (int c0 = 0; c0 < NC; c0 += CH) {
        if (c0 >= T || narrow) break;
        uint32_t gv[CH], uv[CH];
        if constexpr (CH == 16) {
          tmem_ld_32x32b_x16(d + c0, gv);
          tmem_ld_32x32b_x16(d + TR::dn + c0, uv);
        } else {
          tmem_ld_32x32b_x8(d + c0, gv);
          tmem_ld_32x32b_x8(d + TR::dn + c0, uv);
        }
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < CH; j += 2) {
          const int t = c0 + j;
          if (t < T) {
            const float gg = __uint_as_float(gv[j]) * gsc, uu = __uint_as_float(uv[j]) * usc;
            const float g2 = __uint_as_float(gv[j + 1]) * gsc, u2 = __uint_as_float(uv[j + 1]) * usc;
            if (whole) {
              if (in) put_act(t, swiglu(gg, uu), swiglu(g2, u2));
            } else {
              mine[t * 256] = gg;
              mine[t * 256 + 128] = uu;
              if (t + 1 < T) {
                mine[t * 256 + 256] = g2;
                mine[t * 256 + 384] = u2;
              }
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive_warp(t_empty(acc));
      bool done = whole;
      if (!whole) {
        // the CTAs with a part of this tile; only the first can have begun
        // before it (its second partial then)
        const int t0 = tile * KB1, c_lo = cta_of(U1, t0, G1), c_hi = cta_of(U1, t0 + KB1 - 1, G1);
        done = arrive_last(cnt1 + tile, c_hi - c_lo + 1);
        if (done && in) {
          const float* q0 = part + ((size_t)c_lo * 2 + (first_unit(U1, c_lo, G1) < t0 ? 1 : 0)) * pstride;
          const float* q1 = part + (size_t)(c_lo + 1) * 2 * pstride;
          const int more = c_hi - c_lo;
          // 8 tokens of 2 parts at a time: their loads are in flight together
          for (int t = 0; t < T; t += 8) {
            float gg[8], uu[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              gg[j] = t + j < T ? __ldcg(q0 + (t + j) * 256) : 0.f;
              uu[j] = t + j < T ? __ldcg(q0 + (t + j) * 256 + 128) : 0.f;
            }
            for (int c = 0; c < more; c += 2) {
              float g2[2][8], u2[2][8];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float* q = q1 + (size_t)(c + k) * 2 * pstride + t * 256;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const bool on = c + k < more && t + j < T;
                  g2[k][j] = on ? __ldcg(q + j * 256) : 0.f;
                  u2[k][j] = on ? __ldcg(q + j * 256 + 128) : 0.f;
                }
              }
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) gg[j] += g2[k][j], uu[j] += u2[k][j];
            }
#pragma unroll
            for (int j = 0; j < 8; j += 2)
              if (t + j < T) put_act(t + j, swiglu(gg[j], uu[j]), swiglu(gg[j + 1], uu[j + 1]));
          }
        }
      }
      if (done) {
        asm volatile("fence.proxy.async.global;" ::: "memory");
        epi_sync();
        if (lead) (void)add_acq_rel(ready + a);
      }
    }
    // Phase 2: the two warps of a quarter take 128 of the tile's 256 rows each,
    // and all columns.
    constexpr int CP = 16;  // columns read at a time
    const int rset = (warp - 2) >> 2, r2 = rset * 128 + r;
    const uint32_t tq2 = tmem + ((uint32_t)(quarter * 32) << 16) + rset * TR::dn;
    const size_t pstride = (size_t)p.T * 256;  // floats of a partial
    const int n = A * KB2;                      // units of a tile
    auto put = [&](int t, int h, float y) {
      const size_t at = (size_t)t * p.H + h;
      if (p.shared_x) y += __bfloat162float(p.shared_x[at]);
      p.out[at] = __float2bfloat16_rn(y);
    };
    float sum[NP];
#pragma unroll
    for (int t = 0; t < NP; ++t) sum[t] = 0.f;
    for (int u = run ? lo2 : hi2; u < hi2; ++it) {
      const int ta = u / KB2, kb = u - ta * KB2, len = min(KB2 - kb, hi2 - u);
      const int tile = ta / A, a = ta - tile * A, e = list[a], h = tile * 256 + r2;
      const bool in = h < p.H;
      // the tokens that chose the expert, and their weights: lane, lane + 32
      float w0 = 0.f, w1 = 0.f;
      bool m0 = false, m1 = false;
      for (int k = 0; k < p.K; ++k) {
        if (lane < p.T && slot[lane * p.K + k] == e) m0 = true, w0 = prob[lane * p.K + k];
        if (NP > 32 && lane + 32 < p.T && slot[(lane + 32) * p.K + k] == e)
          m1 = true, w1 = prob[(lane + 32) * p.K + k];
      }
      const uint32_t b0 = __ballot_sync(0xffffffffu, m0), b1 = NP > 32 ? __ballot_sync(0xffffffffu, m1) : 0u;
      const float dsc = I8 && in ? p.ds[(size_t)e * p.H + h] : 1.f;
      const int acc = it & 1;
      // (a warp whose wait ran out still comes to the tile's barrier)
      run = run && mbar_wait_warp(t_full(acc), (it >> 1) & 1, abort_flag, p.status);
      tc_fence_after();
      const uint32_t d = tq2 + acc * 2 * TR::dn;
#pragma unroll
      for (int c0 = 0; c0 < NP; c0 += CP) {
        const uint32_t bits = ((c0 < 32 ? b0 : b1) >> (c0 & 31)) & ((1u << CP) - 1u);
        if (bits == 0u) continue;
        uint32_t v[CP];
        tmem_ld_32x32b_x16(d + c0, v);
        if constexpr (TR::side) {
#pragma unroll
          for (int q = 0; q < CP; q += 8) {
            uint32_t low[8];
            tmem_ld_32x32b_x8(d + NP + c0 + q, low);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) v[q + j] = __float_as_uint(__uint_as_float(v[q + j]) + __uint_as_float(low[j]));
          }
        }
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < CP; ++j) {
          const float w = __shfl_sync(0xffffffffu, c0 < 32 ? w0 : w1, (c0 + j) & 31);
          if ((bits >> j) & 1u) sum[c0 + j] = fmaf(w, __uint_as_float(v[j]) * dsc, sum[c0 + j]);
        }
      }
      tc_fence_before();
      mbar_arrive_warp(t_empty(acc));
      u += len;
      const int t0 = tile * n;
      if (u == t0 + n || u == hi2) {
        run = epi_all(run);
        if (!run) break;
        const bool whole = lo2 <= t0 && u == t0 + n;
        float* mine = p.part2 + ((size_t)cta * 2 + (lo2 >= t0 ? 0 : 1)) * pstride + r2;
#pragma unroll
        for (int t = 0; t < NP; ++t) {
          if (t < p.T) {
            if (!whole) mine[t * 256] = sum[t];
            else if (in) put(t, h, sum[t]);
          }
          sum[t] = 0.f;
        }
        if (!whole) {
          epi_sync();
          if (lead) (void)add_acq_rel(cnt2 + tile);
        }
      }
    }
    // Tiles that this CTA shared: its share of their sums, once all parts are
    // there.  (At most two: the first and the last of its run.)
    for (int k = 0; run && lo2 < hi2 && k < 2; ++k) {
      const int tile = k == 0 ? lo2 / n : (hi2 - 1) / n, t0 = tile * n;
      if ((k == 1 && tile == lo2 / n) || (lo2 <= t0 && hi2 >= t0 + n)) continue;
      const int c_lo = cta_of(U2, t0, G2), c_hi = cta_of(U2, t0 + n - 1, G2), parts = c_hi - c_lo + 1;
      run = epi_all(poll_warp([&]() { return ld_relaxed(cnt2 + tile) == (uint32_t)parts; }, abort_flag, p.status));
      if (!run) break;
      const float4* q0 = reinterpret_cast<const float4*>(
          p.part2 + ((size_t)c_lo * 2 + (first_unit(U2, c_lo, G2) < t0 ? 1 : 0)) * pstride);
      const float4* q1 = reinterpret_cast<const float4*>(p.part2 + (size_t)(c_lo + 1) * 2 * pstride);
      const int total = 64 * p.T, end = (int)((long long)total * (cta - c_lo + 1) / parts);
      for (int i = (int)((long long)total * (cta - c_lo) / parts) + (int)threadIdx.x - 64; i < end; i += 256) {
        float4 y = __ldcg(q0 + i);
        for (int c = 0; c < parts - 1; c += 6) {  // loads of six parts in flight
          float4 v[6];
#pragma unroll
          for (int j = 0; j < 6; ++j)
            v[j] = c + j < parts - 1 ? __ldcg(q1 + (size_t)(c + j) * (pstride / 2) + i)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 6; ++j) y.x += v[j].x, y.y += v[j].y, y.z += v[j].z, y.w += v[j].w;
        }
        const int t = i >> 6, h = tile * 256 + (i & 63) * 4;  // (H is a multiple of 64)
        if (h < p.H) {
          const size_t at = (size_t)t * p.H + h;
          if (p.shared_x) {
            const uint2 x = *reinterpret_cast<const uint2*>(p.shared_x + at);
            float f[4];
            VecTraits<__nv_bfloat16>::unpack2(x.x, f);
            VecTraits<__nv_bfloat16>::unpack2(x.y, f + 2);
            y.x += f[0], y.y += f[1], y.z += f[2], y.w += f[3];
          }
          *reinterpret_cast<uint2*>(p.out + at) = make_uint2(VecTraits<__nv_bfloat16>::pack2(y.x, y.y),
                                                             VecTraits<__nv_bfloat16>::pack2(y.z, y.w));
        }
      }
    }
  } else if (I8 && warp >= 12) {
    // ---------------- expand: 8-bit rows to bf16 in tensor memory ----------------
    // A lane takes one row of one of the unit's two boxes.
    const int quarter = warp & 3, j = (warp - 12) >> 2, r = quarter * 32 + lane;
    const uint32_t row = base + j * kBox16 + r * 128 + ((r & 7) << 4);
    const uint32_t dst = tmem + 256 + j * 64 + ((uint32_t)(quarter * 32) << 16);
    const int n = hi1 - lo1 + hi2 - lo2;
    int s = 0, c = 0;
    uint32_t ph = 0, cph = 0;
    for (int i = 0; i < n; ++i) {
      if (!mbar_wait_warp(full(s), ph, abort_flag, p.status)) break;
      const uint32_t src = row + s * TR::stage, a = dst + c * 128;
      uint4 v[4];
      uint32_t f[32];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = ld_shared_v4(src ^ (q << 4));
#pragma unroll
      for (int q = 0; q < 4; ++q) expand16_bf16(v[q], f + 8 * q);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = ld_shared_v4(src ^ ((4 + q) << 4));
      if (!mbar_wait_warp(c_empty(c), cph ^ 1u, abort_flag, p.status)) break;
      tc_fence_after();
      tmem_st_32x32b_x32(a, f);
#pragma unroll
      for (int q = 0; q < 4; ++q) expand16_bf16(v[q], f + 8 * q);
      tmem_st_32x32b_x32(a + 32, f);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_warp(c_full(c));
      mbar_arrive_warp(empty(s));
      c ^= 1;
      if (c == 0) cph ^= 1u;
      if (++s == S) s = 0, ph ^= 1u;
    }
  } else if (I4 && warp >= 12) {
    // ---------------- expand: 4-bit rows to bf16 in tensor memory ----------------
    // A lane takes one row of one of the unit's two boxes, 64 of its k at a time:
    // both quarters of a buffer's 128 k, or with 16 warps one of them.
    constexpr int kParts = TR::expand == 16 ? 1 : 2;
    const int quarter = warp & 3, j = ((warp - 12) >> 2) & 1, r = quarter * 32 + lane;
    const int part = kParts == 1 ? (warp - 12) >> 3 : 0;
    const uint32_t row = base + j * kBox16 + r * 128 + (((r & 7) ^ (2 * part)) << 4);
    const uint32_t dst = tmem + 512 - 128 * TR::bufs + j * 64 + part * 32 + ((uint32_t)(quarter * 32) << 16);
    const int n1 = hi1 - lo1, n = n1 + hi2 - lo2;
    int s = 0, c = 0;
    uint32_t ph = 0, cph = 0;
    const uint32_t mask = int4_mask();
    uint32_t sc_at = 0, sc_off[2][2 * kParts];  // where a lane's scales are in a stage
    bool run = true;
    for (int i = 0; run && i < n; ++i) {
      if (i == 0 || i == n1) {  // (a phase begins)
        const int per = i < n1 ? p.per1 : p.per2;
        const int shift = per == 8 ? 0 : per == 4 ? 1 : 2;  // chunks of 32 k to groups
        const bool half = narrow && i < n1;  // rows of 64 channels: gate's, up's
        sc_at = base + TR::scales + j * per * 256 + (half && r >= 64 ? per * 128 + (r - 64) * 2 : r * 2);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < 2 * kParts; ++q) sc_off[h][q] = ((4 * h + 2 * part + q) >> shift) << (half ? 7 : 8);
      }
      run = mbar_wait_warp(full(s), ph, abort_flag, p.status);
      if (!run) break;
      const uint32_t src = row + s * TR::stage, scs = sc_at + s * TR::stage;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f[32];
        auto expand = [&](int q) {  // two chunks: 64 of k
          const uint32_t at = src ^ (h << 6) ^ (q << 4);
          expand_int4_row(ld_shared_v4(at), ld_shared_u16(scs + sc_off[h][q]), mask, f);
          expand_int4_row(ld_shared_v4(at ^ 16), ld_shared_u16(scs + sc_off[h][q + 1]), mask, f + 16);
        };
        expand(0);
        run = mbar_wait_warp(c_empty(c), cph ^ 1u, abort_flag, p.status);
        if (!run) break;
        tc_fence_after();
        tmem_st_32x32b_x32(dst + c * 128, f);
        if constexpr (kParts == 2) {
          expand(2);
          tmem_st_32x32b_x32(dst + c * 128 + 32, f);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(c_full(c));
        if (++c == TR::bufs) c = 0, cph ^= 1u;
      }
      if (!run) break;
      mbar_arrive_warp(empty(s));
      if (++s == S) s = 0, ph ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct FewLayout {
  size_t words, counts, part1, part2, act, total;
};

// bits: of a weight.  act comes last, so that other weights' calls find everything
// else where 4-bit ones, which keep act in two bf16, have it.
FewLayout few_layout(int T, int K, int H, int I, int E, int bits) {
  const size_t A = (size_t)(T * K < E ? T * K : E);
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  FewLayout l;
  l.words = up(8 * (1 + kMaxCtas));
  l.counts = up(4 * (A + A * ((I + 127) / 128) + (H + 255) / 256 + 1));
  l.part1 = (size_t)kMaxCtas * 2 * T * 256 * 4;
  l.part2 = (size_t)kMaxCtas * 2 * T * 256 * 4;
  l.act = up(A * T * I * (bits == 4 ? 4 : 2));
  l.total = l.words + l.counts + l.part1 + l.part2 + l.act;
  return l;
}

// What the weights and their scales are: of 4-bit weights the bf16 scales (the
// others' float32 ones are in FewParams).
struct FewWeights {
  const void *gate, *up, *down, *gs, *us, *ds;
};

template <int NP, int BITS>
int launch_few(FewParams p, const void* x, const FewWeights& w, cudaStream_t s) {
  using TR = FewTraits<NP, BITS>;
  constexpr int esz = BITS == 16 ? 2 : 1, pack = BITS == 4 ? 2 : 1;
  const void *Wg = w.gate, *Wu = w.up, *Wd = w.down;
  CUtensorMap mg, mu, mg64, mu64, md, mx, ma, mgs = {}, mus = {}, mgs64 = {}, mus64 = {}, mds = {};
  const uint64_t d1[3] = {(uint64_t)p.H / pack, (uint64_t)p.I, (uint64_t)p.E};
  const uint64_t d2[3] = {(uint64_t)p.I / pack, (uint64_t)p.H, (uint64_t)p.E};
  const uint32_t bw[3] = {128 / esz, 128, 1}, bw64[3] = {128 / esz, 64, 1};
  const uint64_t dx[2] = {(uint64_t)p.H, (uint64_t)p.T};
  const uint64_t da[3] = {(uint64_t)p.I, (uint64_t)p.T, (uint64_t)p.A_max * (BITS == 4 ? 2 : 1)};
  const uint32_t bx[3] = {64, NP, 1}, bx2[3] = {64, NP, 2};  // (4-bit: both halves)
  if (!make_map_sw128(&mg, Wg, esz, 3, d1, bw) || !make_map_sw128(&mu, Wu, esz, 3, d1, bw) ||
      !make_map_sw128(&mg64, Wg, esz, 3, d1, bw64) || !make_map_sw128(&mu64, Wu, esz, 3, d1, bw64) ||
      !make_map_sw128(&md, Wd, esz, 3, d2, bw) || !make_map_sw128(&mx, x, 2, 2, dx, bx) ||
      !make_map_sw128(&ma, p.act, 2, 3, da, BITS == 4 ? bx2 : bx))
    return MOE_ERR_CUDA;
  if constexpr (BITS == 4) {
    const uint64_t s1[3] = {(uint64_t)p.I, (uint64_t)p.H * p.per1 / 256, (uint64_t)p.E};
    const uint64_t s2[3] = {(uint64_t)p.H, (uint64_t)p.I * p.per2 / 256, (uint64_t)p.E};
    const uint32_t b1[3] = {128, (uint32_t)p.per1, 1}, b2[3] = {128, (uint32_t)p.per2, 1};
    const uint32_t b64[3] = {64, (uint32_t)p.per1, 1};
    if (!make_map(&mgs, w.gs, 2, 3, s1, b1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map(&mus, w.us, 2, 3, s1, b1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map(&mgs64, w.gs, 2, 3, s1, b64, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map(&mus64, w.us, 2, 3, s1, b64, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map(&mds, w.ds, 2, 3, s2, b2, CU_TENSOR_MAP_SWIZZLE_NONE))
      return MOE_ERR_CUDA;
  }
  static PerDevice smem_allowed;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const int allowed = smem_allowed.get(dev, [] {
    return cudaFuncSetAttribute(few_tokens_kernel<NP, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)TR::smem) == cudaSuccess;
  });
  if (!allowed) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  cfg.gridDim = dim3(sm_count() < kMaxCtas ? sm_count() : kMaxCtas, 1, 1);
  cfg.blockDim = dim3(TR::threads, 1, 1);
  cfg.dynamicSmemBytes = TR::smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, few_tokens_kernel<NP, BITS>, mg, mu, mg64, mu64, md, mx, ma, mgs,
                         mus, mgs64, mus64, mds, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  count_launches(1);
  return MOE_OK;
}

// A call's checks and its launch.
template <int BITS>
int few_tokens(const void* tokens, const int32_t* expert_ids, const float* probs, int T, int H, int K,
               int I, int E, int num_special, const uint8_t* active_mask, int mask_dims, int group1, int group2,
               const FewWeights& w, const void* shared_x, void* out, void* workspace, size_t workspace_bytes,
               int32_t* dev_status, cudaStream_t stream) {
  if (T < 0 || H <= 0 || K <= 0 || I <= 0 || E <= 0 || num_special < 0) return MOE_ERR_INVALID_ARG;
  if (active_mask != nullptr && mask_dims != 1 && mask_dims != 2) return MOE_ERR_INVALID_ARG;
  if (T > MOE_FEW_TOKENS || K > kMaxK || E > kMaxExperts) return MOE_ERR_SHAPE;
  if ((long long)E + num_special > 0x7fffffffLL || (long long)K > (long long)E + num_special)
    return MOE_ERR_SHAPE;
  if (H % 64 || I % 64) return MOE_ERR_SHAPE;
  if (H > MOE_FEW_MAX_SIZE || I > MOE_FEW_MAX_SIZE) return MOE_ERR_SHAPE;  // (T H, a tile's bytes: 31 bits)
  if (BITS == 4) {
    for (int g : {group1, group2})
      if (g != 32 && g != 64 && g != 128) return MOE_ERR_INVALID_ARG;
    if (H % group1 || I % group2) return MOE_ERR_SHAPE;
  }
  if (T == 0) return MOE_OK;
  if (!tokens || !expert_ids || !probs || !w.gate || !w.up || !w.down || !out || !workspace)
    return MOE_ERR_INVALID_ARG;
  const bool scaled = BITS < 16;
  if (scaled != (w.gs != nullptr) || scaled != (w.us != nullptr) || scaled != (w.ds != nullptr))
    return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {tokens, w.gate, w.up, w.down, shared_x, out, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (BITS == 4 && (!aligned16(w.gs) || !aligned16(w.us) || !aligned16(w.ds))) return MOE_ERR_INVALID_ARG;
  const FewLayout l = few_layout(T, K, H, I, E, BITS);
  if (workspace_bytes < l.total) return MOE_ERR_INVALID_ARG;  // (what these weights use)
  if (int rc = device_ok()) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  FewParams p{};
  p.ids = expert_ids;
  p.probs = probs;
  p.mask = active_mask;
  if (BITS == 8) {
    p.gs = static_cast<const float*>(w.gs);
    p.us = static_cast<const float*>(w.us);
    p.ds = static_cast<const float*>(w.ds);
  }
  if (BITS == 4) {
    p.per1 = 256 / group1;
    p.per2 = 256 / group2;
  }
  p.shared_x = static_cast<const __nv_bfloat16*>(shared_x);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.epoch = reinterpret_cast<unsigned long long*>(ws);
  p.count = reinterpret_cast<uint32_t*>(ws += l.words);
  p.part1 = reinterpret_cast<float*>(ws += l.counts);
  p.part2 = reinterpret_cast<float*>(ws += l.part1);
  p.act = reinterpret_cast<__nv_bfloat16*>(ws += l.part2);
  p.status = dev_status;
  p.mask_dims = mask_dims;
  p.T = T;
  p.H = H;
  p.K = K;
  p.I = I;
  p.E = E;
  p.E_all = E + num_special;
  p.A_max = T * K < E ? T * K : E;
  if (T <= 16) return launch_few<16, BITS>(p, tokens, w, stream);
  if (T <= 32) return launch_few<32, BITS>(p, tokens, w, stream);
  return launch_few<64, BITS>(p, tokens, w, stream);
}

}  // namespace
}  // namespace tc
}  // namespace moe

using namespace moe;
using namespace moe::tc;

extern "C" size_t moe_layer_few_tokens_workspace_size(int T, int K, int H, int I, int E) {
  if (T <= 0 || K <= 0 || H <= 0 || I <= 0 || E <= 0 || T > MOE_FEW_TOKENS || K > kMaxK) return 0;
  if (H > MOE_FEW_MAX_SIZE || I > MOE_FEW_MAX_SIZE) return 0;
  return few_layout(T, K, H, I, E, 4).total;  // (any weights)
}

extern "C" int moe_layer_few_tokens(const void* tokens, const int32_t* expert_ids,
                                    const float* probs, int T, int H, int K, int I, int E,
                                    int num_special, const uint8_t* active_mask, int mask_dims,
                                    int weight_dtype, const void* W_gate, const void* W_up,
                                    const void* W_down, const float* gate_scale,
                                    const float* up_scale, const float* down_scale,
                                    const void* shared_x, void* out, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_status,
                                    cudaStream_t stream) {
  if (weight_dtype != MOE_BF16 && weight_dtype != MOE_INT8) return MOE_ERR_INVALID_ARG;
  const FewWeights w{W_gate, W_up, W_down, gate_scale, up_scale, down_scale};
  return (weight_dtype == MOE_INT8 ? few_tokens<8> : few_tokens<16>)(
      tokens, expert_ids, probs, T, H, K, I, E, num_special, active_mask, mask_dims, 0, 0, w, shared_x, out,
      workspace, workspace_bytes, dev_status, stream);
}

extern "C" int moe_layer_few_tokens_int4(const void* tokens, const int32_t* expert_ids,
                                         const float* probs, int T, int H, int K, int I, int E,
                                         int num_special, const uint8_t* active_mask, int mask_dims,
                                         int group, int down_group, const uint8_t* W_gate_q,
                                         const void* gate_scale, const uint8_t* W_up_q,
                                         const void* up_scale, const uint8_t* W_down_q,
                                         const void* down_scale, const void* shared_x, void* out,
                                         void* workspace, size_t workspace_bytes,
                                         int32_t* dev_status, cudaStream_t stream) {
  return few_tokens<4>(tokens, expert_ids, probs, T, H, K, I, E, num_special, active_mask, mask_dims, group,
                    down_group, FewWeights{W_gate_q, W_up_q, W_down_q, gate_scale, up_scale, down_scale}, shared_x,
                    out, workspace, workspace_bytes, dev_status, stream);
}
