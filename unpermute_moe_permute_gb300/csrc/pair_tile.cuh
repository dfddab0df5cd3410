// What the grouped products on CTA pairs with weights in tensor memory share:
// their tiles and their epilogue.
#pragma once

#include "sched.cuh"
#include "tc_warp.cuh"

namespace moe {
namespace tc {
namespace {

constexpr int kTmaWarp = 0, kMmaWarp = 1, kEpiWarp = 2;

struct PairTile {
  int e, row0, hi;  // expert, first row, end of the tile's rows
  int subs;         // accumulators the rows take: 1 or 2
  int n, n1;        // MMA N of the first and of the second: multiples of 32
  int ch0;          // first channel of this CTA
  __device__ __forceinline__ int b_rows() const { return (n + n1) / 2; }  // of this CTA
};

// Tile t is channel tile (t mod ch_tiles) of row tile t / ch_tiles; the rows
// of an expert are split evenly over its ceil(rows / (2 kSub)) row tiles, the rows
// of a row tile over its accumulators in steps of 32.
template <bool kSwiglu, int kSub, typename P>
__device__ __forceinline__ PairTile pair_tile(int t, const P& p, const int32_t* prefix,
                                          const int32_t* offs, int rank) {
  PairTile x;
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

// A tile that one pair of CTAs sums alone.
struct WholeTile {
  __device__ __forceinline__ bool begin() { return true; }
  // v: 32 accumulator columns from column c of the tile on.  Whether this CTA
  // goes on to write them.
  __device__ __forceinline__ bool piece(uint32_t (&)[32], int) { return true; }
  __device__ __forceinline__ void end() {}
};

// The epilogue warps' part of a kernel: every tile's accumulators to rows of
// p.out, with SwiGLU where a tile holds gate and up channels.  kScaled: a scale
// for each channel (p.s0, p.s1) and each row (p.rs).  rank: of the CTA in its
// pair; leader: of the pair's leading CTA in the cluster.  split: how a tile's
// sums are put together (WholeTile, or pairs that share its inputs).
template <typename C, bool kSwiglu, bool kScaled, typename O, typename P, typename S>
__device__ __forceinline__ void pair_epilogue(const P& p, uint32_t base, uint8_t* g, uint32_t tmem, int warp,
                                              int lane, int rank, int leader, int t0, int dt, int total,
                                              uint32_t t_full, uint32_t t_empty,
                                              volatile int* abort_flag, const int32_t* prefix,
                                              const int32_t* offs, S&& split) {
  constexpr int kSub = C::kSub, kEpi = C::kEpi;
  // Lanes are channels, accumulator columns are rows; the warps of a quarter take
  // pieces of 32 columns in turn.  A piece is scaled, turned through the warp's
  // staging rows and written in 16-byte chunks of 8 channels.
  const int quarter = warp & 3, part = (warp - kEpiWarp) >> 2;
  constexpr int kCh = kSwiglu ? 16 : 32;  // channels per warp
  O* out = static_cast<O*>(p.out);
  const uint32_t stage_u = base + C::kStage + (uint32_t)(warp - kEpiWarp) * C::kStageWarp;
  float* scale = reinterpret_cast<float*>(g + C::kStage + (warp - kEpiWarp) * C::kStageWarp + 2048);
  const int ch_l = kSwiglu ? quarter * 16 + (lane & 15) : quarter * 32 + lane;
  int it = 0;
  bool run = true;
  for (int t = t0; run && t < total; t += dt) {
   const PairTile x = pair_tile<kSwiglu, kSub>(t, p, prefix, offs, rank);
   const int ch = x.ch0 + ch_l;
   float cs = 1.f;
   if constexpr (kScaled)
     cs = ch >= p.Nout ? 0.f : ((kSwiglu && lane >= 16) ? p.s1 : p.s0)[(size_t)x.e * p.Nout + ch];
   // two neighbouring rows of this lane's channel
   auto scaled = [&](uint32_t a, uint32_t b, int j) {
     if constexpr (kScaled) return mul2(mul2(a, b, cs, cs), *reinterpret_cast<const float2*>(scale + j));
     else return make_float2(__uint_as_float(a), __uint_as_float(b));
   };
   // row scales of the first pieces (the second accumulator's ahead of its
   // wait, which is short)
   const int r_first = x.row0 + part * 32 + lane, r_second = r_first + x.n;
   float rs_first = 1.f, rs_second = 1.f;
   if constexpr (kScaled) {
     rs_first = part * 32 + lane < min(x.hi - x.row0, x.n) ? p.rs[r_first] : 0.f;
     rs_second = x.subs > 1 && r_second < x.hi ? p.rs[r_second] : 0.f;
   }
   run = split.begin();
   for (int sub = 0; run && sub < x.subs; ++sub, ++it) {
    const int acc = it & 1, row0 = x.row0 + sub * x.n;
    const int rows = min(x.hi - row0, sub ? x.n1 : x.n);
    float rs = sub ? rs_second : rs_first;
    run = mbar_wait_warp(t_full + 8u * acc, (it >> 1) & 1, abort_flag, p.status);
    if (!run) break;
    tc_fence_after();
    const uint32_t d = tmem + acc * kSub + ((uint32_t)(quarter * 32) << 16);
    auto give_back = [&]() {
      tc_fence_before();
      mbar_arrive_cluster_warp(mapa_shared(t_empty + 8u * acc, leader));
    };
    for (int c0 = part * 32; c0 < rows; c0 += 8 * kEpi) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(d + c0, v);
      if constexpr (kScaled) {
        scale[lane] = rs;
        rs = c0 + 8 * kEpi + lane < rows ? p.rs[row0 + c0 + 8 * kEpi + lane] : 0.f;
        __syncwarp();
      }
      tmem_ld_wait();
      if (c0 + 8 * kEpi >= rows) give_back();  // the warp's last piece is in registers
      if (!split.piece(v, sub * x.n + c0)) continue;
      if constexpr (sizeof(O) == 4) {
        // fp32: staging rows of 32 channels, 16 columns at a time
#pragma unroll
        for (int p0 = 0; p0 < 32; p0 += 16) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            st_shared_u32(stage_u + lane * 4 + j * 128,
                          kScaled ? __float_as_uint(__uint_as_float(v[p0 + j]) * cs * scale[p0 + j]) : v[p0 + j]);
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
            const float2 f = scaled(v[j], v[j + 1], j);
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
            const float2 f = scaled(v[2 * j], v[2 * j + 1], 2 * j);
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
   if (run) split.end();
  }
}

}  // namespace
}  // namespace tc
}  // namespace moe
