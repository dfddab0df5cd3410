// 4-bit weights: eight of them in a 32-bit word, expanded to bf16.
//
// Bits 4 i .. 4 i + 3 hold element 2 i of the eight and bits 16 + 4 i .. element
// 2 i + 1, as two's complement, so that a shift and a mask leave two neighbours
// in the lower bits of the two halves of a word: a packed pair of bf16 after two
// more operations.
#pragma once

#include "common.cuh"

namespace moe {

// 2^7 + u in bf16 for u in 0..15 (the exponent leaves steps of 1); q = u - 8
// with the sign bit of the nibble turned over.
constexpr uint32_t kInt4Mask = 0x000f000fu, kInt4Magic = 0x43084308u, kInt4Zero = 0x43084308u;

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v) {
  return *reinterpret_cast<__nv_bfloat162*>(&v);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

// The eight q * scale of a word in order, each a bf16 rounded once (exact where
// the scale has at most five significant bits).  scale2: the scale twice.
__device__ __forceinline__ void expand_int4(uint32_t w, uint32_t scale2, uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t;  // (shifted & mask) ^ magic in one operation: left to the compiler it takes two
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(t) : "r"(w >> (4 * i)), "r"(kInt4Mask), "r"(kInt4Magic));
    r[i] = as_u32(__hmul2(__hsub2(as_bf162(t), as_bf162(kInt4Zero)), as_bf162(scale2)));
  }
}

}  // namespace moe
