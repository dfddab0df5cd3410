// 4-bit weights: eight of them in a 32-bit word, expanded to bf16.
//
// Bits 4 i .. 4 i + 3 hold element 2 i of the eight and bits 16 + 4 i .. element
// 2 i + 1, as two's complement, so that a shift and a mask leave two neighbours
// in the lower bits of the two halves of a word: a packed pair of bf16 after two
// more operations.
#pragma once

#include "common.cuh"

namespace moe {

// The mask, in a register that the assembler cannot see through (a three-input
// operation takes one constant).
__device__ __forceinline__ uint32_t int4_mask() { return __shfl_sync(0xffffffffu, 0x000f000fu, 0); }

// The eight q * scale of a word in order, each a bf16 rounded once (exact where
// the scale has at most five significant bits).  scale2: the scale twice.
// 128 + u, u = q + 8, is a bf16 with u in its lowest bits; less 136 it is q.
// Written in the machine's own operations: from the compiler's types of two bf16,
// mask and magic take two.
//
// A scale of five bits would allow q * scale = (16 + u) scale - 24 scale in one
// multiply-add, every term exact: 4 % faster where nothing else is compiled in
// (16 tokens, H=7168 I=512: 136 us against 142), but not beside this form, which
// other scales need (144).
__device__ __forceinline__ void expand_int4(uint32_t w, uint32_t scale2, uint32_t mask, uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b32 t;\n\tlop3.b32 t, %1, %4, 0x43084308, 0x6a;\n\t"  // (and, exclusive or)
        "sub.rn.bf16x2 t, t, %2;\n\tmul.rn.bf16x2 %0, t, %3;\n\t}"
        : "=r"(r[i])
        : "r"(w >> (4 * i)), "r"(0x43084308u), "r"(scale2), "r"(mask));
}

// A lane's 16 bytes: 32 inputs of a row, 16 registers.
__device__ __forceinline__ void expand_int4_row(uint4 v, uint32_t scale, uint32_t mask, uint32_t* r) {
  const uint32_t s = scale * 0x10001u;
  expand_int4(v.x, s, mask, r);
  expand_int4(v.y, s, mask, r + 4);
  expand_int4(v.z, s, mask, r + 8);
  expand_int4(v.w, s, mask, r + 12);
}

}  // namespace moe
