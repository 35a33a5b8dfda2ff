// The 4-bit weight format and its conversions to bf16 pairs.
//
// A weight row of K values is K / 2 bytes, column 2i in the low half of byte i
// and column 2i + 1 in the high half; a half byte u stands for (u - 8) * s with
// one bf16 scale s for each 128 columns.
#pragma once

#include "internal.cuh"

namespace mla {

constexpr int kW4Group = MLA_W4_GROUP;
__host__ __device__ inline int w4_groups(int K) { return (K + kW4Group - 1) / kW4Group; }

// (v & mask) | bits as the one instruction it is (left to itself the compiler made two, and this conversion is what
// bounds a projection of few tokens).
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
  return d;
}

// The eight half bytes u_0 .. u_7 of a word as four bf16 pairs (u_i - 8, u_{i+4} - 8),
// i = 0 .. 3: 0x4300 is 128, whose bf16 unit in the last place is 1, so 0x4300 | u
// is 128 + u, and the difference to 136 is exact.
__device__ __forceinline__ void w4_pairs(uint32_t v, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t biased = and_or(v >> (4 * i), 0x000f000fu, 0x43004300u);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(biased), "r"(0x43084308u));
  }
}


// The same pairs in f16: 0x6400 is 1024, whose unit in the last place is 1, so a half byte
// in the low bits adds u and one four bits up adds 16 u; both ways back are exact.
__device__ __forceinline__ void w4_pairs_f16(uint32_t v, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = and_or(v >> (8 * i), 0x000f000fu, 0x64006400u);  // 1024 + u
    const uint32_t hi = and_or(v >> (8 * i), 0x00f000f0u, 0x64006400u);  // 1024 + 16 u
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2 * i]) : "r"(lo), "r"(0x64086408u));                       // - 1032
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[2 * i + 1]) : "r"(hi), "r"(0x2c002c00u), "r"(0xd480d480u));  // / 16 - 72
  }
}

}  // namespace mla
