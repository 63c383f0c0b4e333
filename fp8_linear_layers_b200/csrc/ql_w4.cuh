// ql_w4.cuh -- device helpers of the 4-bit weight kernels (sm_100a).
//
// A weight is w = (q - z) * s: q a 4-bit code (two to a byte along K, the low
// nibble the even input), z the group's zero point (8 where none is kept), s the
// group's bf16 scale.  A 32-bit word of codes holds inputs k .. k+7 of one row.
#pragma once

#include "ql_common.cuh"
#include "ql_tc.cuh"

namespace ql {
namespace w4 {

// (w & mask) | bits in one instruction.
template <uint32_t kMask, uint32_t kBits>
QL_DEVINL uint32_t and_or(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(kMask), "n"(kBits));
  return r;
}

QL_DEVINL uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes -> four bf16 pairs (q - z), exact.  A nibble in the low mantissa
// bits of bf16 128.0 reads as 128 + q; zz = (128 + z, 128 + z).  Pair i holds
// inputs (i, i + 4): the order in which the nibbles sit in the two halves.
QL_DEVINL void codes_to_bf16(uint32_t w, uint32_t zz, uint32_t (&p)[4]) {
  p[0] = sub_bf16x2(and_or<0x000F000Fu, 0x43004300u>(w), zz);
  p[1] = sub_bf16x2(and_or<0x000F000Fu, 0x43004300u>(w >> 4), zz);
  p[2] = sub_bf16x2(and_or<0x000F000Fu, 0x43004300u>(w >> 8), zz);
  p[3] = sub_bf16x2(and_or<0x000F000Fu, 0x43004300u>(w >> 12), zz);
}

// D[16x8] += A[16x16] * B[16x8], bf16 x bf16 -> f32.
QL_DEVINL void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weight loads: read once by this launch, so they do not displace x in L1.
template <int kWords>
QL_DEVINL void load_words(const uint8_t* p, uint32_t (&w)[kWords]) {
  if constexpr (kWords == 4) {
    asm("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
        : "l"(p));
  } else if constexpr (kWords == 2) {
    asm("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  } else {
    asm("ld.global.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
}

QL_DEVINL void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

}  // namespace w4
}  // namespace ql
