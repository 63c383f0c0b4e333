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

// ---- f16 pairs of scaled weights (the tcgen05 path)
QL_DEVINL uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
QL_DEVINL uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
QL_DEVINL uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
QL_DEVINL uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
QL_DEVINL uint32_t f32x2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight codes -> four f16 pairs (q - 8) s in the order of codes_to_bf16.  A nibble in
// bits 6-9 of f16 16.0 reads as 16 + q, so (q - 8) s = (16 + q) s - 24 s in one fma:
// 24 s is exact (2 + 8 significant bits), and so is the result (at most 3 + 8).
QL_DEVINL void codes_to_f16(uint32_t w, uint32_t s, uint32_t m24s, uint32_t* p) {
  p[0] = fma_f16x2(and_or<0x03C003C0u, 0x4C004C00u>(w << 6), s, m24s);
  p[1] = fma_f16x2(and_or<0x03C003C0u, 0x4C004C00u>(w << 2), s, m24s);
  p[2] = fma_f16x2(and_or<0x03C003C0u, 0x4C004C00u>(w >> 2), s, m24s);
  p[3] = fma_f16x2(and_or<0x03C003C0u, 0x4C004C00u>(w >> 6), s, m24s);
}

// With a zero point (16 + z) s may need 13 bits, so q - z comes first, exactly: a nibble
// in bits 0-3 of f16 1024.0 reads as 1024 + q, one in bits 4-7 as 1024 + 16 q (one shift
// serves four pairs); zlo = (1024 + z) twice, zhi = -(64 + z) twice.  The product with
// s, up to 12 significant bits, is rounded to 11.
QL_DEVINL void codes_to_f16_zero(uint32_t w, uint32_t zlo, uint32_t zhi, uint32_t s, uint32_t* p) {
  constexpr uint32_t kSixteenth = 0x2C002C00u;
  const uint32_t v = w >> 8;
  p[0] = mul_f16x2(sub_f16x2(and_or<0x000F000Fu, 0x64006400u>(w), zlo), s);
  p[1] = mul_f16x2(fma_f16x2(and_or<0x00F000F0u, 0x64006400u>(w), kSixteenth, zhi), s);
  p[2] = mul_f16x2(sub_f16x2(and_or<0x000F000Fu, 0x64006400u>(v), zlo), s);
  p[3] = mul_f16x2(fma_f16x2(and_or<0x00F000F0u, 0x64006400u>(v), kSixteenth, zhi), s);
}

// mbar_wait_bounded for a whole warp, whose lanes arrive together.  It polls every few
// dozen cycles before the bounded wait, whose timer costs 700 cycles to start, takes over.
QL_DEVINL bool wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  bool ok = mbar_try_wait(a, parity);
#pragma unroll 1
  for (int i = 0; i < 4096 && !__all_sync(0xffffffffu, ok); ++i) {
    __nanosleep(20);
    ok = mbar_try_wait(a, parity);
  }
  if (!__all_sync(0xffffffffu, ok)) ok = mbar_wait_bounded(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

// ---- tcgen05 with the A operand in TMEM
// kind::f16 with f16 operands: the fields of tc::idesc_bf16 with A and B format 0.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One lane of a converged warp (the same one each time).
QL_DEVINL uint32_t elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, K = 16: A holds row i in lane i, two inputs to a
// column.  Called by the whole warp, issued by its elected lane: the operands are then
// warp-uniform and live in uniform registers.  Inside a one-lane branch each issue
// took 60 to 80 cycles to move them there, more than the MMA itself up to 128 tokens.
QL_DEVINL void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t id, uint32_t accumulate,
                          uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(id), "r"(accumulate), "r"(elected)
      : "memory");
}
QL_DEVINL void commit(uint64_t* bar, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}

// Lane i of the warp stores its 32 registers to TMEM lane (taddr.lane + i), columns
// [taddr.col, taddr.col + 32).
QL_DEVINL void st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
QL_DEVINL void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns of one lane quarter.
QL_DEVINL void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// One column of it.
QL_DEVINL float ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  tc::ld_wait();
  return __uint_as_float(r);
}

// ---- clusters
QL_DEVINL void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes of the shared memory of the cluster's CTA `rank`, at this CTA's address saddr.
QL_DEVINL float4 ld_cluster(uint32_t saddr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [ra];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(saddr), "r"(rank)
      : "memory");
  return v;
}

}  // namespace w4
}  // namespace ql
