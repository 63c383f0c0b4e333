// ql_w4_gemm.cu -- products with 4-bit weights for many tokens on tcgen05, dense and
// by routed expert.
//
//   y[m, n] = bf16( sum_k x[m, k] (q[n, k] - z) s )
//
// Weights are the MMA's 128-row A operand, tokens its N columns.  The codes come by
// TMA into shared memory, eight warps turn them into f16 and store them straight
// into TMEM, where the MMA reads its A operand: thread = weight row, one 32-bit
// column = two inputs, so no swizzled shared-memory store is needed and the shared
// memory serves only the tokens' operand.
//
// f16 has 11 significant bits.  x is bf16, 8 bits, and fits; so does a scaled weight
// (q - 8) s, 3 + 8 bits.  With zero points (q - z) s may need 4 + 8: it is rounded once to
// 11, off by at most 2^-11 of itself.  That is a choice: the two halves of a 12-bit weight
// would take two MMAs, twice the tensor time, for an eighth of what bf16 weights lose.
// Exponents are brought into f16's range by powers of two: each token is scaled so that its
// largest |x| lies in [2^14, 2^15), each weight row so that its largest |s| lies in [2^10,
// 2^11).  Inputs more than 2^31 below their token's largest and scales more than 2^27 below
// their row's do not fit; they are zero for the tensor cores, and the epilogue adds their
// products (left_out: of tokens of 4096 N(0, 1) inputs with outliers 20 times larger about one
// in 10,000 has such an input; a tile with all of them, K = 16384, takes 0.2 s).  Sums are f32,
// and the powers of two come off in the epilogue.  Scaling in f16 before the product leaves
// nothing to do at a group's end, so 32-input groups cost what 128-input groups do.
//
// A prepare kernel makes the f16 tokens (the inputs of each eight in the order 0 4 1 5
// 2 6 3 7 in which codes_to_f16 gives the weights) and, for experts, sorts the (token,
// slot) pairs by expert and cuts each expert's pairs into token tiles.
//
// Two kernels.  The narrow one (a 128-row tile, up to 128 tokens, K split over a cluster)
// gives every SM a share of the weights where there are few tokens; the wide one (256 rows
// x up to 192 tokens, persistent) converts each weight once for more tokens.  The tensor
// pipe alone takes 97 cycles for an MMA of 192 columns (96 at its rate); a granule of 64
// inputs of a wide tile, 640 cycles of MMA at 160 tokens, takes about 760: conversion,
// tcgen05.st and the four hand-overs between the warps follow one another through two TMEM
// slots.  Leaving out the conversion saved 19 % of a prompt's time, the stores 29 %, the
// products 21 %, the token loads 10 %: no single part bounds it.  Tried and slower: four
// slots (128 tokens), 16 converting warps, outputs held in the epilogue's registers, a
// store's completion awaited one granule later, one-lane waits.
// 14336 x 4096, group 128: 2048 tokens 188 us (1.28 PFLOP/s), 512 tokens 63 us, 128 tokens
// 32 us, 24 tokens 20 us; 64 experts of 1536 x 2048, 2048 tokens x 8: 126 us.
#include "ql_internal.h"
#include "ql_w4.cuh"

namespace ql {

constexpr unsigned int KID_W4 = 4;  // KernelId of this file's GEMM in the device status word

constexpr int kG4DequantWarps = 8;
constexpr int kG4StageK = 256;   // inputs of a weight stage (128 bytes of codes a row)
constexpr int kG4GranK = 64;     // inputs of a token stage and of a TMEM weight slot
constexpr int kG4WStages = 3;
constexpr int kG4MaxXStages = 8;
constexpr int kG4PrepThreads = 128;
constexpr int kG4PlanThreads = 1024;
constexpr int kG4MaxSplit = 8;
constexpr int64_t kG4CountPairs = 2048;  // experts: up to here each pair's place is counted by its own warp

// Wide kernel: two 128-row weight tiles share up to 192 tokens; one CTA to an SM, which
// takes tile after tile.  An MMA issuer to each weight tile (one for both: 2048 tokens
// 14336 x 4096 197 against 188 us).  TMEM: 2 x 192 accumulator columns, 2 slots x 2 tiles x 32.
constexpr int kWideTok = 192;
constexpr int kWideRing = 110592;  // bytes of token stages
constexpr int kWideProducer = kG4DequantWarps;
constexpr int kWideMma = kWideProducer + 1;
constexpr int kWideFirstEpi = kWideMma + 2;
constexpr int kWideEpiWarps = 8;
constexpr int kWideThreads = (kWideFirstEpi + kWideEpiWarps) * 32;
constexpr int kWideBarriers = 2 * kG4WStages + 2 * kG4MaxXStages + 12;
constexpr int kWideStageRow = 80;  // bytes of a token in an epilogue warp's staging (32 outputs and a pad)
constexpr int kWideStageRowF32 = 144;  // the same of f32 outputs, 8 tokens at a time
constexpr int kWideWBytes = 2 * 128 * 128;
static_assert(8 * kWideStageRowF32 <= 16 * kWideStageRow, "staging");

// Narrow kernel: one weight tile, up to 128 tokens, K split over a cluster; two CTAs to
// an SM.  TMEM: 128 accumulator columns, 4 slots x 32.
constexpr int kNarrowTok = 128;
constexpr int kNarrowRing = 57344;
constexpr int kNarrowSlots = 4;
constexpr int kNarrowThreads = (kG4DequantWarps + 2) * 32;
constexpr int kNarrowWBytes = 128 * 128;

struct G4Tile {
  int expert, start, count, pad;
};

struct G4Params {
  const uint16_t* x;     // the tokens as given (left_out)
  const uint8_t* wq;
  const uint16_t* sw;
  const uint8_t* wz;
  uint16_t* y;           // dense, gather: the result
  float* yp;             // combine: the pairs' products; else null
  const int* ex;         // G4Row::exponent of the prepared tokens (experts: of the sorted pairs)
  const int* order;      // experts: pairs sorted by expert
  int slots;             // experts: pairs of an x row
  const G4Tile* tiles;   // experts: token tiles
  const int* ntiles;
  int64_t N, K;
  int64_t M;             // dense: tokens
  int groups;
  int ntok;              // tokens of a tile (a multiple of 16)
  int row_tiles, tok_tiles;  // wide, dense
  int xstage;            // bytes of a token stage
  int xstages;           // token stages
  int splits;            // CTAs of a cluster along K
  DevStatus* status;
};

QL_DEVINL float exp2i(int e) {  // 2^e, e in [-149, 127]
  return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}
QL_DEVINL float scale2(float v, int e) {  // v 2^e, e in [-298, 254]
  const int h = e / 2;
  return v * exp2i(h) * exp2i(e - h);
}

// Position of the largest set exponent of a bf16 magnitude (floor of its log2); 0 -> zero.
QL_DEVINL int log2_bf16(uint32_t mag, int zero) {
  return mag >= 0x80u ? (int)(mag >> 7) - 127 : mag ? -133 + (31 - __clz(mag)) : zero;
}

// A value whose scaled magnitude is below 2^-17 may not fit f16 (8 significant bits down to
// 2^-24): it is "left out", zero for the tensor cores, and its products are added by the
// epilogue (left_out).  The bf16 magnitude from which on a value scaled by 2^e stays in.
QL_DEVINL uint32_t left_out_below(int e) {
  const int t = -17 - e;  // in [-164, 100]
  return t >= -126 ? (uint32_t)(t + 127) << 7 : t >= -133 ? 1u << (t + 133) : 0u;
}
// low: the smallest nonzero magnitude less one.
QL_DEVINL bool leaves_out(uint32_t low, int e) {
  const uint32_t thr = left_out_below(e);
  return low < thr && low + 1u < thr;
}

// 2 f + 1 if scales are left out, else 2 f: f the power of two that brings a row's largest
// |s| over groups [g0, g1) to [2^10, 2^11).
QL_DEVINL int row_exponent(const uint16_t* sw, int g0, int g1, bool vec) {
  uint32_t top = 0, low = 0xFFFFFFFFu;
  auto add = [&](uint32_t mag) {
    top = max(top, mag);
    low = min(low, mag - 1u);
  };
  if (vec) {  // whole 16-byte pieces; a neighbour's scales do no harm beyond range
    const uint4* v4 = reinterpret_cast<const uint4*>(sw);
#pragma unroll 4
    for (int i = g0 >> 3; i < (g1 + 7) >> 3; ++i) {
      const uint4 v = __ldg(v4 + i);
      add(v.x & 0x7FFFu), add(v.x >> 16 & 0x7FFFu);
      add(v.y & 0x7FFFu), add(v.y >> 16 & 0x7FFFu);
      add(v.z & 0x7FFFu), add(v.z >> 16 & 0x7FFFu);
      add(v.w & 0x7FFFu), add(v.w >> 16 & 0x7FFFu);
    }
  } else {
#pragma unroll 8
    for (int i = g0; i < g1; ++i) add((uint32_t)__ldg(sw + i) & 0x7FFFu);
  }
  const int f = 10 - log2_bf16(min(top, 0x7F7Fu), 10);
  return 2 * f + leaves_out(low, f);
}

template <class T>
QL_DEVINL const T* shfl_pointer(const T* p, int lane) {
  return reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), lane));
}

// What the tensor cores left out of one token's product with each lane's weight row, over
// inputs [k0, k1): the token's values below its threshold, and the groups whose scales are
// below their row's, in f32 from the original operands.  For a whole warp; x and ex are the
// same in all lanes.  ex and f as G4Row::exponent and row_exponent give them.  Rare (a value
// 2^31 below its token's largest, a scale 2^27 below its row's), so a walk over the token
// will do.
template <int kGroup, bool kZero>
__device__ __noinline__ float left_out(const uint16_t* x, const uint8_t* wq, const uint16_t* sw, const uint8_t* wz,
                                       int ex, int f, int k0, int k1) {
  const int lane = threadIdx.x & 31;
  const uint32_t xthr = left_out_below(ex >> 1);
  float sum = 0.0f;
  if (ex & 1) {
    for (int base = k0; base < k1; base += 256) {
      const int k = base + lane * 8;
      uint32_t v[4] = {0, 0, 0, 0};
      if (k < k1) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + k));
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // the nonzero values below the threshold, else 0
          v[i] = ((v[i] & 0x7FFFu) - 1u < xthr - 1u ? v[i] & 0xFFFFu : 0u) |
                 ((v[i] >> 16 & 0x7FFFu) - 1u < xthr - 1u ? v[i] & 0xFFFF0000u : 0u);
      }
      unsigned pieces = __ballot_sync(0xffffffffu, (v[0] | v[1] | v[2] | v[3]) != 0);
      while (pieces) {
        const int src = __ffs(pieces) - 1, kk = base + src * 8, g = kk / kGroup;
        pieces &= pieces - 1;
        const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(wq + (kk >> 1)));
        const float s = __uint_as_float((uint32_t)__ldg(sw + g) << 16);
        const int z = kZero ? __ldg(wz + g) : 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = __shfl_sync(0xffffffffu, v[i], src);
          const int q0 = (int)(c >> (8 * i) & 15u) - z, q1 = (int)(c >> (8 * i + 4) & 15u) - z;
          if (u & 0xFFFFu) sum = fmaf(bf16_lo(u) * (float)q0, s, sum);
          if (u >> 16) sum = fmaf(bf16_hi(u) * (float)q1, s, sum);
        }
      }
    }
  }
  unsigned rows = __ballot_sync(0xffffffffu, f & 1);
  while (rows) {
    const int r = __ffs(rows) - 1;
    rows &= rows - 1;
    const uint32_t sthr = left_out_below(__shfl_sync(0xffffffffu, f, r) >> 1);
    const uint8_t* rw = shfl_pointer(wq, r);
    const uint16_t* rs = shfl_pointer(sw, r);
    const uint8_t* rz = shfl_pointer(wz, r);
    float part = 0.0f;
#pragma unroll 4
    for (int k = k0 + lane * 8; k < k1; k += 256) {
      const uint32_t s16 = __ldg(rs + k / kGroup);
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + k));
      const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(rw + (k >> 1))), v[4] = {u.x, u.y, u.z, u.w};
      const int z = kZero ? __ldg(rz + k / kGroup) : 8;
      const float s = __uint_as_float(s16 << 16);
      const bool out = (s16 & 0x7FFFu) - 1u < sthr - 1u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (the token's own were added above)
        const int q0 = (int)(c >> (8 * i) & 15u) - z, q1 = (int)(c >> (8 * i + 4) & 15u) - z;
        if (out && (v[i] & 0x7FFFu) >= xthr) part = fmaf(bf16_lo(v[i]), (float)q0 * s, part);
        if (out && (v[i] >> 16 & 0x7FFFu) >= xthr) part = fmaf(bf16_hi(v[i]), (float)q1 * s, part);
      }
    }
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == r) sum += part;
  }
  return sum;
}

// A row's scales and zero points of a weight stage's granules kStep i + first, loaded a
// stage ahead.
template <int kGroup, bool kZero, int kStep>
struct G4Scales {
  static constexpr int kStage = kG4StageK / kGroup;   // groups of a stage
  static constexpr int kPer = kGroup == 32 ? 2 : 1;   // groups in a granule
  static constexpr int kOwn = 4 / kStep;
  static constexpr int kN = kGroup == 128 ? 2 : kOwn * kPer;
  uint32_t sraw[kN], zraw[kZero ? kN : 1];
  uint32_t s2[kN], z0[kN], z1[kZero ? kN : 1];  // kZero: zlo, zhi; else z0 = -24 s

  QL_DEVINL void load(const uint16_t* sw, const uint8_t* wz, int w, int first, int groups) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int gi = w * kStage + (kGroup == 128 ? i : (kStep * (i / kPer) + first) * kPer + i % kPer);
      sraw[i] = gi < groups ? __ldg(sw + gi) : 0;
      if constexpr (kZero) zraw[i] = gi < groups ? __ldg(wz + gi) : 8;
    }
  }
  QL_DEVINL void convert(int f, uint32_t below) {  // below: left_out_below(f)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float s = (sraw[i] & 0x7FFFu) < below ? 0.0f : scale2(__uint_as_float(sraw[i] << 16), f);
      s2[i] = w4::f32x2_to_f16x2(s, s);
      if constexpr (kZero) {
        z0[i] = 0x64006400u + zraw[i] * 0x10001u;
        const float zf = -(64.0f + (float)zraw[i]);
        z1[i] = w4::f32x2_to_f16x2(zf, zf);
      } else {
        z0[i] = w4::f32x2_to_f16x2(-24.0f * s, -24.0f * s);
      }
    }
  }
  // A row's 32 bytes of codes of granule gq, from the row's 128 swizzled bytes.
  static QL_DEVINL void codes(const uint8_t* row, int gq, uint32_t rsw, uint32_t (&c)[8]) {
    const uint4 c0 = *reinterpret_cast<const uint4*>(row + (((uint32_t)(2 * gq) ^ rsw) << 4));
    const uint4 c1 = *reinterpret_cast<const uint4*>(row + (((uint32_t)(2 * gq + 1) ^ rsw) << 4));
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w;
    c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
  }
  // The weights of granule kStep own + first.
  QL_DEVINL void granule(const uint32_t (&c)[8], int own, uint32_t (&h)[32]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int gi = kGroup == 128 ? own * kStep / 2 : own * kPer + i * kPer / 8;
      if constexpr (kZero)
        w4::codes_to_f16_zero(c[i], z0[gi], z1[gi], s2[gi], h + 4 * i);
      else
        w4::codes_to_f16(c[i], s2[gi], z0[gi], h + 4 * i);
    }
  }
};

// What the K range of a CTA looks like: weight stages [w0, w0 + n), taken in rotated
// order.  The CTAs start at different stages: marching through K together they would
// all read the same few token lines of L2 at a time.
struct G4Range {
  int w0, n, rot, nk64;
  QL_DEVINL int stage(int j) const {
    const int w = j + rot;
    return w0 + (w < n ? w : w - n);
  }
  QL_DEVINL int granules(int w) const { return min(4, nk64 - w * 4); }
  QL_DEVINL int total() const { return min((w0 + n) * 4, nk64) - w0 * 4; }
};

// ---------------------------------------------------------------------------- narrow

template <int kGroup, bool kZero>
__global__ void __launch_bounds__(kNarrowThreads, 2)
    w4_narrow_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const G4Params p) {
  constexpr int kMmaWarp = kG4DequantWarps + 1;
  constexpr int kThreads = kNarrowThreads;
  constexpr int kSlots = kNarrowSlots;
  const int xs_n = p.xstages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* wring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* xring = wring + kG4WStages * kNarrowWBytes;
  uint64_t* wfull = reinterpret_cast<uint64_t*>(xring + xs_n * p.xstage);
  uint64_t* wempty = wfull + kG4WStages;
  uint64_t* xfull = wempty + kG4WStages;
  uint64_t* xempty = xfull + kG4MaxXStages;
  uint64_t* afull = xempty + kG4MaxXStages;
  uint64_t* aempty = afull + kSlots;
  uint64_t* done = aempty + kSlots;
  int* s_ex = reinterpret_cast<int*>(done + 2);               // the columns' exponents (16-byte aligned)
  float* s_fac = reinterpret_cast<float*>(s_ex + kNarrowTok); // 2^-exponent
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(s_fac + kNarrowTok);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_wide = reinterpret_cast<int*>(tmem_holder + 2);  // an exponent that one factor cannot take, or values left out

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % p.splits;
  const int64_t n0 = (int64_t)(blockIdx.x / p.splits) * 128;
  const int nkw = (int)((p.K + kG4StageK - 1) / kG4StageK);
  G4Range kr;
  kr.nk64 = (int)((p.K + kG4GranK - 1) / kG4GranK);
  kr.w0 = (int)((int64_t)split * nkw / p.splits);
  kr.n = (int)((int64_t)(split + 1) * nkw / p.splits) - kr.w0;
  kr.rot = (int)((blockIdx.x / p.splits * 5u + blockIdx.y * 3u) % (unsigned)kr.n);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kG4WStages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], kG4DequantWarps);
    }
    for (int s = 0; s < xs_n; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&afull[s], 4);
      mbar_init(&aempty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    *s_wide = 0;
    fence_barrier_init();
    tc::prefetch_tmap(&tmW);
    tc::prefetch_tmap(&tmX);
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_holder, 256);
    tc::tmem_relinquish();
  }
  __syncthreads();
  tc::grid_dependency_wait();  // the prepare kernel's tokens, pairs and tiles
  tc::launch_dependents();

  // this CTA's tokens: exponent, and as a factor 2^-ex
  const int64_t m0 = (int64_t)blockIdx.y * p.ntok;
  const int count = (int)min((int64_t)p.ntok, p.M - m0);
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const int ex = p.ex[m0 + i], e = ex >> 1;
    s_ex[i] = ex;
    s_fac[i] = exp2i(max(-126, min(126, -e)));
    if (abs(e) > 60 || (ex & 1)) *s_wide = 1;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tmem_a = tmem + 128;
  const int mma_n = (count + 15) & ~15;

  if (warp == kG4DequantWarps) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t pol_w = l2_policy_evict_first();
    const uint64_t pol_x = l2_policy_evict_last();
    const int wrow = (int)n0;
    bool ok = true;
    int jw = 0, jx = 0;  // issued stages
    int s = 0;           // token stage of the next granule, and how often it was filled
    uint32_t fill = 0;
    for (; jw < kr.n && ok; ++jw) {
      const int v = jw % kG4WStages, w = kr.stage(jw);
      if (jw >= kG4WStages) ok = w4::wait(&wempty[v], ((jw / kG4WStages) - 1) & 1, abort_flag);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&wfull[v], kNarrowWBytes);
        tc::tma_load_2d(wring + v * kNarrowWBytes, &tmW, w * 128, wrow, &wfull[v], pol_w);
      }
      __syncwarp();
      const int ng = kr.granules(w);
      for (int gq = 0; gq < ng; ++gq) {
        if (fill > 0) ok = w4::wait(&xempty[s], (fill - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&xfull[s], (uint32_t)p.ntok * 128u);
          tc::tma_load_2d(xring + s * p.xstage, &tmX, (w * 4 + gq) * 128, (int)m0, &xfull[s], pol_x);
        }
        __syncwarp();
        ++jx;
        if (++s == xs_n) {
          s = 0;
          ++fill;
        }
      }
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_timeout(p.status, KID_W4, 1);
      *abort_flag = 1;
      // the copies in flight land before the CTA leaves (step jw's weights may be among them)
      for (int j = max(0, jw - kG4WStages + 1); j < min(jw + 1, kr.n); ++j)
        mbar_wait_bounded(&wfull[j % kG4WStages], (j / kG4WStages) & 1, nullptr);
      for (int j = max(0, jx - xs_n); j < jx; ++j) mbar_wait_bounded(&xfull[j % xs_n], (j / xs_n) & 1, nullptr);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t id = w4::idesc_f16(128, mma_n);
    const uint32_t elected = w4::elect_one();
    const uint32_t d = __shfl_sync(0xffffffffu, tmem, 0), a = d + 128;  // warp-uniform
    const uint32_t x0 = smem_u32(xring);
    const int ngran = kr.total();
    bool ok = true;
    int xs = 0;
    uint32_t xphase = 0;
    for (int j = 0; j < ngran; ++j) {
      const int slot = j % kSlots;
      ok = w4::wait(&xfull[xs], xphase, abort_flag);
      ok = ok && w4::wait(&afull[slot], (j / kSlots) & 1, abort_flag);
      if (!ok) break;
      tc::fence_after();
      const uint64_t bdesc = tc::sw128_desc(x0 + xs * p.xstage);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w4::mma_f16_ts(d, a + slot * 32 + k * 8, bdesc + 2 * k, id, j > 0 || k > 0, elected);
      w4::commit(&aempty[slot], elected);
      w4::commit(&xempty[xs], elected);
      if (++xs == xs_n) {
        xs = 0;
        xphase ^= 1;
      }
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_timeout(p.status, KID_W4, 2);
      *abort_flag = 1;
    }
    w4::commit(done, elected);
    w4::wait(done, 0, nullptr);
  } else if (warp < kG4DequantWarps) {
    // ------------------------------------------------------------ codes -> TMEM
    // Warps 0-3 take a stage's even granules, 4-7 the odd ones; thread = weight row.
    const int wg = warp >> 2, q = warp & 3;
    const int64_t n = n0 + q * 32 + lane;
    const int64_t wr = min(n, p.N - 1);
    const uint16_t* sw = p.sw + wr * p.groups;
    const uint8_t* wz = kZero ? p.wz + wr * p.groups : nullptr;
    G4Scales<kGroup, kZero, 2> sc;
    const int fl = row_exponent(sw, kr.w0 * sc.kStage, min(p.groups, (kr.w0 + kr.n) * sc.kStage), (p.groups & 7) == 0);
    const int f = fl >> 1;
    const uint32_t below = left_out_below(f);
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    const uint32_t row_off = (uint32_t)((q * 32 + lane) * 128);
    sc.load(sw, wz, kr.stage(0), wg, p.groups);
    bool ok = true;
    int j0 = 0;  // the stage's first granule
    for (int jw = 0; jw < kr.n && ok; ++jw) {
      const int ws = jw % kG4WStages, ng = kr.granules(kr.stage(jw));
      sc.convert(f, below);
      if (jw + 1 < kr.n) sc.load(sw, wz, kr.stage(jw + 1), wg, p.groups);
      ok = w4::wait(&wfull[ws], (jw / kG4WStages) & 1, abort_flag);
      if (!ok) break;
      const uint8_t* src = wring + ws * kNarrowWBytes + row_off;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int gq = 2 * i + wg, j = j0 + gq;
        if (gq >= ng) break;
        uint32_t c[8], h[32];
        sc.codes(src, gq, (uint32_t)(lane & 7), c);
        sc.granule(c, i, h);
        const int slot = j % kSlots, use = j / kSlots;
        if (use > 0) ok = w4::wait(&aempty[slot], (use - 1) & 1, abort_flag);
        if (!ok) break;
        tc::fence_after();
        w4::st32(tmem_a + slot * 32 + lane_addr, h);
        w4::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[slot]);
      }
      if (!ok) break;
      j0 += ng;
      __syncwarp();
      if (lane == 0) mbar_arrive(&wempty[ws]);
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_timeout(p.status, KID_W4, 3);
      *abort_flag = 1;
    }
    // ------------------------------------------------------------ epilogue
    ok = ok && w4::wait(done, 0, abort_flag);
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    if (ok) {
      tc::fence_after();
      // Staged in the rings, which every MMA has left behind: split K, [tok][128]
      // partial sums; else [tok][128] bf16 (rows padded by 16 bytes), so that the rows
      // leave in 16-byte stores.
      constexpr int kRow = 128 * 2 + 16;
      float* part = reinterpret_cast<float*>(wring);
      const int col = q * 32 + lane;
      const int half = ((mma_n / 16 + 1) / 2) * 16;
      const int c_lo = wg ? half : 0, c_hi = wg ? mma_n : half;
      const bool rows_out = __any_sync(0xffffffffu, fl & 1);
      const bool wide = __any_sync(0xffffffffu, *s_wide || abs(f) > 60) || rows_out;
      const float rf = exp2i(max(-126, min(126, -f)));
      for (int c = c_lo; c < c_hi; c += 16) {
        float o[16];
        uint32_t v[16];
        w4::ld16(tmem + lane_addr + c, v);
        tc::ld_wait();
        if (!wide) {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(v[i]) * rf * s_fac[c + i];
        } else {  // the two factors may leave f32's range where their product does not
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = scale2(__uint_as_float(v[i]), -(f + (c + i < count ? s_ex[c + i] >> 1 : 0)));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i >= count) continue;
          if (p.splits > 1)
            part[(c + i) * 128 + col] = o[i];
          else
            *reinterpret_cast<uint16_t*>(wring + (c + i) * kRow + col * 2) = f32_to_bf16_rn(o[i]);
        }
      }
      if (wide) {  // tokens with something left out once more
        __syncwarp();
#pragma unroll 1
        for (int c = c_lo; c < min(c_hi, count); ++c) {
          const int ex = s_ex[c];
          if (!(ex & 1) && !rows_out) continue;
          const float o = scale2(w4::ld1(tmem + lane_addr + c), -(f + (ex >> 1))) +
                          left_out<kGroup, kZero>(p.x + (m0 + c) * p.K, p.wq + wr * (p.K >> 1), sw, wz, ex, fl,
                                                  kr.w0 * kG4StageK, min((int)p.K, (kr.w0 + kr.n) * kG4StageK));
          if (p.splits > 1)
            part[c * 128 + col] = o;
          else
            *reinterpret_cast<uint16_t*>(wring + c * kRow + col * 2) = f32_to_bf16_rn(o);
          __syncwarp();  // ld1 is a whole-warp instruction
        }
      }
      tc::fence_before();
    }
  }

  __syncwarp();
  if (p.splits > 1) {
    // the cluster's partial sums, added in the order of their K ranges
    w4::cluster_sync();
    if (warp == kMmaWarp) {
      tc::fence_after();
      tc::tmem_dealloc(tmem, 256);
    }
    if (!*abort_flag) {
      const uint32_t part = smem_u32(wring);
      const bool vec = (p.N & 3) == 0;
      for (int i = threadIdx.x; i < 32 * ((count - split + p.splits - 1) / p.splits); i += kThreads) {
        const int c = (i / 32) * p.splits + split, col = i % 32 * 4;
        if (n0 + col >= p.N) continue;
        float4 v[kG4MaxSplit];
#pragma unroll
        for (int s = 0; s < kG4MaxSplit; ++s)
          if (s < p.splits) v[s] = w4::ld_cluster(part + (uint32_t)(c * 128 + col) * 4u, (uint32_t)s);
        float4 sum = v[0];
#pragma unroll
        for (int s = 1; s < kG4MaxSplit; ++s)
          if (s < p.splits) sum.x += v[s].x, sum.y += v[s].y, sum.z += v[s].z, sum.w += v[s].w;
        uint16_t* out = p.y + (m0 + c) * p.N + n0 + col;
        if (vec) {
          *reinterpret_cast<uint2*>(out) =
              make_uint2(w4::f32x2_to_bf16x2(sum.x, sum.y), w4::f32x2_to_bf16x2(sum.z, sum.w));
        } else {
          const float o[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n0 + col + j < p.N) out[j] = f32_to_bf16_rn(o[j]);
        }
      }
    }
    __syncwarp();
    w4::cluster_sync();  // no CTA leaves while another reads its sums
  } else {
    __syncthreads();
    // before the copies below, in which a warp's lanes may part: dealloc is a
    // whole-warp instruction
    if (warp == kMmaWarp) {
      tc::fence_after();
      tc::tmem_dealloc(tmem, 256);
    }
    if (!*abort_flag) {
      constexpr int kRow = 128 * 2 + 16;
      const int cols = (int)min((int64_t)128, p.N - n0);
      if ((p.N & 7) == 0) {
        for (int i = threadIdx.x; i < count * 16; i += kThreads) {
          const int c = i / 16, b = i % 16;
          const int64_t row = m0 + c;
          if (b * 8 < cols)
            *reinterpret_cast<uint4*>(p.y + row * p.N + n0 + b * 8) =
                *reinterpret_cast<const uint4*>(wring + c * kRow + b * 16);
        }
      } else {
        for (int i = threadIdx.x; i < count * 128; i += kThreads) {
          const int c = i / 128, b = i % 128;
          const int64_t row = m0 + c;
          if (b < cols) p.y[row * p.N + n0 + b] = *reinterpret_cast<const uint16_t*>(wring + c * kRow + b * 2);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------- wide

// One tile of the persistent kernel: a row tile of 256 weights and up to ntok tokens.
struct WideTile {
  int64_t e, m0;  // expert; first token row
  int count, rt, tt;
  unsigned by;    // experts: the expert; dense: the token tile
  // The first of n weight stages (G4Range): by the expert and not by the token tile, since
  // which of its expert's tiles a pair stands in may depend on timing (w4_plan_kernel), and
  // the order of a sum must not.
  QL_DEVINL int rot(int n) const { return (int)((rt * 5 + by * 3) % (unsigned)n); }
};

template <bool kExperts>
QL_DEVINL WideTile wide_tile(const G4Params& p, int t) {
  WideTile w;
  w.tt = t / p.row_tiles;
  w.rt = t - w.tt * p.row_tiles;
  if constexpr (kExperts) {
    const G4Tile g = p.tiles[w.tt];
    w.e = g.expert;
    w.m0 = g.start;
    w.count = g.count;
    w.by = (unsigned)g.expert;
  } else {
    w.e = 0;
    w.by = (unsigned)w.tt;
    w.m0 = (int64_t)w.tt * p.ntok;
    w.count = (int)min((int64_t)p.ntok, p.M - w.m0);
  }
  return w;
}

// Any of the epilogue's threads (a barrier among them).
QL_DEVINL bool wide_epi_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "n"(kWideEpiWarps * 32)
      : "memory");
  return r != 0;
}

template <int kGroup, bool kZero, bool kExperts>
__global__ void __launch_bounds__(kWideThreads, 1)
    w4_wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const G4Params p) {
  const int xs_n = p.xstages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* wring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* xring = wring + kG4WStages * kWideWBytes;
  uint8_t* staging = xring + xs_n * p.xstage;
  uint64_t* wfull = reinterpret_cast<uint64_t*>(staging + kWideEpiWarps * 16 * kWideStageRow);
  uint64_t* wempty = wfull + kG4WStages;
  uint64_t* xfull = wempty + kG4WStages;
  uint64_t* xempty = xfull + kG4MaxXStages;
  uint64_t* afull = xempty + kG4MaxXStages;
  uint64_t* aempty = afull + 4;  // (afull, aempty: [row tile][slot]; dfull, dempty: [row tile])
  uint64_t* dfull = aempty + 4;
  uint64_t* dempty = dfull + 2;
  // [4][256] the rows' exponents: with short K the dequantizing warps are up to three
  // tiles ahead of the epilogue
  int* s_f = reinterpret_cast<int*>(wfull + kWideBarriers);
  int* s_out = s_f + 4 * 256;                                     // [2][kWideTok] experts: pairs
  int* s_ex = s_out + 2 * kWideTok;                               // [2][kWideTok] the columns' exponents
  float* s_fac = reinterpret_cast<float*>(s_ex + 2 * kWideTok);   // [2][kWideTok] 2^-exponent
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(s_fac + 2 * kWideTok);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  G4Range kr;
  kr.nk64 = (int)((p.K + kG4GranK - 1) / kG4GranK);
  kr.w0 = 0;
  kr.n = (int)((p.K + kG4StageK - 1) / kG4StageK);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kG4WStages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], kG4DequantWarps);
    }
    for (int s = 0; s < xs_n; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 2);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&afull[s], 4);
      mbar_init(&aempty[s], 1);
    }
    for (int r = 0; r < 2; ++r) {
      mbar_init(&dfull[r], 1);
      mbar_init(&dempty[r], kWideEpiWarps / 2);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tc::prefetch_tmap(&tmW);
    tc::prefetch_tmap(&tmX);
  }
  if (warp == kWideMma) {
    tc::tmem_alloc(tmem_holder, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tmem_a = tmem + 2 * kWideTok;
  tc::grid_dependency_wait();  // the prepare kernel's tokens, pairs and tiles
  tc::launch_dependents();
  const int tiles = p.row_tiles * (kExperts ? *p.ntiles : p.tok_tiles);
  bool ok = true;

  if (warp == kWideProducer) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t pol_w = l2_policy_evict_first();
    const uint64_t pol_x = l2_policy_evict_last();
    int jw = 0, jx = 0;  // issued stages
    int s = 0;           // token stage of the next granule, and how often it was filled
    uint32_t fill = 0;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const WideTile w = wide_tile<kExperts>(p, t);
      kr.rot = w.rot(kr.n);
      const int wrow = (int)(w.e * p.N + (int64_t)w.rt * 256);
      for (int j = 0; j < kr.n && ok; ++j) {
        const int v = jw % kG4WStages, ws = kr.stage(j);
        if (jw >= kG4WStages) ok = w4::wait(&wempty[v], ((jw / kG4WStages) - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&wfull[v], kWideWBytes);
          tc::tma_load_2d(wring + v * kWideWBytes, &tmW, ws * 128, wrow, &wfull[v], pol_w);
          tc::tma_load_2d(wring + v * kWideWBytes + 16384, &tmW, ws * 128, wrow + 128, &wfull[v], pol_w);
        }
        __syncwarp();
        ++jw;
        const int ng = kr.granules(ws);
        for (int gq = 0; gq < ng; ++gq) {
          if (fill > 0) ok = w4::wait(&xempty[s], (fill - 1) & 1, abort_flag);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&xfull[s], (uint32_t)p.ntok * 128u);
            tc::tma_load_2d(xring + s * p.xstage, &tmX, (ws * 4 + gq) * 128, (int)w.m0, &xfull[s], pol_x);
          }
          __syncwarp();
          ++jx;
          if (++s == xs_n) {
            s = 0;
            ++fill;
          }
        }
      }
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_timeout(p.status, KID_W4, 4);
      *abort_flag = 1;
      // the copies in flight land before the CTA leaves
      for (int j = max(0, jw - kG4WStages); j < jw; ++j)
        mbar_wait_bounded(&wfull[j % kG4WStages], (j / kG4WStages) & 1, nullptr);
      for (int j = max(0, jx - xs_n); j < jx; ++j) mbar_wait_bounded(&xfull[j % xs_n], (j / xs_n) & 1, nullptr);
    }
  } else if (warp == kWideMma || warp == kWideMma + 1) {
    // ------------------------------------------------------------ MMA issuers, one to a row tile
    const int r = warp - kWideMma;
    const uint32_t elected = w4::elect_one();
    const uint32_t tmem_a0 = __shfl_sync(0xffffffffu, tmem_a, 0);
    const uint32_t d = __shfl_sync(0xffffffffu, tmem, 0) + r * kWideTok, a = tmem_a0 + r * 64;  // warp-uniform
    const uint32_t x0 = smem_u32(xring);
    const int ngran = kr.total();
    int xs = 0, g = 0, it = 0;  // g: granules over all tiles
    uint32_t xphase = 0;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++it) {
      const WideTile w = wide_tile<kExperts>(p, t);
      const uint32_t id = w4::idesc_f16(128, (w.count + 15) & ~15);
      if (it > 0) ok = w4::wait(&dempty[r], (it - 1) & 1, abort_flag);  // the last tile's sums are read
      for (int j = 0; j < ngran && ok; ++j, ++g) {
        const int slot = g & 1;
        ok = w4::wait(&xfull[xs], xphase, abort_flag);
        ok = ok && w4::wait(&afull[r * 2 + slot], (g >> 1) & 1, abort_flag);
        if (!ok) break;
        tc::fence_after();
        const uint64_t bdesc = tc::sw128_desc(x0 + xs * p.xstage);
#pragma unroll
        for (int k = 0; k < 4; ++k) w4::mma_f16_ts(d, a + slot * 32 + k * 8, bdesc + 2 * k, id, j > 0 || k > 0, elected);
        w4::commit(&aempty[r * 2 + slot], elected);
        w4::commit(&xempty[xs], elected);
        if (++xs == xs_n) {
          xs = 0;
          xphase ^= 1;
        }
      }
      if (!ok) break;
      w4::commit(&dfull[r], elected);
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_timeout(p.status, KID_W4, 5);
      *abort_flag = 1;
      // the products in flight end before the CTA leaves
      w4::commit(&dfull[r], elected);
      w4::wait(&dfull[r], it & 1, nullptr);
    }
  } else if (warp < kG4DequantWarps) {
    // ------------------------------------------------------------ codes -> TMEM
    // Each four warps take a row tile; thread = weight row.
    const int r = warp >> 2, q = warp & 3;
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    const uint32_t row = (uint32_t)(r * 128 + q * 32 + lane);
    int g = 0, jw = 0, it = 0;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++it) {
      const WideTile w = wide_tile<kExperts>(p, t);
      kr.rot = w.rot(kr.n);
      const int64_t wr = w.e * p.N + min((int64_t)w.rt * 256 + row, p.N - 1);
      const uint16_t* sw = p.sw + wr * p.groups;
      const uint8_t* wz = kZero ? p.wz + wr * p.groups : nullptr;
      G4Scales<kGroup, kZero, 1> sc;
      sc.load(sw, wz, kr.stage(0), 0, p.groups);
      const int fl = row_exponent(sw, 0, p.groups, (p.groups & 7) == 0), f = fl >> 1;
      const uint32_t below = left_out_below(f);
      s_f[(it & 3) * 256 + row] = fl;
      for (int j = 0; j < kr.n && ok; ++j, ++jw) {
        const int ws = jw % kG4WStages, ng = kr.granules(kr.stage(j));
        sc.convert(f, below);
        if (j + 1 < kr.n) sc.load(sw, wz, kr.stage(j + 1), 0, p.groups);
        ok = w4::wait(&wfull[ws], (jw / kG4WStages) & 1, abort_flag);
        if (!ok) break;
        const uint8_t* src = wring + ws * kWideWBytes + row * 128;
        uint32_t c[8];
        sc.codes(src, 0, (uint32_t)(lane & 7), c);
#pragma unroll
        for (int gq = 0; gq < 4; ++gq) {
          if (gq >= ng) break;
          uint32_t h[32];
          sc.granule(c, gq, h);
          if (gq < 3) sc.codes(src, gq + 1, (uint32_t)(lane & 7), c);
          const int slot = g & 1, use = g >> 1;
          if (use > 0) ok = w4::wait(&aempty[r * 2 + slot], (use - 1) & 1, abort_flag);
          if (!ok) break;
          tc::fence_after();
          w4::st32(tmem_a + (r * 2 + slot) * 32 + lane_addr, h);
          w4::st_wait();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&afull[r * 2 + slot]);
          ++g;
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[ws]);
      }
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_timeout(p.status, KID_W4, 6);
      *abort_flag = 1;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // While the next tile's first weights are dequantized: a warp's 32 rows, 16 tokens
    // at a time, through its own staging so that they leave in 16-byte stores.
    const int ew = warp - kWideFirstEpi, r = ew >> 2, q = warp & 3;
    const int et = threadIdx.x - kWideFirstEpi * 32;
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    uint8_t* stg = staging + ew * 16 * kWideStageRow;
    const bool vec = (p.N & 7) == 0;
    int it = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
      const WideTile w = wide_tile<kExperts>(p, t);
      const int buf = (it & 1) * kWideTok;
      bool wide = false;
      if (et < w.count) {
        const int ex = p.ex[w.m0 + et];
        if constexpr (kExperts) s_out[buf + et] = p.order[w.m0 + et];
        s_ex[buf + et] = ex;
        s_fac[buf + et] = exp2i(max(-126, min(126, -(ex >> 1))));
        wide = abs(ex >> 1) > 60 || (ex & 1);
      }
      wide = wide_epi_any(wide);  // an exponent that one factor cannot take, or values left out
      ok = w4::wait(&dfull[r], it & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok && !*abort_flag);
      if (wide_epi_any(!ok)) break;
      tc::fence_after();
      const int fl = s_f[(it & 3) * 256 + r * 128 + q * 32 + lane], f = fl >> 1;
      const bool rows_out = __any_sync(0xffffffffu, fl & 1);
      wide = __any_sync(0xffffffffu, wide || abs(f) > 60) || rows_out;
      const float rf = exp2i(max(-126, min(126, -f)));
      const int64_t nw = (int64_t)w.rt * 256 + r * 128 + q * 32;  // the warp's first output
      uint16_t* yb = p.y + nw + (lane & 3) * 8;                    // this lane's piece of an output row
      const bool inside = nw + (lane & 3) * 8 < p.N;
      const uint8_t* src = stg + (lane >> 2) * kWideStageRow + (lane & 3) * 16;
      const int mma_n = (w.count + 15) & ~15;
      for (int c = 0; c < mma_n; c += 16) {
        uint32_t v[16];
        w4::ld16(tmem + r * kWideTok + lane_addr + c, v);
        tc::ld_wait();
        if (c + 16 >= mma_n && !wide) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&dempty[r]);
        }
        float o[16];
        if (!wide) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 fac = *reinterpret_cast<const float4*>(s_fac + buf + c + i);
            o[i] = __uint_as_float(v[i]) * rf * fac.x;
            o[i + 1] = __uint_as_float(v[i + 1]) * rf * fac.y;
            o[i + 2] = __uint_as_float(v[i + 2]) * rf * fac.z;
            o[i + 3] = __uint_as_float(v[i + 3]) * rf * fac.w;
          }
        } else {  // the two factors may leave f32's range where their product does not
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = scale2(__uint_as_float(v[i]), -(f + (c + i < w.count ? s_ex[buf + c + i] >> 1 : 0)));
        }
        if (kExperts && p.yp) {  // f32: half the tokens at a time fit the staging
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) *reinterpret_cast<float*>(stg + i * kWideStageRowF32 + lane * 4) = o[h + i];
            __syncwarp();
            if (p.N & 3) {
              for (int i = 0; i < 8; ++i)
                if (c + h + i < w.count && nw + lane < p.N)
                  p.yp[s_out[buf + c + h + i] * p.N + nw + lane] =
                      *reinterpret_cast<const float*>(stg + i * kWideStageRowF32 + lane * 4);
            } else if (nw + (lane & 7) * 4 < p.N) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int row = i * 4 + (lane >> 3), tok = c + h + row;
                if (tok < w.count)
                  *reinterpret_cast<float4*>(p.yp + s_out[buf + tok] * p.N + nw + (lane & 7) * 4) =
                      *reinterpret_cast<const float4*>(stg + row * kWideStageRowF32 + (lane & 7) * 16);
              }
            }
            __syncwarp();
          }
        } else if (vec) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<uint16_t*>(stg + i * kWideStageRow + lane * 2) = f32_to_bf16_rn(o[i]);
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int tok = c + h * 8 + (lane >> 2);
            if (tok < w.count && inside) {
              uint16_t* out = kExperts ? yb + s_out[buf + tok] * p.N : yb + (w.m0 + tok) * p.N;
              *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(src + h * 8 * kWideStageRow);
            }
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i >= w.count || nw + lane >= p.N) continue;
            const int64_t orow = kExperts ? s_out[buf + c + i] : w.m0 + c + i;
            p.y[orow * p.N + nw + lane] = f32_to_bf16_rn(o[i]);
          }
        }
      }
      if (wide) {  // tokens with something left out once more, then the accumulators are free
        __syncwarp();  // (other lanes wrote these outputs above)
#pragma unroll 1
        for (int c = 0; c < w.count; ++c) {
          const int ex = s_ex[buf + c];
          if (!(ex & 1) && !rows_out) continue;
          const int64_t wr = w.e * p.N + min(nw + lane, p.N - 1), orow = kExperts ? s_out[buf + c] : w.m0 + c;
          const float o = scale2(w4::ld1(tmem + r * kWideTok + lane_addr + c), -(f + (ex >> 1))) +
                          left_out<kGroup, kZero>(p.x + (kExperts ? orow / p.slots : orow) * p.K, p.wq + wr * (p.K >> 1),
                                                  p.sw + wr * p.groups, kZero ? p.wz + wr * p.groups : nullptr, ex, fl,
                                                  0, (int)p.K);
          if (nw + lane < p.N) {
            if (kExperts && p.yp)
              p.yp[orow * p.N + nw + lane] = o;
            else
              p.y[orow * p.N + nw + lane] = f32_to_bf16_rn(o);
          }
          __syncwarp();  // ld1 is a whole-warp instruction
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&dempty[r]);
      }
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_timeout(p.status, KID_W4, 7);
      *abort_flag = 1;
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == kWideMma) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------- prepare

struct G4PrepParams {
  const uint16_t* x;
  uint16_t* x16;
  int* ex;
  int64_t K;
  // experts
  const int32_t* ids;
  int64_t pairs;
  int E, ntok;
  int slots;             // pairs of an x row: topk (gather) or 1 (combine)
  int* order;            // [pairs] the pairs by expert
  int* pos;              // [pairs] many pairs: their places in `order` (-1: id out of range); else null
  G4Tile* tiles;
  int* ntiles;
  uint16_t* zero_y;      // gather: the result, whose rows of an id out of range are zeroed
  int64_t N;
};

// do_(pair, its expert or -1) for this thread's pairs, eight loads in flight.
template <class Do>
QL_DEVINL void each_id(const G4PrepParams& p, Do do_) {
  for (int64_t i0 = threadIdx.x; i0 < p.pairs; i0 += 8 * kG4PlanThreads) {
    int e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = i0 + j * kG4PlanThreads < p.pairs ? __ldg(p.ids + i0 + j * kG4PlanThreads) : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j * kG4PlanThreads < p.pairs) do_(i0 + j * kG4PlanThreads, e[j] < p.E ? e[j] : -1);
  }
}

// Cuts the experts' pairs, in expert order, into token tiles; one thread per expert.
// Returns the first place of expert threadIdx.x's pairs.
QL_DEVINL int plan_tiles(const G4PrepParams& p, int* hist) {
  __shared__ int warp_sums[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  hist[tid] = 0;
  __syncthreads();
  each_id(p, [&](int64_t, int e) {
    if (e >= 0) atomicAdd(&hist[e], 1);
  });
  __syncthreads();
  // exclusive sums of the pairs and of the tiles
  const int c = hist[tid], t = (c + p.ntok - 1) / p.ntok;
  int ci = c, ti = t;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, ci, o), b = __shfl_up_sync(0xffffffffu, ti, o);
    if (lane >= o) {
      ci += a;
      ti += b;
    }
  }
  if (lane == 31) {
    warp_sums[0][warp] = ci;
    warp_sums[1][warp] = ti;
  }
  __syncthreads();
  if (warp == 0) {
    int a = warp_sums[0][lane], b = warp_sums[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, a, o), v = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) {
        a += u;
        b += v;
      }
    }
    warp_sums[0][lane] = a;
    warp_sums[1][lane] = b;
  }
  __syncthreads();
  if (warp > 0) {
    ci += warp_sums[0][warp - 1];
    ti += warp_sums[1][warp - 1];
  }
  const int per = t ? ((c + t - 1) / t + 15) & ~15 : 0;  // an expert's tiles are alike
  for (int i = 0; i < t; ++i) p.tiles[ti - t + i] = G4Tile{tid, ci - c + i * per, min(per, c - i * per), 0};
  if (tid == kG4PlanThreads - 1) *p.ntiles = ti;
  return ci - c;
}

// Many pairs: one block plans and gives every pair its place.  The order inside an
// expert depends on timing; results do not, since a pair is one MMA column wherever it
// stands, and all of an expert's tiles take K in the same order (WideTile::rot).
__global__ void __launch_bounds__(kG4PlanThreads) w4_plan_kernel(const G4PrepParams p) {
  __shared__ int hist[kG4PlanThreads];
  tc::grid_dependency_wait();
  tc::launch_dependents();
  const int base = plan_tiles(p, hist);
  __syncthreads();
  hist[threadIdx.x] = base;
  __syncthreads();
  each_id(p, [&](int64_t i, int e) { p.pos[i] = e >= 0 ? atomicAdd(&hist[e], 1) : -1; });
}

// The largest finite magnitude, and the smallest nonzero one less one.
struct G4Span {
  uint32_t top = 0, low = 0xFFFFFFFFu;
  QL_DEVINL void add(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = w[j] & 0x7FFFu, b = w[j] >> 16 & 0x7FFFu;
      if (a < 0x7F80u) top = max(top, a);
      if (b < 0x7F80u) top = max(top, b);
      low = min(low, min(a - 1u, b - 1u));
    }
  }
};

// A row of x for the threads of a warp (kBlock false) or of a block, held in registers
// (kHold pieces a thread) from the search for its largest value to its conversion; a
// longer row's rest is read twice.
template <bool kBlock, int kHold>
struct G4Row {
  const uint4* src;
  int chunks, first, step;  // pieces of 8 inputs, this thread's first, and from one to the next
  uint4 v[kHold];

  QL_DEVINL G4Row(const uint16_t* row, int64_t K)
      : src(reinterpret_cast<const uint4*>(row)),
        chunks((int)(K / 8)),
        first(kBlock ? threadIdx.x : threadIdx.x & 31),
        step(kBlock ? blockDim.x : 32) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (first + i * step < chunks) v[i] = __ldg(src + first + i * step);
    }
  }
  // 2 e + 1 if values are left out, else 2 e: e the power of two that brings the row's largest
  // finite |x| to [2^14, 2^15).
  QL_DEVINL int exponent(uint32_t (*red)[2]) const {
    G4Span a;
#pragma unroll
    for (int i = 0; i < kHold; ++i) a.add(v[i]);
    for (int i = first + kHold * step; i < chunks; i += step) a.add(__ldg(src + i));
    a.top = __reduce_max_sync(0xffffffffu, a.top);
    a.low = __reduce_min_sync(0xffffffffu, a.low);
    if constexpr (kBlock) {
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][0] = a.top, red[threadIdx.x >> 5][1] = a.low;
      __syncthreads();
      for (int i = 0; i < (int)blockDim.x / 32; ++i) a.top = max(a.top, red[i][0]), a.low = min(a.low, red[i][1]);
    }
    const int e = 14 - log2_bf16(a.top, 14);
    return 2 * e + leaves_out(a.low, e);
  }
  // store(piece, its number) for this thread's pieces.
  template <class Store>
  QL_DEVINL void each(Store store) const {
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (first + i * step < chunks) store(v[i], first + i * step);
    for (int i = first + kHold * step; i < chunks; i += step) store(__ldg(src + i), i);
  }
};

// Scales eight inputs by a token's 2^e, in the order 0 4 1 5 2 6 3 7.
struct G4Scaler {
  float f0, f1;
  uint32_t below;  // magnitudes that are left out: 0 where none is

  QL_DEVINL explicit G4Scaler(int ex)
      : f0(exp2i((ex >> 1) / 2)), f1(exp2i((ex >> 1) - (ex >> 1) / 2)), below(ex & 1 ? left_out_below(ex >> 1) : 0u) {}
  QL_DEVINL uint4 operator()(const uint4& v) const {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (below) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if ((w[j] & 0x7FFFu) < below) w[j] &= 0xFFFF0000u;
        if ((w[j] >> 16 & 0x7FFFu) < below) w[j] &= 0xFFFFu;
      }
    }
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16_lo(w[j]) * f0 * f1;
      x[2 * j + 1] = bf16_hi(w[j]) * f0 * f1;
    }
    return make_uint4(w4::f32x2_to_f16x2(x[0], x[4]), w4::f32x2_to_f16x2(x[1], x[5]),
                      w4::f32x2_to_f16x2(x[2], x[6]), w4::f32x2_to_f16x2(x[3], x[7]));
  }
};

__global__ void __launch_bounds__(kG4PrepThreads) w4_prepare_kernel(const G4PrepParams p) {
  __shared__ uint32_t red[32][2];
  tc::grid_dependency_wait();
  tc::launch_dependents();
  const int64_t row = blockIdx.x;
  const G4Row<true, 4> x(p.x + row * p.K, p.K);
  const int e = x.exponent(red);
  if (threadIdx.x == 0) p.ex[row] = e;
  const G4Scaler scaled(e);
  uint4* dst = reinterpret_cast<uint4*>(p.x16 + row * p.K);
  x.each([&](const uint4& v, int i) { dst[i] = scaled(v); });
}

// A pair's place in expert order (-1: no expert), counted by its warp.
QL_DEVINL int count_place(const G4PrepParams& p, int pair) {
  const int e = __ldg(p.ids + pair);
  int before = 0;
#pragma unroll 8
  for (int i = threadIdx.x & 31; i < (int)p.pairs; i += 32) {
    const int o = __ldg(p.ids + i);
    before += (o >= 0 && o < e) || (o == e && i < pair);
  }
  before = __reduce_add_sync(0xffffffffu, before);
  return e >= 0 && e < p.E ? before : -1;
}

// Experts: a block takes an x row and writes it once for each of its pairs, in expert
// order, so that a tile's tokens are one box for TMA.  (Gathering them in the product
// instead, with TMA's gather of four rows or with 16-byte asynchronous copies, took 1100
// and 1700 cycles for a granule of 170 tokens whose MMAs take 680.)  Few pairs: every
// warp counts its pair's place itself, and block 0 plans the tiles beside the others.
__global__ void __launch_bounds__(kG4PlanThreads) w4_prepare_experts_kernel(const G4PrepParams p) {
  __shared__ int hist[kG4PlanThreads];
  __shared__ uint32_t red[32][2];
  __shared__ int s_pos[32];
  tc::grid_dependency_wait();
  tc::launch_dependents();
  int64_t row = blockIdx.x;
  if (!p.pos) {
    if (row == 0) {
      plan_tiles(p, hist);
      return;
    }
    --row;
    for (int j = threadIdx.x >> 5; j < p.slots; j += blockDim.x / 32) {
      const int pos = count_place(p, (int)row * p.slots + j);
      if ((threadIdx.x & 31) == 0) s_pos[j] = pos;
    }
  } else if (threadIdx.x < p.slots) {
    s_pos[threadIdx.x] = p.pos[row * p.slots + threadIdx.x];
  }
  const G4Row<true, 1> x(p.x + row * p.K, p.K);
  const int e = x.exponent(red);  // (and a barrier behind s_pos)
  const G4Scaler scaled(e);
  if (threadIdx.x < p.slots && s_pos[threadIdx.x] >= 0) {
    p.ex[s_pos[threadIdx.x]] = e;
    p.order[s_pos[threadIdx.x]] = (int)row * p.slots + threadIdx.x;
  }
  x.each([&](const uint4& v, int i) {
    const uint4 h = scaled(v);
    for (int j = 0; j < p.slots; ++j)
      if (s_pos[j] >= 0) reinterpret_cast<uint4*>(p.x16 + (int64_t)s_pos[j] * p.K)[i] = h;
  });
  if (p.zero_y) {
    for (int j = 0; j < p.slots; ++j) {
      if (s_pos[j] >= 0) continue;
      for (int64_t n = threadIdx.x; n < p.N; n += blockDim.x) p.zero_y[(row * p.slots + j) * p.N + n] = 0;
    }
  }
}

// Pairs with an x row each: a warp takes a row.
__global__ void __launch_bounds__(kG4PlanThreads) w4_prepare_pairs_kernel(const G4PrepParams p) {
  __shared__ int hist[kG4PlanThreads];
  tc::grid_dependency_wait();
  tc::launch_dependents();
  if (!p.pos && blockIdx.x == 0) {
    plan_tiles(p, hist);
    return;
  }
  const int64_t row = (int64_t)(blockIdx.x - (p.pos ? 0 : 1)) * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (row >= p.pairs) return;
  const int pos = p.pos ? p.pos[row] : count_place(p, (int)row);
  const G4Row<false, 4> x(p.x + row * p.K, p.K);
  if (pos < 0) return;
  const int e = x.exponent(nullptr);
  const G4Scaler scaled(e);
  if ((threadIdx.x & 31) == 0) {
    p.ex[pos] = e;
    p.order[pos] = (int)row;
  }
  uint4* dst = reinterpret_cast<uint4*>(p.x16 + (int64_t)pos * p.K);
  x.each([&](const uint4& v, int i) { dst[i] = scaled(v); });
}

// y[t] = sum_j weights[t, j] yp[t, j] in the order of j, all in f32: the terms of a token may
// cancel, so a rounded term could be off by more than the whole result's rounding.  A thread
// takes kVec neighbouring outputs; bound by the pairs' bytes.
template <int kVec>
__global__ void __launch_bounds__(256, 5) w4_combine_kernel(const float* __restrict__ yp, const int32_t* __restrict__ ids,
                                                         const float* __restrict__ weights, int topk, int E, int64_t N,
                                                         int64_t T, uint16_t* __restrict__ y) {
  tc::grid_dependency_wait();
  tc::launch_dependents();
  const int64_t per = N / kVec, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= T * per) return;
  const int64_t t = at / per, n = (at - t * per) * kVec;
  const int32_t* id = ids + t * topk;
  const float *wt = weights + t * topk, *first = yp + t * topk * N + n;
  float sum[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) sum[i] = 0.0f;
  constexpr int kAhead = 4;  // pairs whose products are loaded before the first is added (8: fewer warps fit, 3 % of a call)
  for (int j0 = 0; j0 < topk; j0 += kAhead) {
    float w[kAhead];
    bool use[kAhead];
    float4 v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int e = j0 + j < topk ? __ldg(id + j0 + j) : -1;
      use[j] = e >= 0 && e < E;
      w[j] = use[j] ? __ldg(wt + j0 + j) : 0.0f;
      if (!use[j]) continue;  // (not a product with zero: the place holds anything)
      const float* src = first + (j0 + j) * N;
      if constexpr (kVec == 4)
        v[j] = *reinterpret_cast<const float4*>(src);
      else
        v[j].x = *src;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!use[j]) continue;
      sum[0] = fmaf(w[j], v[j].x, sum[0]);
      if constexpr (kVec == 4) {
        sum[1] = fmaf(w[j], v[j].y, sum[1]);
        sum[2] = fmaf(w[j], v[j].z, sum[2]);
        sum[3] = fmaf(w[j], v[j].w, sum[3]);
      }
    }
  }
  if constexpr (kVec == 4) {
    *reinterpret_cast<uint2*>(y + t * N + n) =
        make_uint2(w4::f32x2_to_bf16x2(sum[0], sum[1]), w4::f32x2_to_bf16x2(sum[2], sum[3]));
  } else {
    y[t * N + n] = f32_to_bf16_rn(sum[0]);
  }
}

// ---------------------------------------------------------------------------- host

namespace {

struct G4Plan {
  bool wide;
  int ntok, splits;
  unsigned row_tiles, tok_tiles;
};

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One weight tile and K split over clusters: as many CTAs as the SMs hold, two each.
G4Plan plan_narrow(int64_t M, const ql_w4_weight& w, int sms) {
  G4Plan g;
  g.wide = false;
  g.row_tiles = (unsigned)div_up(w.N, 128);
  g.tok_tiles = (unsigned)div_up(M, kNarrowTok);
  g.ntok = (int)div_up(div_up(M, g.tok_tiles), 16) * 16;
  g.splits = 1;
  const int64_t stages = div_up(w.K, kG4StageK);
  while (g.splits < kG4MaxSplit && g.splits * 2 <= stages &&
         (int64_t)g.row_tiles * g.tok_tiles * g.splits * 2 <= 2 * sms)
    g.splits *= 2;
  return g;
}

G4Plan plan_wide(int64_t M, const ql_w4_weight& w, int sms) {
  G4Plan g;
  g.wide = true;
  g.row_tiles = (unsigned)div_up(w.N, 256);
  g.splits = 1;
  // tokens of a tile: fewest rounds of the SMs, each round's time about its tokens
  g.ntok = kWideTok;
  double best = 1e30;
  for (int n = kWideTok; n >= 96; n -= 16) {
    const double cost = (double)div_up(g.row_tiles * div_up(M, n), sms) * (n + 16);
    if (cost < best) {
      best = cost;
      g.ntok = n;
    }
  }
  g.tok_tiles = (unsigned)div_up(M, g.ntok);
  return g;
}

G4Plan plan_dense(int64_t M, const ql_w4_weight& w, int sms) {
  const G4Plan n = plan_narrow(M, w, sms);
  if (M <= kNarrowTok) return n;
  // Few wide tiles leave SMs without work while each of them walks all of K, whatever its
  // tokens (about 0.44 us a granule); two narrow tiles on an SM take about 1.25 times that
  // for theirs (K = 4096, narrow against wide: 129 tokens 4096 rows 17.5 and 33 us, 512
  // tokens 30.7 and 37.2, 1000 tokens 41.0 and 38.8; 512 tokens 1024 rows 19.9 and 35.2).
  const G4Plan g = plan_wide(M, w, sms);
  const int64_t gran = div_up(w.K, kG4GranK);
  const double wide = (double)div_up((int64_t)g.row_tiles * g.tok_tiles, sms) * gran;
  const double narrow = 1.25 * div_up((int64_t)n.row_tiles * n.tok_tiles * n.splits, 2 * sms) * div_up(gran, n.splits);
  return narrow < wide && n.tok_tiles <= 65535u ? n : g;
}

// Experts always take wide tiles (64 experts, 8 to a token: 2048 x 768 combined 20 tokens
// 26 us against 32 in narrow ones, 256 tokens 41 against 48; 1536 x 2048 512 tokens 62
// against 82).  A tile's token loads are ntok rows whatever its expert has, and an expert
// with more takes another tile: four times the mean of the pairs up to 128 (1536 x 2048,
// 256 tokens, mean 32: 48 rows 67 us, 128 rows 56; 64 tokens, mean 8: 32 rows 50), then 192
// (2048 x 768, mean 127: 128 rows 69 us, 192 rows 66).
G4Plan plan_experts(int64_t pairs, const ql_w4_weight& w) {
  G4Plan g;
  const int64_t per = div_up(pairs, w.experts);
  g.splits = 1;
  g.wide = true;
  g.row_tiles = (unsigned)div_up(w.N, 256);
  g.ntok = per > 80 ? kWideTok : (int)std::min<int64_t>(128, std::max<int64_t>(32, div_up(per, 4) * 16));
  g.tok_tiles = (unsigned)(std::min<int64_t>(w.experts, pairs) + pairs / g.ntok);
  return g;
}

struct G4Layout {
  size_t x16, ex, order, pos, tiles, ntiles, yp, total;
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

G4Layout g4_layout(int64_t rows, int64_t K, int64_t pairs, unsigned tiles, int64_t yp_elems) {
  G4Layout L;
  size_t off = 0;
  L.x16 = off;
  off += up256((size_t)rows * K * 2);
  L.ex = off;
  off += up256((size_t)rows * 4);
  L.order = off;
  off += up256((size_t)pairs * 4);
  L.pos = off;
  off += up256((size_t)pairs * 4);
  L.tiles = off;
  off += up256((size_t)tiles * sizeof(G4Tile));
  L.ntiles = off;
  off += 256;
  L.yp = off;
  off += up256((size_t)yp_elems * 4);
  L.total = off + kWorkspaceTail;  // not ours to write
  return L;
}

template <auto kKernel>
cudaError_t launch_g4_kernel(const CUtensorMap& tw, const CUtensorMap& tx, const G4Params& p, dim3 grid, int threads,
                             int smem, cudaStream_t st) {
  cudaError_t e = ensure_smem<kKernel>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kKernel, tw, tx, p);
}

template <int kGroup, bool kZero, bool kExperts>
cudaError_t launch_g4_t(const CUtensorMap& tw, const CUtensorMap& tx, const G4Params& p, const G4Plan& g, int sms,
                        cudaStream_t st) {
  const int ring = kG4WStages * (g.wide ? kWideWBytes : kNarrowWBytes) + p.xstages * p.xstage;
  if constexpr (!kExperts) {
    if (!g.wide) {
      const int smem = 1024 + ring + 8 * (2 * kG4WStages + 2 * kG4MaxXStages + 2 * kNarrowSlots + 2) + 8 * kNarrowTok + 16;
      return launch_g4_kernel<w4_narrow_kernel<kGroup, kZero>>(tw, tx, p, dim3(g.row_tiles * g.splits, g.tok_tiles),
                                                               kNarrowThreads, smem, st);
    }
  }
  const int smem = 1024 + ring + kWideEpiWarps * 16 * kWideStageRow + kWideBarriers * 8 + 4 * 256 * 4 + 6 * kWideTok * 4 + 16;
  const unsigned grid = (unsigned)std::min<int64_t>(sms, (int64_t)g.row_tiles * g.tok_tiles);
  return launch_g4_kernel<w4_wide_kernel<kGroup, kZero, kExperts>>(tw, tx, p, dim3(grid), kWideThreads, smem, st);
}

template <bool kExperts>
cudaError_t launch_g4(const ql_w4_weight& w, const uint16_t* x16, int64_t rows, G4Params p, const G4Plan& g, int sms,
                      cudaStream_t st) {
  if ((int64_t)g.tok_tiles * g.row_tiles >= (int64_t(1) << 31)) return cudaErrorNotSupported;
  CUtensorMap tw, tx;
  cudaError_t e = make_tmap_u8_sw128(&tw, w.wq, (uint64_t)w.K / 2, (uint64_t)w.experts * w.N, (uint64_t)w.K / 2, 128, 128);
  if (e != cudaSuccess) return e;
  e = make_tmap_u8_sw128(&tx, x16, (uint64_t)w.K * 2, (uint64_t)rows, (uint64_t)w.K * 2, 128, g.ntok);
  if (e != cudaSuccess) return e;
  p.wq = static_cast<const uint8_t*>(w.wq);
  p.sw = w.sw;
  p.wz = w.wz;
  p.N = w.N;
  p.K = w.K;
  p.groups = (int)div_up(w.K, w.group);
  p.ntok = g.ntok;
  p.row_tiles = (int)g.row_tiles;
  p.tok_tiles = (int)g.tok_tiles;
  p.xstage = (int)div_up(g.ntok * 128, 1024) * 1024;
  p.splits = g.splits;
  p.xstages = std::min(kG4MaxXStages, std::max(3, (g.wide ? kWideRing : kNarrowRing) / p.xstage));
  if (w.group == 128)
    return w.wz ? launch_g4_t<128, true, kExperts>(tw, tx, p, g, sms, st)
                : launch_g4_t<128, false, kExperts>(tw, tx, p, g, sms, st);
  if (w.group == 64)
    return w.wz ? launch_g4_t<64, true, kExperts>(tw, tx, p, g, sms, st)
                : launch_g4_t<64, false, kExperts>(tw, tx, p, g, sms, st);
  return w.wz ? launch_g4_t<32, true, kExperts>(tw, tx, p, g, sms, st)
              : launch_g4_t<32, false, kExperts>(tw, tx, p, g, sms, st);
}

cudaError_t launch_pdl(void (*kernel)(const G4PrepParams), unsigned grid, unsigned block, const G4PrepParams& p,
                       cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

// Up to here the mma.sync kernel.  Dense, 14336 x 4096: 16 tokens 17.4 us against 20.4, 24
// tokens 34 against 21.  64 experts of which a token takes 8, 16 tokens: 2048 x 768
// combined 26.9 against 31.7, 1536 x 2048 45.1 against 44.3; 32 tokens 50 against 35 and
// 86 against 52.
constexpr int64_t kW4StreamMaxTokens = 16;
constexpr int64_t kW4StreamMaxExpertTokens = 16;
// And the mma.sync kernel, a block of tokens after the other, for rows longer than any
// layer's: where all of a tile is left out (left_out), its epilogue walks every token's row
// for every weight row, and that must end well within the 2 s that other warps wait for it.
constexpr int64_t kW4TensorMaxK = 65536;

size_t w4_workspace_bytes(int64_t M, const ql_w4_weight& w, int sms) {
  if (M <= kW4StreamMaxTokens || w.K > kW4TensorMaxK) return 0;
  return g4_layout(M, w.K, 0, 0, 0).total;
}

cudaError_t launch_w4(const uint16_t* x, const ql_w4_weight& w, int64_t M, uint16_t* y, void* workspace, int sms,
                      DevStatus* status, cudaStream_t st) {
  if (M <= kW4StreamMaxTokens) return launch_w4_stream(x, w, M, y, sms, st);
  if (w.K > kW4TensorMaxK) {
    cudaError_t e = cudaSuccess;
    for (int64_t m = 0; m < M && e == cudaSuccess; m += kW4StreamMaxTokens)
      e = launch_w4_stream(x + m * w.K, w, std::min(M - m, kW4StreamMaxTokens), y + m * w.N, sms, st);
    return e;
  }
  const G4Plan g = plan_dense(M, w, sms);
  const G4Layout L = g4_layout(M, w.K, 0, 0, 0);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  G4PrepParams q = {};
  q.x = x;
  q.x16 = reinterpret_cast<uint16_t*>(ws + L.x16);
  q.ex = reinterpret_cast<int*>(ws + L.ex);
  q.K = w.K;
  cudaError_t e = launch_pdl(w4_prepare_kernel, (unsigned)M, kG4PrepThreads, q, st);
  if (e != cudaSuccess) return e;
  G4Params p = {};
  p.x = x;
  p.y = y;
  p.ex = q.ex;
  p.M = M;
  p.status = status;
  return launch_g4<false>(w, q.x16, M, p, g, sms, st);
}

size_t w4_experts_workspace_bytes(int64_t T, int64_t topk, const ql_w4_weight& w, bool combine, int sms) {
  if (T <= kW4StreamMaxExpertTokens || w.K > kW4TensorMaxK) return 0;
  const int64_t pairs = T * topk;
  const G4Plan g = plan_experts(pairs, w);
  return g4_layout(pairs, w.K, pairs, g.tok_tiles, combine ? pairs * w.N : 0).total;
}

cudaError_t launch_w4_experts(const uint16_t* x, const int32_t* ids, const float* weights, const ql_w4_weight& w,
                              int64_t T, int64_t topk, uint16_t* y, void* workspace, int sms, DevStatus* status,
                              cudaStream_t st) {
  const bool combine = weights != nullptr;
  if (T <= kW4StreamMaxExpertTokens || w.K > kW4TensorMaxK) {
    constexpr int64_t kBlock = 1 << 18;  // tokens of a launch: its grid
    cudaError_t e = cudaSuccess;
    for (int64_t t = 0; t < T && e == cudaSuccess; t += kBlock)
      e = launch_w4_stream_experts(x + t * w.K * (combine ? topk : 1), ids + t * topk,
                                   combine ? weights + t * topk : nullptr, w, std::min(T - t, kBlock), topk,
                                   y + t * w.N * (combine ? 1 : topk), sms, st);
    return e;
  }
  const int64_t pairs = T * topk;
  const G4Plan g = plan_experts(pairs, w);
  const G4Layout L = g4_layout(pairs, w.K, pairs, g.tok_tiles, combine ? pairs * w.N : 0);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  G4PrepParams q = {};
  q.x = x;
  q.x16 = reinterpret_cast<uint16_t*>(ws + L.x16);
  q.ex = reinterpret_cast<int*>(ws + L.ex);
  q.K = w.K;
  q.ids = ids;
  q.pairs = pairs;
  q.E = (int)w.experts;
  q.ntok = g.ntok;
  q.slots = combine ? 1 : (int)topk;
  q.order = reinterpret_cast<int*>(ws + L.order);
  q.tiles = reinterpret_cast<G4Tile*>(ws + L.tiles);
  q.ntiles = reinterpret_cast<int*>(ws + L.ntiles);
  q.zero_y = combine ? nullptr : y;
  q.N = w.N;
  cudaError_t e;
  if (pairs > kG4CountPairs) {
    q.pos = reinterpret_cast<int*>(ws + L.pos);
    if ((e = launch_pdl(w4_plan_kernel, 1, kG4PlanThreads, q, st)) != cudaSuccess) return e;
    e = combine ? launch_pdl(w4_prepare_pairs_kernel, (unsigned)div_up(pairs, 8), 256, q, st)
                : launch_pdl(w4_prepare_experts_kernel, (unsigned)T, 256, q, st);
  } else {
    e = combine ? launch_pdl(w4_prepare_pairs_kernel, (unsigned)div_up(pairs, kG4PlanThreads / 32) + 1, kG4PlanThreads, q, st)
                : launch_pdl(w4_prepare_experts_kernel, (unsigned)T + 1, kG4PlanThreads, q, st);
  }
  if (e != cudaSuccess) return e;
  G4Params p = {};
  p.y = y;
  p.x = x;
  p.slots = q.slots;
  p.yp = combine ? reinterpret_cast<float*>(ws + L.yp) : nullptr;
  p.ex = q.ex;
  p.order = q.order;
  p.tiles = q.tiles;
  p.ntiles = q.ntiles;
  p.status = status;
  e = launch_g4<true>(w, q.x16, pairs, p, g, sms, st);
  if (e != cudaSuccess || !combine) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t threads = w.N % 4 ? T * w.N : T * (w.N / 4);
  if (div_up(threads, 256) >= (int64_t(1) << 31)) return cudaErrorNotSupported;
  cfg.gridDim = dim3((unsigned)div_up(threads, 256));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, w.N % 4 ? w4_combine_kernel<1> : w4_combine_kernel<4>, (const float*)p.yp, ids,
                            weights, (int)topk, (int)w.experts, w.N, T, y);
}

}  // namespace ql
