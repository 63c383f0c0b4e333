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
// f16 carries both operands without loss.  A scaled weight (q - z) s has at most 3 + 8
// significant bits for z = 8 and 4 + 8 with zero points, f16 has 11; x is bf16, 8
// bits.  Their exponents are brought into f16's range by powers of two: each token is
// scaled so that its largest |x| lies in [2^14, 2^15) (values more than 2^31 below it
// lose bits), each weight row so that its largest |s| lies in [2^10, 2^11).  Sums are
// f32, and the powers of two come off in the epilogue.  Scaling in f16 before the
// product leaves nothing to do at a group's end, so 32-input groups cost what
// 128-input groups do.
//
// A prepare kernel makes the f16 tokens (the inputs of each eight in the order 0 4 1 5
// 2 6 3 7 in which codes_to_f16 gives the weights) and, for experts, sorts the (token,
// slot) pairs by expert and cuts each expert's pairs into token tiles.
#include "ql_internal.h"
#include "ql_w4.cuh"

namespace ql {

constexpr unsigned int KID_W4 = 4;  // KernelId of this file's GEMM in the device status word

constexpr int kG4DequantWarps = 8;
constexpr int kG4TmaWarp = 8;
constexpr int kG4MmaWarp = 9;
constexpr int kG4Threads = 320;
constexpr int kG4StageK = 256;   // inputs of a weight stage (128 bytes of codes a row)
constexpr int kG4GranK = 64;     // inputs of a token stage and of a TMEM weight slot
constexpr int kG4WStages = 3;
constexpr int kG4Slots = 4;      // TMEM weight slots of 32 columns, over all row tiles
constexpr int kG4MaxXStages = 8;
constexpr int kG4PrepThreads = 128;
constexpr int kG4PlanThreads = 1024;
constexpr int kG4MaxSplit = 8;

// RT 128-row weight tiles share the CTA's tokens.
template <int RT>
struct G4Cfg {
  static constexpr int kTok = RT == 2 ? 192 : 128;  // largest token tile
  static constexpr int kRing = RT == 2 ? 110592 : 57344;  // bytes of token stages, 3 to 8 of them
  static constexpr int kTmem = RT == 2 ? 512 : 256;
  static constexpr int kDCols = RT == 2 ? 192 : 128;  // columns of one accumulator
  static constexpr int kWBytes = RT * 128 * 128;
};

struct G4Tile {
  int expert, start, count, pad;
};

struct G4Params {
  const uint16_t* sw;
  const uint8_t* wz;
  uint16_t* y;           // dense, gather: the result; combine: the pairs' products
  const int* ex;         // tokens' exponents
  const int* order;      // experts: pairs sorted by expert
  const G4Tile* tiles;   // experts: token tiles
  const int* ntiles;
  int64_t N, K;
  int64_t M;             // dense: tokens
  int groups;
  int ntok;              // tokens of a tile (a multiple of 16)
  int xstage;            // bytes of a token stage
  int xstages;           // token stages
  int rows_per_token;    // experts: pairs that share an x row (topk for gather, else 1)
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

template <int RT, int kGroup, bool kZero, bool kExperts>
__global__ void __launch_bounds__(kG4Threads, RT == 2 ? 1 : 2)
    w4_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const G4Params p) {
  using Cfg = G4Cfg<RT>;
  const int xs_n = p.xstages;
  constexpr int kPerStage = kG4StageK / kGroup;  // scales of a row in a weight stage
  extern __shared__ uint8_t smem_raw[];
  uint8_t* wring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* xring = wring + kG4WStages * Cfg::kWBytes;
  uint64_t* wfull = reinterpret_cast<uint64_t*>(xring + xs_n * p.xstage);
  uint64_t* wempty = wfull + kG4WStages;
  uint64_t* xfull = wempty + kG4WStages;
  uint64_t* xempty = xfull + kG4MaxXStages;
  uint64_t* afull = xempty + kG4MaxXStages;
  uint64_t* aempty = afull + kG4Slots;
  uint64_t* done = aempty + kG4Slots;
  int* s_ex = reinterpret_cast<int*>(done + 2);     // [kTok] the columns' exponents (16-byte aligned)
  int* s_row = s_ex + Cfg::kTok;                    // [kTok] experts: x rows
  int* s_out = s_row + Cfg::kTok;                   // [kTok] experts: pairs
  float* s_fac = reinterpret_cast<float*>(s_out + Cfg::kTok);  // [kTok] 2^-exponent
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(s_fac + Cfg::kTok);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_wide = reinterpret_cast<int*>(tmem_holder + 2);  // an exponent that one factor cannot take

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % p.splits;
  const int64_t n0 = (int64_t)(blockIdx.x / p.splits) * (RT * 128);
  const int nk64 = (int)((p.K + kG4GranK - 1) / kG4GranK);
  const int nkw = (int)((p.K + kG4StageK - 1) / kG4StageK);
  const int w0 = (int)((int64_t)split * nkw / p.splits), w1 = (int)((int64_t)(split + 1) * nkw / p.splits);
  const int ngran = min(w1 * 4, nk64) - w0 * 4;  // this CTA's granules

  if (threadIdx.x == 0) {
    for (int s = 0; s < kG4WStages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], kG4DequantWarps);
    }
    for (int s = 0; s < xs_n; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int s = 0; s < kG4Slots; ++s) {
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
  if (warp == kG4MmaWarp) {
    tc::tmem_alloc(tmem_holder, Cfg::kTmem);
    tc::tmem_relinquish();
  }
  __syncthreads();
  tc::grid_dependency_wait();  // the prepare kernel's tokens, pairs and tiles
  tc::launch_dependents();

  // this CTA's tokens: exponent, and as a factor 2^-ex
  int64_t e = 0, m0 = 0;
  int count;
  if constexpr (kExperts) {
    const bool live = (int)blockIdx.y < *p.ntiles;
    const G4Tile tile = live ? p.tiles[blockIdx.y] : G4Tile{0, 0, 0, 0};
    e = tile.expert;
    count = tile.count;
    for (int i = threadIdx.x; i < p.ntok && count > 0; i += kG4Threads) {
      const int pair = p.order[tile.start + min(i, count - 1)];
      const int row = pair / p.rows_per_token;
      const int ex = p.ex[row];
      s_out[i] = pair;
      s_row[i] = row;
      s_ex[i] = ex;
      s_fac[i] = exp2i(max(-126, min(126, -ex)));
      if (abs(ex) > 60) *s_wide = 1;
    }
  } else {
    m0 = (int64_t)blockIdx.y * p.ntok;
    count = (int)min((int64_t)p.ntok, p.M - m0);
    for (int i = threadIdx.x; i < count; i += kG4Threads) {
      const int ex = p.ex[m0 + i];
      s_ex[i] = ex;
      s_fac[i] = exp2i(max(-126, min(126, -ex)));
      if (abs(ex) > 60) *s_wide = 1;
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tmem_a = tmem + RT * Cfg::kDCols;
  const int mma_n = (count + 15) & ~15;

  if (count > 0 && warp == kG4TmaWarp) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_w = l2_policy_evict_first();
      const uint64_t pol_x = l2_policy_evict_last();
      const int wrow = (int)(e * p.N + n0);
      const uint32_t xbytes = kExperts ? (uint32_t)((count + 3) / 4) * 512u : (uint32_t)p.ntok * 128u;
      bool ok = true;
      int jw = 0, jx = 0;  // issued stages
      int s = 0;           // token stage of granule j, and how often it was filled
      uint32_t fill = 0;
      for (int j = 0; j < ngran && ok; ++j) {
        if (j % 4 == 0) {
          const int v = jw % kG4WStages;
          if (jw >= kG4WStages) ok = mbar_wait_bounded(&wempty[v], ((jw / kG4WStages) - 1) & 1, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(&wfull[v], Cfg::kWBytes);
#pragma unroll
          for (int r = 0; r < RT; ++r)
            tc::tma_load_2d(wring + v * Cfg::kWBytes + r * 16384, &tmW, (w0 + jw) * 128, wrow + r * 128, &wfull[v],
                            pol_w);
          ++jw;
        }
        if (fill > 0) ok = mbar_wait_bounded(&xempty[s], (fill - 1) & 1, abort_flag);
        if (!ok) break;
        mbar_arrive_expect_tx(&xfull[s], xbytes);
        uint8_t* dst = xring + s * p.xstage;
        const int xb = (w0 * 4 + j) * 128;
        if constexpr (kExperts) {
          for (int i = 0; i < count; i += 4)
            w4::tma_gather4(dst + i * 128, &tmX, xb, *reinterpret_cast<const int4*>(s_row + i), &xfull[s]);
        } else {
          tc::tma_load_2d(dst, &tmX, xb, (int)m0, &xfull[s], pol_x);
        }
        ++jx;
        if (++s == xs_n) {
          s = 0;
          ++fill;
        }
      }
      if (!ok) {
        if (!*abort_flag) record_timeout(p.status, KID_W4, 1);
        *abort_flag = 1;
        // the copies in flight land before the CTA leaves
        for (int j = max(0, jw - kG4WStages); j < jw; ++j)
          mbar_wait_bounded(&wfull[j % kG4WStages], (j / kG4WStages) & 1, nullptr);
        for (int j = max(0, jx - xs_n); j < jx; ++j) mbar_wait_bounded(&xfull[j % xs_n], (j / xs_n) & 1, nullptr);
      }
    }
  } else if (count > 0 && warp == kG4MmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id = w4::idesc_f16(128, mma_n);
      bool ok = true;
      int xs = 0;
      uint32_t xphase = 0;
      for (int j = 0; j < ngran && ok; ++j) {
        ok = mbar_wait_bounded(&xfull[xs], xphase, abort_flag);
        const uint64_t bdesc = tc::sw128_desc(smem_u32(xring + xs * p.xstage));
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int use = RT == 2 ? j / 2 : j / 4;              // how often the slot was used before
          const int slot = RT == 2 ? r * 2 + (j & 1) : j & 3;
          ok = ok && mbar_wait_bounded(&afull[slot], use & 1, abort_flag);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w4::mma_f16_ts(tmem + r * Cfg::kDCols, tmem_a + slot * 32 + k * 8, bdesc + 2 * k, id, j > 0 || k > 0);
          tc::commit(&aempty[slot]);
        }
        if (ok) tc::commit(&xempty[xs]);
        if (++xs == xs_n) {
          xs = 0;
          xphase ^= 1;
        }
      }
      if (!ok) {
        if (!*abort_flag) record_timeout(p.status, KID_W4, 2);
        *abort_flag = 1;
      }
      tc::commit(done);
      mbar_wait_bounded(done, 0, nullptr);
    }
  } else if (count > 0 && warp < kG4DequantWarps) {
    // ------------------------------------------------------------ codes -> TMEM
    // RT = 2: each four warps take a row tile; RT = 1: they take alternate granules.
    const int wg = warp >> 2, q = warp & 3;
    const int r = RT == 2 ? wg : 0;
    const int64_t n = n0 + r * 128 + q * 32 + lane;
    const int64_t wr = e * p.N + min(n, p.N - 1);
    const uint16_t* sw = p.sw + wr * p.groups;
    const uint8_t* wz = kZero ? p.wz + wr * p.groups : nullptr;
    const int g0 = w0 * kPerStage, g1 = min(p.groups, w1 * kPerStage);
    // the row's exponent: its largest |s| to [2^10, 2^11)
    uint32_t top = 0;
    if ((p.groups & 7) == 0) {
      const uint4* v4 = reinterpret_cast<const uint4*>(sw);
#pragma unroll 4
      for (int i = g0 >> 3; i < (g1 + 7) >> 3; ++i) {
        const uint4 v = __ldg(v4 + i);
        top = max(max(max(top, v.x & 0x7FFFu), max(v.x >> 16 & 0x7FFFu, v.y & 0x7FFFu)),
                  max(max(v.y >> 16 & 0x7FFFu, v.z & 0x7FFFu),
                      max(v.z >> 16 & 0x7FFFu, max(v.w & 0x7FFFu, v.w >> 16 & 0x7FFFu))));
      }
    } else {
#pragma unroll 8
      for (int i = g0; i < g1; ++i) top = max(top, (uint32_t)__ldg(sw + i) & 0x7FFFu);
    }
    top = min(top, 0x7F7Fu);
    // exponent of a bf16: the biased field, or for a subnormal the place of its top bit
    const int p2 = top >= 0x80u ? (int)(top >> 7) - 127 : top ? -133 + (31 - __clz(top)) : 10;
    const int f = 10 - p2;
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    const uint32_t rsw = (uint32_t)(lane & 7);
    const uint32_t row_off = (uint32_t)(r * 16384 + (q * 32 + lane) * 128);

    uint32_t sraw[kPerStage], zraw[kPerStage];
    auto load_scales = [&](int w) {
#pragma unroll
      for (int i = 0; i < kPerStage; ++i) {
        const int gi = w * kPerStage + i;
        sraw[i] = gi < p.groups ? __ldg(sw + gi) : 0;
        if constexpr (kZero) zraw[i] = gi < p.groups ? __ldg(wz + gi) : 8;
      }
    };
    load_scales(w0);
    bool ok = true;
    for (int w = w0; w < w1 && ok; ++w) {
      const int jw = w - w0, ws = jw % kG4WStages;
      uint32_t s2[kPerStage], zlo[kPerStage], zhi[kPerStage];
#pragma unroll
      for (int i = 0; i < kPerStage; ++i) {
        const float s = scale2(__uint_as_float(sraw[i] << 16), f);
        s2[i] = w4::f32x2_to_f16x2(s, s);
        if constexpr (kZero) {
          zlo[i] = 0x64006400u + zraw[i] * 0x10001u;
          const float zf = -(64.0f + (float)zraw[i]);
          zhi[i] = w4::f32x2_to_f16x2(zf, zf);
        } else {
          zlo[i] = 0x64086408u;  // 1032
          zhi[i] = 0xD480D480u;  // -72
        }
      }
      if (w + 1 < w1) load_scales(w + 1);
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&wfull[ws], (jw / kG4WStages) & 1, abort_flag));
      if (!ok) break;
      const uint8_t* src = wring + ws * Cfg::kWBytes + row_off;
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) {
        const int j = jw * 4 + gq;
        if (j >= ngran) break;
        if (RT == 1 && (gq & 1) != wg) continue;
        const uint4 c0 = *reinterpret_cast<const uint4*>(src + (((uint32_t)(2 * gq) ^ rsw) << 4));
        const uint4 c1 = *reinterpret_cast<const uint4*>(src + (((uint32_t)(2 * gq + 1) ^ rsw) << 4));
        const uint32_t c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        uint32_t h[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int gi = (gq * 64 + i * 8) / kGroup;
          w4::codes_to_f16(c[i], zlo[gi], zhi[gi], s2[gi], h + 4 * i);
        }
        const int use = RT == 2 ? j / 2 : j / 4;
        const int slot = RT == 2 ? r * 2 + (j & 1) : j & 3;
        if (use > 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&aempty[slot], (use - 1) & 1, abort_flag));
        if (!ok) break;
        tc::fence_after();
        w4::st32(tmem_a + slot * 32 + lane_addr, h);
        w4::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[slot]);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&wempty[ws]);
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_timeout(p.status, KID_W4, 3);
      *abort_flag = 1;
    }
    // ------------------------------------------------------------ epilogue
    ok = ok && mbar_wait_bounded(done, 0, abort_flag) && !*abort_flag;
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc::fence_after();
      // Staged in the rings, which every MMA has left behind: split K, [tok][128 RT]
      // partial sums; else [tok][128 RT] bf16 (rows padded by 16 bytes), so that the
      // rows leave in 16-byte stores, 512 or 256 bytes of a token together.
      constexpr int kRow = RT * 128 * 2 + 16;
      float* part = reinterpret_cast<float*>(wring);
      const int col = r * 128 + q * 32 + lane;
      const int half = ((mma_n / 16 + 1) / 2) * 16;
      const int c_lo = RT == 2 ? 0 : wg ? half : 0, c_hi = RT == 2 ? mma_n : wg ? mma_n : half;
      const bool wide = __any_sync(0xffffffffu, *s_wide || abs(f) > 60);
      const float rf = exp2i(max(-126, min(126, -f)));
      for (int c = c_lo; c < c_hi; c += 16) {
        uint32_t v[16];
        w4::ld16(tmem + r * Cfg::kDCols + lane_addr + c, v);
        tc::ld_wait();
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(v[i]) * rf * s_fac[c + i];
        if (wide) {  // the two factors together may leave f32's range where their product does not
#pragma unroll 1
          for (int i = 0; i < 16; ++i)
            if (c + i < count) {
              uint32_t one[1];
              w4::ld1(tmem + r * Cfg::kDCols + lane_addr + c + i, one);
              tc::ld_wait();
              const float t = scale2(__uint_as_float(one[0]), -(f + s_ex[c + i]));
              if (p.splits > 1)
                part[(c + i) * (RT * 128) + col] = t;
              else
                *reinterpret_cast<uint16_t*>(wring + (c + i) * kRow + col * 2) = f32_to_bf16_rn(t);
            }
        } else if (p.splits > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < count) part[(c + i) * (RT * 128) + col] = o[i];
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < count) *reinterpret_cast<uint16_t*>(wring + (c + i) * kRow + col * 2) = f32_to_bf16_rn(o[i]);
        }
      }
      tc::fence_before();
    }
  }

  __syncwarp();
  if (p.splits > 1) {
    // the cluster's partial sums, added in the order of their K ranges
    w4::cluster_sync();
    if (warp == kG4MmaWarp) {
      tc::fence_after();
      tc::tmem_dealloc(tmem, Cfg::kTmem);
    }
    if (!*abort_flag) {
      const uint32_t part = smem_u32(wring);
      for (int i = threadIdx.x; i < RT * 128 * ((count - split + p.splits - 1) / p.splits); i += kG4Threads) {
        const int c = (i / (RT * 128)) * p.splits + split, col = i % (RT * 128);
        if (n0 + col >= p.N) continue;
        float sum = 0.0f;
        for (int s = 0; s < p.splits; ++s)
          sum += w4::ld_cluster(part + (uint32_t)(c * (RT * 128) + col) * 4u, (uint32_t)s);
        p.y[(m0 + c) * p.N + n0 + col] = f32_to_bf16_rn(sum);
      }
    }
    __syncwarp();
    w4::cluster_sync();  // no CTA leaves while another reads its sums
  } else {
    __syncthreads();
    // before the copies below, in which a warp's lanes may part: dealloc is a
    // whole-warp instruction
    if (warp == kG4MmaWarp) {
      tc::fence_after();
      tc::tmem_dealloc(tmem, Cfg::kTmem);
    }
    if (count > 0 && !*abort_flag) {
      constexpr int kRow = RT * 128 * 2 + 16;
      constexpr int kVecs = RT * 16;  // 16-byte pieces of a token's row
      const int cols = (int)min((int64_t)(RT * 128), p.N - n0);
      if ((p.N & 7) == 0) {
        for (int i = threadIdx.x; i < count * kVecs; i += kG4Threads) {
          const int c = i / kVecs, b = i % kVecs;
          const int64_t row = kExperts ? s_out[c] : m0 + c;
          if (b * 8 < cols)
            *reinterpret_cast<uint4*>(p.y + row * p.N + n0 + b * 8) =
                *reinterpret_cast<const uint4*>(wring + c * kRow + b * 16);
        }
      } else {
        for (int i = threadIdx.x; i < count * RT * 128; i += kG4Threads) {
          const int c = i / (RT * 128), b = i % (RT * 128);
          const int64_t row = kExperts ? s_out[c] : m0 + c;
          if (b < cols) p.y[row * p.N + n0 + b] = *reinterpret_cast<const uint16_t*>(wring + c * kRow + b * 2);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------- prepare

struct G4PrepParams {
  const uint16_t* x;
  uint16_t* x16;
  int* ex;
  int64_t rows, K;
  // experts
  const int32_t* ids;
  int64_t pairs;
  int E, ntok, topk;
  int* order;
  G4Tile* tiles;
  int* ntiles;
  uint16_t* zero_y;  // gather: the result, whose rows of an id out of range are zeroed
  int64_t N;
};

// Block 0 of an experts launch: the pairs in expert order and the token tiles.  The
// order inside an expert depends on timing; results do not, since a pair is one MMA
// column wherever it stands.
QL_DEVINL void plan_experts(const G4PrepParams& p, int* hist) {
  int* base = hist + 1024;
  __shared__ int warp_sums[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 1024; i += kG4PlanThreads) hist[i] = 0;
  __syncthreads();
  for (int64_t i = tid; i < p.pairs; i += kG4PlanThreads) {
    const int e = p.ids[i];
    if (e >= 0 && e < p.E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  // exclusive sums of the pairs and of the tiles; one thread per expert
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
  base[tid] = ci - c;
  for (int i = 0; i < t; ++i)
    p.tiles[ti - t + i] = G4Tile{tid, ci - c + i * p.ntok, min(p.ntok, c - i * p.ntok), 0};
  if (tid == kG4PlanThreads - 1) *p.ntiles = ti;
  __syncthreads();
  for (int64_t i = tid; i < p.pairs; i += kG4PlanThreads) {
    const int e = p.ids[i];
    if (e >= 0 && e < p.E) p.order[atomicAdd(&base[e], 1)] = (int)i;
  }
}

// One row of tokens: the exponent of its largest finite |x| and the scaled f16 values.
QL_DEVINL void prepare_row(const G4PrepParams& p, int64_t row, int tid, int threads, float* red) {
  const uint4* src = reinterpret_cast<const uint4*>(p.x + row * p.K);
  uint4* dst = reinterpret_cast<uint4*>(p.x16 + row * p.K);
  const int chunks = (int)(p.K / 8);
  uint32_t top = 0;
  for (int i = tid; i < chunks; i += threads) {
    const uint4 v = __ldg(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = w[j] & 0x7FFFu, b = w[j] >> 16 & 0x7FFFu;
      if (a < 0x7F80u) top = max(top, a);
      if (b < 0x7F80u) top = max(top, b);
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  uint32_t* r = reinterpret_cast<uint32_t*>(red);
  if ((tid & 31) == 0) r[tid >> 5] = top;
  __syncthreads();
  top = 0;
  for (int i = 0; i < threads / 32; ++i) top = max(top, r[i]);
  const int p2 = top >= 0x80u ? (int)(top >> 7) - 127 : top ? -133 + (31 - __clz(top)) : 14;
  const int e = 14 - p2;
  if (tid == 0) p.ex[row] = e;
  const float f0 = exp2i(e / 2), f1 = exp2i(e - e / 2);
  for (int i = tid; i < chunks; i += threads) {
    const uint4 v = __ldg(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16_lo(w[j]) * f0 * f1;
      x[2 * j + 1] = bf16_hi(w[j]) * f0 * f1;
    }
    dst[i] = make_uint4(w4::f32x2_to_f16x2(x[0], x[4]), w4::f32x2_to_f16x2(x[1], x[5]),
                        w4::f32x2_to_f16x2(x[2], x[6]), w4::f32x2_to_f16x2(x[3], x[7]));
  }
}

__global__ void __launch_bounds__(kG4PrepThreads) w4_prepare_kernel(const G4PrepParams p) {
  __shared__ float red[32];
  tc::grid_dependency_wait();
  tc::launch_dependents();
  prepare_row(p, blockIdx.x, threadIdx.x, kG4PrepThreads, red);
}

// Experts: block 0 plans, the others take eight groups of 128 threads' rows in turn.
__global__ void __launch_bounds__(kG4PlanThreads) w4_prepare_experts_kernel(const G4PrepParams p) {
  __shared__ int hist[2048];
  tc::grid_dependency_wait();
  tc::launch_dependents();
  if (blockIdx.x == 0) {
    plan_experts(p, hist);
    return;
  }
  for (int64_t row = blockIdx.x - 1; row < p.rows; row += gridDim.x - 1) {
    prepare_row(p, row, threadIdx.x, kG4PlanThreads, reinterpret_cast<float*>(hist));
    __syncthreads();
    if (p.zero_y) {
      for (int j = 0; j < p.topk; ++j) {
        const int e = p.ids[row * p.topk + j];
        if (e >= 0 && e < p.E) continue;
        for (int64_t n = threadIdx.x; n < p.N; n += kG4PlanThreads) p.zero_y[(row * p.topk + j) * p.N + n] = 0;
      }
    }
  }
}

// y[t] = sum_j weights[t, j] yp[t, j], the pairs' products rounded to bf16 (half the
// traffic of f32 between the two kernels; one more rounding of each term).
__global__ void __launch_bounds__(128) w4_combine_kernel(const uint16_t* __restrict__ yp, const int32_t* __restrict__ ids,
                                                         const float* __restrict__ weights, int topk, int E, int64_t N,
                                                         uint16_t* __restrict__ y) {
  tc::grid_dependency_wait();
  tc::launch_dependents();
  const int64_t t = blockIdx.x;
  for (int64_t n = (int64_t)blockIdx.y * 128 + threadIdx.x; n < N; n += (int64_t)gridDim.y * 128) {
    float sum = 0.0f;
    for (int j = 0; j < topk; ++j) {
      const int e = __ldg(ids + t * topk + j);
      if (e < 0 || e >= E) continue;
      sum = fmaf(__ldg(weights + t * topk + j), bf16_lo(yp[(t * topk + j) * N + n]), sum);
    }
    y[t * N + n] = f32_to_bf16_rn(sum);
  }
}

// ---------------------------------------------------------------------------- host

namespace {

struct G4Plan {
  int rt, ntok, splits;
  unsigned row_tiles, tok_tiles;
};

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

G4Plan plan_dense(int64_t M, const ql_w4_weight& w, int sms) {
  G4Plan g;
  if (M > 128) {
    g.rt = 2;
    g.row_tiles = (unsigned)div_up(w.N, 256);
    g.ntok = 192;
    double best = 1e30;
    for (int n = 192; n >= 96; n -= 16) {
      const int64_t tt = div_up(M, n);
      const double cost = (double)div_up(g.row_tiles * tt, sms) * (n + 16);
      if (cost < best) {
        best = cost;
        g.ntok = n;
      }
    }
    g.tok_tiles = (unsigned)div_up(M, g.ntok);
    g.splits = 1;
  } else {
    g.rt = 1;
    g.row_tiles = (unsigned)div_up(w.N, 128);
    g.ntok = (int)div_up(M, 16) * 16;
    g.tok_tiles = 1;
    g.splits = 1;
    const int64_t stages = div_up(w.K, kG4StageK);
    while (g.splits < kG4MaxSplit && g.splits * 2 <= stages && (int64_t)g.row_tiles * g.splits * 2 <= 2 * sms)
      g.splits *= 2;
  }
  return g;
}

G4Plan plan_experts_host(int64_t pairs, const ql_w4_weight& w) {
  G4Plan g;
  const int64_t per = div_up(pairs, w.experts);
  g.splits = 1;
  if (per > 64) {
    g.rt = 2;
    g.row_tiles = (unsigned)div_up(w.N, 256);
    g.ntok = 128;
  } else {
    g.rt = 1;
    g.row_tiles = (unsigned)div_up(w.N, 128);
    g.ntok = per > 16 ? 64 : 32;
  }
  g.tok_tiles = (unsigned)(std::min<int64_t>(w.experts, pairs) + pairs / g.ntok);
  return g;
}

struct G4Layout {
  size_t x16, ex, order, tiles, ntiles, yp, total;
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
  L.tiles = off;
  off += up256((size_t)tiles * sizeof(G4Tile));
  L.ntiles = off;
  off += 256;
  L.yp = off;
  off += up256((size_t)yp_elems * 2);
  L.total = off;
  return L;
}

template <int RT, int kGroup, bool kZero, bool kExperts>
cudaError_t launch_g4_t(const CUtensorMap& tw, const CUtensorMap& tx, const G4Params& p, const G4Plan& g,
                        cudaStream_t st) {
  using Cfg = G4Cfg<RT>;
  const int smem = 1024 + kG4WStages * Cfg::kWBytes + p.xstages * p.xstage +
                   8 * (2 * kG4WStages + 2 * kG4MaxXStages + 2 * kG4Slots + 2) + 16 * Cfg::kTok + 16;
  cudaError_t e = ensure_smem<w4_gemm_kernel<RT, kGroup, kZero, kExperts>>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.row_tiles * g.splits, g.tok_tiles);
  cfg.blockDim = dim3(kG4Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = g.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, w4_gemm_kernel<RT, kGroup, kZero, kExperts>, tw, tx, p);
}

template <int RT, bool kExperts>
cudaError_t launch_g4_group(const CUtensorMap& tw, const CUtensorMap& tx, const G4Params& p, const G4Plan& g,
                            int group, cudaStream_t st) {
  if (p.wz) {
    if (group == 128) return launch_g4_t<RT, 128, true, kExperts>(tw, tx, p, g, st);
    if (group == 64) return launch_g4_t<RT, 64, true, kExperts>(tw, tx, p, g, st);
    return launch_g4_t<RT, 32, true, kExperts>(tw, tx, p, g, st);
  }
  if (group == 128) return launch_g4_t<RT, 128, false, kExperts>(tw, tx, p, g, st);
  if (group == 64) return launch_g4_t<RT, 64, false, kExperts>(tw, tx, p, g, st);
  return launch_g4_t<RT, 32, false, kExperts>(tw, tx, p, g, st);
}

template <bool kExperts>
cudaError_t launch_g4(const ql_w4_weight& w, const uint16_t* x16, int64_t rows, G4Params p, const G4Plan& g,
                      cudaStream_t st) {
  if (g.tok_tiles > 65535u) return cudaErrorNotSupported;  // grid.y
  CUtensorMap tw, tx;
  cudaError_t e = make_tmap_u8_sw128(&tw, w.wq, (uint64_t)w.K / 2, (uint64_t)w.experts * w.N, (uint64_t)w.K / 2, 128, 128);
  if (e != cudaSuccess) return e;
  e = make_tmap_u8_sw128(&tx, x16, (uint64_t)w.K * 2, (uint64_t)rows, (uint64_t)w.K * 2, 128, kExperts ? 1 : g.ntok);
  if (e != cudaSuccess) return e;
  p.sw = w.sw;
  p.wz = w.wz;
  p.N = w.N;
  p.K = w.K;
  p.groups = (int)div_up(w.K, w.group);
  p.ntok = g.ntok;
  p.xstage = (int)div_up(g.ntok * 128, 1024) * 1024;
  p.splits = g.splits;
  p.xstages = std::min(kG4MaxXStages, std::max(3, (g.rt == 2 ? G4Cfg<2>::kRing : G4Cfg<1>::kRing) / p.xstage));
  return g.rt == 2 ? launch_g4_group<2, kExperts>(tw, tx, p, g, (int)w.group, st)
                   : launch_g4_group<1, kExperts>(tw, tx, p, g, (int)w.group, st);
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

constexpr int64_t kW4StreamMaxTokens = 16;        // dense: up to here the mma.sync kernel
constexpr int64_t kW4StreamMaxExpertTokens = 8;

size_t w4_workspace_bytes(int64_t M, const ql_w4_weight& w, int sms) {
  if (M <= kW4StreamMaxTokens) return 0;
  return g4_layout(M, w.K, 0, 0, 0).total;
}

cudaError_t launch_w4(const uint16_t* x, const ql_w4_weight& w, int64_t M, uint16_t* y, void* workspace, int sms,
                      DevStatus* status, cudaStream_t st) {
  if (M <= kW4StreamMaxTokens) return launch_w4_stream(x, w, M, y, st);
  const G4Plan g = plan_dense(M, w, sms);
  const G4Layout L = g4_layout(M, w.K, 0, 0, 0);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  G4PrepParams q = {};
  q.x = x;
  q.x16 = reinterpret_cast<uint16_t*>(ws + L.x16);
  q.ex = reinterpret_cast<int*>(ws + L.ex);
  q.rows = M;
  q.K = w.K;
  cudaError_t e = launch_pdl(w4_prepare_kernel, (unsigned)M, kG4PrepThreads, q, st);
  if (e != cudaSuccess) return e;
  G4Params p = {};
  p.y = y;
  p.ex = q.ex;
  p.M = M;
  p.status = status;
  return launch_g4<false>(w, q.x16, M, p, g, st);
}

size_t w4_experts_workspace_bytes(int64_t T, int64_t topk, const ql_w4_weight& w, bool combine, int sms) {
  if (T <= kW4StreamMaxExpertTokens) return 0;
  const int64_t pairs = T * topk;
  const G4Plan g = plan_experts_host(pairs, w);
  return g4_layout(combine ? pairs : T, w.K, pairs, g.tok_tiles, combine ? pairs * w.N : 0).total;
}

cudaError_t launch_w4_experts(const uint16_t* x, const int32_t* ids, const float* weights, const ql_w4_weight& w,
                              int64_t T, int64_t topk, uint16_t* y, void* workspace, int sms, DevStatus* status,
                              cudaStream_t st) {
  if (T <= kW4StreamMaxExpertTokens) return launch_w4_stream_experts(x, ids, weights, w, T, topk, y, st);
  const bool combine = weights != nullptr;
  const int64_t pairs = T * topk, rows = combine ? pairs : T;
  const G4Plan g = plan_experts_host(pairs, w);
  const G4Layout L = g4_layout(rows, w.K, pairs, g.tok_tiles, combine ? pairs * w.N : 0);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  G4PrepParams q = {};
  q.x = x;
  q.x16 = reinterpret_cast<uint16_t*>(ws + L.x16);
  q.ex = reinterpret_cast<int*>(ws + L.ex);
  q.rows = rows;
  q.K = w.K;
  q.ids = ids;
  q.pairs = pairs;
  q.E = (int)w.experts;
  q.ntok = g.ntok;
  q.topk = (int)topk;
  q.order = reinterpret_cast<int*>(ws + L.order);
  q.tiles = reinterpret_cast<G4Tile*>(ws + L.tiles);
  q.ntiles = reinterpret_cast<int*>(ws + L.ntiles);
  q.zero_y = combine ? nullptr : y;
  q.N = w.N;
  cudaError_t e = launch_pdl(w4_prepare_experts_kernel, (unsigned)std::min<int64_t>(rows + 1, 4 * sms), kG4PlanThreads, q, st);
  if (e != cudaSuccess) return e;
  uint16_t* yp = combine ? reinterpret_cast<uint16_t*>(ws + L.yp) : y;
  G4Params p = {};
  p.y = yp;
  p.ex = q.ex;
  p.order = q.order;
  p.tiles = q.tiles;
  p.ntiles = q.ntiles;
  p.rows_per_token = combine ? 1 : (int)topk;
  p.status = status;
  e = launch_g4<true>(w, q.x16, rows, p, g, st);
  if (e != cudaSuccess || !combine) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)T, (unsigned)std::min<int64_t>(div_up(w.N, 128), 64));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, w4_combine_kernel, (const uint16_t*)yp, ids, weights, (int)topk, (int)w.experts, w.N, y);
}

}  // namespace ql
