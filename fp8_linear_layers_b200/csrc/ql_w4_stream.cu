// ql_w4_stream.cu -- products with 4-bit weights for few tokens (mma.sync), dense
// and by routed expert.
//
//   y[m, n] = bf16( sum_k x[m, k] (q[n, k] - z[n, k / g]) s[n, k / g] )
//
// For one token the floor is the weight stream, N K / 2 bytes of codes and
// N ceil(K / g) scales; everything else is small.  The products run on the tensor
// cores: 16 weight rows are the MMA's A operand, up to 8 tokens its columns, so
// the weight stream costs the same for 1 and for 8 tokens.  Codes convert exactly
// to bf16 integers and x stays bf16, so every product is exact and the sums are
// f32; a group's sum is scaled in f32 when the group is complete.
//
// An MMA must not mix groups.  Lane (g, t) of a warp holds rows g and g + 8 and
// the words [t V, (t + 1) V) of every 4 V words of a row, V = group / 32: the 16
// inputs that one MMA takes from the four lanes of a row then lie in one group.
// The order of the inputs inside a group is the same for x and W, and a dot
// product does not depend on it.
//
// A CTA owns 16 or 32 output rows and splits K over its warps, each a run of chunks of
// 128 inputs, the next chunk's loads in flight while one is multiplied; the warps' sums
// meet in shared memory and are added in warp order, so a result does not depend on
// timing.
//
// What bounds it: no one unit (SM throughput 27 to 33 %, DRAM 17 to 22 %, a fifth of the
// warps, first stall the long scoreboard; the weights in L2 or in HBM: the same time).  A
// launch's start, fill and drain are a third of the time; CTAs do not divide by the SMs (4096
// rows: 256 CTAs, so 40 of 148 SMs hold one and 108 two); and a word of eight codes takes 11
// instructions to become bf16 and 1 to be multiplied, with the loads, addresses and scales
// about 16.  Fewer of those did help: one address a row and chunk, bounds only at a row's
// end, and scales of neighbouring groups in one load (one token, group 128: 4096 x 14336
// 14.7 -> 12.2 us, a combined product of 7 tokens with 8 experts 2048 x 768 18.5 -> 14.1 us).
// The variants of 32 rows and zero points and of 16 tokens spill 8 to 104 bytes a thread.
// 14336 x 4096, group 128: 1 token 11.2 us (2.7 TB/s), 8 tokens 12.3 us, 16 tokens 17.4 us;
// 1024 x 4096 1 token 2.6 us.
#include "ql_internal.h"
#include "ql_w4.cuh"

namespace ql {

constexpr int kW4Chunk = 128;   // inputs per unit of a warp's work
constexpr int kW4Rows = 16;     // output rows of a CTA
constexpr int kW4Tokens = 8;    // columns of one MMA
constexpr int kW4Pad = 2;       // floats behind a row of sums: a warp reads a column of rows
constexpr int kW4MaxTopK = 32;

enum W4Mode { kW4Dense = 0, kW4Gather = 1, kW4Combine = 2 };

struct W4StreamParams {
  const uint16_t* x;
  const uint8_t* wq;
  const uint16_t* sw;
  const uint8_t* wz;
  uint16_t* y;
  const int32_t* ids;   // experts: [T, topk]
  const float* wts;     // combine: [T, topk]
  int64_t N, K;
  int groups;           // groups per row
  int nchunk;           // chunks per row
  int M;                // tokens
  int topk, E;
};

// A lane's rows (g + 8 i) of a tile; rows past N repeat row N - 1: loaded, not stored.
template <int RT>
struct W4Lane {
  uint32_t woff[2 * RT];  // bytes from the tile's first row to the lane's first word
  uint32_t soff[2 * RT];  // scales from the tile's first row's

  QL_DEVINL void rows(const W4StreamParams& p, int64_t n0, int g, int lane_bytes) {
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) {
      const uint32_t r = (uint32_t)min((int64_t)(g + 8 * i), p.N - 1 - n0);
      woff[i] = r * (uint32_t)(p.K >> 1) + lane_bytes;
      soff[i] = r * (uint32_t)p.groups;
    }
  }
};

// The next chunk a warp loads: its place in the tile's first row of codes and scales, and
// in the row of x of the lane's token.
struct W4Cursor {
  const uint8_t* w;
  const uint16_t* s;
  const uint8_t* z;
  const uint16_t* x;
  int k;  // the chunk's first input

  QL_DEVINL void set(const W4StreamParams& p, int64_t row0, int c, int kloads) {
    w = p.wq + row0 * (p.K >> 1) + c * (kW4Chunk / 2);
    s = p.sw + row0 * p.groups + c * kloads;
    z = p.wz + row0 * p.groups + c * kloads;
    k = c * kW4Chunk;
  }
  QL_DEVINL void next(int kloads) {
    w += kW4Chunk / 2;
    s += kloads;
    z += kloads;
    k += kW4Chunk;
    x += kW4Chunk;
  }
};

// A chunk's operands: weight words of the lane's 2 RT rows, and x of its tokens.  x of 16
// tokens comes only when the chunk is multiplied: two chunks of it do not fit the
// registers.
template <int V, int RT, int NT, bool kZero>
struct W4Unit {
  static constexpr int kLoads = 4 / V;
  static constexpr bool kHeld = NT == 1;
  uint32_t w[2 * RT][4];
  uint32_t s[2 * RT][(kLoads + 1) / 2];  // scales, two to a word
  uint32_t z[kZero ? 2 * RT : 1];        // zero points, a byte each
  uint4 x[kHeld ? 4 : 1];
  int k;

  // has: this lane has a token.
  QL_DEVINL void load(const W4StreamParams& p, const W4Lane<RT>& l, const W4Cursor& at, bool has, int t) {
    k = at.k;
    if (at.k + kW4Chunk <= (int)p.K && (kLoads == 1 || p.groups % kLoads == 0)) {
      // every chunk but, where K % 128, the last: no bounds, scales in one load
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          uint32_t u[V];
          w4::load_words<V>(at.w + l.woff[r] + i * 16 * V, u);
#pragma unroll
          for (int j = 0; j < V; ++j) w[r][i * V + j] = u[j];
        }
        const uint16_t* sw = at.s + l.soff[r];
        const uint8_t* wz = at.z + l.soff[r];
        if constexpr (kLoads == 1) {
          s[r][0] = __ldg(sw);
          if constexpr (kZero) z[r] = __ldg(wz);
        } else if constexpr (kLoads == 2) {
          s[r][0] = __ldg(reinterpret_cast<const uint32_t*>(sw));
          if constexpr (kZero) z[r] = __ldg(reinterpret_cast<const uint16_t*>(wz));
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(sw));
          s[r][0] = v.x, s[r][kLoads / 2 - 1] = v.y;
          if constexpr (kZero) z[r] = __ldg(reinterpret_cast<const uint32_t*>(wz));
        }
      }
      if constexpr (kHeld)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = make_uint4(0, 0, 0, 0);
          if (has) x[j] = __ldg(piece(at.x, j, t));
        }
    } else {
      const int gi = at.k / (32 * V);
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
#pragma unroll
        for (int i = 0; i < (kLoads + 1) / 2; ++i) s[r][i] = 0;
        if constexpr (kZero) z[r] = 0;
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
          uint32_t u[V];
#pragma unroll
          for (int j = 0; j < V; ++j) u[j] = 0;
          if (at.k + i * 32 * V + t * 8 * V < (int)p.K) w4::load_words<V>(at.w + l.woff[r] + i * 16 * V, u);
#pragma unroll
          for (int j = 0; j < V; ++j) w[r][i * V + j] = u[j];
          if (gi + i < p.groups) {
            s[r][i / 2] |= (uint32_t)__ldg(at.s + l.soff[r] + i) << (16 * (i % 2));
            if constexpr (kZero) z[r] |= (uint32_t)__ldg(at.z + l.soff[r] + i) << (8 * i);
          }
        }
        if constexpr (kHeld)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            x[i * V + j] = make_uint4(0, 0, 0, 0);
            if (has && at.k + i * 32 * V + t * 8 * V < (int)p.K) x[i * V + j] = __ldg(piece(at.x, i * V + j, t));
          }
      }
    }
  }

  // The 8 inputs of lane t's word q (load q / V, word q % V) of the chunk at x.
  static QL_DEVINL const uint4* piece(const uint16_t* x, int q, int t) {
    return reinterpret_cast<const uint4*>(x + (q / V) * 32 * V + t * 8 * V) + q % V;
  }

  // acc += the chunk's products, each group's sum times its scale.  xo: where x of the
  // lane's tokens is if it is not held (-1: no token).  Weighted: times
  // `cw`, the weights of the two columns this lane holds, a column without a pair
  // (use0, use1) left alone.
  template <bool kWeighted>
  QL_DEVINL void accumulate(float (&acc)[RT][NT][4], const W4StreamParams& p, const int (&xo)[NT], int t,
                            float2 cw = {}, bool use0 = true, bool use1 = true) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint32_t zb[2 * RT];  // 128 + z in both halves
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r)
        zb[r] = kZero ? __byte_perm(z[kZero ? r : 0], 0x43004300u, 0x7070u | i * 0x0101u) : 0x43084308u;
      float d[RT][NT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) d[r][n][k] = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        uint32_t xb[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 v;
          if constexpr (kHeld)
            v = x[i * V + j];
          else
            v = xo[n] >= 0 && k + i * 32 * V + t * 8 * V < (int)p.K ? __ldg(piece(p.x + xo[n] + k, i * V + j, t))
                                                                    : make_uint4(0, 0, 0, 0);
          xb[n][0] = __byte_perm(v.x, v.z, 0x5410);
          xb[n][1] = __byte_perm(v.x, v.z, 0x7632);
          xb[n][2] = __byte_perm(v.y, v.w, 0x5410);
          xb[n][3] = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          uint32_t a[4], b[4];
          w4::codes_to_bf16(w[2 * r][i * V + j], zb[2 * r], a);
          w4::codes_to_bf16(w[2 * r + 1][i * V + j], zb[2 * r + 1], b);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            w4::mma_bf16_16816(d[r][n], a[0], b[0], a[1], b[1], xb[n][0], xb[n][1]);
            w4::mma_bf16_16816(d[r][n], a[2], b[2], a[3], b[3], xb[n][2], xb[n][3]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint32_t s0 = s[2 * r][i / 2], s1 = s[2 * r + 1][i / 2];
        const float f0 = __uint_as_float(i % 2 ? s0 & 0xFFFF0000u : s0 << 16);
        const float f1 = __uint_as_float(i % 2 ? s1 & 0xFFFF0000u : s1 << 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float(&o)[4] = acc[r][n];
          const float(&q)[4] = d[r][n];
          if constexpr (kWeighted) {
            if (use0) {
              o[0] = fmaf(q[0] * f0, cw.x, o[0]);
              o[2] = fmaf(q[2] * f1, cw.x, o[2]);
            }
            if (use1) {
              o[1] = fmaf(q[1] * f0, cw.y, o[1]);
              o[3] = fmaf(q[3] * f1, cw.y, o[3]);
            }
          } else {
            o[0] = fmaf(q[0], f0, o[0]);
            o[1] = fmaf(q[1], f0, o[1]);
            o[2] = fmaf(q[2], f1, o[2]);
            o[3] = fmaf(q[3], f1, o[3]);
          }
        }
      }
    }
  }
};

// Units [u, end), the next one's loads in flight while one is multiplied: load(unit) in
// order, multiply(unit, index).
template <class Unit, class Load, class Multiply>
QL_DEVINL void run_units(int u, int end, Load load, Multiply multiply) {
  Unit u0, u1;
  if (u < end) load(u0);
#pragma unroll 1
  while (u < end) {
    if (u + 1 < end) load(u1);
    multiply(u0, u);
    if (++u >= end) break;
    if (u + 1 < end) load(u0);
    multiply(u1, u);
    ++u;
  }
}

template <int V, int RT, int NT, bool kZero, W4Mode kMode>
__global__ void __launch_bounds__(512) w4_stream_kernel(const W4StreamParams p) {
  extern __shared__ float red[];     // [warps][16 RT rows][kPitch]
  __shared__ int s_pair[kW4Tokens];  // gather: the columns' pairs
  using Unit = W4Unit<V, RT, NT, kZero>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  constexpr int kCols = NT * kW4Tokens, kRows = RT * kW4Rows;
  constexpr int kPitch = kCols + kW4Pad;
  const int64_t n0 = (int64_t)blockIdx.x * kRows;
  constexpr int kLoads = 4 / V;
  W4Lane<RT> l;
  l.rows(p, n0, g, t * 4 * V);
  // the warp's chunks of a row: neighbours, so that a line of scales or x serves several
  const int c0 = (int)((int64_t)warp * p.nchunk / warps), c1 = (int)((int64_t)(warp + 1) * p.nchunk / warps);
  W4Cursor at;

  if constexpr (kMode == kW4Dense) {
    // The warp's weights to L2 while the previous kernel on the stream ends.  (L2 is where
    // that kernel's own writes go, so weights it may still be writing are read correctly
    // below.)
    at.set(p, n0, c0, kLoads);
    for (int c = 2 * t; c < c1 - c0; c += 8) {  // two chunks to a line
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) {
        w4::prefetch_l2(at.w + l.woff[i] - t * 4 * V + c * (kW4Chunk / 2));
        if (c == 0) w4::prefetch_l2(at.s + l.soff[i]);
      }
    }
  }
  tc::grid_dependency_wait();
  tc::launch_dependents();

  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[r][n][k] = 0.0f;

  if constexpr (kMode == kW4Dense) {
    int xo[NT];  // (16 rows of at most 2^24)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int m = n * kW4Tokens + g;
      xo[n] = m < p.M ? m * (int)p.K : -1;
    }
    const bool has = xo[0] >= 0;
    at.x = p.x + max(xo[0], 0) + c0 * kW4Chunk;
    run_units<Unit>(
        c0, c1,
        [&](Unit& u) {
          u.load(p, l, at, has, t);
          at.next(kLoads);
        },
        [&](const Unit& u, int) { u.template accumulate<false>(acc, p, xo, t); });
  } else {
    // the CTA's block of up to 8 tokens and their (token, slot) pairs
    const int t0 = blockIdx.z * kW4Tokens;
    const int pairs = min(kW4Tokens, p.M - t0) * p.topk;
    const int64_t pair0 = (int64_t)t0 * p.topk;
    if constexpr (kMode == kW4Gather) {
      // CTA (n tile, pair): a pair whose expert was chosen 8 r times before it in
      // the block leads that expert's next 8 pairs; the other pairs' CTAs leave.
      // Every warp finds the columns' pairs by itself.
      const int me = blockIdx.y;
      if (me >= pairs) return;
      const int e = __ldg(p.ids + pair0 + me);
      const bool valid = e >= 0 && e < p.E;
      int rank = 0, mine = -1, column = -1;  // column: the pair of column `lane`
      for (int b = 0; b < pairs; b += 32) {
        const bool in = b + lane < pairs;
        const int o = in ? __ldg(p.ids + pair0 + b + lane) : -1;
        unsigned hits = __ballot_sync(0xffffffffu, in && (valid ? o == e : b + lane == me));
        if (me >= b + 32)
          rank += __popc(hits);
        else if (me >= b) {
          rank += __popc(hits & ((1u << (me - b)) - 1u));
          hits &= ~((1u << (me - b)) - 1u);
        }
        if (me < b + 32) {  // the pairs from me on take the columns in order
          const int want = lane - __popc(__ballot_sync(0xffffffffu, column >= 0));
          for (int i = 0; i < want && i < kW4Tokens; ++i) hits &= hits - 1;
          if (want >= 0 && lane < kW4Tokens && hits) column = b + __ffs(hits) - 1;
        }
      }
      if (valid && rank % kW4Tokens) return;
      if (warp == 0 && lane < kW4Tokens) s_pair[lane] = column;
      mine = __shfl_sync(0xffffffffu, column, g);
      if (valid) {
        at.set(p, e * p.N + n0, c0, kLoads);
        at.x = p.x + (int64_t)(t0 + max(mine, 0) / p.topk) * p.K + c0 * kW4Chunk;
        run_units<Unit>(
            c0, c1,
            [&](Unit& u) {
              u.load(p, l, at, mine >= 0, t);
              at.next(kLoads);
            },
            [&](const Unit& u, int) { u.template accumulate<false>(acc, p, {}, t); });
      }
    } else {
      // The block's experts in the order of their first pair; an entry is one expert
      // with, for each token, the pair that chose it.  A token that names an expert
      // again gets an entry of its own for that pair.
      constexpr int kMax = kW4Tokens * kW4MaxTopK;
      __shared__ int s_first[QL_ROUTE_MAX_EXPERTS];  // an expert's first pair, then its entry
      __shared__ int s_entry[kMax], s_slot[kMax][kW4Tokens];
      __shared__ int s_leaders[16];
      for (int i = threadIdx.x; i < p.E; i += blockDim.x) s_first[i] = kMax;
      __syncthreads();
      const int me = threadIdx.x;  // (blockDim >= kMax)
      const int tok = me / p.topk;
      const int e = me < pairs ? __ldg(p.ids + pair0 + me) : -1;
      bool valid = e >= 0 && e < p.E, again = false;
      if (valid) {
        for (int i = tok * p.topk; i < me; ++i) again |= __ldg(p.ids + pair0 + i) == e;
        if (!again) atomicMin(&s_first[e], me);
      }
      __syncthreads();
      const bool leads = valid && (again || s_first[e] == me);
      const unsigned ballot = __ballot_sync(0xffffffffu, leads);
      if (lane == 0) s_leaders[warp] = __popc(ballot);
      __syncthreads();
      int spot = __popc(ballot & ((1u << lane) - 1u)), count = 0;
      for (int w = 0; w < warps; ++w) {
        if (w < warp) spot += s_leaders[w];
        count += s_leaders[w];
      }
      if (leads) {
        s_entry[spot] = e;
        for (int q = 0; q < kW4Tokens; ++q) s_slot[spot][q] = -1;
        if (again) s_slot[spot][tok] = me;
      }
      __syncthreads();
      if (leads && !again) s_first[e] = spot;
      __syncthreads();
      if (valid && !again) s_slot[s_first[e]][tok] = me;
      __syncthreads();
      const float* wts = p.wts + pair0;
      // units: the chunks of all entries, in order; a warp takes a run of them
      const int units = count * p.nchunk;
      const int q0 = (int)((int64_t)warp * units / warps), q1 = (int)((int64_t)(warp + 1) * units / warps);
      int le = q0 / p.nchunk, lc = q0 - le * p.nchunk, me_ = le, mc = lc;  // entry and chunk to load, to multiply
      bool has = false;
      auto enter = [&] {
        at.set(p, s_entry[le] * p.N + n0, lc, kLoads);
        const int mine = s_slot[le][g];
        has = mine >= 0;
        at.x = p.x + (pair0 + max(mine, 0)) * p.K + lc * kW4Chunk;
      };
      float2 cw = make_float2(0.0f, 0.0f);
      bool use0 = false, use1 = false;
      auto weigh = [&] {
        const int ca = s_slot[me_][2 * t], cb = s_slot[me_][2 * t + 1];
        use0 = ca >= 0, use1 = cb >= 0;
        cw = make_float2(use0 ? __ldg(wts + ca) : 0.0f, use1 ? __ldg(wts + cb) : 0.0f);
      };
      if (q0 < q1) {
        enter();
        weigh();
      }
      run_units<Unit>(
          q0, q1,
          [&](Unit& u) {
            if (lc == p.nchunk) {
              lc = 0;
              ++le;
              enter();
            }
            u.load(p, l, at, has, t);
            at.next(kLoads);
            ++lc;
          },
          [&](const Unit& u, int) {
            if (mc == p.nchunk) {
              mc = 0;
              ++me_;
              weigh();
            }
            u.template accumulate<true>(acc, p, {}, t, cw, use0, use1);
            ++mc;
          });
    }
  }

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float* base = red + (warp * kRows + r * kW4Rows) * kPitch + n * kW4Tokens + 2 * t;
      *reinterpret_cast<float2*>(base + g * kPitch) = make_float2(acc[r][n][0], acc[r][n][1]);
      *reinterpret_cast<float2*>(base + (g + 8) * kPitch) = make_float2(acc[r][n][2], acc[r][n][3]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kCols; i += blockDim.x) {
    const int row = i % kRows, col = i / kRows;
    int64_t out = -1;  // y row of this column
    if constexpr (kMode == kW4Dense) {
      if (col < p.M) out = col;
    } else if constexpr (kMode == kW4Gather) {
      if (s_pair[col] >= 0) out = (int64_t)blockIdx.z * kW4Tokens * p.topk + s_pair[col];
    } else {
      if (blockIdx.z * kW4Tokens + col < p.M) out = (int64_t)blockIdx.z * kW4Tokens + col;
    }
    if (out < 0 || n0 + row >= p.N) continue;
    float sum = 0.0f;
    for (int w = 0; w < warps; ++w) sum += red[(w * kRows + row) * kPitch + col];
    p.y[out * p.N + n0 + row] = f32_to_bf16_rn(sum);
  }
}

// ---------------------------------------------------------------------------- host

template <int V, int RT, int NT, bool kZero, W4Mode kMode>
static cudaError_t launch_t(const W4StreamParams& p, dim3 grid, int warps, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = (size_t)warps * RT * kW4Rows * (NT * kW4Tokens + kW4Pad) * sizeof(float);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, w4_stream_kernel<V, RT, NT, kZero, kMode>, p);
}

template <int RT, int NT, W4Mode kMode>
static cudaError_t launch_group(const W4StreamParams& p, int group, dim3 grid, int warps, cudaStream_t st) {
  const bool z = p.wz != nullptr;
  if (group == 128)
    return z ? launch_t<4, RT, NT, true, kMode>(p, grid, warps, st) : launch_t<4, RT, NT, false, kMode>(p, grid, warps, st);
  if (group == 64)
    return z ? launch_t<2, RT, NT, true, kMode>(p, grid, warps, st) : launch_t<2, RT, NT, false, kMode>(p, grid, warps, st);
  if constexpr (RT == 1 || NT == 2)
    return z ? launch_t<1, RT, NT, true, kMode>(p, grid, warps, st)
             : launch_t<1, RT, NT, false, kMode>(p, grid, warps, st);
  return cudaErrorInvalidValue;  // (wide_tiles)
}

static W4StreamParams stream_params(const uint16_t* x, const ql_w4_weight& w, int64_t M, uint16_t* y) {
  W4StreamParams p = {};
  p.x = x;
  p.wq = static_cast<const uint8_t*>(w.wq);
  p.sw = w.sw;
  p.wz = w.wz;
  p.y = y;
  p.N = w.N;
  p.K = w.K;
  p.groups = (int)((w.K + w.group - 1) / w.group);
  p.nchunk = (int)((w.K + kW4Chunk - 1) / kW4Chunk);
  p.M = (int)M;
  return p;
}

// Warps of a CTA: as many as fill the SMs' 16 (32-row tiles) or 20 (16-row tiles) warps
// with one round of CTAs, so that a warp has as many units as the size allows and none
// waits for another round.
static int stream_warps(int64_t ctas, int nunit, int64_t fill, int least) {
  int w = 16;
  while (w > least && (ctas * w > fill || w > nunit)) w /= 2;
  return w;
}

// 32 rows to a tile or 16.  Up to 8 tokens 32 rows halve the work per code on x, but leave
// half the CTAs: better from two 16-row tiles an SM on (K = 4096, one token: 6144 rows 6.1
// against 8.0 us, 4096 rows 4.4 against 4.2).  With groups of 32 inputs the scales and zero
// points of 32 rows do not fit the registers (14336 rows, zero points: 20.9 against 17.3).
static bool wide_tiles(int64_t tiles, int64_t group, int sms) { return tiles >= 2 * sms && group > 32; }

cudaError_t launch_w4_stream(const uint16_t* x, const ql_w4_weight& w, int64_t M, uint16_t* y, int sms,
                             cudaStream_t st) {
  const W4StreamParams p = stream_params(x, w, M, y);
  const int64_t tiles = (w.N + kW4Rows - 1) / kW4Rows, wide = (w.N + 2 * kW4Rows - 1) / (2 * kW4Rows);
  if (M > kW4Tokens) {
    // 16 tokens' x is read by every tile and is more than its codes: 32 rows as soon as 16
    // leave SMs with two tiles (16 tokens, K = 4096: 4096 rows 6.0 against 10.5 us, 2048
    // rows 5.5 against 5.1).
    if (tiles > sms)
      return launch_group<2, 2, kW4Dense>(p, (int)w.group, dim3((unsigned)wide),
                                          stream_warps(wide, p.nchunk, 16 * sms, 4), st);
    return launch_group<1, 2, kW4Dense>(p, (int)w.group, dim3((unsigned)tiles),
                                        stream_warps(tiles, p.nchunk, 20 * sms, 4), st);
  }
  if (wide_tiles(tiles, w.group, sms))
    return launch_group<2, 1, kW4Dense>(p, (int)w.group, dim3((unsigned)wide),
                                        stream_warps(wide, p.nchunk, 16 * sms, 4), st);
  return launch_group<1, 1, kW4Dense>(p, (int)w.group, dim3((unsigned)tiles),
                                      stream_warps(tiles, p.nchunk, 20 * sms, 4), st);
}

cudaError_t launch_w4_stream_experts(const uint16_t* x, const int32_t* ids, const float* weights,
                                     const ql_w4_weight& w, int64_t T, int64_t topk, uint16_t* y, int sms,
                                     cudaStream_t st) {
  W4StreamParams p = stream_params(x, w, T, y);
  p.ids = ids;
  p.wts = weights;
  p.topk = (int)topk;
  p.E = (int)w.experts;
  const int64_t tiles = (w.N + kW4Rows - 1) / kW4Rows;
  const unsigned blocks = (unsigned)((T + kW4Tokens - 1) / kW4Tokens);
  if (weights) return launch_group<1, 1, kW4Combine>(p, (int)w.group, dim3((unsigned)tiles, 1, blocks), 16, st);
  const int64_t pairs = std::min<int64_t>(T, kW4Tokens) * topk;
  const int64_t busy = std::min<int64_t>(pairs, w.experts);  // CTAs of a tile that do not leave at once, at most
  if (wide_tiles(tiles * busy, w.group, sms)) {
    const int64_t wide = (w.N + 2 * kW4Rows - 1) / (2 * kW4Rows);
    const int warps = stream_warps(wide * busy, p.nchunk, 16 * sms, 4);
    return launch_group<2, 1, kW4Gather>(p, (int)w.group, dim3((unsigned)wide, (unsigned)pairs, blocks), warps, st);
  }
  const int warps = stream_warps(tiles * busy, p.nchunk, 20 * sms, 4);
  return launch_group<1, 1, kW4Gather>(p, (int)w.group, dim3((unsigned)tiles, (unsigned)pairs, blocks), warps, st);
}

}  // namespace ql
