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
// A CTA owns 16 output rows and splits K over its warps in chunks of 128 inputs;
// the warps' sums meet in shared memory and are added in warp order, so a result
// does not depend on timing.
#include "ql_internal.h"
#include "ql_w4.cuh"

namespace ql {

constexpr int kW4Chunk = 128;   // inputs per unit of a warp's work
constexpr int kW4Rows = 16;     // output rows of a CTA
constexpr int kW4Tokens = 8;    // columns of one MMA
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

// A chunk's operands: weight words of rows g and g + 8, and x of the lane's tokens,
// which for 16 tokens comes only when the chunk is multiplied (held ahead, two chunks
// of it do not fit the registers).
template <int V, int NT, bool kZero>
struct W4Unit {
  static constexpr int kLoads = 4 / V;
  static constexpr int kHeld = NT == 1 ? 4 : 1;
  uint32_t w0[4], w1[4];
  uint4 x[kHeld];
  uint32_t s0[kLoads], s1[kLoads], z0[kZero ? kLoads : 1], z1[kZero ? kLoads : 1];

  static QL_DEVINL uint4 load_x(const W4StreamParams& p, const uint16_t* xr, int c, int i, int j, int t) {
    const int64_t k = (int64_t)c * kW4Chunk + i * 32 * V + t * 8 * V;
    return k < p.K && xr ? __ldg(reinterpret_cast<const uint4*>(xr + k) + j) : make_uint4(0, 0, 0, 0);
  }

  QL_DEVINL void load(const W4StreamParams& p, int64_t row0, int64_t row1, const uint16_t* const (&xr)[NT],
                      int c, int t) {
    const uint8_t* a = p.wq + row0 * (p.K >> 1);
    const uint8_t* b = p.wq + row1 * (p.K >> 1);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int64_t k = (int64_t)c * kW4Chunk + i * 32 * V + t * 8 * V;  // this lane's first input
      const int gi = c * kLoads + i;
      uint32_t u[V], v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) u[j] = v[j] = 0;
      s0[i] = s1[i] = 0;
      if constexpr (kZero) z0[i] = z1[i] = 8;
      if (gi < p.groups) {
        s0[i] = __ldg(p.sw + row0 * p.groups + gi);
        s1[i] = __ldg(p.sw + row1 * p.groups + gi);
        if constexpr (kZero) {
          z0[i] = __ldg(p.wz + row0 * p.groups + gi);
          z1[i] = __ldg(p.wz + row1 * p.groups + gi);
        }
      }
      const bool in = k < p.K;
      if (in) {
        w4::load_words<V>(a + (k >> 1), u);
        w4::load_words<V>(b + (k >> 1), v);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        w0[i * V + j] = u[j];
        w1[i * V + j] = v[j];
        if constexpr (NT == 1) x[i * V + j] = load_x(p, xr[0], c, i, j, t);
      }
    }
  }

  // acc += the chunk's products, each group's sum times its scale; weighted: times
  // `cw`, the weights of the two columns this lane holds, a column without a pair
  // (use0, use1) left alone.
  template <bool kWeighted>
  QL_DEVINL void accumulate(float (&acc)[NT][4], const W4StreamParams& p, const uint16_t* const (&xr)[NT], int c, int t,
                            float2 cw = {}, bool use0 = true, bool use1 = true) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      float d[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) d[n][r] = 0.0f;
      const uint32_t zz0 = kZero ? 0x43004300u | z0[i] * 0x10001u : 0x43084308u;
      const uint32_t zz1 = kZero ? 0x43004300u | z1[i] * 0x10001u : 0x43084308u;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        uint32_t a[4], b[4];
        uint4 xn[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (NT == 1)
            xn[n] = x[i * V + j];
          else
            xn[n] = load_x(p, xr[n], c, i, j, t);
        }
        w4::codes_to_bf16(w0[i * V + j], zz0, a);
        w4::codes_to_bf16(w1[i * V + j], zz1, b);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 xv = xn[n];
          w4::mma_bf16_16816(d[n], a[0], b[0], a[1], b[1], __byte_perm(xv.x, xv.z, 0x5410),
                             __byte_perm(xv.x, xv.z, 0x7632));
          w4::mma_bf16_16816(d[n], a[2], b[2], a[3], b[3], __byte_perm(xv.y, xv.w, 0x5410),
                             __byte_perm(xv.y, xv.w, 0x7632));
        }
      }
      const float f0 = __uint_as_float(s0[i] << 16), f1 = __uint_as_float(s1[i] << 16);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (kWeighted) {
          if (use0) {
            acc[n][0] = fmaf(d[n][0] * f0, cw.x, acc[n][0]);
            acc[n][2] = fmaf(d[n][2] * f1, cw.x, acc[n][2]);
          }
          if (use1) {
            acc[n][1] = fmaf(d[n][1] * f0, cw.y, acc[n][1]);
            acc[n][3] = fmaf(d[n][3] * f1, cw.y, acc[n][3]);
          }
        } else {
          acc[n][0] = fmaf(d[n][0], f0, acc[n][0]);
          acc[n][1] = fmaf(d[n][1], f0, acc[n][1]);
          acc[n][2] = fmaf(d[n][2], f1, acc[n][2]);
          acc[n][3] = fmaf(d[n][3], f1, acc[n][3]);
        }
      }
    }
  }
};

// A warp's units first, first + step, ... below n, the next one's loads in flight while
// one is multiplied: load(unit, index) and multiply(unit, index).
template <class Unit, class Load, class Multiply>
QL_DEVINL void run_units(int first, int step, int n, Load load, Multiply multiply) {
  Unit u0, u1;
  int c = first;
  if (c < n) load(u0, c);
#pragma unroll 1
  while (c < n) {
    if (c + step < n) load(u1, c + step);
    multiply(u0, c);
    c += step;
    if (c >= n) break;
    if (c + step < n) load(u0, c + step);
    multiply(u1, c);
    c += step;
  }
}

template <int V, int NT, bool kZero, W4Mode kMode>
__global__ void __launch_bounds__(512) w4_stream_kernel(const W4StreamParams p) {
  extern __shared__ float red[];     // [warps][16 rows][8 NT columns]
  __shared__ int s_pair[kW4Tokens];  // gather: the columns' pairs
  using Unit = W4Unit<V, NT, kZero>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * kW4Rows;
  const int64_t r0 = min(n0 + g, p.N - 1), r1 = min(n0 + g + 8, p.N - 1);  // rows past N: loaded, not stored
  constexpr int kCols = NT * kW4Tokens;

  if constexpr (kMode == kW4Dense) {
    // The warp's first weights to L2 while the previous kernel on the stream ends.  (L2
    // is where that kernel's own writes go, so weights it may still be writing are
    // read correctly below.)
    const int64_t k = ((int64_t)warp * kW4Chunk + t * 32) >> 1;
    if (k < p.K >> 1) {
      w4::prefetch_l2(p.wq + r0 * (p.K >> 1) + k);
      w4::prefetch_l2(p.wq + r1 * (p.K >> 1) + k);
    }
  }
  tc::grid_dependency_wait();
  tc::launch_dependents();

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[n][r] = 0.0f;

  if constexpr (kMode == kW4Dense) {
    const int m0 = blockIdx.y * kCols;
    const uint16_t* xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int m = m0 + n * kW4Tokens + g;
      xr[n] = m < p.M ? p.x + (int64_t)m * p.K : nullptr;
    }
    run_units<Unit>(
        warp, warps, p.nchunk, [&](Unit& u, int c) { u.load(p, r0, r1, xr, c, t); },
        [&](const Unit& u, int c) { u.template accumulate<false>(acc, p, xr, c, t); });
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
        const uint16_t* xr[1] = {mine >= 0 ? p.x + (int64_t)(t0 + mine / p.topk) * p.K : nullptr};
        run_units<Unit>(
            warp, warps, p.nchunk, [&](Unit& u, int c) { u.load(p, e * p.N + r0, e * p.N + r1, xr, c, t); },
            [&](const Unit& u, int c) { u.template accumulate<false>(acc, p, xr, c, t); });
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
      int at = __popc(ballot & ((1u << lane) - 1u)), count = 0;
      for (int w = 0; w < warps; ++w) {
        if (w < warp) at += s_leaders[w];
        count += s_leaders[w];
      }
      if (leads) {
        s_entry[at] = e;
        for (int q = 0; q < kW4Tokens; ++q) s_slot[at][q] = -1;
        if (again) s_slot[at][tok] = me;
      }
      __syncthreads();
      if (leads && !again) s_first[e] = at;
      __syncthreads();
      if (valid && !again) s_slot[s_first[e]][tok] = me;
      __syncthreads();
      const float* wts = p.wts + pair0;
      run_units<Unit>(
          warp, warps, count * p.nchunk,
          [&](Unit& u, int q) {
            const int i = q / p.nchunk;
            const int64_t row = (int64_t)s_entry[i] * p.N;
            const int mine = s_slot[i][g];
            const uint16_t* xr[1] = {mine >= 0 ? p.x + (pair0 + mine) * p.K : nullptr};
            u.load(p, row + r0, row + r1, xr, q - i * p.nchunk, t);
          },
          [&](const Unit& u, int q) {
            const int i = q / p.nchunk;
            const int ca = s_slot[i][2 * t], cb = s_slot[i][2 * t + 1];
            const uint16_t* none[1] = {nullptr};  // x is held
            u.template accumulate<true>(
                acc, p, none, q, t, make_float2(ca >= 0 ? __ldg(wts + ca) : 0.0f, cb >= 0 ? __ldg(wts + cb) : 0.0f), ca >= 0, cb >= 0);
          });
    }
  }

#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* base = red + warp * kW4Rows * kCols + n * kW4Tokens + 2 * t;
    *reinterpret_cast<float2*>(base + g * kCols) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(base + (g + 8) * kCols) = make_float2(acc[n][2], acc[n][3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kW4Rows * kCols; i += blockDim.x) {
    const int row = i % kW4Rows, col = i / kW4Rows;
    int64_t out = -1;  // y row of this column
    if constexpr (kMode == kW4Dense) {
      if (blockIdx.y * kCols + col < p.M) out = (int64_t)blockIdx.y * kCols + col;
    } else if constexpr (kMode == kW4Gather) {
      if (s_pair[col] >= 0) out = (int64_t)blockIdx.z * kW4Tokens * p.topk + s_pair[col];
    } else {
      if (blockIdx.z * kW4Tokens + col < p.M) out = (int64_t)blockIdx.z * kW4Tokens + col;
    }
    if (out < 0 || n0 + row >= p.N) continue;
    float sum = 0.0f;
    for (int w = 0; w < warps; ++w) sum += red[(w * kW4Rows + row) * kCols + col];
    p.y[out * p.N + n0 + row] = f32_to_bf16_rn(sum);
  }
}

// ---------------------------------------------------------------------------- host

template <int V, int NT, bool kZero, W4Mode kMode>
static cudaError_t launch_t(const W4StreamParams& p, dim3 grid, int warps, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = (size_t)warps * kW4Rows * NT * kW4Tokens * sizeof(float);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, w4_stream_kernel<V, NT, kZero, kMode>, p);
}

template <int NT, W4Mode kMode>
static cudaError_t launch_group(const W4StreamParams& p, int group, dim3 grid, int warps, cudaStream_t st) {
  const bool z = p.wz != nullptr;
  if (group == 128)
    return z ? launch_t<4, NT, true, kMode>(p, grid, warps, st) : launch_t<4, NT, false, kMode>(p, grid, warps, st);
  if (group == 64)
    return z ? launch_t<2, NT, true, kMode>(p, grid, warps, st) : launch_t<2, NT, false, kMode>(p, grid, warps, st);
  return z ? launch_t<1, NT, true, kMode>(p, grid, warps, st) : launch_t<1, NT, false, kMode>(p, grid, warps, st);
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

// Warps of a CTA: as many as fill the SMs' 24 to 32 warps with one round of CTAs, so that
// a warp has as many units as the size allows and none waits for another round.
static int stream_warps(int64_t ctas, int nunit, int sms, int least) {
  int w = 16;
  while (w > least && (ctas * w > (int64_t)sms * 28 || w > nunit)) w /= 2;
  return w;
}

cudaError_t launch_w4_stream(const uint16_t* x, const ql_w4_weight& w, int64_t M, uint16_t* y, int sms,
                             cudaStream_t st) {
  const W4StreamParams p = stream_params(x, w, M, y);
  const int64_t tiles = (w.N + kW4Rows - 1) / kW4Rows;
  const int warps = stream_warps(tiles, p.nchunk, sms, 4);
  if (M <= kW4Tokens) return launch_group<1, kW4Dense>(p, (int)w.group, dim3((unsigned)tiles, 1), warps, st);
  return launch_group<2, kW4Dense>(p, (int)w.group, dim3((unsigned)tiles, (unsigned)((M + 15) / 16)), warps, st);
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
  if (weights) return launch_group<1, kW4Combine>(p, (int)w.group, dim3((unsigned)tiles, 1, blocks), 16, st);
  const int64_t pairs = std::min<int64_t>(T, kW4Tokens) * topk;
  const int64_t busy = std::min<int64_t>(pairs, w.experts);  // CTAs of a tile that do not leave at once, at most
  const int warps = stream_warps(tiles * busy, p.nchunk, sms, 4);
  return launch_group<1, kW4Gather>(p, (int)w.group, dim3((unsigned)tiles, (unsigned)pairs, blocks), warps, st);
}

}  // namespace ql
