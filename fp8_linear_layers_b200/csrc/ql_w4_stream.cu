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

// A chunk's operands: weight words of rows g and g + 8, x of the lane's tokens.
template <int V, int NT, bool kZero>
struct W4Unit {
  static constexpr int kLoads = 4 / V;
  uint32_t w0[4], w1[4];
  uint4 x[NT][4];
  uint32_t s0[kLoads], s1[kLoads], z0[kLoads], z1[kLoads];

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
      z0[i] = z1[i] = 8;
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
#pragma unroll
        for (int n = 0; n < NT; ++n)
          x[n][i * V + j] = in && xr[n] ? __ldg(reinterpret_cast<const uint4*>(xr[n] + k) + j) : make_uint4(0, 0, 0, 0);
      }
    }
  }

  // acc += the chunk's products, each group's sum times its scale; weighted: times
  // `cw`, the weights of the two columns this lane holds, a column without a pair
  // (use0, use1) left alone.
  template <bool kWeighted>
  QL_DEVINL void accumulate(float (&acc)[NT][4], float2 cw = {}, bool use0 = true, bool use1 = true) const {
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
        w4::codes_to_bf16(w0[i * V + j], zz0, a);
        w4::codes_to_bf16(w1[i * V + j], zz1, b);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 xv = x[n][i * V + j];
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

template <int V, int NT, bool kZero, W4Mode kMode>
__global__ void __launch_bounds__(512) w4_stream_kernel(const W4StreamParams p) {
  extern __shared__ float red[];  // [warps][16 rows][8 NT columns]
  __shared__ int s_pair[kW4Tokens];  // gather: the columns' pairs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * kW4Rows;
  const int64_t r0 = min(n0 + g, p.N - 1), r1 = min(n0 + g + 8, p.N - 1);  // rows past N: loaded, not stored
  constexpr int kCols = NT * kW4Tokens;

  tc::grid_dependency_wait();
  tc::launch_dependents();

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[n][r] = 0.0f;
  W4Unit<V, NT, kZero> u;

  if constexpr (kMode == kW4Dense) {
    const int m0 = blockIdx.y * kCols;
    const uint16_t* xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int m = m0 + n * kW4Tokens + g;
      xr[n] = m < p.M ? p.x + (int64_t)m * p.K : nullptr;
    }
    for (int c = warp; c < p.nchunk; c += warps) {
      u.load(p, r0, r1, xr, c, t);
      u.template accumulate<false>(acc);
    }
  } else {
    // the CTA's block of up to 8 tokens and their (token, slot) pairs
    __shared__ int s_id[kW4Tokens * kW4MaxTopK], s_entry[kW4Tokens * kW4MaxTopK];
    __shared__ int s_slot[kW4Tokens * kW4MaxTopK][kW4Tokens];
    __shared__ int s_count;
    const int t0 = blockIdx.z * kW4Tokens;
    const int pairs = min(kW4Tokens, p.M - t0) * p.topk;
    const int64_t pair0 = (int64_t)t0 * p.topk;
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) s_id[i] = p.ids[pair0 + i];
    if (threadIdx.x < kW4Tokens) s_pair[threadIdx.x] = -1;
    __syncthreads();
    if constexpr (kMode == kW4Gather) {
      // CTA (n tile, pair): a pair whose expert was chosen 8 r times before it in
      // the block leads that expert's next 8 pairs; the other pairs' CTAs leave.
      const int me = blockIdx.y;
      if (me >= pairs) return;
      const int e = s_id[me];
      const bool valid = e >= 0 && e < p.E;
      int rank = 0;
      for (int i = 0; i < me; ++i) rank += s_id[i] == e;
      if (valid && rank % kW4Tokens) return;
      if (warp == 0) {
        int seen = 0;
        for (int b = 0; b < pairs; b += 32) {
          const bool hit = b + lane < pairs && (valid ? s_id[b + lane] == e : b + lane == me);
          const unsigned mask = __ballot_sync(0xffffffffu, hit);
          const int r = seen + __popc(mask & ((1u << lane) - 1u)) - (valid ? rank : 0);
          if (hit && r >= 0 && r < kW4Tokens) s_pair[r] = b + lane;
          seen += __popc(mask);
        }
      }
      __syncthreads();
      if (valid) {
        const int mine = s_pair[g];
        const uint16_t* xr[1] = {mine >= 0 ? p.x + (int64_t)(t0 + mine / p.topk) * p.K : nullptr};
        for (int c = warp; c < p.nchunk; c += warps) {
          u.load(p, e * p.N + r0, e * p.N + r1, xr, c, t);
          u.template accumulate<false>(acc);
        }
      }
    } else {
      // The block's experts in the order of their first pair; an entry is one
      // expert with, for each token, the pair that chose it.  A token that names
      // an expert twice gets an entry of its own for the second.
      if (threadIdx.x == 0) {
        int count = 0;
        for (int i = 0; i < pairs; ++i) {
          const int e = s_id[i], tok = i / p.topk;
          if (e < 0 || e >= p.E) continue;
          int at = 0;
          while (at < count && (s_entry[at] != e || s_slot[at][tok] >= 0)) ++at;
          if (at == count) {
            s_entry[count++] = e;
            for (int q = 0; q < kW4Tokens; ++q) s_slot[at][q] = -1;
          }
          s_slot[at][tok] = i;
        }
        s_count = count;
      }
      __syncthreads();
      const int units = s_count * p.nchunk;
      for (int q = warp; q < units; q += warps) {
        const int at = q / p.nchunk, c = q - at * p.nchunk;
        const int64_t e = s_entry[at];
        const int mine = s_slot[at][g], ca = s_slot[at][2 * t], cb = s_slot[at][2 * t + 1];
        const uint16_t* xr[1] = {mine >= 0 ? p.x + (pair0 + mine) * p.K : nullptr};
        const float2 cw = make_float2(ca >= 0 ? __ldg(p.wts + pair0 + ca) : 0.0f,
                                      cb >= 0 ? __ldg(p.wts + pair0 + cb) : 0.0f);
        u.load(p, e * p.N + r0, e * p.N + r1, xr, c, t);
        u.template accumulate<true>(acc, cw, ca >= 0, cb >= 0);
      }
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

cudaError_t launch_w4_stream(const uint16_t* x, const ql_w4_weight& w, int64_t M, uint16_t* y, cudaStream_t st) {
  const W4StreamParams p = stream_params(x, w, M, y);
  const unsigned tiles = (unsigned)((w.N + kW4Rows - 1) / kW4Rows);
  if (M <= kW4Tokens) return launch_group<1, kW4Dense>(p, (int)w.group, dim3(tiles, 1), 8, st);
  return launch_group<2, kW4Dense>(p, (int)w.group, dim3(tiles, (unsigned)((M + 15) / 16)), 8, st);
}

cudaError_t launch_w4_stream_experts(const uint16_t* x, const int32_t* ids, const float* weights,
                                     const ql_w4_weight& w, int64_t T, int64_t topk, uint16_t* y,
                                     cudaStream_t st) {
  W4StreamParams p = stream_params(x, w, T, y);
  p.ids = ids;
  p.wts = weights;
  p.topk = (int)topk;
  p.E = (int)w.experts;
  const unsigned tiles = (unsigned)((w.N + kW4Rows - 1) / kW4Rows), blocks = (unsigned)((T + kW4Tokens - 1) / kW4Tokens);
  if (weights) return launch_group<1, kW4Combine>(p, (int)w.group, dim3(tiles, 1, blocks), 8, st);
  const unsigned pairs = (unsigned)(std::min<int64_t>(T, kW4Tokens) * topk);
  return launch_group<1, kW4Gather>(p, (int)w.group, dim3(tiles, pairs, blocks), 8, st);
}

}  // namespace ql
