// ql_route.cu -- routing of tokens to experts: scores, balance bias, groups, top-k
// and the chosen experts' weights, one kernel.
//
//   p = softmax(l) or sigmoid(l);  c = p + bias, or without a bias c = l (both
//   scores rise with the logit, so the order is the same);  experts outside the
//   best groups leave;  ids = the k largest c, ties to the lower index;
//   w_j = p[id_j], divided by their sum when renormalized, times a scale.
//
// The floor is the logits' bytes (T E of 2 or 4 bytes); the selection's
// instructions are what bounds the kernel.  One warp takes one token and keeps
// its logits in registers, E / 32 to a lane, as unsigned keys that sort like the
// values (0 = not available); a round of the selection is one warp-wide integer
// maximum and one minimum of the indices that hold it.
//
// Order must not depend on rounding.  Without a bias the keys are the logits
// themselves.  With one (or when two scores are summed for a group) the f32 values
// carry an error, so neighbours in the selected order, and the last chosen against
// the best left out, are compared with a bound on it; a token with a pair inside
// the bound is selected again from f64 values.  That is about one token in a few
// hundred, so the common path stays f32.
#include "ql_internal.h"
#include "ql_w4.cuh"

namespace ql {

constexpr int kRouteWarps = 4;
constexpr unsigned kFull = 0xffffffffu;

// Bound on the relative error of an f32 score: expf and the division are within
// a few ulp and a softmax sum of up to 1024 terms within 2^-20; 2^-18 covers both.
constexpr float kScoreErr = 0x1p-18f;
constexpr float kRoundErr = 0x1p-22f;

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t T;
  int E, k;
  int sigmoid;
  int G, top_groups, group_top, gsize;
  uint32_t gmagic;  // e / gsize == e * gmagic >> 20 for e, gsize <= 1024
  int renormalize;
  float scale;
};

// Order-preserving key of a float that is not a NaN; never 0.
QL_DEVINL uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 and +0 are equal
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
QL_DEVINL float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

QL_DEVINL float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
QL_DEVINL double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

template <bool kBf16>
QL_DEVINL float load_logit(const void* row, int e) {
  if constexpr (kBf16) return bf16_lo(__ldg(static_cast<const uint16_t*>(row) + e));
  return __ldg(static_cast<const float*>(row) + e);
}

// A logit that can be chosen: not NaN, not -inf; +inf reads as the largest f32.
QL_DEVINL bool usable(float l) { return l > -__int_as_float(0x7f800000); }
QL_DEVINL float finite(float l) { return fminf(l, 3.402823466e38f); }

QL_DEVINL float sigmoid(float l) {
  const float e = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}
QL_DEVINL double sigmoid(double l) {
  const double e = exp(-fabs(l));
  return (l >= 0.0 ? 1.0 : e) / (1.0 + e);
}

// The lane-wide winner (value, index): largest value, then lowest index.
QL_DEVINL void warp_argmax(double& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(kFull, v, o);
    const int oi = __shfl_xor_sync(kFull, i, o);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

// The selection from f64 values; `c` is the warp's row of E doubles.
template <int VPL, bool kBf16>
__device__ __noinline__ void select_f64(const RouteParams& p, const void* row, float lmax, double* c, int lane,
                                        int& my_id) {
  const double kNone = -__longlong_as_double(0x7ff0000000000000ll);
  double sum = 0.0;
  if (!p.sigmoid) {
    for (int e = lane; e < p.E; e += 32) {
      const float l = load_logit<kBf16>(row, e);
      if (usable(l)) sum += exp((double)finite(l) - (double)lmax);
    }
    sum = warp_sum(sum);
  }
  for (int pass = 0; pass < 2; ++pass) {
    // pass 0: the groups' values; pass 1: the members' (the logits, without a bias)
    const bool by_logit = !p.bias && (pass == 1 || p.group_top == 1);
    if (pass == 0 && p.G == 1) continue;
    uint32_t kept = kFull;
    if (pass == 1 && p.G > 1) kept = (uint32_t)my_id;
    __syncwarp();
    for (int e = lane; e < p.E; e += 32) {
      const float l = load_logit<kBf16>(row, e);
      double v = kNone;
      if (usable(l)) {
        const double d = (double)finite(l);
        v = by_logit ? d : p.sigmoid ? sigmoid(d) : exp(d - (double)lmax) / sum;
        if (p.bias) {
          const float b = __ldg(p.bias + e);
          v = usable(b) ? v + (double)b : kNone;
        }
        if (pass == 1 && p.G > 1 && !((kept >> (((e * p.gmagic) >> 20) & 31)) & 1u)) v = kNone;
      }
      c[e] = v;
    }
    __syncwarp();
    if (pass == 0) {
      double gs = kNone;
      if (lane < p.G) {
        double a = kNone, b = kNone;
        for (int i = 0; i < p.gsize; ++i) {
          const double v = c[lane * p.gsize + i];
          if (v > a) {
            b = a;
            a = v;
          } else if (v > b) {
            b = v;
          }
        }
        gs = p.group_top == 1 ? a : a + b;
      }
      uint32_t mask = 0;
      bool taken = lane >= p.G;
      for (int r = 0; r < p.top_groups; ++r) {
        double v = taken ? kNone : gs;
        int i = taken ? 64 + lane : lane;
        warp_argmax(v, i);
        // all that is left may be -inf: the lowest group not taken yet
        mask |= 1u << (i & 31);
        if (i == lane) taken = true;
      }
      my_id = (int)mask;
    } else {
      int out = -1;
      for (int j = 0; j < p.k; ++j) {
        double v = kNone;
        int i = 0x7fffffff;
        for (int e = lane; e < p.E; e += 32)
          if (c[e] > v) {
            v = c[e];
            i = e;
          }
        warp_argmax(v, i);
        if (i == 0x7fffffff) break;
        if (lane == j) out = i;
        __syncwarp();
        if (lane == 0) c[i] = kNone;
        __syncwarp();
      }
      my_id = out;
    }
  }
}

template <int VPL, bool kBf16>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams p) {
  extern __shared__ double route_smem[];  // kRouteWarps rows of E doubles (scores by group or f64)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tc::grid_dependency_wait();
  tc::launch_dependents();
  const int64_t tok = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (tok >= p.T) return;
  const void* row = static_cast<const char*>(p.logits) + tok * p.E * (kBf16 ? 2 : 4);

  // logits, their maximum and (softmax) the sum
  float l[VPL];
  float mx = -__int_as_float(0x7f800000);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    l[i] = e < p.E ? load_logit<kBf16>(row, e) : -__int_as_float(0x7f800000);
    if (usable(l[i])) mx = fmaxf(mx, l[i] = finite(l[i]));
  }
  mx = warp_max(mx);
  const bool scores = p.bias || (p.G > 1 && p.group_top == 2);  // values beyond the logits are compared
  float sum = 1.0f;
  if (!p.sigmoid && (scores || !p.renormalize)) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (usable(l[i])) s += expf(l[i] - mx);
    sum = warp_sum(s);
  }

  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = 0;
    if (usable(l[i])) {
      float v = l[i];
      if (p.bias) {
        const float b = __ldg(p.bias + i * 32 + lane);
        v = (p.sigmoid ? sigmoid(v) : expf(v - mx) / sum) + b;
        if (!usable(b)) v = __int_as_float(0x7fffffff);
      }
      if (v == v) key[i] = order_key(v);
    }
  }

  bool unsure = false;
  if (p.G > 1) {
    float* c = reinterpret_cast<float*>(route_smem + warp * p.E);
    const float none = -__int_as_float(0x7f800000);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      if (e < p.E) {
        float v = none;
        if (key[i])
          v = p.bias || p.group_top == 1 ? key_value(key[i]) : p.sigmoid ? sigmoid(l[i]) : expf(l[i] - mx) / sum;
        c[e] = v;
      }
    }
    __syncwarp();
    uint32_t gkey = 0;
    float gerr = 0.0f;
    if (lane < p.G) {
      float a = none, b = none;
      int off = lane % p.gsize;  // rotated: the groups' rows start on different banks
      for (int i = 0; i < p.gsize; ++i) {
        const float v = c[lane * p.gsize + off];
        off = off + 1 == p.gsize ? 0 : off + 1;
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
      const float gs = p.group_top == 1 ? a : a + b;
      gkey = order_key(gs);
      gerr = usable(gs) ? 2.0f * kScoreErr + kRoundErr * (fabsf(a) + fabsf(b)) : 0.0f;
      if (p.group_top == 1) gerr = p.bias ? kScoreErr + kRoundErr * fabsf(a) : 0.0f;
      if (!usable(gs)) gerr = 0.0f;
    }
    __syncwarp();
    uint32_t kept = 0;
    float low = 0.0f;  // the smallest value kept, less its error
    for (int r = 0; r < p.top_groups; ++r) {
      const uint32_t m = __reduce_max_sync(kFull, gkey);
      const int win = __ffs(__ballot_sync(kFull, gkey == m)) - 1;
      kept |= 1u << win;
      const float v = key_value(m) - __shfl_sync(kFull, gerr, win);
      low = r == 0 ? v : fminf(low, v);
      if (lane == win) gkey = 0;
    }
    if (scores) {
      const bool close = gkey && gerr > 0.0f && key_value(gkey) + gerr >= low;
      unsure = __any_sync(kFull, close);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!((kept >> ((((i * 32 + lane) * p.gmagic) >> 20) & 31)) & 1u)) key[i] = 0;
  }

  // k rounds (one more where the choice may have to be confirmed); lane j keeps round j's winner
  uint32_t best = 0;
  int best_i = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (key[i] > best) {
      best = key[i];
      best_i = i;
    }
  int my_id = -1;
  uint32_t my_key = 0, next_key = 0;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t m = __reduce_max_sync(kFull, best);
    if (m == 0) break;
    const int win = (int)__reduce_min_sync(kFull, best == m ? (unsigned)(best_i * 32 + lane) : kFull);
    if (lane == j) {
      my_id = win;
      my_key = m;
    }
    if ((win & 31) == lane) {
      best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i == (win >> 5)) key[i] = 0;
        if (key[i] > best) {
          best = key[i];
          best_i = i;
        }
      }
    }
  }
  if (p.bias && !unsure) {
    // neighbours in the order whose f32 distance does not settle it
    const uint32_t left = __reduce_max_sync(kFull, best);
    next_key = __shfl_down_sync(kFull, my_key, 1);
    if (lane == p.k - 1) next_key = left;
    float mine = 0.0f, b = 0.0f;
    if (my_id >= 0) {
      mine = load_logit<kBf16>(row, my_id);
      b = __ldg(p.bias + my_id);
    }
    const float next_l = __shfl_down_sync(kFull, mine, 1), next_b = __shfl_down_sync(kFull, b, 1);
    bool close = false;
    if (my_id >= 0 && next_key) {
      const float c0 = key_value(my_key), c1 = key_value(next_key);
      const bool same = lane < p.k - 1 && mine == next_l && b == next_b;
      const float nb = lane < p.k - 1 ? fabsf(next_b) : fabsf(c1) + 1.0f;
      close = !same && !(c0 - c1 > kScoreErr * (fabsf(c0) + fabsf(b) + fabsf(c1) + nb));
    }
    unsure = __any_sync(kFull, close);
  }
  if (unsure) select_f64<VPL, kBf16>(p, row, mx, route_smem + warp * p.E, lane, my_id);

  // weights of the chosen experts, one to a lane
  const bool has = lane < p.k && my_id >= 0;
  const float lj = has ? finite(load_logit<kBf16>(row, my_id)) : 0.0f;
  float w = 0.0f;
  if (p.renormalize) {
    // scaled by a common factor so that the largest is near 1: w_j / sum does not underflow
    const float top = warp_max(has ? (p.sigmoid ? fminf(lj, 0.0f) : lj) : -__int_as_float(0x7f800000));
    if (has) w = p.sigmoid ? expf(fminf(lj, 0.0f) - top) / (1.0f + expf(-fabsf(lj))) : expf(lj - top);
    const float s = warp_sum(w);
    if (has) w = w / s;
  } else if (has) {
    w = p.sigmoid ? sigmoid(lj) : expf(lj - mx) / sum;
  }
  if (lane < p.k) {
    p.ids[tok * p.k + lane] = my_id;
    p.weights[tok * p.k + lane] = w * p.scale;
  }
}

// ---------------------------------------------------------------------------- host

template <int VPL, bool kBf16>
static cudaError_t launch_route_t(const RouteParams& p, cudaStream_t st) {
  const bool rows = p.bias || p.G > 1;
  const size_t smem = rows ? (size_t)kRouteWarps * p.E * sizeof(double) : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.T + kRouteWarps - 1) / kRouteWarps));
  cfg.blockDim = dim3(kRouteWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_kernel<VPL, kBf16>, p);
}

template <bool kBf16>
static cudaError_t launch_route_e(const RouteParams& p, cudaStream_t st) {
  const int vpl = (p.E + 31) / 32;
  if (vpl <= 1) return launch_route_t<1, kBf16>(p, st);
  if (vpl <= 2) return launch_route_t<2, kBf16>(p, st);
  if (vpl <= 4) return launch_route_t<4, kBf16>(p, st);
  if (vpl <= 8) return launch_route_t<8, kBf16>(p, st);
  if (vpl <= 16) return launch_route_t<16, kBf16>(p, st);
  return launch_route_t<32, kBf16>(p, st);
}

cudaError_t launch_route(const void* logits, bool bf16, const ql_route_config& c, const float* bias, int64_t T,
                         int32_t* ids, float* weights, cudaStream_t st) {
  RouteParams p = {};
  p.logits = logits;
  p.bias = bias;
  p.ids = ids;
  p.weights = weights;
  p.T = T;
  p.E = (int)c.experts;
  p.k = (int)c.top_k;
  p.sigmoid = c.score == QL_ROUTE_SIGMOID;
  p.G = (int)c.groups;
  p.top_groups = (int)c.top_groups;
  p.group_top = (int)c.group_top;
  p.gsize = p.E / p.G;
  p.gmagic = (uint32_t)(((1u << 20) + p.gsize - 1) / p.gsize);
  p.renormalize = c.renormalize != 0;
  p.scale = c.scale;
  return bf16 ? launch_route_e<true>(p, st) : launch_route_e<false>(p, st);
}

}  // namespace ql
