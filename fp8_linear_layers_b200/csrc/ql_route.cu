// ql_route.cu -- routing of tokens to experts: scores, balance bias, groups, top-k
// and the chosen experts' weights, one kernel.
//
//   p = softmax(l) or sigmoid(l);  c = p + bias, or without a bias c = l (both
//   scores rise with the logit, so the order is the same);  experts outside the
//   best groups leave;  ids = the k largest c, ties to the lower index;
//   w_j = p[id_j], divided by their sum when renormalized, times a scale.
//
// The floor is the logits' bytes (T E of 2 or 4 bytes); the selection's instructions are
// what bounds the kernel.  One warp takes one token.  Lane i keeps the experts
// [i VPL, (i + 1) VPL) in registers, as unsigned keys that sort like the values (0 = not
// available), so that a row is read in 16-byte pieces, the lowest lane that holds a
// maximum holds its lowest index, and a group of experts is a run of lanes: all groups'
// values come from one local pass and a few shuffles.  A round of the selection is one
// warp-wide integer maximum, a ballot, and a new local maximum for the lane that lost
// its own.
//
// Order must not depend on rounding.  Without a bias the keys are the logits
// themselves.  With one (or when two scores are summed for a group) the f32 values
// carry an error, for which there is a bound.  Where two neighbours in the order, or the
// last chosen and the best left out, are closer than that, the candidates that can
// matter (at most 32, one to a lane) get their f64 values and are ranked by those; where
// groups are that close, or more than 32 candidates, the token is selected again from
// f64 values throughout (4099 x 256, sigmoid, bias, groups: 13.4 us, 18 to 20 with such a
// token).  Up to 128 experts, and from 257 to 512, 8 to 16 bytes a thread spill.
#include "ql_internal.h"
#include "ql_w4.cuh"

namespace ql {

constexpr int kRouteWarps = 4;
constexpr unsigned kFull = 0xffffffffu;

// Bounds on the relative error of an f32 score of at least 1e-37 (what is below is always
// compared in f64).  Sigmoid: expf is within 2^-23, 1 + e rounds to 2^-24, the
// approximate reciprocal is within 2^-23 and the product rounds to 2^-24.  Softmax: the
// difference d of two logits rounds to |d| 2^-24, of which |d| <= 88 matters, expf and
// two roundings add 2^-22, and the sum's terms are off by the mean of that |d| (at most
// 8 for 1024 terms) and its 37 additions by 2^-24 each.
constexpr float kSigmoidErr = 0x1p-20f;
constexpr float kSoftmaxErr = 0x1p-16f;
constexpr float kScoreFloor = 1e-37f;
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
  int glanes;  // lanes of a group where groups are runs of 2^n lanes, else 0
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

// For comparisons: see kSigmoidErr.
QL_DEVINL float sigmoid_fast(float l) {
  const float e = expf(-fabsf(l));
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return l >= 0.0f ? r : e * r;
}
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
    const bool again = pass == 1 && p.G > 1 && (p.bias || p.group_top == 1);  // the groups' pass made these values
    for (int e = lane; again && e < p.E; e += 32)
      if (!((kept >> (((e * p.gmagic) >> 20) & 31)) & 1u)) c[e] = kNone;
#pragma unroll 4
    for (int e = lane; !again && e < p.E; e += 32) {
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
        gs = p.group_top == 1 ? a : b == kNone ? kNone : a + b;  // (a may be +inf)
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

// A candidate's exact choice (f64).
template <bool kBf16>
QL_DEVINL double choice_f64(const RouteParams& p, const void* row, int e, float lmax, double sum) {
  const double d = (double)finite(load_logit<kBf16>(row, e));
  const double v = p.sigmoid ? sigmoid(d) : exp(d - (double)lmax) / sum;
  return v + (double)__ldg(p.bias + e);
}

template <int VPL, bool kBf16>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams p) {
  extern __shared__ double route_smem[];  // kRouteWarps rows of E doubles (scores by group or f64)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float none = -__int_as_float(0x7f800000);
  tc::grid_dependency_wait();
  tc::launch_dependents();
  const int64_t tok = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (tok >= p.T) return;
  const void* row = static_cast<const char*>(p.logits) + tok * p.E * (kBf16 ? 2 : 4);

  // logits (this lane's VPL, in 16-byte pieces where the row is whole) and their maximum
  float l[VPL];
  const bool whole = p.E == 32 * VPL && VPL >= 4;
  if (whole) {
    if constexpr (kBf16 && VPL >= 8) {
#pragma unroll
      for (int i = 0; i < VPL / 8; ++i) {
        const uint4 v = __ldg(static_cast<const uint4*>(row) + lane * (VPL / 8) + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          l[8 * i + 2 * j] = bf16_lo(w[j]);
          l[8 * i + 2 * j + 1] = bf16_hi(w[j]);
        }
      }
    } else if constexpr (kBf16 && VPL == 4) {
      const uint2 v = __ldg(static_cast<const uint2*>(row) + lane);
      l[0] = bf16_lo(v.x), l[1] = bf16_hi(v.x), l[2] = bf16_lo(v.y), l[3] = bf16_hi(v.y);
    } else if constexpr (!kBf16 && VPL >= 4) {
#pragma unroll
      for (int i = 0; i < VPL / 4; ++i) {
        const float4 v = __ldg(static_cast<const float4*>(row) + lane * (VPL / 4) + i);
        l[4 * i] = v.x, l[4 * i + 1] = v.y, l[4 * i + 2] = v.z, l[4 * i + 3] = v.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      l[i] = e < p.E ? load_logit<kBf16>(row, e) : none;
    }
  }
  float mx = none;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (usable(l[i])) mx = fmaxf(mx, l[i] = finite(l[i]));
  const bool scores = p.bias || (p.G > 1 && p.group_top == 2);  // values beyond the logits are compared
  float sum = 1.0f;
  if (!p.sigmoid && (scores || !p.renormalize)) {
    mx = warp_max(mx);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (usable(l[i])) s += expf(l[i] - mx);
    sum = warp_sum(s);
  }
  const float inv = 1.0f / sum;
  const float err = p.sigmoid ? kSigmoidErr : kSoftmaxErr;
  auto score = [&](float v) { return p.sigmoid ? sigmoid_fast(v) : expf(v - mx) * inv; };

  uint32_t key[VPL];
  if (p.bias) {
    float b[VPL];
    if (whole) {
      if constexpr (VPL >= 4)
#pragma unroll
        for (int i = 0; i < VPL / 4; ++i) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(p.bias) + lane * (VPL / 4) + i);
          b[4 * i] = v.x, b[4 * i + 1] = v.y, b[4 * i + 2] = v.z, b[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) b[i] = lane * VPL + i < p.E ? __ldg(p.bias + lane * VPL + i) : none;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = usable(l[i]) && usable(b[i]) ? order_key(score(l[i]) + b[i]) : 0;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = usable(l[i]) ? order_key(l[i]) : 0;
  }

  bool unsure = false;
  if (p.G > 1) {
    // every group's value and a bound on its error, on the lane of the group's number or
    // (runs of lanes) on all of the group's lanes
    uint32_t gkey = 0;
    float gerr = 0.0f;
    float a = none, b = none;  // the group's two largest
    auto add = [&](float v) {
      b = fmaxf(b, fminf(a, v));
      a = fmaxf(a, v);
    };
    const bool by_key = p.bias || p.group_top == 1;
    bool member;  // this lane stands for a group
    if (p.glanes) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) add(!key[i] ? none : by_key ? key_value(key[i]) : score(l[i]));
      for (int o = 1; o < p.glanes; o <<= 1) {
        const float oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
        add(oa);
        add(ob);
      }
      member = lane < p.G * p.glanes;
    } else {
      float* c = reinterpret_cast<float*>(route_smem + warp * p.E);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane * VPL + i < p.E) c[lane * VPL + i] = !key[i] ? none : by_key ? key_value(key[i]) : score(l[i]);
      __syncwarp();
      member = lane < p.G;
      if (member) {
        int off = lane % p.gsize;  // rotated: the groups' rows start on different banks
        for (int i = 0; i < p.gsize; ++i) {
          add(c[lane * p.gsize + off]);
          off = off + 1 == p.gsize ? 0 : off + 1;
        }
      }
      __syncwarp();
    }
    if (member) {
      // the mean of two stands for their sum: it is in range wherever they are (a mask may be
      // the lowest f32); short of two, -inf, though the one be +inf
      const float gs = p.group_top == 1 ? a : usable(b) ? 0.5f * a + 0.5f * b : none;
      gkey = order_key(gs);
      // scores are at most 1; without a bias a single largest is a logit, and exact; so are
      // infinities
      if (scores && fabsf(gs) < -none)
        gerr = err + kRoundErr * (p.group_top == 1 ? fabsf(a) : 0.5f * fabsf(a) + 0.5f * fabsf(b));
    }
    uint32_t kept = 0;  // by group
    float low = 0.0f;   // the smallest value kept, less its error
    for (int r = 0; r < p.top_groups; ++r) {
      const uint32_t m = __reduce_max_sync(kFull, gkey);
      const int win = __ffs(__ballot_sync(kFull, gkey == m)) - 1;
      const int group = p.glanes ? win / p.glanes : win;
      kept |= 1u << group;
      const float v = key_value(m) - __shfl_sync(kFull, gerr, win);
      low = r == 0 ? v : fminf(low, v);
      if ((p.glanes ? lane / p.glanes : lane) == group) gkey = 0;
    }
    if (scores) unsure = __any_sync(kFull, gkey && gerr > 0.0f && key_value(gkey) + gerr >= low);
    if (p.glanes) {
      if (!((kept >> (lane / p.glanes & 31)) & 1u)) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!((kept >> ((((lane * VPL + i) * p.gmagic) >> 20) & 31)) & 1u)) key[i] = 0;
    }
  }

  // k rounds; lane j keeps round j's winner
  uint32_t best = 0;
  int best_i = 0;
  auto local_best = [&] {
    best = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) {
        best = key[i];
        best_i = i;
      }
  };
  local_best();
  __shared__ uint2 s_won[kRouteWarps][32];  // the rounds' winners: key, expert
  auto round = [&](int j) {  // false: none left
    const uint32_t m = __reduce_max_sync(kFull, best);
    if (m == 0) return false;
    const unsigned at = __ballot_sync(kFull, best == m);
    if (best == m && (at & ((1u << lane) - 1u)) == 0) {  // the lowest lane has the lowest index
      s_won[warp][j] = make_uint2(m, (unsigned)(lane * VPL + best_i));
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == best_i) key[i] = 0;
      local_best();
    }
    return true;
  };
  int n = 0;
#pragma unroll 1
  while (n < p.k && round(n)) ++n;
  int my_id = -1;
  uint32_t my_key = 0;
  auto collect = [&] {  // lane j takes round j's winner
    __syncwarp();
    if (lane < n) {
      my_key = s_won[warp][lane].x;
      my_id = (int)s_won[warp][lane].y;
    }
  };
  collect();
  if (p.bias && !unsure) {
    // neighbours in the order whose f32 distance does not settle it
    const uint32_t left = __reduce_max_sync(kFull, best);
    float mine = 0.0f, b = 0.0f;
    if (my_id >= 0) {
      mine = load_logit<kBf16>(row, my_id);
      b = __ldg(p.bias + my_id);
    }
    uint32_t next = __shfl_down_sync(kFull, my_key, 1);
    const float next_l = __shfl_down_sync(kFull, mine, 1), next_b = __shfl_down_sync(kFull, b, 1);
    const bool border = lane == p.k - 1;
    if (border) next = left;
    bool close = false;
    const float c0 = key_value(my_key);
    if (my_id >= 0 && next) {
      const float c1 = key_value(next);
      const bool same = !border && mine == next_l && b == next_b;
      const float nb = border ? fabsf(c1) + 1.0f : fabsf(next_b);
      close = !same && !(c0 - c1 > err * (fabsf(c0) + fabsf(b) + fabsf(c1) + nb) + kScoreFloor);
    }
    if (__any_sync(kFull, close)) {
      // more candidates, while they may reach the last chosen one; then all by their f64 values
      const uint32_t kth = __shfl_sync(kFull, my_key, p.k - 1);
      bool more = kth != 0;
      const float cut = key_value(kth) - 2.0f * err * (2.0f * fabsf(key_value(kth)) + 2.0f) - kScoreFloor;
      while (n < 32 && more) {
        const uint32_t m = __reduce_max_sync(kFull, best);
        more = m != 0 && !(key_value(m) < cut);
        if (more && round(n)) ++n;
      }
      collect();
      unsure = more;
      if (!unsure) {
        double total = 1.0;
        if (!p.sigmoid) {
          double s = 0.0;
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (usable(l[i])) s += exp((double)l[i] - (double)mx);
          total = warp_sum(s);
        }
        const double c = my_id >= 0 ? choice_f64<kBf16>(p, row, my_id, mx, total) : 0.0;
        int rank = 0;
        for (int i = 0; i < n; ++i) {
          const double oc = __shfl_sync(kFull, c, i);
          const int oid = __shfl_sync(kFull, my_id, i);
          rank += oc > c || (oc == c && oid < my_id);
        }
        int out = -1;
        for (int i = 0; i < n; ++i) {
          const int orank = __shfl_sync(kFull, rank, i), oid = __shfl_sync(kFull, my_id, i);
          if (orank == lane) out = oid;
        }
        my_id = lane < p.k ? out : -1;
      }
    }
  }
  if (unsure) {
    select_f64<VPL, kBf16>(p, row, mx, route_smem + warp * p.E, lane, my_id);
    if (!p.bias && my_id >= 0) my_key = order_key(finite(load_logit<kBf16>(row, my_id)));
  }

  // weights of the chosen experts, one to a lane
  const bool has = lane < p.k && my_id >= 0;
  float lj = 0.0f;  // without a bias the key is the logit
  if (has) lj = p.bias ? finite(load_logit<kBf16>(row, my_id)) : key_value(my_key);
  float w = 0.0f;
  if (p.renormalize) {
    // scaled by a common factor so that the largest is near 1: w_j / sum does not underflow
    float top = p.sigmoid ? fminf(lj, 0.0f) : lj;
    top = p.bias ? warp_max(has ? top : none) : __shfl_sync(kFull, top, 0);
    if (has) w = p.sigmoid ? expf(fminf(lj, 0.0f) - top) / (1.0f + expf(-fabsf(lj))) : expf(lj - top);
    float s = w;
    for (int o = 1; o < p.k; o <<= 1) s += __shfl_xor_sync(kFull, s, o);
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
  const int vpl = p.E <= 32 ? 1 : p.E <= 64 ? 2 : p.E <= 128 ? 4 : p.E <= 256 ? 8 : p.E <= 512 ? 16 : 32;
  if (p.gsize % vpl == 0 && ((p.gsize / vpl) & (p.gsize / vpl - 1)) == 0) p.glanes = p.gsize / vpl;
  p.gmagic = (uint32_t)(((1u << 20) + p.gsize - 1) / p.gsize);
  p.renormalize = c.renormalize != 0;
  p.scale = c.scale;
  return bf16 ? launch_route_e<true>(p, st) : launch_route_e<false>(p, st);
}

}  // namespace ql
