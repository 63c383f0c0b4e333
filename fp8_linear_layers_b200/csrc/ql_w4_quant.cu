// ql_w4_quant.cu -- 4-bit weight quantization in groups along K (offline).
//
//   no zero points:  s = bf16(absmax / 7),        q = clamp(rne(w / s), -7, 7) + 8
//   zero points:     s = bf16((hi - lo) / 15),    z = clamp(rne(-lo / s), 0, 15),
//                    q = clamp(rne(w / s) + z, 0, 15),  lo <= 0 <= hi the group's range
//
// with IEEE f32 divisions; a group whose scale is zero gets codes (and zero
// points) 8.  One thread takes 8 inputs (16 bytes), group / 8 neighbouring lanes
// take a group.  Offline: 14336 x 4096 101 us, with zero points 106 (1.4 TB/s read and
// written); a division to a weight, not the bytes, takes the time.
#include "ql_internal.h"
#include "ql_w4.cuh"

namespace ql {

template <bool kZero>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const uint16_t* __restrict__ w, int64_t N, int64_t K,
                                                          int group, int64_t groups, uint8_t* __restrict__ wq,
                                                          uint16_t* __restrict__ sw, uint8_t* __restrict__ wz) {
  const int per = group / 8;  // lanes of a group: 4, 8 or 16
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t gi = id / per;
  const bool live = gi < N * groups;
  const int64_t n = live ? gi / groups : 0, gg = live ? gi - n * groups : 0;
  const int64_t k = gg * group + (id % per) * 8;
  const bool in = live && k < K;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (in) v = *reinterpret_cast<const uint4*>(w + n * K + k);
  const uint32_t words[4] = {v.x, v.y, v.z, v.w};
  float f[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(words[j]);
    f[2 * j + 1] = bf16_hi(words[j]);
    lo = fminf(lo, fminf(f[2 * j], f[2 * j + 1]));
    hi = fmaxf(hi, fmaxf(f[2 * j], f[2 * j + 1]));
  }
  for (int o = per >> 1; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint16_t s16 = f32_to_bf16_rn(kZero ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
  const float s = __uint_as_float((uint32_t)s16 << 16);
  float z = 8.0f;
  if (kZero && s > 0.0f) z = fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f);
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float q = s > 0.0f ? rintf(f[j] / s) : 0.0f;
    if (kZero)
      q = fminf(fmaxf(q + z, 0.0f), 15.0f);
    else
      q = fminf(fmaxf(q, -7.0f), 7.0f) + 8.0f;
    out |= (uint32_t)q << (4 * j);
  }
  if (in) *reinterpret_cast<uint32_t*>(wq + n * (K >> 1) + (k >> 1)) = out;
  if (live && id % per == 0) {
    sw[gi] = s16;
    if (kZero) wz[gi] = (uint8_t)z;
  }
}

cudaError_t launch_quantize_w4(const uint16_t* w, int64_t N, int64_t K, int64_t group, uint8_t* wq, uint16_t* sw,
                               uint8_t* wz, cudaStream_t st) {
  const int64_t groups = (K + group - 1) / group;
  const int64_t threads = N * groups * (group / 8);
  const unsigned blocks = (unsigned)((threads + 255) / 256);
  if (wz)
    quantize_w4_kernel<true><<<blocks, 256, 0, st>>>(w, N, K, (int)group, groups, wq, sw, wz);
  else
    quantize_w4_kernel<false><<<blocks, 256, 0, st>>>(w, N, K, (int)group, groups, wq, sw, nullptr);
  return cudaGetLastError();
}

}  // namespace ql
