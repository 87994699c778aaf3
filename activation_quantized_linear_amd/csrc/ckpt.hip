// Activation checkpoints in 8 bits: per row and group of 128 columns
//   s = max |x| / 127 (1 where that is not positive), code = clamp(rint(x / s), -127, 127)
// and back, x' = code * s. One pass over the data each way, bound by memory:
// 3 bytes a value (bf16) plus 4 bytes a group.
//
// 32 lanes hold a group, 4 values a lane, so a group's maximum takes 5 lane
// exchanges and no LDS, a wave works on two groups at a time, and a lane packs
// its four codes into one dword store. Groups are numbered over the whole
// matrix; a half wave takes kIlp of them at once to keep enough loads in flight.
#include "ckpt.h"

namespace aql {
namespace {

constexpr int kIlp = 4;

template <bool BF16>
__device__ __forceinline__ f32x4 load4(const void *x, int64_t i) {
  if constexpr (BF16) {
    const i32x2 d = *reinterpret_cast<const i32x2 *>(static_cast<const uint16_t *>(x) + i);
    return f32x4{__uint_as_float((uint32_t)d[0] << 16), __uint_as_float((uint32_t)d[0] & 0xffff0000u),
                 __uint_as_float((uint32_t)d[1] << 16), __uint_as_float((uint32_t)d[1] & 0xffff0000u)};
  } else {
    return *reinterpret_cast<const f32x4 *>(static_cast<const float *>(x) + i);
  }
}

// rint(v / s) for |v| <= 127 s, s a normal float with a normal reciprocal r:
// v r carries two roundings (2^-24 each) and lies within 2^-16 of the IEEE
// quotient (at most 127), so unless it is within 2^-10 of a half integer both
// round to the same code; those few take the division itself.
__device__ __forceinline__ float code_of(float v, float s, float r) {
  const float t = v * r;
  float c = rintf(t);
  if (fabsf(t - c) > 0.5f - 0x1p-10f) c = rintf(v / s);
  return c;
}

// First element of group t's four of lane l, and whether they lie in the matrix:
// (m, gi) is group t's row and place in it.
__device__ __forceinline__ void next_group(int64_t &m, int64_t &gi, int64_t G) {
  if (++gi == G) {
    gi = 0;
    ++m;
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_act_checkpoint(const void *__restrict__ x, int64_t groups,
                                                        int64_t K, int64_t G,
                                                        int8_t *__restrict__ xq,
                                                        float *__restrict__ xs) {
  const int l = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kIlp;
  int64_t m = t0 / G, gi = t0 - m * G;
  f32x4 v[kIlp];
  int64_t at[kIlp];
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    const int64_t c = gi * kCkptGroup + 4 * l;
    const bool in = t0 + u < groups && c < K;  // whole fours: K is a multiple of 4
    at[u] = in ? m * K + c : -1;
    v[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (in) v[u] = load4<BF16>(x, at[u]);
    next_group(m, gi, G);
  }
  float mine = 1.0f;  // lane u keeps group t0 + u's scale
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    float mx = fmaxf(fmaxf(fabsf(v[u][0]), fabsf(v[u][1])), fmaxf(fabsf(v[u][2]), fabsf(v[u][3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    float s = mx / 127.0f;
    s = s > 0.0f ? s : 1.0f;
    if (l == u) mine = s;
    if (at[u] >= 0) {
      uint32_t w = 0;
      // scales from 2^-100 to 2^100 have a normal reciprocal
      if (s >= 0x1p-100f && s <= 0x1p100f) {
        const float r = 1.0f / s;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w |= ((uint32_t)(int)clamp_code(code_of(v[u][e], s, r), -127.0f, 127.0f) & 255u) << (8 * e);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w |= ((uint32_t)(int)clamp_code(rintf(v[u][e] / s), -127.0f, 127.0f) & 255u) << (8 * e);
      }
      *reinterpret_cast<uint32_t *>(xq + at[u]) = w;
    }
  }
  if (l < kIlp && t0 + l < groups) xs[t0 + l] = mine;
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_act_restore(const int8_t *__restrict__ xq,
                                                     const float *__restrict__ xs, int64_t groups,
                                                     int64_t K, int64_t G, void *__restrict__ x) {
  const int l = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kIlp;
  int64_t m = t0 / G, gi = t0 - m * G;
  int w[kIlp];
  float s[kIlp];
  int64_t at[kIlp];
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    const int64_t c = gi * kCkptGroup + 4 * l;
    const bool in = t0 + u < groups && c < K;
    at[u] = in ? m * K + c : -1;
    w[u] = in ? *reinterpret_cast<const int *>(xq + at[u]) : 0;
    s[u] = in ? xs[t0 + u] : 0.0f;
    next_group(m, gi, G);
  }
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    if (at[u] < 0) continue;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)(int8_t)(w[u] >> (8 * e)) * s[u];
    if constexpr (BF16) {
      const uint32_t lo = f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16);
      const uint32_t hi = f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16);
      *reinterpret_cast<i32x2 *>(static_cast<uint16_t *>(x) + at[u]) = i32x2{(int)lo, (int)hi};
    } else {
      *reinterpret_cast<f32x4 *>(static_cast<float *>(x) + at[u]) = v;
    }
  }
}

}  // namespace

hipError_t launch_act_checkpoint(const void *x, bool bf16, int64_t M, int64_t K, int8_t *xq,
                                 float *xs, hipStream_t st) {
  const int64_t G = (K + kCkptGroup - 1) / kCkptGroup, groups = M * G;
  const dim3 grid((unsigned)((groups + 8 * kIlp - 1) / (8 * kIlp)));
  if (bf16)
    hipLaunchKernelGGL(k_act_checkpoint<true>, grid, dim3(256), 0, st, x, groups, K, G, xq, xs);
  else
    hipLaunchKernelGGL(k_act_checkpoint<false>, grid, dim3(256), 0, st, x, groups, K, G, xq, xs);
  return hipGetLastError();
}

hipError_t launch_act_restore(const int8_t *xq, const float *xs, int64_t M, int64_t K, void *x,
                              bool bf16, hipStream_t st) {
  const int64_t G = (K + kCkptGroup - 1) / kCkptGroup, groups = M * G;
  const dim3 grid((unsigned)((groups + 8 * kIlp - 1) / (8 * kIlp)));
  if (bf16)
    hipLaunchKernelGGL(k_act_restore<true>, grid, dim3(256), 0, st, xq, xs, groups, K, G, x);
  else
    hipLaunchKernelGGL(k_act_restore<false>, grid, dim3(256), 0, st, xq, xs, groups, K, G, x);
  return hipGetLastError();
}

}  // namespace aql
