// Activation checkpoints in 8 bits: per row and group of 128 columns
//   s = max |x| / 127 (1 where that is 0), code = clamp(rint(x / s), -127, 127)
// and back, x' = code * s. One pass over the data each way, bound by memory:
// 3 bytes a value (bf16) plus 4 bytes a group (8192 x 14336 bf16: 68 us, 5.2 TB/s to
// codes, 64 us, 5.6 TB/s back, each in a run of its own; in turn 81 and 56, the save
// behind the restore's writes and the restore on codes still in cache. 4096 x 14336
// float32 in turn: 69 and 46. A copy of such a size runs at 5.0).
//
// 16 lanes hold a group, 8 values a lane (16 bytes of bf16), so a group's maximum
// takes four DPP moves and no LDS, and a lane packs its codes into one 8-byte
// store. Groups are numbered over the whole matrix; 16 lanes take kIlp of them at
// once to keep enough loads in flight. Where K is an odd multiple of 4, a row's last
// lane moves 4 values, and odd rows begin at half of such an access's size, which
// global memory takes as it is; the types below say so.
#include "ckpt.h"

namespace aql {
namespace {

typedef int i32x4_8 __attribute__((ext_vector_type(4), aligned(8)));  // 8 bf16 of such a row
typedef int i32x2_4 __attribute__((ext_vector_type(2), aligned(4)));  // 8 codes of one

constexpr int kIlp = 4;  // groups in flight for 16 lanes

// Groups of one launch, 4 threads each. A grid holds fewer than 2^32 threads, and of
// a larger one only what is left over past 2^32 runs, without an error (2^30 + 5
// rows of 4 values: all but the first 64 groups were left as they were).
constexpr int64_t kSlice = 1 << 28;
static_assert(kSlice % (16 * kIlp) == 0 && kSlice / (16 * kIlp) * 256 < (1LL << 32), "one grid");

constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The maximum over a row of 16 lanes, in every lane. Magnitudes are compared as
// their bits, which order like the values and put a NaN above an infinity, so a
// group with either gets a scale that is none and does not restore as if it held
// numbers.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = umax(v, dpp<kDppXor1>(v));
  v = umax(v, dpp<kDppXor2>(v));
  v = umax(v, dpp<kDppHalfMirror>(v));
  return umax(v, dpp<kDppMirror>(v));
}

// n (8, 4 or 0) values from element i on; the others zero.
template <bool BF16>
__device__ __forceinline__ void load8(const void *x, int64_t i, int n, float (&v)[8]) {
  if constexpr (BF16) {
    const uint16_t *p = static_cast<const uint16_t *>(x) + i;
    i32x4 d = {0, 0, 0, 0};
    if (n == 8) {
      d = *reinterpret_cast<const i32x4_8 *>(p);
    } else if (n) {
      const i32x2 h = *reinterpret_cast<const i32x2 *>(p);
      d[0] = h[0];
      d[1] = h[1];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float((uint32_t)d[e] << 16);
      v[2 * e + 1] = __uint_as_float((uint32_t)d[e] & 0xffff0000u);
    }
  } else {
    const float *p = static_cast<const float *>(x) + i;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    if (n) a = *reinterpret_cast<const f32x4 *>(p);
    if (n == 8) b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
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

__device__ __forceinline__ void next_group(int64_t &m, int64_t &gi, int64_t G) {
  if (++gi == G) {
    gi = 0;
    ++m;
  }
}

// A lane's place in group (m, gi): its first element and how many of its eight
// lie in the row (K is a multiple of 4).
__device__ __forceinline__ int place(bool live, int64_t m, int64_t gi, int l, int64_t K,
                                     int64_t &at) {
  const int64_t c = gi * kCkptGroup + 8 * l;
  at = m * K + c;
  return !live || c >= K ? 0 : (c + 8 <= K ? 8 : 4);
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_act_checkpoint(const void *__restrict__ x, int64_t first,
                                                        int64_t groups, int64_t K, int64_t G,
                                                        int8_t *__restrict__ xq,
                                                        float *__restrict__ xs) {
  const int l = threadIdx.x & 15;
  const int64_t t0 = first + ((int64_t)blockIdx.x * 16 + (threadIdx.x >> 4)) * kIlp;
  int64_t m = t0 / G, gi = t0 - m * G;
  float v[kIlp][8];
  int64_t at[kIlp];
  int n[kIlp];
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    n[u] = place(t0 + u < groups, m, gi, l, K, at[u]);
    load8<BF16>(x, at[u], n[u], v[u]);
    next_group(m, gi, G);
  }
  float mine = 1.0f;  // lane u keeps group t0 + u's scale
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    uint32_t mx = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = umax(mx, __float_as_uint(v[u][e]) & 0x7fffffffu);
    float s = __uint_as_float(max16(mx)) / 127.0f;
    s = s == 0.0f ? 1.0f : s;
    if (l == u) mine = s;
    uint32_t w[2] = {0, 0};
    // scales from 2^-100 to 2^100 have a normal reciprocal
    if (s >= 0x1p-100f && s <= 0x1p100f) {
      const float r = 1.0f / s;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e >> 2] |= ((uint32_t)(int)clamp_code(code_of(v[u][e], s, r), -127.0f, 127.0f) & 255u)
                     << (8 * (e & 3));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e >> 2] |= ((uint32_t)(int)clamp_code(rintf(v[u][e] / s), -127.0f, 127.0f) & 255u)
                     << (8 * (e & 3));
    }
    if (n[u] == 8)
      *reinterpret_cast<i32x2_4 *>(xq + at[u]) = i32x2{(int)w[0], (int)w[1]};
    else if (n[u])
      *reinterpret_cast<uint32_t *>(xq + at[u]) = w[0];
  }
  if (l < kIlp && t0 + l < groups) xs[t0 + l] = mine;
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_act_restore(const int8_t *__restrict__ xq,
                                                     const float *__restrict__ xs, int64_t first,
                                                     int64_t groups, int64_t K, int64_t G,
                                                     void *__restrict__ x) {
  const int l = threadIdx.x & 15;
  const int64_t t0 = first + ((int64_t)blockIdx.x * 16 + (threadIdx.x >> 4)) * kIlp;
  int64_t m = t0 / G, gi = t0 - m * G;
  int w[kIlp][2];
  float s[kIlp];
  int64_t at[kIlp];
  int n[kIlp];
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    n[u] = place(t0 + u < groups, m, gi, l, K, at[u]);
    w[u][0] = w[u][1] = 0;
    if (n[u] == 8) {
      const i32x2 d = *reinterpret_cast<const i32x2_4 *>(xq + at[u]);
      w[u][0] = d[0];
      w[u][1] = d[1];
    } else if (n[u]) {
      w[u][0] = *reinterpret_cast<const int *>(xq + at[u]);
    }
    s[u] = n[u] ? xs[t0 + u] : 0.0f;
    next_group(m, gi, G);
  }
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    if (n[u] == 0) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)(w[u][e >> 2] >> (8 * (e & 3))) * s[u];
    if constexpr (BF16) {
      i32x4 d;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        d[e] = (int)((uint32_t)f32_to_bf16_rne(v[2 * e]) |
                     ((uint32_t)f32_to_bf16_rne(v[2 * e + 1]) << 16));
      uint16_t *p = static_cast<uint16_t *>(x) + at[u];
      if (n[u] == 8) *reinterpret_cast<i32x4_8 *>(p) = d;
      else *reinterpret_cast<i32x2 *>(p) = i32x2{d[0], d[1]};
    } else {
      float *p = static_cast<float *>(x) + at[u];
      *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
      if (n[u] == 8) *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
}

// launch(first, grid) for slices of kSlice groups.
template <class F>
hipError_t slices(int64_t groups, F &&launch) {
  for (int64_t first = 0; first < groups; first += kSlice) {
    const int64_t n = groups - first < kSlice ? groups - first : kSlice;
    launch(first, dim3((unsigned)((n + 16 * kIlp - 1) / (16 * kIlp))));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_act_checkpoint(const void *x, bool bf16, int64_t M, int64_t K, int8_t *xq,
                                 float *xs, hipStream_t st) {
  const int64_t G = (K + kCkptGroup - 1) / kCkptGroup, groups = M * G;
  const auto kern = bf16 ? k_act_checkpoint<true> : k_act_checkpoint<false>;
  return slices(groups, [&](int64_t first, dim3 grid) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, x, first, groups, K, G, xq, xs);
  });
}

hipError_t launch_act_restore(const int8_t *xq, const float *xs, int64_t M, int64_t K, void *x,
                              bool bf16, hipStream_t st) {
  const int64_t G = (K + kCkptGroup - 1) / kCkptGroup, groups = M * G;
  const auto kern = bf16 ? k_act_restore<true> : k_act_restore<false>;
  return slices(groups, [&](int64_t first, dim3 grid) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, xq, xs, first, groups, K, G, x);
  });
}

}  // namespace aql
