// Gradient of the W8A16 linear to its input (internal to libaql.so).
#pragma once

#include "common.h"
#include "lora.h"

namespace aql {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kDgradStage = 64;  // channels of a stage: d's rows are padded to whole ones
constexpr int kDgradTop = 14;    // exponent of a row's largest scaled product

// The scaling of dy, the product's first operand: d[m, n] = dy[m, n] scale[n]
// 2^ex[m] in float16, [M, NP], NP = N rounded up to whole stages, zeros past N.
struct DgradScale {
  const uint16_t *dy;
  const float *scale;
  int64_t M, N, NP;
  uint16_t *d;
  int32_t *ex;
};

// Row m by 256 threads (t of them; rows past M take part and write nothing), 8
// values a thread and round. NI rounds are held in registers between the maximum
// and the scaling, so dy is read once (NI = 0: any N, read twice). Bound by
// memory: 4 bytes a value (M = 2048, N = 14336: 23 us, 5.1 TB/s).
// red: a float for each wave of the workgroup.
template <int NI>
__device__ __forceinline__ void dgrad_scale_row(const DgradScale &a, int64_t m, int t,
                                                float *red) {
  const bool live = m < a.M;
  const int64_t N = live ? a.N : 0, NP = live ? a.NP : 0;
  const uint16_t *row = a.dy + m * a.N;
  auto load = [&](int64_t n, float (&v)[8]) {
    const i32x4 w = *reinterpret_cast<const i32x4 *>(row + n);
    const f32x4 s0 = *reinterpret_cast<const f32x4 *>(a.scale + n);
    const f32x4 s1 = *reinterpret_cast<const f32x4 *>(a.scale + n + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = (uint32_t)w[i];
      v[2 * i] = __uint_as_float(u << 16) * (i < 2 ? s0[2 * i] : s1[2 * i - 4]);
      v[2 * i + 1] = __uint_as_float(u & 0xffff0000u) * (i < 2 ? s0[2 * i + 1] : s1[2 * i - 3]);
    }
  };
  float mx = 0.0f;
  constexpr int NR = NI > 0 ? NI : 1;
  float v[NR][8];
  if constexpr (NI > 0) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t n = 8 * (int64_t)(t + 256 * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      if (n < N) load(n, v[i]);  // whole chunks: N is a multiple of 8
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[i][e]));
  } else {
    for (int64_t n = 8 * (int64_t)t; n < N; n += 8 * 256) {
      load(n, v[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[0][e]));
    }
  }
  mx = group_reduce_max<256>(mx, red);
  const int e2 = kDgradTop - __builtin_amdgcn_frexp_expf(mx);
  if (t == 0 && live) a.ex[m] = e2;
  auto store = [&](int64_t n, const float (&x)[8]) {
    f16x8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (_Float16)ldexpf(x[e], e2);
    *reinterpret_cast<f16x8 *>(a.d + m * NP + n) = o;
  };
  if constexpr (NI > 0) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t n = 8 * (int64_t)(t + 256 * i);
      if (n < NP) store(n, v[i]);
    }
  } else {
    for (int64_t n = 8 * (int64_t)t; n < NP; n += 8 * 256) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[0][e] = 0.0f;
      if (n < N) load(n, v[0]);
      store(n, v[0]);
    }
  }
}

// What a split product leaves: dx = bf16(part[0] + ... + part[S - 1] + u A).
struct DgradParts {
  const float *part;  // [S, M, K]
  int S;
  int64_t M, K;
  uint16_t *dx;
  int64_t blocks() const { return (M * (K / 4) + 255) / 256; }
};

// Its sums in split order by M K / 4 threads, of which i takes 4 consecutive
// columns, so the rows of A are read as whole lines.
template <class LT>
__device__ __forceinline__ void dgrad_reduce(const DgradParts &p, const LT &lt, int64_t i) {
  const int64_t M = p.M, K = p.K, ng = K / 4;
  if (i >= M * ng) return;
  const int64_t m = i / ng, k = (i - m * ng) * 4;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.S; ++s)
    acc += *reinterpret_cast<const f32x4 *>(p.part + ((int64_t)s * M + m) * K + k);
  if constexpr (LT::on) {
    const int a = lt.idx[m];
    if (a >= 0 && lt.T) {
      acc += *reinterpret_cast<const f32x4 *>(lt.T + m * K + k);
    } else if (a >= 0) {
      const uint16_t *w = lt.W + (int64_t)a * lt.R * K + k;
      const float *u = lt.h + m * lt.R;
      f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int j = 0; j < lt.R; ++j) {
        const i32x2 d = *reinterpret_cast<const i32x2 *>(w + (int64_t)j * K);
        t[0] = fmaf(u[j], __uint_as_float((uint32_t)d[0] << 16), t[0]);
        t[1] = fmaf(u[j], __uint_as_float((uint32_t)d[0] & 0xffff0000u), t[1]);
        t[2] = fmaf(u[j], __uint_as_float((uint32_t)d[1] << 16), t[2]);
        t[3] = fmaf(u[j], __uint_as_float((uint32_t)d[1] & 0xffff0000u), t[3]);
      }
      acc += t;
    }
  }
  const uint32_t lo = f32_to_bf16_rne(acc[0]) | ((uint32_t)f32_to_bf16_rne(acc[1]) << 16);
  const uint32_t hi = f32_to_bf16_rne(acc[2]) | ((uint32_t)f32_to_bf16_rne(acc[3]) << 16);
  *reinterpret_cast<i32x2 *>(p.dx + m * K + k) = i32x2{(int)lo, (int)hi};
}

// Bytes of the workspace: dy times the scales in float16 [M, N rounded up to 64],
// an exponent a row, and the partial sums of shapes that split the contraction.
size_t w8a16_dgrad_bytes(int64_t M, int64_t N, int64_t K);
// Whether such a shape splits it.
bool w8a16_dgrad_split(int64_t M, int64_t N, int64_t K);

// The scaling's arguments for a call with this workspace.
DgradScale w8a16_dgrad_scale_args(const uint16_t *dy, const float *scale, int64_t M, int64_t N,
                                  int64_t K, void *ws);

// dx[m, k] = bf16(sum_n dy[m, n] scale[n] q[n, k]); N % 8 == 0, K % 16 == 0,
// K <= 2^24, N <= 2^22. ws: as above.
hipError_t launch_w8a16_dgrad(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q,
                              const float *scale, int64_t K, uint16_t *dx, void *ws,
                              hipStream_t st);
// The same plus sum_j u[m, j] A[a][j, k] (lt: h = u [M, R], W = A [L, R, K], N = K),
// the scaling done by an earlier launch. later (may be NULL): a shape that splits
// the contraction leaves its last sum to the caller.
hipError_t launch_w8a16_dgrad_scaled(const DgradScale &a, const int8_t *q, int64_t K, uint16_t *dx,
                                     void *ws, hipStream_t st, const LoraTerm &lt,
                                     DgradParts *later);

}  // namespace aql
