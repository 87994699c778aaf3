// Low-rank adapters beside the int8 linear (internal to libaql.so): the batch
// plan, the adapter term that the W8A16 kernels add in their epilogues, and the
// launchers of the adapter kernels. Arguments are validated by the C ABI layer.
#pragma once

#include "common.h"

namespace aql {

// ------------------------------------------------------------------ the plan
//
// Device buffer of int32 that orders a batch's rows by adapter: a header, the
// rows' adapters (-1: none), then tiles of 16 positions. A tile holds rows of
// one adapter, adapters ascending, rows ascending within one; the rows without
// an adapter come last as adapter -1. A segment's last tile is padded with -1.
constexpr int kLoraTile = 16;
constexpr int kLoraMaxAdapters = 1024;
constexpr int kLoraHeader = 16;  // [0] tiles in use
constexpr int kLoraMaxRank = 128;

struct LoraPlanLayout {
  int64_t tiles;     // tiles a batch of M rows over L adapters can need
  int64_t idx;       // [M] adapter of each row
  int64_t perm;      // [16 tiles] row at each sorted position, -1: padding
  int64_t owner;     // [tiles] adapter of a tile, -1: rows without one, -2: unused
  int64_t first;     // [L + 1] first tile of adapter a; [L]: of the rows without one
  int64_t total;     // int32 elements in all
};
constexpr LoraPlanLayout lora_plan_layout(int64_t M, int64_t L) {
  LoraPlanLayout p{};
  p.tiles = M / kLoraTile + (M < L + 1 ? M : L + 1);
  p.idx = kLoraHeader;
  p.perm = p.idx + (M + 15) / 16 * 16;
  p.owner = p.perm + p.tiles * kLoraTile;
  p.first = p.owner + (p.tiles + 15) / 16 * 16;
  p.total = p.first + (L + 1 + 15) / 16 * 16;
  return p;
}

hipError_t launch_lora_plan(const int32_t *idx, int64_t M, int64_t L, int32_t *plan,
                            hipStream_t st);

// --------------------------------------------------- the term in an epilogue

// No adapters: the epilogues compile to what they are without this parameter.
struct NoLora {
  static constexpr bool on = false;
  __device__ __forceinline__ float add(int64_t, int64_t, float v) const { return v; }
};

// v + sum_j h[m, j] W[a][n, j], a = idx[m]: the low-rank product of one output.
// h is float32 and the sum is taken in float32, so the output is rounded to
// bf16 once, with the projection's sum in it. Rows without an adapter read
// neither h nor W.
struct LoraTerm {
  static constexpr bool on = true;
  const float *h;        // [M, R]
  const uint16_t *W;     // [L, N, R] bf16
  const int32_t *idx;    // [M]
  int32_t R;             // a multiple of 8
  int64_t N;
  __device__ __forceinline__ float add(int64_t m, int64_t n, float v) const {
    const int a = idx[m];
    if (a < 0) return v;
    const uint16_t *w = W + ((int64_t)a * N + n) * R;
    const float *hm = h + m * R;
    float s0 = 0.0f, s1 = 0.0f;
    for (int j = 0; j < R; j += 8) {
      const i32x4 wv = *reinterpret_cast<const i32x4 *>(w + j);
      const f32x4 h0 = *reinterpret_cast<const f32x4 *>(hm + j);
      const f32x4 h1 = *reinterpret_cast<const f32x4 *>(hm + j + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t d = (uint32_t)wv[e];
        const float a0 = e < 2 ? h0[2 * e] : h1[2 * e - 4];
        const float a1 = e < 2 ? h0[2 * e + 1] : h1[2 * e - 3];
        s0 = fmaf(__uint_as_float(d << 16), a0, s0);
        s1 = fmaf(__uint_as_float(d & 0xffff0000u), a1, s1);
      }
    }
    return v + (s0 + s1);
  }
};

// Eight floats -> bf16 parts with v = hi + lo up to 2^-16 |v| (both rounded to
// nearest, 2^-8 each): products with bf16 operands then cost two matrix instructions and
// keep the float32 operand's precision well below the output's rounding.
__device__ __forceinline__ void split_bf16(const float (&v)[8], bf16x8 &hi, bf16x8 &lo) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = (__bf16)v[e];
    lo[e] = (__bf16)(v[e] - (float)hi[e]);
  }
}

// The same in three parts (v = hi + mid + lo up to 2^-24 |v|, float32's own
// rounding), for the weight gradients, whose outputs are float32.
__device__ __forceinline__ void split_bf16(const float (&v)[8], bf16x8 &hi, bf16x8 &mid,
                                           bf16x8 &lo) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = (__bf16)v[e];
    const float r = v[e] - (float)hi[e];
    mid[e] = (__bf16)r;
    lo[e] = (__bf16)(r - (float)mid[e]);
  }
}

// The 16 x 32 contraction block of h that lane (r, g) holds for a matrix
// instruction: row r of the block, ranks j0 .. j0 + 7, in two bf16 parts.
__device__ __forceinline__ void lora_h_frag(const float *h, bool in, bf16x8 &hi, bf16x8 &lo) {
  f32x4 h0 = {0.f, 0.f, 0.f, 0.f}, h1 = h0;
  if (in) {
    h0 = *reinterpret_cast<const f32x4 *>(h);
    h1 = *reinterpret_cast<const f32x4 *>(h + 4);
  }
  const float v[8] = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
  split_bf16(v, hi, lo);
}

// Its other operand, for a wave's TJ blocks of columns: ranks j0 .. j0 + 7 of
// adapter a. W [L, N, R]: block j's column is n + 16 j, its ranks lie together.
// KMAJOR, W [L, R, N] (contraction rows): block j's column is n + j, so the four
// blocks' values of a rank are one 8-byte load, and pairs of ranks are packed.
template <bool KMAJOR, int TJ>
__device__ __forceinline__ void lora_w_frags(const LoraTerm &t, int a, int64_t n, int j0,
                                             bf16x8 (&w)[TJ]) {
  const bool jin = j0 < t.R;  // whole chunks of 8: R is a multiple of 8
  if constexpr (KMAJOR) {
    static_assert(TJ == 4, "four columns a lane");
    i32x2 d[8];
    const uint16_t *p = t.W + ((int64_t)a * t.R + j0) * t.N + n;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      d[e] = i32x2{0, 0};
      if (jin && n < t.N) d[e] = *reinterpret_cast<const i32x2 *>(p + (int64_t)e * t.N);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      i32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = (int)__builtin_amdgcn_perm((uint32_t)d[2 * e + 1][j >> 1], (uint32_t)d[2 * e][j >> 1],
                                          j & 1 ? 0x07060302u : 0x05040100u);
      w[j] = __builtin_bit_cast(bf16x8, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int64_t nj = n + 16 * j;
      i32x4 v = {0, 0, 0, 0};
      if (jin && nj < t.N)
        v = *reinterpret_cast<const i32x4 *>(t.W + ((int64_t)a * t.N + nj) * t.R + j0);
      w[j] = __builtin_bit_cast(bf16x8, v);
    }
  }
}

// acc[i][j] += h . W_a^T over a wave's tile of MFMA blocks: 16 TI rows from m0
// by 16 TJ columns from n0, accumulators in the 16x16x32 layout (lane 16 g + r
// holds rows 4 g + v of one column: n0 + 16 j + r, or with KMAJOR n0 + TJ r + j).
// All 64 lanes must be active.
// Where all the tile's rows are of one adapter (a prefill, a training batch)
// its operand is loaded once for the tile. Else each block of 16 rows walks its
// distinct adapters in ascending order; in a block of several the products of
// the other rows are computed and dropped by a select, so no value of one
// adapter (an infinity or a NaN in it among them) reaches a row of another.
template <bool KMAJOR, int TI, int TJ>
__device__ __forceinline__ void lora_add_tile(f32x4 (&acc)[TI][TJ], const LoraTerm &t, int64_t m0,
                                              int64_t M, int64_t n0) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t n = KMAJOR ? n0 + TJ * r : n0 + r;
  int id[TI];
  bool same = true;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int64_t m = m0 + 16 * i + r;
    id[i] = m < M ? t.idx[m] : -1;
  }
  const int a0 = __builtin_amdgcn_readfirstlane(id[0]);
#pragma unroll
  for (int i = 0; i < TI; ++i) same = same && (id[i] == a0 || m0 + 16 * i + r >= M);
  if (__all(same)) {
    if (a0 < 0) return;
    for (int c = 0; c < t.R; c += 32) {
      const int j0 = c + 8 * g;
      bf16x8 w[TJ];
      lora_w_frags<KMAJOR>(t, a0, n, j0, w);
      const float *h = t.h + m0 * t.R;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int row = 16 * i + r;
        bf16x8 hi, lo;
        lora_h_frag(h + row * t.R + j0, j0 < t.R && m0 + row < M, hi, lo);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, w[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, w[j], acc[i][j], 0, 0, 0);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    int prev = -1;
    for (;;) {
      int next = id[i] > prev ? id[i] : 0x7fffffff;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const int other = __shfl_xor(next, o);
        next = other < next ? other : next;
      }
      const int a = __builtin_amdgcn_readfirstlane(next);
      if (a == 0x7fffffff) break;
      prev = a;
      const uint32_t own = (uint32_t)(__ballot(id[i] == a) >> (4 * g));  // bit v: row 4 g + v
      for (int c = 0; c < t.R; c += 32) {
        const int j0 = c + 8 * g;
        bf16x8 hi, lo;
        lora_h_frag(t.h + (m0 + 16 * i + r) * t.R + j0, j0 < t.R && id[i] == a, hi, lo);
        bf16x8 w[TJ];
        lora_w_frags<KMAJOR>(t, a, n, j0, w);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          f32x4 d = {0.f, 0.f, 0.f, 0.f};
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, w[j], d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, w[j], d, 0, 0, 0);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] += own & (1u << v) ? d[v] : 0.0f;
        }
      }
    }
  }
}

// ---------------------------------------------------------------- launchers

// h[m, :] = alpha[a] A_a x[m] (float32 [M, R]); rows without an adapter get
// zeros. x [M, K] bf16, A [L, R, K] bf16.
hipError_t launch_lora_shrink(const uint16_t *x, int64_t M, int64_t K, const uint16_t *A,
                              const float *alpha, int64_t L, int64_t R, const int32_t *plan,
                              float *h, hipStream_t st);

// u[m, :] = alpha[a] B_a^T dy[m] (float32 [M, R]); rows without an adapter get
// zeros. dy [M, N] bf16, B [L, N, R] bf16, N % 8 == 0.
hipError_t launch_lora_shrink_t(const uint16_t *dy, int64_t M, int64_t N, const uint16_t *B,
                                const float *alpha, int64_t L, int64_t R, const int32_t *plan,
                                float *u, hipStream_t st);

// dB[a][n, j] = sum_{m in a} dy[m, n] h[m, j] and
// dA[a][j, k] = sum_{m in a} u[m, j] xq[m, k] xs[m, k / 128], both float32;
// accumulate adds to what the outputs hold. Either output may be NULL.
struct LoraWgradArgs {
  const uint16_t *dy;
  const int8_t *xq;
  const float *xs;
  const float *h, *u;
  const int32_t *plan;
  float *dA, *dB;
  int64_t M, N, K, L, R;
  bool accumulate;
};
hipError_t launch_lora_wgrad(const LoraWgradArgs &a, hipStream_t st);

}  // namespace aql
