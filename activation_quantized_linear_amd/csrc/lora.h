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
// Last, for each group of 128 rows as the batch has them: whether more than
// kLoraFew adapters share it.
constexpr int kLoraTile = 16;
constexpr int kLoraMaxAdapters = 1024;
constexpr int kLoraHeader = 16;  // [0] tiles in use
constexpr int kLoraMaxRank = 128;
constexpr int kLoraGroup = 128;  // rows of the largest tile of the tiled kernels
// Adapters of a group that they take in their epilogues; with more the products are
// computed ahead. Both sides, walked and ahead, us a call in a graph, R = 16: M = 128,
// N = 14336, K = 4096, 3 adapters 45.2, 47.4, 4 47.8, 47.3, 5 50.4, 47.5, 8 59.0, 47.5;
// M = 2048, N = K = 4096, 3 84.8, 89.6, 4 88.5, 90.4, 6 96.1, 90.2, 8 102.6, 91.2; backward
// there, 2 93.3, 101.9, 4 100.6, 101.4, 6 111.9, 105.1.
constexpr int kLoraFew = 4;

struct LoraPlanLayout {
  int64_t tiles;     // tiles a batch of M rows over L adapters can need
  int64_t idx;       // [M] adapter of each row
  int64_t perm;      // [16 tiles] row at each sorted position, -1: padding
  int64_t owner;     // [tiles] adapter of a tile, -1: rows without one, -2: unused
  int64_t first;     // [L + 1] first tile of adapter a; [L]: of the rows without one
  int64_t mixed;     // [M / 128] 1: more than kLoraFew adapters in the group
  int64_t total;     // int32 elements in all
};
constexpr LoraPlanLayout lora_plan_layout(int64_t M, int64_t L) {
  LoraPlanLayout p{};
  p.tiles = M / kLoraTile + (M < L + 1 ? M : L + 1);
  p.idx = kLoraHeader;
  p.perm = p.idx + (M + 15) / 16 * 16;
  p.owner = p.perm + p.tiles * kLoraTile;
  p.first = p.owner + (p.tiles + 15) / 16 * 16;
  p.mixed = p.first + (L + 1 + 15) / 16 * 16;
  p.total = p.mixed + ((M + kLoraGroup - 1) / kLoraGroup + 15) / 16 * 16;
  return p;
}

hipError_t launch_lora_plan(const int32_t *idx, int64_t M, int64_t L, int32_t *plan,
                            hipStream_t st);

// --------------------------------------------------- the term in an epilogue

// No adapters: the epilogues compile to what they are without this parameter.
struct NoLora {
  static constexpr bool on = false, act = false;
  __device__ __forceinline__ float add(int64_t, int64_t, float v) const { return v; }
};

// v + sum_j h[m, j] W[a][n, j], a = idx[m]: the low-rank product of one output.
// h is float32 and the sum is taken in float32, so the output is rounded to
// bf16 once, with the projection's sum in it. Rows without an adapter read
// neither h nor W.
struct LoraTerm {
  static constexpr bool on = true, act = false;
  const float *h;        // [M, R]
  const uint16_t *W;     // [L, N, R] bf16
  const int32_t *idx;    // [M]
  int32_t R;             // a multiple of 8
  int64_t N;
  // not NULL: h is not there yet, the launch that leaves the projection's partial
  // sums computes it beside them (lora_shrink_rows; A [L, R, K], alpha [L])
  const uint16_t *A = nullptr;
  const float *alpha = nullptr;
  // not NULL: the products themselves [M, N], of the rows in the plan's mixed
  // groups, or of all rows where mixed is NULL (launch_lora_products)
  const float *T = nullptr;
  const int32_t *mixed = nullptr;
  __device__ __forceinline__ bool ready(int64_t m0) const {  // the group of m0's products
    return T && (!mixed || mixed[m0 / kLoraGroup]);
  }
  __device__ __forceinline__ float add(int64_t m, int64_t n, float v) const {
    const int a = idx[m];
    if (a < 0) return v;
    if (T) return v + T[m * N + n];  // (where outputs come one at a time: all rows)
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

__device__ __forceinline__ float bf16_lo(int d) { return __uint_as_float((uint32_t)d << 16); }
__device__ __forceinline__ float bf16_hi(int d) {
  return __uint_as_float((uint32_t)d & 0xffff0000u);
}

// h of few rows, by a workgroup of 4 waves: J ranks from j0 on of row m. J rows of
// the adapter's A are read once, the waves taking 512-element steps of K in turn.
// Bound by latency (M = 1, K = 4096, R = 16: 2.7 us, a launch's own time) and, with many
// adapters, by reading them (2 R K bytes each).
// red: 4 J floats of LDS.
template <int J>
__device__ __forceinline__ void lora_shrink_rows(const uint16_t *x, int64_t K, const uint16_t *A,
                                                 const float *alpha, int R, const int32_t *idx,
                                                 float *h, int64_t m, int j0, float *red) {
  const int a = idx[m];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (a < 0) {  // uniform over the workgroup
    if (threadIdx.x < J) h[m * R + j0 + threadIdx.x] = 0.0f;
    return;
  }
  const uint16_t *xr = x + m * K, *ar = A + ((int64_t)a * R + j0) * K;
  float acc[J][2];
#pragma unroll
  for (int j = 0; j < J; ++j) acc[j][0] = acc[j][1] = 0.0f;
  constexpr int U = J == 1 ? 4 : 2;
  for (int64_t k0 = 8 * (int64_t)threadIdx.x; k0 < K; k0 += 2048 * U) {
    i32x4 xv[U], av[U][J];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = k0 + 2048 * u;
      xv[u] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < J; ++j) av[u][j] = i32x4{0, 0, 0, 0};
      if (k < K) {
        xv[u] = *reinterpret_cast<const i32x4 *>(xr + k);
#pragma unroll
        for (int j = 0; j < J; ++j) av[u][j] = *reinterpret_cast<const i32x4 *>(ar + j * K + k);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = bf16_lo(xv[u][e]), x1 = bf16_hi(xv[u][e]);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          acc[j][0] = fmaf(x0, bf16_lo(av[u][j][e]), acc[j][0]);
          acc[j][1] = fmaf(x1, bf16_hi(av[u][j][e]), acc[j][1]);
        }
      }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float s = acc[j][0] + acc[j][1];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) red[wave * J + j] = s;
  }
  __syncthreads();
  if (threadIdx.x < J) {
    const int j = threadIdx.x;
    h[m * R + j0 + j] = alpha[a] * ((red[j] + red[J + j]) + (red[2 * J + j] + red[3 * J + j]));
  }
}

// Eight floats -> bf16 parts with v = hi + lo up to 2^-16 |v| (both rounded to
// nearest, 2^-8 each): products with bf16 operands then cost two matrix instructions and
// keep the float32 operand's precision well below the output's rounding. (A finite
// value past bfloat16's largest, 3.396e38 and more, rounds to an infinity and counts
// as one.)
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

// The adapter terms of a workgroup's output tile, after its own sums: acc[i][j]
// += h . W_a^T for the blocks of 16 x 16 that a wave holds (16x16x32 layout, lane
// 16 g + r holding rows 4 g + v of one column). The tile's distinct adapters are
// walked in ascending order (one, in a prefill or a training batch), 32 NS ranks at
// a step: the rows' h goes to LDS split into two bf16 parts, once for all waves,
// with the adapter's ranks of the tile's columns beside it, and every block takes
// two matrix instructions for 32 ranks. Products are added through a select by
// row, so no value of one adapter (an infinity or a NaN in it among them) reaches
// a row of another. A step costs 4 to 5 us (input gradient's kernel at M = 500, N = 4096,
// K = 14336: 55.9 us without adapters, 60.2 with one of 64 ranks, 65.0 with two in a
// tile): its
// loads, their split and the products follow each other, and neither loading a
// step ahead nor interleaving the blocks by hand shortened the whole, the first
// for want of registers beside the accumulators.
// KMAJOR: W is [L, R, N] (contraction rows) and block j's column is col0 + TJ r
// + j; else W is [L, N, R] and the column is col0 + 16 j + r.

// The tile's adapters in LDS, found before the main loop, under its first loads.
template <int BM>
struct LoraRows {
  int ids[BM];   // of the rows, -1: none
  int list[BM];  // the distinct ones, ascending
  int count;
};

template <int BM, int NT>
__device__ __forceinline__ void lora_rows(LoraRows<BM> &s, const LoraTerm &t, int64_t m0,
                                          int64_t M) {
  const int tid = threadIdx.x;
  for (int i = tid; i < BM; i += NT) s.ids[i] = m0 + i < M ? t.idx[m0 + i] : -1;
  __syncthreads();
  if (t.ready(m0)) {
    if (tid == 0) s.count = 0;
  } else if (tid < 64) {
    int n = 0;
    for (int prev = -1;; ++n) {
      int next = 0x7fffffff;
      for (int i = tid; i < BM; i += 64) {
        const int v = s.ids[i];
        next = v > prev && v < next ? v : next;
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int other = __shfl_xor(next, o);
        next = other < next ? other : next;
      }
      prev = __builtin_amdgcn_readfirstlane(next);
      if (prev == 0x7fffffff) break;
      if (tid == 0) s.list[n] = prev;
    }
    if (tid == 0) s.count = n;
  }
}

template <int BM, int BN, bool KMAJOR, int NS>
struct LoraLds {
  static constexpr int H = BM * 128;                        // rows of 32 high, 32 low parts
  static constexpr int W = KMAJOR ? 32 * BN * 2 : BN * 64;  // 32 ranks of BN columns
  static constexpr int BYTES = NS * (H + W);
};

// smem: LoraLds<BM, BN, KMAJOR, NS>::BYTES bytes that nothing uses once every
// wave of the workgroup's NT threads has entered; lora_rows has filled s. The wave's
// blocks begin at row row0 and column col0 of the tile. The accumulators are touched
// in one counted loop without branches around them: in loops that leave early or
// skip blocks the compiler keeps a second copy of them, in scratch memory.
template <int BM, int BN, int NT, bool KMAJOR, int NS, int TI, int TJ>
__device__ __forceinline__ void lora_add_tile(char *smem, const LoraRows<BM> &s,
                                              f32x4 (&acc)[TI][TJ], const LoraTerm &t, int64_t m0,
                                              int64_t n0, int row0, int col0) {
  using S = LoraLds<BM, BN, KMAJOR, NS>;
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  auto hswz = [](int row) { return (row >> 1) & 7; };
  auto wswz = [](int row) { return (row >> 2) & 3; };
  __syncthreads();
  const int nc = (t.R + 32 * NS - 1) / (32 * NS);
  const int steps = __builtin_amdgcn_readfirstlane(s.count) * nc;
  for (int q = 0; q < steps; ++q) {
    const int a = __builtin_amdgcn_readfirstlane(s.list[q / nc]);
    const int c0 = q % nc * (32 * NS);
    // both operands' loads are out before the first is used
    constexpr int TH = BM * 4, NH = (TH + NT - 1) / NT, NW = S::W / 16 / NT;
    static_assert((NH == 1 || NH * NT == TH) && NW * NT == S::W / 16, "staged evenly");
    f32x4 hv[NS][NH][2];
    i32x4 wv[NS][NW];
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      const int c = c0 + 32 * b;
#pragma unroll
      for (int i = 0; i < NH; ++i) {  // a row's ranks c + 8 k .. + 7
        const int u = tid + NT * i, row = u >> 2, k = u & 3;
        hv[b][i][0] = hv[b][i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (u < TH && s.ids[row] == a && c + 8 * k < t.R) {  // whole chunks of 8 ranks
          const float *h = t.h + (m0 + row) * t.R + c + 8 * k;
          hv[b][i][0] = *reinterpret_cast<const f32x4 *>(h);
          hv[b][i][1] = *reinterpret_cast<const f32x4 *>(h + 4);
        }
      }
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const int u = tid + NT * i;
        wv[b][i] = i32x4{0, 0, 0, 0};
        if constexpr (KMAJOR) {
          const int j = u / (BN / 8), k = u % (BN / 8);  // rank c + j, columns 8 k .. + 7
          if (c + j < t.R && n0 + 8 * k < t.N)  // whole chunks: N is a multiple of 8
            wv[b][i] = *reinterpret_cast<const i32x4 *>(
                t.W + ((int64_t)a * t.R + c + j) * t.N + n0 + 8 * k);
        } else {
          const int row = u >> 2, k = u & 3;  // column n0 + row, ranks c + 8 k .. + 7
          if (c + 8 * k < t.R && n0 + row < t.N)
            wv[b][i] = *reinterpret_cast<const i32x4 *>(
                t.W + ((int64_t)a * t.N + n0 + row) * t.R + c + 8 * k);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      char *hs = smem + b * (S::H + S::W);
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const int u = tid + NT * i, row = u >> 2, k = u & 3;
        const f32x4 v0 = hv[b][i][0], v1 = hv[b][i][1];
        const float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
        bf16x8 hi, lo;
        split_bf16(v, hi, lo);
        if (u < TH) {
          *reinterpret_cast<bf16x8 *>(hs + row * 128 + 16 * (k ^ hswz(row))) = hi;
          *reinterpret_cast<bf16x8 *>(hs + row * 128 + 16 * ((4 + k) ^ hswz(row))) = lo;
        }
      }
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const int u = tid + NT * i, row = u >> 2, k = u & 3;
        *reinterpret_cast<i32x4 *>(hs + S::H + (KMAJOR ? 16 * u : row * 64 + 16 * (k ^ wswz(row)))) =
            wv[b][i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      const char *hs = smem + b * (S::H + S::W);
      bf16x8 w[TJ];
      if constexpr (KMAJOR) {
        static_assert(!KMAJOR || TJ == 4, "four columns a lane");
        i32x2 d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          d[e] = *reinterpret_cast<const i32x2 *>(hs + S::H + (8 * g + e) * BN * 2 +
                                                  2 * (col0 + 4 * r));
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          i32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = (int)__builtin_amdgcn_perm((uint32_t)d[2 * e + 1][j >> 1],
                                              (uint32_t)d[2 * e][j >> 1],
                                              j & 1 ? 0x07060302u : 0x05040100u);
          w[j] = __builtin_bit_cast(bf16x8, v);
        }
      } else {
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          const int row = col0 + 16 * j + r;
          w[j] = *reinterpret_cast<const bf16x8 *>(hs + S::H + row * 64 + 16 * (g ^ wswz(row)));
        }
      }
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const i32x4 id = *reinterpret_cast<const i32x4 *>(s.ids + row0 + 16 * i + 4 * g);
        const int row = row0 + 16 * i + r;
        const bf16x8 hi = *reinterpret_cast<const bf16x8 *>(hs + row * 128 + 16 * (g ^ hswz(row)));
        const bf16x8 lo =
            *reinterpret_cast<const bf16x8 *>(hs + row * 128 + 16 * ((4 + g) ^ hswz(row)));
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          f32x4 d = {0.f, 0.f, 0.f, 0.f};
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, w[j], d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, w[j], d, 0, 0, 0);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] += id[v] == a ? d[v] : 0.0f;
        }
        __builtin_amdgcn_sched_barrier(0);  // one block's operands at a time
      }
    }
    __syncthreads();
  }
  if (t.ready(m0)) {  // no steps: the products lie in memory
    const int c0 = col0 + (KMAJOR ? 4 * r : r);
    const float *p = t.T + (m0 + row0 + 4 * g) * t.N + n0 + c0;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const i32x4 id = *reinterpret_cast<const i32x4 *>(s.ids + row0 + 16 * i + 4 * g);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if constexpr (KMAJOR) {
          f32x4 d = {0.f, 0.f, 0.f, 0.f};
          if (id[v] >= 0 && n0 + c0 < t.N) d = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
          for (int j = 0; j < TJ; ++j) acc[i][j][v] += d[j];
        } else {
#pragma unroll
          for (int j = 0; j < TJ; ++j)
            acc[i][j][v] += id[v] >= 0 && n0 + c0 + 16 * j < t.N ? p[16 * j] : 0.0f;
        }
        p += v < 3 ? t.N : 13 * t.N;
        asm volatile("" : "+v"(p));  // one row's address at a time
      }
    }
  }
}

// ---------------------------------------------------------------- launchers

// Rows from which the shrink of x takes the tiled form, and the most bytes that
// either shrink's partial sums take in the tiled form for up to M rows (C: the length
// of the contraction).
constexpr int64_t kLoraTiledMinM = 64;
size_t lora_shrink_most_bytes(int64_t M, int64_t C, int64_t L, int64_t R);

// h[m, :] = alpha[a] A_a x[m] (float32 [M, R]); rows without an adapter get
// zeros. x [M, K] bf16, A [L, R, K] bf16. part: lora_shrink_most_bytes(M, K, L, R)
// bytes from kLoraTiledMinM rows on.
hipError_t launch_lora_shrink(const uint16_t *x, int64_t M, int64_t K, const uint16_t *A,
                              const float *alpha, int64_t L, int64_t R, const int32_t *plan,
                              float *h, float *part, hipStream_t st);

// u[m, :] = alpha[a] B_a^T dy[m] (float32 [M, R]); rows without an adapter get
// zeros. dy [M, N] bf16, B [L, N, R] bf16, N % 8 == 0. part:
// lora_shrink_most_bytes(M, N, L, R) bytes. sc (may be NULL): dy's scaling for the
// input's gradient, done by further workgroups of the same launch.
struct DgradScale;
hipError_t launch_lora_shrink_t(const uint16_t *dy, int64_t M, int64_t N, const uint16_t *B,
                                const float *alpha, int64_t L, int64_t R, const int32_t *plan,
                                float *u, float *part, const DgradScale *sc, hipStream_t st);

// Whether a split kernel's sum of M x C outputs is better given their products
// than left to compute each, R multiply-adds with R ranks read for it. Whole calls in
// a graph, products given and left, C = 4096, K = 14336: M = 500, R = 64 101.7 us, 143.6;
// M = 128, R = 32 (2^24) 53.2, 56.1; M = 256, R = 16 (2^24) 61.5, 62.5; M = 128, R = 16
// 52.7, 51.9; M = 256, R = 8 61.1, 56.9. With the contraction as W's slow axis (kmajor)
// neighbouring outputs share lines, so later (backward, C = K = 4096: M = 500, R = 128
// 72.0, 98.2; R = 32 (2^26) 48.6, 49.7; M = 256, R = 64 (2^26) 43.3, 44.9; M = 256, R = 32
// 37.2, 35.9; M = 500, R = 16 46.7, 44.1; M = 128, R = 64 (2^25) 37.4, 38.8).
constexpr bool lora_split_products(bool kmajor, int64_t M, int64_t C, int64_t R) {
  return M * C * R >= (kmajor ? 1 << 26 : 1 << 24);
}

// T[m, n] = sum_j h[m, j] W[a][n, j] (float32 [M, N]) for the rows with an adapter,
// where mixed is given only those in its groups; other rows stay as they are.
// kmajor: W is [L, R, N]. 1 <= N <= 2^26.
hipError_t launch_lora_products(const float *h, const uint16_t *W, bool kmajor, int64_t M,
                                int64_t N, int64_t L, int64_t R, const int32_t *plan,
                                const int32_t *mixed, float *T, hipStream_t st);

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
// The same with the last sum of a split input gradient beside it, in workgroups of 4
// waves: for segments of few rows and not too many workgroups (lora_wgrad_beside).
struct DgradParts;
bool lora_wgrad_beside(const LoraWgradArgs &a);
hipError_t launch_lora_wgrad_reduce(const LoraWgradArgs &a, const DgradParts &parts,
                                    const LoraTerm &lt, hipStream_t st);

}  // namespace aql
