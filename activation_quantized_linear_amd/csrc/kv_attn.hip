// Attention over the paged 8-bit KV cache. For a query at position p of a sequence, over
// the tokens t that it sees (max(0, p - window + 1) .. p):
//   y = sum_t e^(a (q . k_t)) v_t / sum_t e^(a (q . k_t)),  k_t = ks code_k, v_t = vs code_v,
// with one ks and vs for each page of 64 tokens and kv head.
//
// The scales never touch the codes. Scores are computed in powers of two and with log2 vs in them,
//   z_t = a log2(e) ks (q . code_k) + log2 vs,   w_t = 2^(z_t - M),
// M a little below the running maximum of z (kTop), so that outputs are sums of w_t code_v and w_t is
// at most 2^15 where it weighs most, whatever the pages' scales; the denominator adds a
// page's w_t times 1 / vs, in which weights down to 2^-20 of the largest count while the scales of V
// that a row sees lie within 2^110 of each other (below 2^-126 w_t is 0). Codes widen to float16
// exactly, and so does q under an exponent of its row that brings the largest value to
// 2^15 .. 2^16 (values down to 2^-32 of the largest keep all of their bits, smaller ones are
// rounded by 2^-40 of it). w is rounded to float16: by 2^-11 of its value, or where it is
// subnormal there by 2^-25, which is 2^-40 of the largest weight in streams and 2^-32 in tiles,
// so that what 2^20 small weights lose together stays far below a bf16 output's 2^-8. Sums,
// M and the denominator are float32.
//
// Scores are computed transposed (tokens as rows), so that a lane ends with 16
// consecutive tokens of one query, which is the operand layout of the second product:
// nothing passes through LDS or other lanes between the two. Of the 16 x 16 x 32
// instructions' lanes 16 g + r, tile tau of a page's 4 takes tokens 16 (r / 4) + 4 tau + r % 4
// as rows, so lane (r, g) holds tokens 16 g + 4 tau + v of query r. The contractions
// over dims and over tokens take 16 consecutive bytes of the cache a lane, in the cache's order.
#include <atomic>
#include <type_traits>

#include "kv.h"

namespace aql {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Two codes, already offset by 128, as the low mantissa bits of float16 1024, less 1152.
__device__ __forceinline__ uint32_t f16x2_from_u8(uint32_t w, uint32_t sel) {
  const f16x2 v = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, sel));
  return __builtin_bit_cast(uint32_t, v - f16x2{(_Float16)1152.0f, (_Float16)1152.0f});
}

// Eight codes -> eight float16, exactly.
__device__ __forceinline__ f16x8 widen_f16(uint32_t w0, uint32_t w1) {
  const uint32_t x0 = w0 ^ 0x80808080u, x1 = w1 ^ 0x80808080u;
  return __builtin_bit_cast(f16x8, u32x4{f16x2_from_u8(x0, 0x04010400u), f16x2_from_u8(x0, 0x04030402u),
                                         f16x2_from_u8(x1, 0x04010400u), f16x2_from_u8(x1, 0x04030402u)});
}

// The power of two that brings a row's largest magnitude to 2^15 .. 2^16, as inv, and its inverse.
// The largest bfloat16 there, 65280, is below float16's 65504. Rows whose largest is below
// 2^-111 take 2^126, the largest power that has an inverse.
__device__ __forceinline__ float row_exponent(float largest, float &inv) {
  const uint32_t e = min(max(__float_as_uint(largest) & 0x7f800000u, 16u << 23), 254u << 23);
  inv = __uint_as_float((269u << 23) - e);
  return __uint_as_float(e - (15u << 23));
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// f over the four lanes that hold a query, without LDS.
template <class F>
__device__ __forceinline__ float across(float v, F &&f) {
  const uint32_t a = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const float w = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const uint32_t b = __float_as_uint(w);
  const auto q = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return f(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// A lane's operands of one row of q, dims 64 c + 16 g + 8 s .. + 7 in q[2 c + s], in float16
// under the row's exponent, which goes into the scores' scale. Dims from D on, and rows that
// are none, are zero.
template <int C>
__device__ __forceinline__ void load_query(const uint16_t *p, bool live, int D, int g, float sm,
                                           f16x8 (&q)[2 * C], float &scale) {
  i32x4 v[2 * C];
  uint32_t mx = 0;
#pragma unroll
  for (int cs = 0; cs < 2 * C; ++cs) {
    const int d = 32 * (cs & ~1) + 16 * g + 8 * (cs & 1);
    v[cs] = i32x4{0, 0, 0, 0};
    if (live && d < D) v[cs] = *reinterpret_cast<const i32x4 *>(p + d);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      mx = max(mx, max((uint32_t)v[cs][e] << 16 & 0x7fffffffu, (uint32_t)v[cs][e] & 0x7fff0000u));
  }
  float inv;
  scale = sm * row_exponent(across(__uint_as_float(mx), [](float x, float y) {
            return __uint_as_float(max(__float_as_uint(x), __float_as_uint(y)));
          }), inv);
#pragma unroll
  for (int cs = 0; cs < 2 * C; ++cs)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[cs][2 * e] = (_Float16)(__uint_as_float((uint32_t)v[cs][e] << 16) * inv);
      q[cs][2 * e + 1] = (_Float16)(__uint_as_float((uint32_t)v[cs][e] & 0xffff0000u) * inv);
    }
}

struct AttnArgs {
  const uint16_t *q;
  int64_t qrow;
  float sm;  // sm_scale log2(e)
  KvCache c;
  const int32_t *table;
  int64_t W;
  const int32_t *plan;
  int64_t at_units, at_joins, window;
  int G, Hq, tile;  // tile: rows of a partial result
  uint16_t *y;
  float *lse;
  float *pm, *po;  // partial results: (M, denominator) and sums of each part, head and row
};

constexpr float kLn2 = 0.693147181f;

// Weights use float16's range: their reference M is the largest score less 15 in the streaming kernel,
// so that the largest weight is 2^15. The tile kernel moves M only when a score passes it by 15, and
// then to 7 below that score.
constexpr float kTop = 15.0f, kTopMoved = 7.0f;

// Outputs of row `row` of a unit's sequence: 4 dims from d on.
__device__ __forceinline__ void store_out(const AttnArgs &a, int tok, int h, int row, int d,
                                          const f32x4 &o) {
  const int64_t at = ((int64_t)(tok + row / a.G) * a.Hq + h * a.G + row % a.G) * a.c.D + d;
  const uint32_t lo = (uint32_t)f32_to_bf16_rne(o[0]) | ((uint32_t)f32_to_bf16_rne(o[1]) << 16);
  const uint32_t hi = (uint32_t)f32_to_bf16_rne(o[2]) | ((uint32_t)f32_to_bf16_rne(o[3]) << 16);
  *reinterpret_cast<uint2 *>(a.y + at) = uint2{lo, hi};
}
__device__ __forceinline__ void store_lse(const AttnArgs &a, int tok, int h, int row, float M,
                                          float l) {
  if (a.lse)
    a.lse[(int64_t)(tok + row / a.G) * a.Hq + h * a.G + row % a.G] =
        l == 0.0f ? -__builtin_inff() : (M + __log2f(l)) * kLn2;
}

// Few rows (decode): 16 NB rows of one kv head against a range of blocks, streamed from
// memory once (loads that leave no copy in the caches: 64 requests of up to 8192 tokens 88 us,
// 103 with them). Bound by memory. The four waves take blocks in turn, each with a
// maximum and sums of its own, and join in LDS at the end. The next block's K is in
// flight from when the present one is used up, V from the same moment one block earlier.
// (With 8 waves on two a SIMD's registers, a block's V is loaded once its K is used up and
// the next K after that: the other waves' loads fill the time.)
template <int NB, int C, int NW>
struct StreamLds {
  static constexpr int DIMS = C > 2 ? 128 : 64 * C;  // joined at a time
  float o[NW][16][DIMS + 4];
  float m[NW][16 * NB], l[NW][16 * NB];
};

// Rows row0 .. row0 + 16 NB - 1 of u's sequence.
template <int NB, int C, int NW>
__device__ __forceinline__ void stream_rows(const AttnArgs &a, const KvUnit &u, int h, int row0,
                                            StreamLds<NB, C, NW> &lds) {
  constexpr int DP = 64 * C, ND = DP / 16, HD = StreamLds<NB, C, NW>::DIMS;
  constexpr bool AHEAD = NW == 4;
  auto &ob = lds.o;
  auto &om = lds.m;
  auto &ol = lds.l;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int rows = min(16 * NB, u.len * a.G - row0);

  f16x8 qf[NB][2 * C];
  int qpos[NB];
  float qs[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int row = row0 + 16 * nb + r;
    const bool live = 16 * nb + r < rows;
    qpos[nb] = u.pos + (live ? row : row0) / a.G;
    const uint16_t *p = a.q + (int64_t)(u.tok + row / a.G) * a.qrow + (h * a.G + row % a.G) * a.c.D;
    load_query<C>(p, live, a.c.D, g, a.sm, qf[nb], qs[nb]);
  }
  const int pmin = u.pos + row0 / a.G, pmax = u.pos + (row0 + rows - 1) / a.G;
  const uint32_t oldest = a.window > 0 ? (uint32_t)a.window - 1 : 0x7fffffffu;

  f32x4 acc[NB][ND];
  float M[NB], l[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    M[nb] = -__builtin_inff();
    l[nb] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[nb][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int32_t *row_table = a.table + u.seq * a.W;
  const int ktok = 16 * (r >> 2) + (r & 3);
  const int64_t kofs = ktok * 64 + 16 * g, vofs = r * 64 + 16 * g;
  i32x4 kb[4][C], vb[ND];
  // a page that is none reads page 0 and counts for nothing
  auto page_at = [&](int b) { return __builtin_amdgcn_readfirstlane(row_table[b]); };
  auto base = [&](int page) {
    return ((int64_t)(page >= 0 && page < a.c.pages ? page : 0) * a.c.Hkv + h) * (64 * DP);
  };
  auto load_k = [&](int page) {
    const int8_t *p = a.c.kq + base(page) + kofs;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        kb[t][c] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(p + c * 4096 + t * 256));
  };
  int b = u.b0 + wave;
  int page = b < u.b1 ? page_at(b) : 0;
  if (b < u.b1) load_k(page);
  while (b < u.b1) {
    const bool more = b + NW < u.b1;
    const int next = more ? page_at(b + NW) : page;
    auto load_v = [&]() {
      const int8_t *p = a.c.vq + base(page) + vofs;
#pragma unroll
      for (int d = 0; d < ND; ++d) vb[d] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(p + d * 1024));
    };
    if constexpr (AHEAD) load_v();
    const bool live = page >= 0 && page < a.c.pages;
    const int64_t at = (live ? (int64_t)page : 0) * a.c.Hkv + h;
    const float ks = a.c.ks[at], vs = a.c.vs[at];
    const float c2 = __builtin_amdgcn_logf(vs), iv = __builtin_amdgcn_rcpf(vs);

    f32x4 s[NB][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) s[nb][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const f16x8 k0 = widen_f16((uint32_t)kb[t][c][0], (uint32_t)kb[t][c][1]);
        const f16x8 k1 = widen_f16((uint32_t)kb[t][c][2], (uint32_t)kb[t][c][3]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          s[nb][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[nb][2 * c], s[nb][t], 0, 0, 0);
          s[nb][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[nb][2 * c + 1], s[nb][t], 0, 0, 0);
        }
      }
    }
    if constexpr (!AHEAD) {
      __builtin_amdgcn_sched_barrier(0);
      load_v();
    } else if (more) {
      load_k(next);
    }

    // tokens past a query or before its window, and those of a page that is none: of the
    // lane's tokens, how far each lies behind its query, as an unsigned number
    const int t0 = b * 64;
    const bool whole = live && t0 + 63 <= pmin && (uint32_t)(pmax - t0) <= oldest;
    f16x8 pf[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int age = live ? qpos[nb] - t0 - 16 * g : -1 - 64;
      const float c1 = ks * qs[nb];
      float mx = -__builtin_inff();
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float z = fmaf(s[nb][t][v], c1, c2);
          if (!whole) z = (uint32_t)(age - 4 * t - v) <= oldest ? z : -__builtin_inff();
          s[nb][t][v] = z;
          mx = fmaxf(mx, z);
        }
      mx = across(mx, [](float x, float y) { return fmaxf(x, y); });
      const float Mn = fmaxf(M[nb], mx - kTop);
      const float off = Mn == -__builtin_inff() ? 0.0f : Mn;
      const float alpha = exp2_hw(M[nb] - off);
      M[nb] = Mn;
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float w = exp2_hw(s[nb][t][v] - off);
          sum += w;
          pf[nb][t >> 1][4 * (t & 1) + v] = (_Float16)w;
        }
      // (a page without a visible token may hold any scale)
      l[nb] = fmaf(l[nb], alpha, sum == 0.0f ? 0.0f : sum * iv);
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[nb][d] *= alpha;
    }
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const f16x8 v0 = widen_f16((uint32_t)vb[d][0], (uint32_t)vb[d][1]);
      const f16x8 v1 = widen_f16((uint32_t)vb[d][2], (uint32_t)vb[d][3]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        acc[nb][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[nb][0], acc[nb][d], 0, 0, 0);
        acc[nb][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[nb][1], acc[nb][d], 0, 0, 0);
      }
    }
    if constexpr (!AHEAD) {
      __builtin_amdgcn_sched_barrier(0);
      if (more) load_k(next);
    }
    page = next;
    b += NW;
  }

  // ---- the waves' results join
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const float sum = across(l[nb], [](float x, float y) { return x + y; });
    if (g == 0) {
      om[wave][16 * nb + r] = M[nb];
      ol[wave][16 * nb + r] = sum;
    }
  }
  __syncthreads();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int row = 16 * nb + r;
    float top = om[0][row];
#pragma unroll
    for (int w = 1; w < NW; ++w) top = fmaxf(top, om[w][row]);
    const float off = top == -__builtin_inff() ? 0.0f : top;
    const float f = exp2_hw(M[nb] - off);
#pragma unroll
    for (int half = 0; half < DP; half += HD) {
#pragma unroll
      for (int d = 0; d < HD / 16; ++d)
        if (half / 16 + d < ND)
          *reinterpret_cast<f32x4 *>(&ob[wave][r][16 * d + 4 * g]) = acc[nb][half / 16 + d] * f;
      __syncthreads();
      // thread (row orow, piece oc): 4 dims at a time
      const int orow = threadIdx.x >> 4, oc = threadIdx.x & 15, lrow = 16 * nb + orow;
      if (orow < 16 && lrow < rows) {
        float t2 = om[0][lrow], L = 0.0f;
#pragma unroll
        for (int w = 1; w < NW; ++w) t2 = fmaxf(t2, om[w][lrow]);
        const float o2 = t2 == -__builtin_inff() ? 0.0f : t2;
#pragma unroll
        for (int w = 0; w < NW; ++w) L = fmaf(ol[w][lrow], exp2_hw(om[w][lrow] - o2), L);
        const int64_t at = ((int64_t)u.part * a.c.Hkv + h) * a.tile + row0 - u.row0 + lrow;
        if (half == 0 && oc == 0) {
          if (u.part < 0) {
            store_lse(a, u.tok, h, row0 + lrow, t2, L);
          } else {
            a.pm[2 * at] = t2;
            a.pm[2 * at + 1] = L;
          }
        }
#pragma unroll
        for (int p = 0; p < HD / 64; ++p) {
          const int d = 4 * (oc + 16 * p);
          if (half + d >= a.c.D) continue;
          f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < NW; ++w) o += *reinterpret_cast<const f32x4 *>(&ob[w][orow][d]);
          if (u.part < 0) store_out(a, u.tok, h, row0 + lrow, half + d, L == 0.0f ? f32x4{0.f, 0.f, 0.f, 0.f} : o * (1.0f / L));
          else *reinterpret_cast<f32x4 *>(a.po + at * DP + half + d) = o;
        }
      }
      __syncthreads();
    }
  }
}

template <int NB, int C>
__global__ __launch_bounds__(256) void k_kv_attn_stream(AttnArgs a) {
  __shared__ __attribute__((aligned(16))) StreamLds<NB, C, 4> lds;
  const int i = blockIdx.x / a.c.Hkv, h = blockIdx.x % a.c.Hkv;
  if (i >= a.plan[kKvUnits]) return;
  const KvUnit u = reinterpret_cast<const KvUnit *>(a.plan + a.at_units)[i];
  const int row0 = u.row0 + (int)blockIdx.y * (16 * NB);
  if (row0 < u.len * a.G) stream_rows<NB, C, 4>(a, u, h, row0, lds);
}

// LDS writes done and every wave here; loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Many rows (prefill): 4 waves of 32 or 8 of 16 rows of one kv head against a range of blocks. A
// block's codes are widened once for all waves, on the way from memory into LDS, where
// they lie as the matrix instructions' operands, fragment by fragment, 16 bytes a lane in the
// order of lanes (the one order that neither reads nor writes conflict on). One barrier a block: while
// block i meets V, block i + 1 meets K, and K of block i + 2 and V of block i + 1
// go to the halves of LDS that the last block has left.
template <int C>
struct TileLds {
  static constexpr int HALF = 8192 * C;       // one block's K, or V
  static constexpr int BYTES = 4 * HALF;      // K, K, V, V
};

template <int NB, int C>
__device__ __forceinline__ void tile_rows(const AttnArgs &a, const KvUnit &u, int h, char *smem) {
  constexpr int DP = 64 * C, ND = DP / 16, HALF = TileLds<C>::HALF;
  constexpr int P = kKvTileRows / (64 * NB), SL = (C + P - 1) / P;  // fours of waves, slices of each
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int four = wave >> 2, kw = wave & 3;
  const int r = lane & 15, g = lane >> 4;
  const int total = u.len * a.G;                  // rows of the sequence
  const int w0 = u.row0 + wave * (16 * NB);       // the wave's first
  const int rows = min(16 * NB, total - w0);      // (none: the wave only loads)

  f16x8 qf[NB][2 * C];
  int qpos[NB];
  float qs[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int row = w0 + 16 * nb + r;
    const bool live = row < total;
    qpos[nb] = u.pos + (live ? row : total - 1) / a.G;
    const uint16_t *p = a.q + (int64_t)(u.tok + row / a.G) * a.qrow + (h * a.G + row % a.G) * a.c.D;
    load_query<C>(p, live, a.c.D, g, a.sm, qf[nb], qs[nb]);
  }
  const int pmin = u.pos + min(w0, total - 1) / a.G, pmax = u.pos + (min(w0 + 16 * NB, total) - 1) / a.G;
  const uint32_t oldest = a.window > 0 ? (uint32_t)a.window - 1 : 0x7fffffffu;

  // ---- blocks from memory into LDS
  const int32_t *row_table = a.table + u.seq * a.W;
  const int n = u.b1 - u.b0;
  auto page_at = [&](int k) { return row_table[u.b0 + min(k, n - 1)]; };
  // a page that is none reads page 0 and counts for nothing
  auto head_at = [&](int page) {
    return (int64_t)(page >= 0 && page < a.c.pages ? page : 0) * a.c.Hkv + h;
  };
  // every wave brings SL KiB of K and of V, in loads whose lanes hold what the lanes of two
  // fragments will: slices c = four, four + P, .. of the dims, of K tile kw, of V dims
  // 16 (kw + 4 c) ..
  const int8_t *ksrc = a.c.kq + (16 * (r >> 2) + 4 * kw + (r & 3)) * 64 + 16 * g;
  const int8_t *vsrc = a.c.vq + kw * 1024 + r * 64 + 16 * g;
  auto slice = [&](int i) { return four + P * i; };
  i32x4 kr[SL], vr[SL];
  auto load_k = [&](int page) {
    const int8_t *p = ksrc + head_at(page) * (64 * DP);
#pragma unroll
    for (int i = 0; i < SL; ++i)
      if (C % P == 0 || slice(i) < C) kr[i] = *reinterpret_cast<const i32x4 *>(p + slice(i) * 4096);
  };
  auto load_v = [&](int page) {
    const int8_t *p = vsrc + head_at(page) * (64 * DP);
#pragma unroll
    for (int i = 0; i < SL; ++i)
      if (C % P == 0 || slice(i) < C) vr[i] = *reinterpret_cast<const i32x4 *>(p + slice(i) * 4096);
  };
  // piece i of the 2 SL that a wave widens of either, into block k's half of LDS
  auto put_k = [&](int k, int i) {
    if (C % P == 0 || slice(i >> 1) < C)
      *reinterpret_cast<f16x8 *>(smem + (k & 1) * HALF + kw * (C * 2048) + lane * 16 +
                                 slice(i >> 1) * 2048 + (i & 1) * 1024) =
          widen_f16((uint32_t)kr[i >> 1][2 * (i & 1)], (uint32_t)kr[i >> 1][2 * (i & 1) + 1]);
  };
  auto put_v = [&](int k, int i) {
    if (C % P == 0 || slice(i >> 1) < C)
      *reinterpret_cast<f16x8 *>(smem + (2 + (k & 1)) * HALF + kw * 2048 + lane * 16 +
                                 slice(i >> 1) * 8192 + (i & 1) * 1024) =
          widen_f16((uint32_t)vr[i >> 1][2 * (i & 1)], (uint32_t)vr[i >> 1][2 * (i & 1) + 1]);
  };
  auto put_all = [&](int k) {  // V is a block behind K
#pragma unroll
    for (int i = 0; i < 2 * SL; ++i) {
      put_v(k + 1, i);
      put_k(k + 2, i);
    }
  };
  const int fo = lane * 16;

  f32x4 acc[NB][ND], s[NB][4];
  float M[NB], off[NB], l[NB];  // off: M, or 0 where no token was seen yet
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    M[nb] = -__builtin_inff();
    off[nb] = l[nb] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[nb][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  constexpr int F = 8 * C;  // fragments of a block's K, and of its V
  auto read = [&](int k, bool v, int f) {
    return *reinterpret_cast<const f16x8 *>(smem + (2 * v + (k & 1)) * HALF + fo + f * 1024);
  };
  // Before block k: the pages of k .. k + 3 and the scales of k and k + 1 are here, and one of each
  // is asked for, so that no load waits for another's result.
  int page0, page1, page2, page3, page4;
  float ks0, vs0, ks1, vs1, ks2, vs2;
  auto ask = [&](int k) {
    page4 = page_at(k + 4);
    ks2 = a.c.ks[head_at(page2)];
    vs2 = a.c.vs[head_at(page2)];
  };
  auto move = [&]() {
    page0 = page1;
    page1 = page2;
    page2 = page3;
    page3 = __builtin_amdgcn_readfirstlane(page4);
    ks0 = ks1;
    vs0 = vs1;
    ks1 = ks2;
    vs1 = vs2;
  };
  // Scores of block k in s become weights and meet V; with `more`, those of block k + 1
  // take their place. The reference M of a row moves only when a score passes it by kTop:
  // weights up to 2^15 lose nothing in float16, and moving it costs every sum a product.
  //
  // Written in the order of issue. Every fragment is read four ahead of its products; the weights'
  // arithmetic goes between the products of the next scores, the widening of the codes
  // to come between those with V. (Left to the compiler, the reads wait for each other: the
  // prefill of 11490 tokens, 32 heads of 128 over 8, takes 474 us.)
  auto step = [&](auto more, int k) {
    const int t0 = 64 * (u.b0 + k);
    const bool live = page0 >= 0 && page0 < a.c.pages;
    const float iv = __builtin_amdgcn_rcpf(vs0);
    constexpr bool MORE = decltype(more)::value;
    f16x8 kf[4], vf[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if constexpr (MORE) kf[f] = read(k + 1, false, f);
      else vf[f] = read(k, true, f);
    }
    __builtin_amdgcn_sched_barrier(0);
    float c1[NB], c2 = __builtin_amdgcn_logf(vs0);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) c1[nb] = ks0 * qs[nb];
    if (!(live && t0 + 63 <= pmin && (uint32_t)(pmax - t0) <= oldest)) {
      // tokens past a query or before its window, and those of a page that is none: of the
      // lane's tokens, how far each lies behind its query, as an unsigned number
      int age[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) age[nb] = live ? qpos[nb] - t0 - 16 * g : -1 - 64;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const bool see = (uint32_t)(age[nb] - 4 * t - v) <= oldest;
            s[nb][t][v] = see ? fmaf(s[nb][t][v], c1[nb], c2) : -__builtin_inff();
          }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) c1[nb] = 1.0f;  // (done, so that a scale that is no number
      c2 = 0.0f;                                       // stays with its tokens)
    }
    float top[NB];
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float mx = s[nb][0][0];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) mx = fmaxf(mx, s[nb][t][v]);
      top[nb] = across(fmaf(mx, c1[nb], c2), [](float x, float y) { return fmaxf(x, y); });
      grow = grow || top[nb] > M[nb] + kTop;
    }
    if (__any(grow)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // (from M, not off: 0 where nothing was seen yet, however far below 0 the new maximum lies)
        const float before = M[nb];
        M[nb] = fmaxf(before, top[nb] - kTopMoved);
        off[nb] = M[nb] == -__builtin_inff() ? 0.0f : M[nb];
        const float alpha = exp2_hw(before - off[nb]);
        l[nb] *= alpha;
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[nb][d] *= alpha;
      }
    }
    f16x8 pf[NB][2];
    float c3[NB], sum[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      c3[nb] = c2 - off[nb];
      sum[nb] = 0.0f;
    }
    f32x4 sn[NB][4];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      if constexpr (MORE) {
        const int t = f / (2 * C), cs = f % (2 * C);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          sn[nb][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              kf[f & 3], qf[nb][cs], cs == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : sn[nb][t], 0, 0, 0);
        if (f + 4 < F) kf[f & 3] = read(k + 1, false, f + 4);
        else vf[f & 3] = read(k, true, f + 4 - F);
      }
#pragma unroll
      for (int e = 16 * NB * f / F; e < 16 * NB * (f + 1) / F; ++e) {
        const int nb = e >> 4, t = e >> 2 & 3, v = e & 3;
        const float w = exp2_hw(fmaf(s[nb][t][v], c1[nb], c3[nb]));
        sum[nb] += w;
        pf[nb][t >> 1][4 * (t & 1) + v] = (_Float16)w;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)  // (a page that is not seen may have any scale)
      l[nb] += sum[nb] == 0.0f ? 0.0f : sum[nb] * iv;
#pragma unroll
    for (int f = 0; f < F; ++f) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        acc[nb][f >> 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[f & 3], pf[nb][f & 1],
                                                                 acc[nb][f >> 1], 0, 0, 0);
      if (f + 4 < F) vf[f & 3] = read(k, true, f + 4);
      if constexpr (MORE)
        if (f & 1) {
          if (f < F / 2 && f / 2 < 2 * SL) put_v(k + 1, f / 2);
          if (f >= F / 2 && f / 2 - 2 * C < 2 * SL) put_k(k + 2, f / 2 - 2 * C);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (MORE) {
      load_v(page2);
      load_k(page3);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int t = 0; t < 4; ++t) s[nb][t] = sn[nb][t];
    }
  };
  page0 = __builtin_amdgcn_readfirstlane(page_at(0));
  page1 = __builtin_amdgcn_readfirstlane(page_at(1));
  page2 = __builtin_amdgcn_readfirstlane(page_at(2));
  page3 = __builtin_amdgcn_readfirstlane(page_at(3));
  ks0 = a.c.ks[head_at(page0)];
  vs0 = a.c.vs[head_at(page0)];
  ks1 = a.c.ks[head_at(page1)];
  vs1 = a.c.vs[head_at(page1)];
  load_k(page0);
  load_v(page0);
#pragma unroll
  for (int i = 0; i < 2 * SL; ++i) put_k(0, i);
  load_k(page1);
  lds_barrier();
  put_all(-1);
  load_v(page1);
  load_k(page2);
  if (rows <= 0) {  // a wave without rows only brings blocks in
    lds_barrier();
    for (int k = 0; k < n - 1; ++k) {
      ask(k);
      put_all(k);
      load_v(page2);
      load_k(page3);
      lds_barrier();
      move();
    }
    return;
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) s[nb][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int cs = 0; cs < 2 * C; ++cs) {
      const f16x8 kf = read(0, false, t * 2 * C + cs);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        s[nb][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[nb][cs], s[nb][t], 0, 0, 0);
    }
  }
  lds_barrier();
  for (int k = 0; k < n - 1; ++k) {
    ask(k);
    step(std::true_type{}, k);
    lds_barrier();
    move();
  }
  step(std::false_type{}, n - 1);

#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int lrow = 16 * nb + r;
    l[nb] = across(l[nb], [](float x, float y) { return x + y; });  // the lanes' own tokens
    if (lrow >= rows) continue;
    const int row = w0 + lrow;
    const float inv = l[nb] == 0.0f ? 0.0f : 1.0f / l[nb];
    if (u.part < 0) {
      if (g == 0) store_lse(a, u.tok, h, row, M[nb], l[nb]);
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (16 * d + 4 * g < a.c.D) store_out(a, u.tok, h, row, 16 * d + 4 * g, acc[nb][d] * inv);
    } else {
      const int64_t at = ((int64_t)u.part * a.c.Hkv + h) * kKvTileRows + (row - u.row0);
      if (g == 0) {
        a.pm[2 * at] = M[nb];
        a.pm[2 * at + 1] = l[nb];
      }
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (16 * d + 4 * g < a.c.D)
          *reinterpret_cast<f32x4 *>(a.po + at * DP + 16 * d + 4 * g) = acc[nb][d];
    }
  }
}

// Units of few rows among them (decoding sequences in a step with a prefill, a
// sequence's last rows) stream instead: a block that 128 rows meet in 2.2 us is read by one of
// their 4 waves in little more than 1.
//
// Heads past 128 leave room for one workgroup's LDS a CU: it has 8 waves of 16 rows, so that
// every SIMD still has two (prefill of 4096 tokens, 32 heads of 256 over 8: 401 us with 4 waves, 323;
// 16 requests and a chunk of 100 tokens behind 8000: 117, 104).
template <int C>
constexpr int kTileWaves = C > 2 ? 8 : 4;
static_assert(kTileWaves<3> == kTileWaves<4> && kTileWaves<1> == 4 && kTileWaves<2> == 4, "the launcher's check");

template <int C>
__global__ __launch_bounds__(64 * kTileWaves<C>, 2) void k_kv_attn_tile(AttnArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  using Stream = StreamLds<1, C, kTileWaves<C>>;
  static_assert(sizeof(Stream) <= TileLds<C>::BYTES, "either's LDS");
  const int i = blockIdx.x / a.c.Hkv, h = blockIdx.x % a.c.Hkv;
  if (i >= a.plan[kKvUnits]) return;
  const KvUnit u = reinterpret_cast<const KvUnit *>(a.plan + a.at_units)[i];
  if (u.len * a.G - u.row0 <= kKvFewRows)
    stream_rows<1, C, kTileWaves<C>>(a, u, h, u.row0, *reinterpret_cast<Stream *>(smem));
  else
    tile_rows<kKvTileRows / (16 * kTileWaves<C>), C>(a, u, h, smem);
}

// The partial results of rows whose blocks were spread over several units. 16 C threads
// take a row's dims; with SPREAD (few rows, up to hundreds of parts) the workgroup's groups of
// threads share a row's parts and add up in LDS, else (many rows, few parts) each takes a
// row. Sums are in one order for a given number of parts.
template <int C, bool SPREAD>
__global__ __launch_bounds__(256) void k_kv_attn_join(AttnArgs a) {
  const int tile = a.tile;
  constexpr int TPR = 16 * C, GROUPS = 256 / TPR, U = 4;  // U: parts in flight
  __shared__ float red[2][GROUPS];
  __shared__ f32x4 sums[SPREAD ? GROUPS : 1][TPR];
  const int i = blockIdx.x / a.c.Hkv, h = blockIdx.x % a.c.Hkv;
  if (i >= a.plan[kKvJoins]) return;
  const KvJoin u = reinterpret_cast<const KvJoin *>(a.plan + a.at_joins)[i];
  const int rows = min(tile, u.len * a.G - u.row0);
  const int gi = threadIdx.x / TPR, d = 4 * (threadIdx.x % TPR);
  const int row = SPREAD ? (int)blockIdx.y : (int)blockIdx.y * GROUPS + gi;
  if (SPREAD ? row >= rows : (int)blockIdx.y * GROUPS >= rows) return;
  const bool live = gi < GROUPS && row < rows && d < a.c.D;
  const int64_t step = (int64_t)a.c.Hkv * tile;
  const int64_t at = ((int64_t)u.part * a.c.Hkv + h) * tile + row;
  const int p0 = SPREAD ? gi : 0, by = SPREAD ? GROUPS : 1;
  float top = -__builtin_inff(), L = 0.0f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  if (live)
    for (int p = p0; p < u.parts; p += U * by) {
      float m[U];
#pragma unroll
      for (int k = 0; k < U; ++k) m[k] = a.pm[2 * (at + min(p + k * by, u.parts - 1) * step)];
#pragma unroll
      for (int k = 0; k < U; ++k) top = fmaxf(top, m[k]);
    }
  if constexpr (SPREAD) {
    if (gi < GROUPS && d == 0) red[0][gi] = top;
    __syncthreads();
    for (int k = 0; k < GROUPS; ++k) top = fmaxf(top, red[0][k]);
  }
  const float off = top == -__builtin_inff() ? 0.0f : top;
  if (live)
    for (int p = p0; p < u.parts; p += U * by) {
      float m[U], l[U];
      f32x4 v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t r = at + min(p + k * by, u.parts - 1) * step;
        m[k] = a.pm[2 * r];
        l[k] = a.pm[2 * r + 1];
        v[k] = *reinterpret_cast<const f32x4 *>(a.po + r * a.c.DP + d);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float f = exp2_hw(m[k] - off);
        if (p + k * by < u.parts) {  // (a part that is none may hold anything)
          L = fmaf(l[k], f, L);
          o += v[k] * f;
        }
      }
    }
  if constexpr (SPREAD) {
    if (live) {
      sums[gi][threadIdx.x % TPR] = o;
      if (d == 0) red[1][gi] = L;
    }
    __syncthreads();
    if (gi != 0 || !live) return;
    L = 0.0f;
    o = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < GROUPS; ++k) {
      L += red[1][k];
      o += sums[k][threadIdx.x];
    }
  }
  if (!live) return;
  if (d == 0) store_lse(a, u.tok, h, u.row0 + row, top, L);
  store_out(a, u.tok, h, u.row0 + row, d, o * (L == 0.0f ? 0.0f : 1.0f / L));
}

template <bool SPREAD>
hipError_t launch_join(const AttnArgs &a, int64_t joins, hipStream_t st) {
  const auto go = [&](auto kern, int groups) {
    hipLaunchKernelGGL(kern, dim3((unsigned)(joins * a.c.Hkv), SPREAD ? a.tile : (a.tile + groups - 1) / groups),
                       dim3(256), 0, st, a);
  };
  switch (a.c.DP / 64) {
    case 1: go(k_kv_attn_join<1, SPREAD>, 16); break;
    case 2: go(k_kv_attn_join<2, SPREAD>, 8); break;
    case 3: go(k_kv_attn_join<3, SPREAD>, 5); break;
    default: go(k_kv_attn_join<4, SPREAD>, 4); break;
  }
  return hipGetLastError();
}

// In units of 16 NB rows, `per` workgroups of them a unit of the plan.
template <int NB>
void launch_stream(const AttnArgs &a, unsigned grid, unsigned per, hipStream_t st) {
  switch (a.c.DP / 64) {
    case 1: hipLaunchKernelGGL((k_kv_attn_stream<NB, 1>), dim3(grid, per), dim3(256), 0, st, a); break;
    case 2: hipLaunchKernelGGL((k_kv_attn_stream<NB, 2>), dim3(grid, per), dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL((k_kv_attn_stream<NB, 3>), dim3(grid, per), dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL((k_kv_attn_stream<NB, 4>), dim3(grid, per), dim3(256), 0, st, a); break;
  }
}

template <int C>
hipError_t launch_tile(const AttnArgs &a, unsigned grid, hipStream_t st) {
  const auto kern = k_kv_attn_tile<C>;
  constexpr int bytes = TileLds<C>::BYTES;
  if constexpr (bytes > 65536) {  // once a device; a launch that the limit refuses reports itself
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    (void)hipGetDevice(&dev);
    if (!(set.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
      (void)hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
      (void)hipGetLastError();
      set.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * kTileWaves<C>), bytes, st, a);
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_bytes(const KvSizes &z, int DP) {
  const int64_t rows = kv_plan_layout(z).parts * z.Hkv * kv_tile_rows(z);
  return (size_t)rows * (8 + 4 * (size_t)DP);
}

hipError_t launch_kv_attention(const uint16_t *q, int64_t qrow, float sm_scale, const KvCache &c,
                               const int32_t *table, const KvSizes &z, const int32_t *plan,
                               uint16_t *y, float *lse, void *ws, hipStream_t st) {
  const KvPlanLayout lay = kv_plan_layout(z);
  const int tile = kv_tile_rows(z);
  AttnArgs a{};
  a.q = q;
  a.qrow = qrow;
  a.sm = sm_scale * 1.44269504f;
  a.c = c;
  a.table = table;
  a.W = z.W;
  a.plan = plan;
  a.at_units = lay.at_units;
  a.at_joins = lay.at_joins;
  a.window = z.window;
  a.G = z.Hq / z.Hkv;
  a.tile = tile;
  a.Hq = z.Hq;
  a.y = y;
  a.lse = lse;
  // sums first: rows of 4 DP bytes keep every access aligned
  a.po = static_cast<float *>(ws);
  a.pm = a.po + lay.parts * z.Hkv * tile * c.DP;
  const bool tiles = tile == kKvTileRows && (c.DP <= 128 || z.most * a.G > 64);
  const int64_t groups = lay.units * z.Hkv;
  // (the rounded grid of two streams a unit below is the largest of 256 threads)
  if (!grid_fits((groups + 7) / 8 * 8, tiles && c.DP > 128 ? 64 * kTileWaves<4> : 256))
    return hipErrorInvalidConfiguration;
  const unsigned grid = (unsigned)groups;
  hipError_t e = hipSuccess;
  if (tiles) {
    switch (c.DP / 64) {
      case 1: e = launch_tile<1>(a, grid, st); break;
      case 2: e = launch_tile<2>(a, grid, st); break;
      case 3: e = launch_tile<3>(a, grid, st); break;
      default: e = launch_tile<4>(a, grid, st); break;
    }
  } else {
    // (33 to 64 rows of a head past 128, whose tiles leave one workgroup a CU, in two streams of
    // 32: one sequence, one kv head of 256, 300 and 1500 tokens 16.7, 17.0 us, as tiles 21.9, 22.2.
    // The two of a unit lie on one XCD and its L2.)
    if (tile == 16) launch_stream<1>(a, grid, 1, st);
    else if (tile == 32) launch_stream<2>(a, grid, 1, st);
    else launch_stream<2>(a, (grid + 7) / 8 * 8, 2, st);
    e = hipGetLastError();
  }
  if (e != hipSuccess || lay.joins == 0) return e;
  // few tiles may be in many parts each (one sequence of 64 rows for one kv head of 128, 30000
  // tokens: 45.5 us with a row a group of threads, 19.9 spread), many are in few (16 requests and a
  // chunk of 509 tokens, 264 joins at most: 90, 105 spread; 256 tokens behind 16000, 72: 94, 99)
  return tile == kKvTileRows && lay.joins * z.Hkv > 64 ? launch_join<false>(a, lay.joins, st)
                                                       : launch_join<true>(a, lay.joins, st);
}

}  // namespace aql
