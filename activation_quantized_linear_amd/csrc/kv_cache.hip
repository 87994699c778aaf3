// A paged 8-bit KV cache: a step's plan, quantising new tokens into their pages, and
// reading them back.
//
// Of a page and kv head, K and V each:  s = max(max |x| / 127, 2^-64),
// code = clamp(rint(x / s), -127, 127), value = code s. A page that a write begins takes
// its scale from the new tokens; behind live tokens the scale only grows, and where
// it does their codes become clamp(rint((code s) / s')), each product and quotient
// rounded once to binary32.
#include "kv.h"

namespace aql {
namespace {

// ------------------------------------------------------------------- the plan

constexpr int kPlanThreads = 1024, kBins = 256;

struct Seq {
  int tok, len, pos;
};

// Sequence s as cu and pos have it; len 0 and bad set where they cannot be served.
__device__ __forceinline__ Seq sequence(const int32_t *cu, const int32_t *pos, const KvSizes &z,
                                        int s, bool &bad) {
  const int64_t a = cu[s], b = cu[s + 1], p = pos[s];
  bad = a < 0 || b < a || b > z.T || b - a > z.most || p < 0 ||
        (b > a && p + (b - a) > z.W * kKvBlock);
  return bad ? Seq{0, 0, 0} : Seq{(int)a, (int)(b - a), (int)p};
}

// The blocks that rows row0 .. row0 + rows - 1 of a sequence see.
__device__ __forceinline__ void tile_blocks(const Seq &q, int G, int64_t window, int row0, int rows,
                                            int &b0, int &b1) {
  const int last = min(row0 + rows, q.len * G) - 1;
  const int64_t first = (int64_t)q.pos + row0 / G - (window - 1);
  b0 = window > 0 && first > 0 ? (int)(first / kKvBlock) : 0;
  b1 = (q.pos + last / G) / kKvBlock + 1;
}

// What one block of these rows costs, in blocks of few rows.
__device__ __forceinline__ int block_cost(const Seq &q, int G, int tile, int row0) {
  return tile < kKvTileRows || q.len * G - row0 <= kKvFewRows ? 1 : kKvTileCost;
}

// Exclusive sum over the workgroup's threads; total to all.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t *lds, int64_t &total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w < wave) before += lds[w];
    total += lds[w];
  }
  __syncthreads();
  return before + x - v;
}

// The sequence whose share of [0, total) holds i: the last s with first[s] <= i.
__device__ __forceinline__ int owner(const int *first, int S, int i) {
  int lo = 0, hi = S;  // first[lo] <= i < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One workgroup. Sequences' pieces and tiles are counted and summed up; every piece and
// tile then finds its sequence by bisection, three times over the tiles: their blocks,
// their units' lengths, the units. A tile's blocks are divided into units of about
// `chunk` = total / target blocks' cost, at most a quarter more, and units are laid out longest
// first (by classes of length: atomics in LDS give the places inside a class, which no
// result depends on), so that the last ones to start are short.
__global__ __launch_bounds__(kPlanThreads) void k_kv_plan(const int32_t *__restrict__ cu,
                                                          const int32_t *__restrict__ pos,
                                                          KvSizes z, int tile, KvPlanLayout lay,
                                                          int64_t target,
                                                          int32_t *__restrict__ plan) {
  __shared__ int first_piece[kKvMaxSeqs + 1], first_tile[kKvMaxSeqs + 1];
  __shared__ int64_t tmp[kPlanThreads / 64];
  __shared__ int count[kBins], cursor[kBins], s_bad, s_parts, s_joins, s_longest;
  const int tid = threadIdx.x, G = z.Hq / z.Hkv, S = (int)z.S;
  if (tid == 0) {
    s_bad = 0x7fffffff;
    s_parts = s_joins = s_longest = 0;
  }
  if (tid < kBins) count[tid] = 0;
  __syncthreads();

  // ---- pieces and tiles of every sequence
  int64_t npieces = 0, ntiles = 0, total;
  for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int64_t p = 0, t = 0;
    if (s < S) {
      bool bad;
      const Seq q = sequence(cu, pos, z, s, bad);
      if (bad) atomicMin(&s_bad, s);
      if (q.len > 0) {
        p = (q.pos + q.len - 1) / kKvBlock - q.pos / kKvBlock + 1;
        t = ((int64_t)q.len * G + tile - 1) / tile;
      }
    }
    const int64_t fp = scan(p, tmp, total) + npieces;
    npieces += total;
    const int64_t ft = scan(t, tmp, total) + ntiles;
    ntiles += total;
    if (s < S) {
      first_piece[s] = (int)fp;
      first_tile[s] = (int)ft;
    }
  }
  // sequences that overlap in the step would have more than the plan holds
  const bool fits = npieces <= lay.pieces && ntiles <= lay.units - lay.parts;
  if (!fits) npieces = ntiles = 0;
  if (tid == 0) {
    first_piece[S] = (int)npieces;
    first_tile[S] = (int)ntiles;
  }
  __syncthreads();

  // ---- blocks of every tile
  int64_t mine = 0, blocks;
  int most = 0;
  for (int i = tid; i < ntiles; i += kPlanThreads) {
    const int s = owner(first_tile, S, i);
    bool bad;
    const Seq q = sequence(cu, pos, z, s, bad);
    int b0, b1;
    const int row0 = (i - first_tile[s]) * tile;
    tile_blocks(q, G, z.window, row0, tile, b0, b1);
    const int cost = (b1 - b0) * block_cost(q, G, tile, row0);
    mine += cost;
    most = max(most, cost);
  }
  atomicMax(&s_longest, most);
  scan(mine, tmp, blocks);
  int64_t chunk = (blocks + target - 1) / target;
  const int64_t least = kKvMinBlocks * (tile < kKvTileRows ? 1 : kKvTileCost);
  chunk = chunk < least ? least : chunk;
  if (lay.parts == 0) chunk = kKvTileCost * z.W;
  const int longest = (int)min(chunk + chunk / 4, (int64_t)s_longest);
  auto bin_of = [&](int len) {  // long units first (a part that may not be smaller is the longest)
    len = min(len, longest);
    return kBins - 1 - (int)((int64_t)len * (kBins - 1) / (longest > 0 ? longest : 1));
  };

  // ---- pieces
  KvPiece *pieces = reinterpret_cast<KvPiece *>(plan + lay.at_pieces);
  for (int i = tid; i < npieces; i += kPlanThreads) {
    const int s = owner(first_piece, S, i);
    bool bad;
    const Seq q = sequence(cu, pos, z, s, bad);
    const int blk = q.pos / kKvBlock + i - first_piece[s];
    const int from = max(q.pos, blk * kKvBlock), to = min(q.pos + q.len, (blk + 1) * kKvBlock);
    pieces[i] = KvPiece{s, blk, q.tok + from - q.pos, to - from, from - blk * kKvBlock, {0, 0, 0}};
  }

  // ---- units: places by length, then the units themselves
  KvUnit *units = reinterpret_cast<KvUnit *>(plan + lay.at_units);
  KvJoin *joins = reinterpret_cast<KvJoin *>(plan + lay.at_joins);
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = tid; i < ntiles; i += kPlanThreads) {
      const int s = owner(first_tile, S, i);
      bool bad;
      const Seq q = sequence(cu, pos, z, s, bad);
      const int row0 = (i - first_tile[s]) * tile;
      int b0, b1;
      tile_blocks(q, G, z.window, row0, tile, b0, b1);
      const int n = b1 - b0;
      const int64_t cost = (int64_t)n * block_cost(q, G, tile, row0);
      // (no more parts than the plan has room for: at least kKvMinBlocks blocks each)
      const int parts = (int)max((int64_t)1, min((cost + chunk - 1 - chunk / 4) / chunk,
                                                 (int64_t)(n + kKvMinBlocks - 1) / kKvMinBlocks));
      const int bin = bin_of((int)((cost + parts - 1) / parts));
      if (pass == 0) {
        atomicAdd(&count[bin], parts);
        continue;
      }
      int at = atomicAdd(&cursor[bin], parts), part = -1;
      if (parts > 1) {
        part = atomicAdd(&s_parts, parts);
        joins[atomicAdd(&s_joins, 1)] = KvJoin{q.tok, q.len, row0, part, parts, {0, 0, 0}};
      }
      for (int u = 0; u < parts; ++u)  // as even as whole blocks are
        units[at + u] = KvUnit{s, q.tok, q.len, q.pos, row0, b0 + (int)((int64_t)n * u / parts),
                               b0 + (int)((int64_t)n * (u + 1) / parts),
                               part < 0 ? -1 : part + u};
    }
    __syncthreads();
    if (pass == 0) {
      const int64_t at = scan(tid < kBins ? count[tid] : 0, tmp, total);
      if (tid < kBins) cursor[tid] = (int)at;
      if (tid == 0) plan[kKvUnits] = (int)total;
      __syncthreads();
    }
  }
  if (tid == 0) {
    plan[kKvInfo] = s_bad != 0x7fffffff ? s_bad + 1 : fits ? 0 : S + 1;
    plan[kKvPieces] = (int)npieces;
    plan[kKvJoins] = s_joins;
  }
}

// ------------------------------------------------------------- write and read

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// rint(v / s) for |v| <= 127 s: v times the reciprocal r is within 2^-16 of the
// quotient, so only values that near a half integer take the division.
__device__ __forceinline__ int code_of(float v, float s, float r) {
  const float t = v * r;
  float c = rintf(t);
  if (fabsf(t - c) > 0.5f - 0x1p-10f) c = rintf(v / s);
  return (int)clamp_code(c, -127.0f, 127.0f);
}
__device__ __forceinline__ int code_far(float v, float s) {
  return (int)clamp_code(rintf(v / s), -127.0f, 127.0f);
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *x, int64_t i, float (&v)[8]) {
  if constexpr (BF16) {
    const i32x4 d = *reinterpret_cast<const i32x4 *>(static_cast<const uint16_t *>(x) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float((uint32_t)d[e] << 16);
      v[2 * e + 1] = __uint_as_float((uint32_t)d[e] & 0xffff0000u);
    }
  } else {
    const float *p = static_cast<const float *>(x) + i;
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  }
}

// A thread's share of a page and head: tokens 4 jq .. 4 jq + 3, dims 8 c .. 8 c + 7.
// Codes lie as one dword (4 tokens) for each dim of V, 8 bytes (dims) for each token of K.
struct Share {
  int jq, c;
  __device__ Share() : jq(threadIdx.x & 15), c(threadIdx.x >> 4) {}
  __device__ int64_t k(int t) const { return (c >> 3) * 4096 + (4 * jq + t) * 64 + (c & 7) * 8; }
  __device__ int64_t v(int e) const { return (8 * c + e) * 64 + 4 * jq; }
};

// code[t] = the 8 codes of token t, one a byte of the two dwords, from either layout.
__device__ __forceinline__ void load_codes(const int8_t *p, bool isv, const Share &sh,
                                           uint32_t (&code)[4][2]) {
  if (!isv) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const i32x2 d = *reinterpret_cast<const i32x2 *>(p + sh.k(t));
      code[t][0] = (uint32_t)d[0];
      code[t][1] = (uint32_t)d[1];
    }
    return;
  }
  uint32_t d[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) d[e] = *reinterpret_cast<const uint32_t *>(p + sh.v(e));
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t r = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) r |= ((d[4 * w + e] >> (8 * t)) & 255u) << (8 * e);
      code[t][w] = r;
    }
}

__device__ __forceinline__ int code_at(const uint32_t (&code)[2], int e) {
  return (int)(int8_t)(code[e >> 2] >> (8 * (e & 3)));
}

// One workgroup of 2 DP threads a piece, kv head and array (blockIdx.y: K, V). The
// page is read only where codes have to be rounded anew, or to complete V's dwords.
// Bound by memory for whole pages (3 bytes a value), by its chain of loads (the piece, the
// page's number, its scale) for single tokens.
template <bool BF16>
__global__ __launch_bounds__(512) void k_kv_write(const void *__restrict__ k, int64_t krow,
                                                  const void *__restrict__ v, int64_t vrow,
                                                  KvCache c, const int32_t *__restrict__ table,
                                                  int64_t W, const int32_t *__restrict__ plan,
                                                  int64_t at_pieces) {
  const int i = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv;
  if (i >= plan[kKvPieces]) return;
  const KvPiece u = reinterpret_cast<const KvPiece *>(plan + at_pieces)[i];
  const int64_t page = table[u.seq * W + u.blk];
  if (page < 0 || page >= c.pages) return;
  const bool isv = blockIdx.y == 1;
  const void *x = isv ? v : k;
  const int64_t row = isv ? vrow : krow;
  float *scale = (isv ? c.vs : c.ks) + page * c.Hkv + h;
  int8_t *codes = (isv ? c.vq : c.kq) + (page * c.Hkv + h) * (kKvBlock * (int64_t)c.DP);
  const Share sh;
  const int end = u.off + u.n;
  const float old = u.off > 0 ? *scale : 0.0f;

  float f[4][8];
  uint32_t mx = 0;
  const bool dims = 8 * sh.c < c.D;  // whole eights: D is a multiple of 8
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int j = 4 * sh.jq + t;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[t][e] = 0.0f;
    if (dims && j >= u.off && j < end) {
      load8<BF16>(x, (u.tok + j - u.off) * row + (int64_t)h * c.D + 8 * sh.c, f[t]);
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = umax(mx, __float_as_uint(f[t][e]) & 0x7fffffffu);
    }
  }
  // the largest magnitude: bits order like magnitudes, a NaN above an infinity, so a page that
  // is given either gets a scale that is no number and restores none
  __shared__ uint32_t part[8];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = umax(mx, (uint32_t)__shfl_xor((int)mx, o));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = mx;
  __syncthreads();
  for (int w = 0; w < (int)blockDim.x >> 6; ++w) mx = umax(mx, part[w]);
  const uint32_t top = umax(__float_as_uint(__uint_as_float(mx) / 127.0f),
                            __float_as_uint(kKvMinScale));
  const float s = __uint_as_float(umax(__float_as_uint(old), top));
  const bool anew = u.off > 0 && __float_as_uint(s) != __float_as_uint(old);
  if (threadIdx.x == 0 && (u.off == 0 || anew)) *scale = s;

  const int from = anew ? 0 : u.off;  // tokens from .. end - 1 are written
  if (4 * sh.jq + 3 < from || 4 * sh.jq >= end) return;
  uint32_t code[4][2] = {};
  if (u.off > 0 && 4 * sh.jq < u.off && (anew || isv)) load_codes(codes, isv, sh, code);
  const bool near = s <= 0x1p100f;  // scales up to 2^100 have a normal reciprocal
  const float r = 1.0f / s;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int j = 4 * sh.jq + t;
    if (j >= end) {
      code[t][0] = code[t][1] = 0;
      continue;
    }
    if (j < from) continue;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x1 = j < u.off ? (float)code_at(code[t], e) * old : f[t][e];
      w[e >> 2] |= ((uint32_t)(near ? code_of(x1, s, r) : code_far(x1, s)) & 255u) << (8 * (e & 3));
    }
    code[t][0] = w[0];
    code[t][1] = w[1];
  }
  if (!isv) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int j = 4 * sh.jq + t;
      if (j >= from && j < end)
        *reinterpret_cast<i32x2 *>(codes + sh.k(t)) = i32x2{(int)code[t][0], (int)code[t][1]};
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t d = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) d |= ((uint32_t)code_at(code[t], e) & 255u) << (8 * t);
    *reinterpret_cast<uint32_t *>(codes + sh.v(e)) = d;
  }
}

template <bool BF16>
__global__ __launch_bounds__(512) void k_kv_read(KvCache c, const int32_t *__restrict__ table,
                                                 int64_t W, const int32_t *__restrict__ plan,
                                                 int64_t at_pieces, void *__restrict__ k,
                                                 void *__restrict__ v) {
  const int i = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv;
  if (i >= plan[kKvPieces]) return;
  const KvPiece u = reinterpret_cast<const KvPiece *>(plan + at_pieces)[i];
  const int64_t page = table[u.seq * W + u.blk];
  const bool live = page >= 0 && page < c.pages;
  const bool isv = blockIdx.y == 1;
  const int64_t at = live ? page * c.Hkv + h : 0;
  const int8_t *codes = (isv ? c.vq : c.kq) + at * (kKvBlock * (int64_t)c.DP);
  const Share sh;
  const int end = u.off + u.n;
  if (8 * sh.c >= c.D || 4 * sh.jq + 3 < u.off || 4 * sh.jq >= end) return;
  uint32_t code[4][2] = {};
  float s = 0.0f;
  if (live) {
    s = (isv ? c.vs : c.ks)[at];
    load_codes(codes, isv, sh, code);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int j = 4 * sh.jq + t;
    if (j < u.off || j >= end) continue;
    const int64_t o = ((int64_t)(u.tok + j - u.off) * c.Hkv + h) * c.D + 8 * sh.c;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)code_at(code[t], e) * s;
    if constexpr (BF16) {
      i32x4 d;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        d[e] = (int)((uint32_t)f32_to_bf16_rne(f[2 * e]) |
                     ((uint32_t)f32_to_bf16_rne(f[2 * e + 1]) << 16));
      *reinterpret_cast<i32x4 *>(static_cast<uint16_t *>(isv ? v : k) + o) = d;
    } else {
      float *p = static_cast<float *>(isv ? v : k) + o;
      *reinterpret_cast<f32x4 *>(p) = f32x4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f32x4 *>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
    }
  }
}

}  // namespace

hipError_t launch_kv_plan(const int32_t *cu, const int32_t *pos, const KvSizes &z, int32_t *plan,
                          hipStream_t st) {
  hipLaunchKernelGGL(k_kv_plan, dim3(1), dim3(kPlanThreads), 0, st, cu, pos, z, kv_tile_rows(z),
                     kv_plan_layout(z), kv_target(z), plan);
  return hipGetLastError();
}

hipError_t launch_kv_write(const void *k, int64_t krow, const void *v, int64_t vrow, bool bf16,
                           const KvCache &c, const int32_t *table, const KvSizes &z,
                           const int32_t *plan, hipStream_t st) {
  const KvPlanLayout lay = kv_plan_layout(z);
  if (!grid_fits(lay.pieces * c.Hkv, 2 * c.DP)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(bf16 ? k_kv_write<true> : k_kv_write<false>,
                     dim3((unsigned)(lay.pieces * c.Hkv), 2), dim3(2 * c.DP), 0, st, k, krow, v,
                     vrow, c, table, z.W, plan, lay.at_pieces);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &c, const int32_t *table, const KvSizes &z,
                          const int32_t *plan, void *k, void *v, bool bf16, hipStream_t st) {
  const KvPlanLayout lay = kv_plan_layout(z);
  if (!grid_fits(lay.pieces * c.Hkv, 2 * c.DP)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(bf16 ? k_kv_read<true> : k_kv_read<false>,
                     dim3((unsigned)(lay.pieces * c.Hkv), 2), dim3(2 * c.DP), 0, st, c, table, z.W,
                     plan, lay.at_pieces, k, v);
  return hipGetLastError();
}

}  // namespace aql
