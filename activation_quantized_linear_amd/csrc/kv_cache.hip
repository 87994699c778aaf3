// A paged 8-bit KV cache: a step's plan, quantising new tokens into their pages, and
// reading them back.
//
// Of a page and kv head, K and V each:  s = max(max |x| / 127, 2^-64),
// code = clamp(rint(x / s), -127, 127), value = code s. A page that a write begins takes
// its scale from the new tokens; behind live tokens the scale only grows, and where
// it does their codes become clamp(rint((code s) / s')), each product and quotient
// rounded once to binary32.
#include <type_traits>

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
// tile then finds its sequence by bisection, with three passes over the tiles: their blocks,
// their units' lengths, the units. Bound by latency (one request 7 us, 27 of them 11, 64 divided
// ones 16). A tile's blocks are divided into units of about `chunk` = total / target blocks'
// cost (and kKvMinBlocks blocks), at most a quarter more, and units are laid out longest
// first (by classes of length: atomics in LDS give the places inside a class, which no result
// depends on), so that the last ones to start are short.
__global__ __launch_bounds__(kPlanThreads) void k_kv_plan(const int32_t *__restrict__ cu,
                                                          const int32_t *__restrict__ pos,
                                                          KvSizes z, int tile, KvPlanLayout lay,
                                                          int64_t target,
                                                          int32_t *__restrict__ plan) {
  __shared__ int first_piece[kKvMaxSeqs + 1], first_tile[kKvMaxSeqs + 1];
  __shared__ int64_t tmp[kPlanThreads / 64];
  __shared__ int count[kBins], cursor[kBins], s_bad, s_parts, s_joins, s_longest;
  __shared__ unsigned long long s_blocks;
  const int tid = threadIdx.x, G = z.Hq / z.Hkv, S = (int)z.S;
  if (tid == 0) {
    s_bad = 0x7fffffff;
    s_parts = s_joins = s_longest = 0;
    s_blocks = 0;
  }
  if (tid < kBins) count[tid] = 0;
  __syncthreads();

  // ---- pieces and tiles of every sequence, summed up as the halves of one number
  int64_t npieces = 0, ntiles = 0;
  for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int64_t both = 0, total;
    if (s < S) {
      bool bad;
      const Seq q = sequence(cu, pos, z, s, bad);
      if (bad) atomicMin(&s_bad, s);
      if (q.len > 0)
        both = (int64_t)((q.pos + q.len - 1) / kKvBlock - q.pos / kKvBlock + 1) << 32 |
               ((int64_t)q.len * G + tile - 1) / tile;
    }
    const int64_t at = scan(both, tmp, total);
    if (s < S) {
      first_piece[s] = (int)(npieces + (at >> 32));
      first_tile[s] = (int)(ntiles + (at & 0xffffffff));
    }
    npieces += total >> 32;
    ntiles += total & 0xffffffff;
  }
  // sequences that overlap in the step would have more than the plan holds
  const bool fits = npieces <= lay.pieces && ntiles <= lay.units - lay.parts;
  if (!fits) npieces = ntiles = 0;
  if (tid == 0) {
    first_piece[S] = (int)npieces;
    first_tile[S] = (int)ntiles;
  }
  __syncthreads();

  // ---- blocks of every tile; a thread keeps its first one's numbers
  struct Tile {
    Seq q;
    int s, row0, b0, b1, cost;
  };
  auto tile_of = [&](int i) {
    Tile t;
    t.s = owner(first_tile, S, i);
    bool bad;
    t.q = sequence(cu, pos, z, t.s, bad);
    t.row0 = (i - first_tile[t.s]) * tile;
    tile_blocks(t.q, G, z.window, t.row0, tile, t.b0, t.b1);
    t.cost = (t.b1 - t.b0) * block_cost(t.q, G, tile, t.row0);
    return t;
  };
  Tile own{};
  if (tid < ntiles) own = tile_of(tid);
  int64_t mine = own.cost;
  int most = own.cost;
  for (int i = tid + kPlanThreads; i < ntiles; i += kPlanThreads) {
    const Tile t = tile_of(i);
    mine += t.cost;
    most = max(most, t.cost);
  }
  if (most > 0) {
    atomicMax(&s_longest, most);
    atomicAdd(&s_blocks, (unsigned long long)mine);
  }
  __syncthreads();
  const int64_t blocks = (int64_t)s_blocks;
  const int64_t share = (blocks + target - 1) / target;
  auto chunk_of = [&](int cost) -> int64_t {  // of a tile whose blocks cost so much each
    if (lay.parts == 0) return kKvTileCost * z.W;
    return share < kKvMinBlocks * cost ? kKvMinBlocks * cost : share;
  };
  const int64_t widest = chunk_of(tile < kKvTileRows ? 1 : kKvTileCost);
  const int longest = (int)min(widest + widest / 4, (int64_t)s_longest);
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
      const Tile t = i == tid ? own : tile_of(i);
      const Seq &q = t.q;
      const int s = t.s, row0 = t.row0, b0 = t.b0, n = t.b1 - t.b0;
      const int64_t cost = t.cost, chunk = chunk_of(block_cost(q, G, tile, row0));
      // (no more parts than the plan has room for: at least kKvMinBlocks blocks each)
      const int parts = (int)max((int64_t)1, min((cost + chunk - 1 - chunk / 4) / chunk,
                                                 (int64_t)(n + kKvMinBlocks - 1) / kKvMinBlocks));
      const int bin = bin_of((int)((cost + parts - 1) / parts));
      if (pass == 0) {
        atomicAdd(&count[bin], parts);
        continue;
      }
      const int at = atomicAdd(&cursor[bin], parts);
      if (parts > 1) {  // (its units below; the join keeps their place and the tile meanwhile)
        const int part = atomicAdd(&s_parts, parts);
        joins[atomicAdd(&s_joins, 1)] = KvJoin{q.tok, q.len, row0, part, parts, {at, i, 0}};
      } else {
        units[at] = KvUnit{s, q.tok, q.len, q.pos, row0, b0, b0 + n, -1};
      }
    }
    __syncthreads();
    if (pass == 0) {
      int64_t total;
      const int64_t at = scan(tid < kBins ? count[tid] : 0, tmp, total);
      if (tid < kBins) cursor[tid] = (int)at;
      if (tid == 0) plan[kKvUnits] = (int)total;
      __syncthreads();
    }
  }
  // a wave a divided tile, a lane a part: as even as whole blocks are
  for (int j = tid >> 6; j < s_joins; j += kPlanThreads / 64) {
    const KvJoin w = joins[j];
    const Tile t = tile_of(w.pad[1]);
    const uint32_t n = (uint32_t)(t.b1 - t.b0), parts = (uint32_t)w.parts;  // n parts < 2^31
    for (uint32_t u = tid & 63; u < parts; u += 64)
      units[w.pad[0] + u] = KvUnit{t.s, t.q.tok, t.q.len, t.q.pos, t.row0,
                                   t.b0 + (int)(n * u / parts), t.b0 + (int)(n * (u + 1) / parts),
                                   w.part + (int)u};
  }
  if (tid == 0) {
    // (overlapping sequences come with one whose rows are not ascending: nothing being done goes first)
    plan[kKvInfo] = !fits ? S + 1 : s_bad != 0x7fffffff ? s_bad + 1 : 0;
    plan[kKvPieces] = (int)npieces;
    plan[kKvJoins] = s_joins;
  }
}

// ------------------------------------------------------------- write and read

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// rint(v / s) for |v| <= 127 s: v times the reciprocal r is within 2^-16 of the
// quotient, so only values near a half integer take the division. (From 2^-10 on, which
// one value in 512 is, and so some value of one wave in eight.)
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

// A thread's share of a page and head: tokens 4 jq .. 4 jq + 3, dims 8 c .. 8 c + 7. Consecutive
// lanes take consecutive dims, so that rows of K and V pass as whole runs (with
// consecutive tokens, 64 bytes of 16 rows a wave, writing and reading 8881 tokens of 8 heads of 128
// back took 32.6 us, 28.5 with runs). Codes: 8 bytes of each token of K; V's page is transposed, its tokens
// contiguous, so its codes change sides in LDS and pass in 16-byte pieces.
template <int C>
struct Share {
  static constexpr int NC = 8 * C, THREADS = 16 * NC;
  static constexpr int ROW = 17;  // dwords of a dim's 64 codes in LDS
  int jq, c;
  __device__ Share() : jq(threadIdx.x / NC), c(threadIdx.x % NC) {}
  __device__ int k(int t) const { return (c >> 3) * 4096 + (4 * jq + t) * 64 + (c & 7) * 8; }
  __device__ int lds(int e) const { return (8 * c + e) * ROW + jq; }
};

// w[e] = the codes of dim e, one token a byte, of code[t] = those of token t, one dim a byte.
__device__ __forceinline__ void transpose(const uint32_t (&code)[4][2], uint32_t (&w)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) w[e] |= (code[t][e >> 2] >> (8 * (e & 3)) & 255u) << (8 * t);
  }
}
__device__ __forceinline__ void transpose(const uint32_t (&w)[8], uint32_t (&code)[4][2]) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      code[t][h] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) code[t][h] |= (w[4 * h + e] >> (8 * t) & 255u) << (8 * e);
    }
}

__device__ __forceinline__ int code_at(const uint32_t (&code)[2], int e) {
  return (int)(int8_t)(code[e >> 2] >> (8 * (e & 3)));
}

// Codes of a page and head as they lie, code[t] those of token 4 jq + t.
template <int C>
__device__ __forceinline__ void load_codes(const int8_t *p, bool isv, const Share<C> &sh,
                                           uint32_t *lds, uint32_t (&code)[4][2]) {
  if (!isv) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const i32x2 d = *reinterpret_cast<const i32x2 *>(p + sh.k(t));
      code[t][0] = (uint32_t)d[0];
      code[t][1] = (uint32_t)d[1];
    }
    return;
  }
  i32x4 d[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    d[i] = *reinterpret_cast<const i32x4 *>(p + 16 * (threadIdx.x + Share<C>::THREADS * i));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int piece = threadIdx.x + Share<C>::THREADS * i;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      lds[(piece >> 2) * Share<C>::ROW + 4 * (piece & 3) + e] = (uint32_t)d[i][e];
  }
  __syncthreads();
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = lds[sh.lds(e)];
  transpose(w, code);
}

// One workgroup a piece, kv head and array (blockIdx.y: K, V). The page is read only where
// codes have to be rounded anew, or to complete V's 16-byte pieces. Bound by memory for
// whole pages (3 bytes a value), by its chain of loads (the piece, the page's number, its
// scale) for single tokens.
template <bool BF16, int C>
__global__ __launch_bounds__(Share<C>::THREADS) void k_kv_write(
    const void *__restrict__ k, int64_t krow, const void *__restrict__ v, int64_t vrow, KvCache c,
    const int32_t *__restrict__ table, int64_t W, const int32_t *__restrict__ plan,
    int64_t at_pieces) {
  __shared__ uint32_t lds[64 * C * Share<C>::ROW];
  __shared__ uint32_t part[8];
  const int i = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv;
  if (i >= plan[kKvPieces]) return;
  const KvPiece u = reinterpret_cast<const KvPiece *>(plan + at_pieces)[i];
  const int64_t page = table[u.seq * W + u.blk];
  const bool isv = blockIdx.y == 1;
  const void *x = isv ? v : k;
  const int64_t row = isv ? vrow : krow;
  const Share<C> sh;
  const int end = u.off + u.n;

  float f[4][8];
  uint32_t mx = 0;
  const bool dims = 8 * sh.c < c.D;  // whole eights: D is a multiple of 8
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int j = 4 * sh.jq + t;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[t][e] = 0.0f;
    if (dims && j >= u.off && j < end)
      load8<BF16>(x, (u.tok + j - u.off) * row + (int64_t)h * c.D + 8 * sh.c, f[t]);
  }
  if (page < 0 || page >= c.pages) return;  // (the tokens' loads are on their way meanwhile)
  float *scale = (isv ? c.vs : c.ks) + page * c.Hkv + h;
  int8_t *codes = (isv ? c.vq : c.kq) + (page * c.Hkv + h) * (kKvBlock * 64 * C);
  const float old = u.off > 0 ? *scale : 0.0f;
  // the largest magnitude: bits order like magnitudes, a NaN above an infinity, so a page that
  // is given either gets a scale that is no number and restores none
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = umax(mx, __float_as_uint(f[t][e]) & 0x7fffffffu);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = umax(mx, (uint32_t)__shfl_xor((int)mx, o));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = mx;
  __syncthreads();
  for (int w = 0; w < Share<C>::THREADS / 64; ++w) mx = umax(mx, part[w]);
  const uint32_t top = umax(__float_as_uint(__uint_as_float(mx) / 127.0f),
                            __float_as_uint(kKvMinScale));
  const float s = __uint_as_float(umax(__float_as_uint(old), top));
  const bool anew = u.off > 0 && __float_as_uint(s) != __float_as_uint(old);
  if (threadIdx.x == 0 && (u.off == 0 || anew)) *scale = s;

  const int from = anew ? 0 : u.off;  // tokens from .. end - 1 are written
  uint32_t code[4][2] = {};
  if (anew) {  // (uniform over the workgroup)
    load_codes(codes, isv, sh, lds, code);
    if (isv) __syncthreads();
  }
  const auto codes_of = [&](auto &&one) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int j = 4 * sh.jq + t;
      uint32_t w[2] = {0, 0};
      if (j >= from && j < end) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x1 = j < u.off ? (float)code_at(code[t], e) * old : f[t][e];
          w[e >> 2] |= ((uint32_t)one(x1) & 255u) << (8 * (e & 3));
        }
        if (!isv) *reinterpret_cast<i32x2 *>(codes + sh.k(t)) = i32x2{(int)w[0], (int)w[1]};
      }
      code[t][0] = w[0];
      code[t][1] = w[1];
    }
  };
  if (s <= 0x1p100f) {  // scales up to 2^100 have a normal reciprocal
    const float r = 1.0f / s;
    codes_of([&](float x1) { return code_of(x1, s, r); });
  } else {
    codes_of([&](float x1) { return code_far(x1, s); });
  }
  if (!isv) return;
  uint32_t w[8];
  transpose(code, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) lds[sh.lds(e)] = w[e];
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {  // 16 tokens of a dim; those before `from` stay
    const int piece = threadIdx.x + Share<C>::THREADS * q, t0 = 16 * (piece & 3);
    if (t0 + 16 <= from || t0 >= end) continue;
    i32x4 d, *to = reinterpret_cast<i32x4 *>(codes + 16 * piece);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = (int)lds[(piece >> 2) * Share<C>::ROW + (piece & 3) * 4 + e];
    if (t0 < from) {
      const i32x4 was = *to;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int keep = min(max(from - t0 - 4 * e, 0), 4);  // bytes
        const uint32_t mask = keep == 4 ? 0xffffffffu : (1u << (8 * keep)) - 1u;
        d[e] = (int)(((uint32_t)was[e] & mask) | ((uint32_t)d[e] & ~mask));
      }
    }
    *to = d;
  }
}

template <bool BF16, int C>
__global__ __launch_bounds__(Share<C>::THREADS) void k_kv_read(
    KvCache c, const int32_t *__restrict__ table, int64_t W, const int32_t *__restrict__ plan,
    int64_t at_pieces, void *__restrict__ k, void *__restrict__ v) {
  __shared__ uint32_t lds[64 * C * Share<C>::ROW];
  const int i = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv;
  if (i >= plan[kKvPieces]) return;
  const KvPiece u = reinterpret_cast<const KvPiece *>(plan + at_pieces)[i];
  const int64_t page = table[u.seq * W + u.blk];
  const bool live = page >= 0 && page < c.pages;
  const bool isv = blockIdx.y == 1;
  const int64_t at = live ? page * c.Hkv + h : 0;
  const Share<C> sh;
  const int end = u.off + u.n;
  uint32_t code[4][2] = {};
  float s = 0.0f;
  if (live) {  // (uniform over the workgroup)
    s = (isv ? c.vs : c.ks)[at];
    load_codes((isv ? c.vq : c.kq) + at * (kKvBlock * 64 * C), isv, sh, lds, code);
  }
  if (8 * sh.c >= c.D) return;
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

template <bool BF16, int C>
void launch_write(unsigned grid, hipStream_t st, const void *k, int64_t krow, const void *v,
                  int64_t vrow, const KvCache &c, const int32_t *table, int64_t W,
                  const int32_t *plan, int64_t at) {
  hipLaunchKernelGGL((k_kv_write<BF16, C>), dim3(grid, 2), dim3(Share<C>::THREADS), 0, st, k, krow,
                     v, vrow, c, table, W, plan, at);
}
template <bool BF16, int C>
void launch_read(unsigned grid, hipStream_t st, const KvCache &c, const int32_t *table, int64_t W,
                 const int32_t *plan, int64_t at, void *k, void *v) {
  hipLaunchKernelGGL((k_kv_read<BF16, C>), dim3(grid, 2), dim3(Share<C>::THREADS), 0, st, c, table,
                     W, plan, at, k, v);
}

// f(bool constant, int constant) for the type and the head's slices of 64.
template <class F>
void dispatch(bool bf16, int slices, F &&f) {
  const auto by_type = [&](auto c) {
    if (bf16) f(std::true_type{}, c);
    else f(std::false_type{}, c);
  };
  switch (slices) {
    case 1: by_type(std::integral_constant<int, 1>{}); break;
    case 2: by_type(std::integral_constant<int, 2>{}); break;
    case 3: by_type(std::integral_constant<int, 3>{}); break;
    default: by_type(std::integral_constant<int, 4>{}); break;
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
  dispatch(bf16, c.DP / 64, [&](auto t, auto n) {
    launch_write<decltype(t)::value, decltype(n)::value>((unsigned)(lay.pieces * c.Hkv), st, k, krow,
                                                         v, vrow, c, table, z.W, plan, lay.at_pieces);
  });
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &c, const int32_t *table, const KvSizes &z,
                          const int32_t *plan, void *k, void *v, bool bf16, hipStream_t st) {
  const KvPlanLayout lay = kv_plan_layout(z);
  if (!grid_fits(lay.pieces * c.Hkv, 2 * c.DP)) return hipErrorInvalidConfiguration;
  dispatch(bf16, c.DP / 64, [&](auto t, auto n) {
    launch_read<decltype(t)::value, decltype(n)::value>((unsigned)(lay.pieces * c.Hkv), st, c, table,
                                                        z.W, plan, lay.at_pieces, k, v);
  });
  return hipGetLastError();
}

}  // namespace aql
