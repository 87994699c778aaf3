// A paged 8-bit KV cache and attention over it (internal to libaql.so): the cache's
// layout, a step's plan, and the launchers. Arguments are validated by the C ABI layer.
#pragma once

#include "common.h"

namespace aql {

// ------------------------------------------------------------------ the cache
//
// Pages of kKvBlock tokens. Head sizes are padded with zero codes to a multiple of 64 (DP).
// Of page p and kv head h, at (p Hkv + h) kKvBlock DP bytes of either array:
//   K  [DP / 64][64 tokens][64 dims]   a 16-byte piece of a token is what a lane of
//   V  [DP][64 tokens]                 a matrix instruction contracts over
// so that every load of the attention kernels is a whole KiB: for scores the
// contraction runs over dims, for outputs over tokens. One scale for each page, head and array.
constexpr int kKvBlock = 64;
constexpr int kKvMaxHead = 256;
constexpr int64_t kKvMaxSeqs = 4096;
constexpr int64_t kKvMaxTokens = 1 << 20;   // of a step
constexpr int64_t kKvMaxBlocks = 1 << 20;   // pages of a sequence
constexpr float kKvMinScale = 0x1p-64f;

struct KvCache {
  int8_t *kq, *vq;
  float *ks, *vs;
  int64_t pages;
  int Hkv, D, DP;
};
constexpr int kv_padded(int64_t D) { return (int)((D + 63) / 64 * 64); }

// ------------------------------------------------------------------- the plan
//
// Device buffer of int32, made once a step for all layers: a header, then units of
// work as structs of 8 words.

// New tokens of one page: rows tok .. tok + n - 1 of the step at places off ..
// off + n - 1 of block blk of sequence seq.
struct KvPiece {
  int32_t seq, blk, tok, n, off, pad[3];
};

// Rows row0 .. row0 + tile - 1 of a sequence (row i: token i / G, head i % G of a kv
// head's G) against blocks b0 .. b1 - 1. The sequence's first token is row tok of the
// step and has position pos; it has len tokens. part: where the partial results
// go, -1: the only unit of its rows, which writes the outputs.
struct KvUnit {
  int32_t seq, tok, len, pos, row0, b0, b1, part;
};

// Rows whose blocks are spread over `parts` units, from partial result `part` on. (pad: the
// plan's own.)
struct KvJoin {
  int32_t tok, len, row0, part, parts, pad[3];
};

enum : int { kKvInfo = 0, kKvPieces = 1, kKvUnits = 2, kKvJoins = 3, kKvHeader = 16 };

struct KvSizes {
  int64_t T, S, W;    // rows of the step, sequences, blocks of the table's rows
  int64_t most;       // most new tokens of a sequence
  int Hq, Hkv;
  int64_t window;     // 0: none
};

// Rows of a unit, by the most that any sequence can have. Up to 32 a block's codes go
// straight to registers and are bound by memory; past that a block serves so many rows
// that widening it once, into LDS, pays (one sequence of 64 rows for 8 kv heads of 128, 20, 300, 30000
// tokens, us: streamed in units of 64 rows 13.6, 17.6, 71.7; tiles 7.2, 12.8, 47.7; of 32 rows, 300 and
// 1500 tokens: streamed 10.5, 11.2; tiles 12.5, 13.0).
constexpr int kKvTileRows = 128;
// Units of at most so many rows stream also in a step of tiles; there a block of theirs
// costs about a quarter of a tile's.
constexpr int kKvFewRows = 16;
constexpr int kKvTileCost = 4;
constexpr int kv_tile_rows(const KvSizes &z) {
  const int64_t rows = z.most * (z.Hq / z.Hkv);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : kKvTileRows;
}
// Units that a step is divided into where there is enough to divide (over all kv heads),
// and the fewest blocks of one. Streams: three workgroups a CU (64 requests of up to 8192
// tokens, one of 131071, us: 512 units 93.9, 50.2; 768 88.2, 50.8; 1024 90.2, 52.1). Tiles:
// fewer than the two a CU that run at once, as each tile's parts are rounded up (16 requests
// and a chunk of 509 tokens behind 6007; 256 behind 16000: 384 units 91, 105; 448 91, 94; 512 107,
// 89; the first comes to 528 units all the same, the longest 1.29 of their mean cost).
constexpr int64_t kv_target(const KvSizes &z) {
  const int64_t t = (kv_tile_rows(z) == kKvTileRows ? 448 : 768) / z.Hkv;
  return t > 1 ? t : 1;
}
constexpr int64_t kKvMinBlocks = 4;
// Tables of at most so many blocks leave nothing to divide: a second launch that joins the parts
// costs what 4 waves take for two more blocks each (one request of 334 tokens, 15 heads
// of 64 over 5: 5.1 us in one unit, 7.0 divided; of 1024 tokens 8.1, 7.1). It is the table's
// width that counts, which the host knows: with wider tables the same request is divided, and
// one of 31 tokens, which is not, has the second launch all the same (5.8 us against 4.3).
constexpr int64_t kKvWhole = 8;

struct KvPlanLayout {
  int64_t pieces, units, joins;        // most of each
  int64_t parts;                       // most partial results (of each kv head)
  int64_t tiles;                       // most tiles
  int64_t at_pieces, at_units, at_joins, total;  // in words
};
constexpr KvPlanLayout kv_plan_layout(const KvSizes &z) {
  const int64_t live = z.S < z.T ? z.S : z.T;  // sequences with tokens
  const int64_t G = z.Hq / z.Hkv;
  const int64_t tiles = z.T * G / kv_tile_rows(z) + live;
  const int64_t target = kv_target(z);
  const int64_t most = z.W <= kKvWhole ? 1 : (z.W + kKvMinBlocks - 1) / kKvMinBlocks;  // of a tile
  KvPlanLayout p{};
  p.pieces = z.T / kKvBlock + 2 * live;
  // a unit has at least total / target blocks, but for the last one of a tile
  p.parts = most < 2 ? 0 : 2 * target < tiles * most ? 2 * target : tiles * most;
  p.tiles = tiles;
  p.units = tiles + p.parts;
  p.joins = p.parts / 2 < tiles ? p.parts / 2 : tiles;
  p.at_pieces = kKvHeader;
  p.at_units = p.at_pieces + 8 * p.pieces;
  p.at_joins = p.at_units + 8 * p.units;
  p.total = p.at_joins + 8 * p.joins;
  return p;
}

hipError_t launch_kv_plan(const int32_t *cu, const int32_t *pos, const KvSizes &z, int32_t *plan,
                          hipStream_t st);

// ------------------------------------------------------------- cache and attention

// k, v: [T, Hkv, D], rows ks and vs elements apart.
hipError_t launch_kv_write(const void *k, int64_t krow, const void *v, int64_t vrow, bool bf16,
                           const KvCache &c, const int32_t *table, const KvSizes &z,
                           const int32_t *plan, hipStream_t st);
hipError_t launch_kv_read(const KvCache &c, const int32_t *table, const KvSizes &z,
                          const int32_t *plan, void *k, void *v, bool bf16, hipStream_t st);

// Bytes of an attention call's partial results.
size_t kv_attention_bytes(const KvSizes &z, int DP);
hipError_t launch_kv_attention(const uint16_t *q, int64_t qrow, float sm_scale, const KvCache &c,
                               const int32_t *table, const KvSizes &z, const int32_t *plan,
                               uint16_t *y, float *lse, void *ws, hipStream_t st);

}  // namespace aql
