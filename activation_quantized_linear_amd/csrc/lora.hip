// Low-rank adapters beside the int8 linear: the batch plan, the shrink
// products (x onto an adapter's A, dy onto its B) and the weight gradients.
//
//   h[m, j]     = alpha[a] sum_k x[m, k] A_a[j, k]            a = idx[m]
//   u[m, j]     = alpha[a] sum_n dy[m, n] B_a[n, j]
//   dB_a[n, j]  = sum_{m in a} dy[m, n] h[m, j]
//   dA_a[j, k]  = sum_{m in a} u[m, j] xq[m, k] xs[m, k / 128]
//
// h and u are float32 [M, R]; the expanding products h B^T and u A are added in
// the epilogues of the projection's own kernels (lora.h), so neither y nor dx
// makes a second trip through memory. All products run on the bf16 matrix
// cores with float32 accumulation (or as float32 FMAs of exact bf16 products);
// float32 operands are split into bf16 parts that add up to them.
// Every sum has one order, so results repeat bit for bit.
#include "lora.h"

#include "ckpt.h"
#include "w8a16_dgrad.h"

namespace aql {
namespace {

// ------------------------------------------------------------------ the plan

// A counting sort of the rows by adapter, by one workgroup: LDS histogram (its
// atomics count, so their order does not matter), tile offsets by a scan over
// the adapters, then chunks of 1024 rows in order. Inside a chunk a row's rank
// is the number of equal rows before it in its wave (ballots) plus the counts
// of the waves before (a byte table), so rows keep their order in a segment.
// One launch a batch, for all its layers: bound by its barriers and round trips
// (M = 500: 6.6 us, M = 2048: 8.4, 17 with 64 adapters at random), which one workgroup
// keeps few.
__global__ __launch_bounds__(1024) void k_lora_plan(const int32_t *__restrict__ idx, int64_t M,
                                                    int64_t L, int32_t *__restrict__ plan) {
  constexpr int NB = kLoraMaxAdapters + 1;  // the last bin: rows without an adapter
  __shared__ int next[NB];                  // counts, then the next free position of a bin
  __shared__ int scan[1024];
  __shared__ int total;
  __shared__ uint8_t cnt[16][NB + 3];
  const LoraPlanLayout p = lora_plan_layout(M, L);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nb = (int)L + 1;
  for (int b = tid; b < nb; b += 1024) next[b] = 0;
  for (int b = tid; b < 16 * (NB + 3); b += 1024) (&cnt[0][0])[b] = 0;
  __syncthreads();
  auto bin_of = [&](int64_t m) {
    const int a = idx[m];
    return a >= 0 && a < L ? a : (int)L;
  };
  for (int64_t m = tid; m < M; m += 1024) {
    const int b = bin_of(m);
    plan[p.idx + m] = b < L ? b : -1;
    atomicAdd(&next[b], 1);
  }
  __syncthreads();
  // tiles of bins 0 .. L - 1, scanned; bin L (at most 1025 bins) comes last
  const int mine = tid < nb && tid < 1024 ? (next[tid] + kLoraTile - 1) / kLoraTile : 0;
  scan[tid] = mine;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int v = tid >= o ? scan[tid - o] : 0;
    __syncthreads();
    scan[tid] += v;
    __syncthreads();
  }
  const int before = scan[tid] - mine;
  if (tid == 0) {
    const int all = scan[1023];
    total = nb > 1024 ? all + (next[1024] + kLoraTile - 1) / kLoraTile : all;
    if (nb > 1024) {  // L = 1024: the bin past the scan
      plan[p.first + 1024] = all;
      next[1024] = all * kLoraTile;
    }
  }
  __syncthreads();
  if (tid < nb && tid < 1024) {
    plan[p.first + tid] = before;
    next[tid] = before * kLoraTile;
  }
  for (int64_t gr = wave; gr * kLoraGroup < M; gr += 16) {  // a wave a group
    const int64_t m = gr * kLoraGroup + lane;
    const int v0 = m < M ? bin_of(m) : (int)L, v1 = m + 64 < M ? bin_of(m + 64) : (int)L;
    int n = 0;
    for (int prev = -1; n <= kLoraFew; ++n) {
      int least = v0 > prev ? v0 : (int)L;
      least = v1 > prev && v1 < least ? v1 : least;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int other = __shfl_xor(least, o);
        least = other < least ? other : least;
      }
      if (least == (int)L) break;
      prev = least;
    }
    if (lane == 0) plan[p.mixed + gr] = n > kLoraFew;
  }
  for (int64_t t = total + tid; t < p.tiles; t += 1024) plan[p.owner + t] = -2;
  for (int64_t i = tid; i < p.tiles * kLoraTile; i += 1024) plan[p.perm + i] = -1;
  if (tid == 0) plan[0] = total;
  __threadfence_block();
  __syncthreads();
  for (int64_t m0 = 0; m0 < M; m0 += 1024) {
    const int64_t m = m0 + tid;
    const bool live = m < M;
    const int b = live ? bin_of(m) : -1;
    uint64_t left = __ballot(live);
    int rank = 0;
    while (left) {
      const int lead = __ffsll((unsigned long long)left) - 1;
      const int bb = __shfl(b, lead);
      const uint64_t same = __ballot(b == bb);
      if (b == bb) rank = __popcll(same & ((1ull << lane) - 1));
      if (lane == lead) cnt[wave][bb] = (uint8_t)__popcll(same);
      left &= ~same;
    }
    __syncthreads();
    if (live) {
      int pos = next[b] + rank;
      for (int w = 0; w < wave; ++w) pos += cnt[w][b];
      plan[p.perm + pos] = (int32_t)m;
      if (pos % kLoraTile == 0) plan[p.owner + pos / kLoraTile] = b < L ? b : -1;
    }
    __syncthreads();
    for (int c = tid; c < nb; c += 1024) {
      int sum = 0;
      for (int w = 0; w < 16; ++w) {
        sum += cnt[w][c];
        cnt[w][c] = 0;
      }
      next[c] += sum;
    }
    __syncthreads();
  }
}

// --------------------------------------------------- shrink, streaming form

template <int J>
__global__ __launch_bounds__(256) void k_lora_shrink_rows(
    const uint16_t *__restrict__ x, int64_t K, const uint16_t *__restrict__ A,
    const float *__restrict__ alpha, int R, const int32_t *__restrict__ idx,
    float *__restrict__ h) {
  __shared__ float red[4 * J];
  lora_shrink_rows<J>(x, K, A, alpha, R, idx, h, blockIdx.y, blockIdx.x * J, red);
}

// ------------------------------------------------------- shrink, tiled form

// A workgroup of W waves takes NT tiles of the plan (16 rows each, mostly of one
// adapter), 16 ranks and one of several ranges of the contraction; its waves
// take steps of 128 in turn and meet in LDS. What it costs is round trips to
// memory (about 1.3 us each with the data in HBM), so all loads of a step are out
// at once, and a CU draws little more than its 1/256 of the memory's rate, so
// what each workgroup reads counts. Two forms:
//  * NT = 4, W = 4, ranges of about one step a wave: 64 rows share a read of the
//    16 ranks (with 16 rows the adapter's bytes equal the rows'), and float32
//    partial sums in sorted order are added in order by k_lora_shrink_sum;
//  * NT = 1, W = 16 over the whole of a short contraction: one launch.
// (x onto A at M = 500, K = 4096, R = 64: 10.4 us; dy onto B at M = 2048, N = 14336, R = 16:
// 15 + 4 us, 32 + 5 with dy's scaling beside it, 59 MB read and written.)
// Operands go from memory to the MFMA registers as they lie: x and A have the
// contraction contiguous. KMAJOR: the adapter matrix is [C, R] (dy onto B); each
// wave then passes its step's 32 x 16 blocks through its own LDS slot and reads
// them back transposed.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kU = 4;           // matrix instructions of a step
constexpr int kStep = 32 * kU;  // of the contraction, per wave

// The scaling's part of a launch: none, or dgrad_scale_row<NI> in the workgroups
// behind the shrink's, W / 4 rows each.
struct NoScale {
  static constexpr bool on = false;
  __device__ void row(int64_t, int, float *) const {}
};
template <int NI>
struct WithScale {
  static constexpr bool on = true;
  DgradScale a;
  __device__ void row(int64_t m, int t, float *red) const { dgrad_scale_row<NI>(a, m, t, red); }
};

template <int NT, int W, bool KMAJOR, class SC>
__global__ __launch_bounds__(64 * W) void k_lora_shrink(
    const uint16_t *__restrict__ x, int64_t C, const uint16_t *__restrict__ A,
    const float *__restrict__ alpha, int R, int64_t M, int64_t L,
    const int32_t *__restrict__ plan, float *__restrict__ h, float *__restrict__ part,
    int64_t range, int tiles, int ranks, int shrink_blocks, SC sc) {
  constexpr int SLOT = (KMAJOR && kU * 1024 > NT * 1024) ? kU * 1024 : NT * 1024;  // a wave's
  __shared__ __attribute__((aligned(16))) char smem[W * SLOT];
  if constexpr (SC::on) {
    if ((int)blockIdx.x >= shrink_blocks) {
      const int64_t m = (int64_t)(blockIdx.x - shrink_blocks) * (W / 4) + threadIdx.x / 256;
      sc.row(m, threadIdx.x % 256, reinterpret_cast<float *>(smem));
      return;
    }
  }
  const LoraPlanLayout p = lora_plan_layout(M, L);
  // the workgroup's first tile, first rank and range
  const int bx = blockIdx.x % tiles, by = blockIdx.x / tiles % ranks;
  const int bz = blockIdx.x / (tiles * ranks);
  const int t0 = bx * NT, rb = by * 16;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c_lo = bz * range, c_hi = c_lo + range < C ? c_lo + range : C;
  int owner[NT], row[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const bool in = t0 + t < p.tiles;
    owner[t] = in ? plan[p.owner + t0 + t] : -2;
    // a padding position computes the tile's first row again; its results are dropped
    const int32_t *perm = plan + p.perm + (int64_t)(in ? t0 + t : t0) * kLoraTile;
    row[t] = perm[r] >= 0 ? perm[r] : perm[0];
  }
  const i32x4 zero = {0, 0, 0, 0};
  char *stage = smem + wave * SLOT;
  f32x4 *red = reinterpret_cast<f32x4 *>(smem);
  int done = -1;
  for (;;) {
    // the tiles' adapters in ascending order (-1 and -2: nothing to compute)
    int a = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < NT; ++t) a = owner[t] > done && owner[t] < a ? owner[t] : a;
    if (a == 0x7fffffff) break;
    done = a;
    int any = 0;
#pragma unroll
    for (int t = NT - 1; t >= 0; --t) any = owner[t] == a ? row[t] : any;
    const uint16_t *xr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)  // another adapter's tile reads one of this one's again
      xr[t] = x + (int64_t)(owner[t] == a ? row[t] : any) * C;
    const uint16_t *ab = A + (int64_t)a * R * C;
    const float al = alpha[a];
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Step {
      i32x4 x[kU][NT], a[kU];
    };
    auto load = [&](int64_t c0, Step &s) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t c = c0 + 32 * u + 8 * g;
        if constexpr (!KMAJOR) {
          const int j = rb + r < R ? rb + r : R - 1;  // past R: dropped columns
          s.a[u] = c < c_hi ? *reinterpret_cast<const i32x4 *>(ab + (int64_t)j * C + c) : zero;
        } else {
          // lane l: row c0 + 32 u + l / 2 of A, ranks rb + 8 (l % 2) .. + 7
          const int64_t cr = c0 + 32 * u + (lane >> 1);
          const int j = rb + 8 * (lane & 1);
          s.a[u] = cr < c_hi && j < R ? *reinterpret_cast<const i32x4 *>(ab + cr * R + j) : zero;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
          s.x[u][t] = c < c_hi ? *reinterpret_cast<const i32x4 *>(xr[t] + c) : zero;
      }
    };
    auto multiply = [&](Step &s) {
      if constexpr (KMAJOR) {
        // a wave's own LDS slot: its stores and loads complete in order
#pragma unroll
        for (int u = 0; u < kU; ++u)
          *reinterpret_cast<i32x4 *>(stage + u * 1024 + 16 * lane) = s.a[u];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          // 16 lanes read 4 rows x 16 ranks and get column r of them
          const uint32_t at = (uint32_t)(uintptr_t)(stage + u * 1024 + (8 * g + (r >> 2)) * 32 +
                                                    8 * (r & 3));
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)at);
          const s16x4 hi =
              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)(at + 128));
          const i32x2 l2 = __builtin_bit_cast(i32x2, lo), h2 = __builtin_bit_cast(i32x2, hi);
          s.a[u] = i32x4{l2[0], l2[1], h2[0], h2[1]};
        }
        __builtin_amdgcn_wave_barrier();
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, s.x[u][t]),
                                                           __builtin_bit_cast(bf16x8, s.a[u]),
                                                           acc[t], 0, 0, 0);
    };
    for (int64_t c0 = c_lo + wave * kStep; c0 < c_hi; c0 += W * kStep) {
      Step s;
      load(c0, s);
      multiply(s);
    }
    __syncthreads();  // the waves' slots become the sums'
#pragma unroll
    for (int t = 0; t < NT; ++t) red[(wave * NT + t) * 64 + lane] = acc[t];
    __syncthreads();
    if (wave < NT) {  // wave t finishes tile t
      const int t = wave;
      int mine = owner[0];
#pragma unroll
      for (int i = 1; i < NT; ++i) mine = t == i ? owner[i] : mine;
      const int j = rb + r;
      if (mine == a && j < R) {
        f32x4 s = red[t * 64 + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) s += red[(w * NT + t) * 64 + lane];
        const int64_t pos = (int64_t)(t0 + t) * kLoraTile + 4 * g;
        if (part) {
          float *dst = part + (bz * p.tiles * kLoraTile + pos) * R + j;
#pragma unroll
          for (int v = 0; v < 4; ++v) dst[(int64_t)v * R] = s[v];
        } else {
          const i32x4 out = *reinterpret_cast<const i32x4 *>(plan + p.perm + pos);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (out[v] >= 0) h[(int64_t)out[v] * R + j] = al * s[v];
        }
      }
    }
    __syncthreads();  // the sums are read before the next adapter's steps
  }
  if (part) return;
  // rows without an adapter
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (owner[t] != -1 || rb != 0) continue;
    const int32_t *perm = plan + p.perm + (int64_t)(t0 + t) * kLoraTile;
    for (int i = threadIdx.x; i < kLoraTile * R; i += 64 * W) {
      const int m = perm[i / R];
      if (m >= 0) h[(int64_t)m * R + i % R] = 0.0f;
    }
  }
}

// h of the rows at each sorted position from Z partial sums; a thread takes 4 ranks.
__global__ __launch_bounds__(256) void k_lora_shrink_sum(const float *__restrict__ part, int Z,
                                                         const float *__restrict__ alpha, int R,
                                                         int64_t M, int64_t L,
                                                         const int32_t *__restrict__ plan,
                                                         float *__restrict__ h) {
  const LoraPlanLayout p = lora_plan_layout(M, L);
  const int q = R / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, pos = i / q;
  const int j = (int)(i - pos * q) * 4;
  const int64_t n = p.tiles * kLoraTile;
  if (pos >= n) return;
  // the sums, the row and its adapter at once (what lies at positions without a
  // row was never written and is not used)
  const int m = plan[p.perm + pos], a = plan[p.owner + pos / kLoraTile];
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  int z = 0;
  for (; z + 4 <= Z; z += 4) {
    f32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = *reinterpret_cast<const f32x4 *>(part + ((z + i) * n + pos) * R + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) s += v[i];
  }
  for (; z < Z; ++z) s += *reinterpret_cast<const f32x4 *>(part + (z * n + pos) * R + j);
  if (m < 0) return;
  s = a >= 0 ? s * alpha[a] : f32x4{0.f, 0.f, 0.f, 0.f};
  *reinterpret_cast<f32x4 *>(h + (int64_t)m * R + j) = s;
}

// ----------------------------------------------------------- weight gradients

// One workgroup of W waves: adapter a, 16 CW columns of dy (dB) or of the
// checkpoint (dA, 128 columns: they share one scale per row) and 16 RT ranks. The
// contraction runs over the adapter's rows in sorted order, 32 at a step, the
// waves taking steps in turn and meeting in LDS at the end. Both operands have
// the contraction as their slow axis: lane (r, g) reads CW columns of the 8 rows
// 8 g .. 8 g + 7 and turns the 8 x CW block in registers into the operands of CW
// MFMAs, MFMA c covering columns CW r + c. The float32 operand (h, or u times
// the row's scale) is split into three bf16 parts. Loads in flight come from the
// waves of a CU rather than from a step ahead in each, whose registers cost as
// many waves. Bound by those round trips: 17 us for the 25 MB of M = 500, N = 4096,
// K = 14336, R = 64, 3 adapters (14 without the input's gradient around it); 21 us, 3.2
// TB/s, for M = 2048, N = 14336, K = 4096, R = 16 (19).

// a.lo16 | b.lo16 << 16 and the high halves
__device__ __forceinline__ int pack_lo(int a, int b) {
  return (int)__builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x05040100u);
}
__device__ __forceinline__ int pack_hi(int a, int b) {
  return (int)__builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x07060302u);
}

template <int W, int RT, bool CODES>
__device__ __forceinline__ void lora_wgrad(const LoraWgradArgs &p, const LoraPlanLayout &pl,
                                           int64_t a, int64_t c0, int j0, char *smem) {
  constexpr int CW = CODES ? 8 : 4;
  static_assert(!CODES || 16 * CW == kCkptGroup, "a workgroup's columns share a scale");
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t C = CODES ? p.K : p.N;
  const int R = (int)p.R;
  const int64_t G = (p.K + kCkptGroup - 1) / kCkptGroup;
  const int32_t *perm = p.plan + pl.perm;
  const int first = p.plan[pl.first + a] * kLoraTile, last = p.plan[pl.first + a + 1] * kLoraTile;
  const float *left = CODES ? p.u : p.h;
  const int64_t col = c0 + CW * r;
  const bool cin = col < C;  // whole chunks: C is a multiple of 8

  f32x4 acc[RT][CW];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int c = 0; c < CW; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  // a step's operands: 8 rows x 8 bytes, their scales, 8 rows x RT ranks; rows
  // of padding are zero on both sides
  struct Step {
    i32x2 d[8];
    float s[CODES ? 8 : 1], v[RT][8];
  };
  auto rows_of = [&](int p0, int (&row)[8]) {
    const int q0 = p0 + 8 * g;
#pragma unroll
    for (int e = 0; e < 8; ++e) row[e] = q0 + e < last ? perm[q0 + e] : -1;
  };
  auto load = [&](const int (&row)[8], Step &b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool in = row[e] >= 0;
      b.d[e] = i32x2{0, 0};
      if (in && cin) {
        if constexpr (CODES)
          b.d[e] = *reinterpret_cast<const i32x2 *>(p.xq + (int64_t)row[e] * C + col);
        else
          b.d[e] = *reinterpret_cast<const i32x2 *>(p.dy + (int64_t)row[e] * C + col);
      }
      if constexpr (CODES) b.s[e] = in ? p.xs[(int64_t)row[e] * G + c0 / kCkptGroup] : 0.0f;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int j = j0 + 16 * t + r;
        b.v[t][e] = in && j < R ? left[(int64_t)row[e] * R + j] : 0.0f;
      }
    }
  };
  auto multiply = [&](Step &b) {
    bf16x8 hi[RT], mid[RT], lo[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if constexpr (CODES)
#pragma unroll
        for (int e = 0; e < 8; ++e) b.v[t][e] *= b.s[e];
      split_bf16(b.v[t], hi[t], mid[t], lo[t]);
    }
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      i32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (CODES) {
          const float f0 = (float)(int8_t)(b.d[2 * e][c >> 2] >> (8 * (c & 3)));
          const float f1 = (float)(int8_t)(b.d[2 * e + 1][c >> 2] >> (8 * (c & 3)));
          o[e] = pack_hi((int)__float_as_uint(f0), (int)__float_as_uint(f1));  // exact
        } else {
          o[e] = (c & 1) ? pack_hi(b.d[2 * e][c >> 1], b.d[2 * e + 1][c >> 1])
                         : pack_lo(b.d[2 * e][c >> 1], b.d[2 * e + 1][c >> 1]);
        }
      }
      const bf16x8 bv = __builtin_bit_cast(bf16x8, o);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[t], bv, acc[t][c], 0, 0, 0);
        acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mid[t], bv, acc[t][c], 0, 0, 0);
        acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[t], bv, acc[t][c], 0, 0, 0);
      }
    }
  };
  int row[8];
  int p0 = first + 32 * wave;
  if (p0 < last) rows_of(p0, row);
  for (; p0 < last; p0 += 32 * W) {
    Step s;
    load(row, s);
    rows_of(p0 + 32 * W, row);
    multiply(s);
  }
  // the waves' sums meet pairwise
  f32x4 *red = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
  for (int half = W / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < CW; ++c)
          red[(((wave - half) * RT + t) * CW + c) * 64 + lane] = acc[t][c];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < CW; ++c) acc[t][c] += red[((wave * RT + t) * CW + c) * 64 + lane];
    }
  }
  if (wave != 0 || !cin) return;
  // acc[t][c] lane: ranks j0 + 16 t + 4 g + v of column col + c
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int j = j0 + 16 * t + 4 * g;
    if (j >= R) continue;  // whole groups of 4
    if constexpr (CODES) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float *dst = p.dA + ((int64_t)a * R + j + v) * C + col;
        f32x4 o0 = {acc[t][0][v], acc[t][1][v], acc[t][2][v], acc[t][3][v]};
        f32x4 o1 = {acc[t][4][v], acc[t][5][v], acc[t][6][v], acc[t][7][v]};
        if (p.accumulate) {
          o0 += *reinterpret_cast<const f32x4 *>(dst);
          o1 += *reinterpret_cast<const f32x4 *>(dst + 4);
        }
        *reinterpret_cast<f32x4 *>(dst) = o0;
        *reinterpret_cast<f32x4 *>(dst + 4) = o1;
      }
    } else {
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        float *dst = p.dB + ((int64_t)a * C + col + c) * R + j;
        f32x4 o = acc[t][c];
        if (p.accumulate) o += *reinterpret_cast<const f32x4 *>(dst);
        *reinterpret_cast<f32x4 *>(dst) = o;
      }
    }
  }
}

template <int W, int RT>
__global__ __launch_bounds__(64 * W) void k_lora_wgrad(LoraWgradArgs p, int tiles_b) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const LoraPlanLayout pl = lora_plan_layout(p.M, p.L);
  const int64_t a = blockIdx.y;
  const int j0 = blockIdx.z * 16 * RT;
  const int tile = blockIdx.x;
  if (tile < tiles_b)
    lora_wgrad<W, RT, false>(p, pl, a, (int64_t)tile * 64, j0, smem);
  else
    lora_wgrad<W, RT, true>(p, pl, a, (int64_t)(tile - tiles_b) * 128, j0, smem);
}

// The same with the last sum of a split input gradient in the workgroups behind
// (blocks of the weight gradients): both are short, and neither waits for the other.
__global__ __launch_bounds__(256) void k_lora_wgrad_reduce(LoraWgradArgs p, int tiles_b, int tiles,
                                                           int blocks, DgradParts parts,
                                                           LoraTerm lt) {
  __shared__ __attribute__((aligned(16))) char smem[4 / 2 * 8 * 64 * 16];
  int b = blockIdx.x;
  if (b >= blocks) {
    dgrad_reduce(parts, lt, (int64_t)(b - blocks) * 256 + threadIdx.x);
    return;
  }
  const LoraPlanLayout pl = lora_plan_layout(p.M, p.L);
  const int tile = b % tiles;
  b /= tiles;
  const int64_t a = b % (int)p.L;
  const int j0 = b / (int)p.L * 16;
  if (tile < tiles_b)
    lora_wgrad<4, 1, false>(p, pl, a, (int64_t)tile * 64, j0, smem);
  else
    lora_wgrad<4, 1, true>(p, pl, a, (int64_t)(tile - tiles_b) * 128, j0, smem);
}

// --------------------------------------------------------- products in memory

// One workgroup: a tile of the plan (16 rows of one adapter) x 256 columns, a wave
// 64 of them. Where many adapters share a tile of the projection's kernel, walking
// them there costs 3 to 5 us each (all 64 or 128 rows take part in each step), so
// their products are computed here, spread over the chip with each adapter read
// once per 16 rows, and the epilogues add them. Bound by memory: the adapters in
// use and the float32 products, written here and read there (whole calls, 64
// adapters at random: M = 128, N = 14336, K = 4096, R = 16: 54 us, 156 walked, of which
// 9.6 are this kernel's; M = 2048, N = K = 4096, 32 adapters: 90, 182). A batch with more
// than kLoraFew adapters stacked but none of its groups mixed pays a launch whose
// workgroups return (M = 128: 3.9 us; M = 2048: 5.4).
template <bool KMAJOR>
__global__ __launch_bounds__(256) void k_lora_products(const float *__restrict__ h,
                                                       const uint16_t *__restrict__ W, int64_t M,
                                                       int64_t N, int64_t L, int R,
                                                       const int32_t *__restrict__ plan,
                                                       const int32_t *__restrict__ mixed,
                                                       int first, int blocks,
                                                       float *__restrict__ T) {
  const LoraPlanLayout p = lora_plan_layout(M, L);
  const int tile = first + blockIdx.x / blocks;  // blocks of columns
  const int a = plan[p.owner + tile];
  if (a < 0) return;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
  const int32_t *perm = plan + p.perm + (int64_t)tile * kLoraTile;
  const int row = perm[r];
  if (mixed && !__any(row >= 0 && mixed[(row < 0 ? 0 : row) / kLoraGroup])) return;
  const i32x4 out = *reinterpret_cast<const i32x4 *>(perm + 4 * g);
  const int64_t n0 = (int64_t)(blockIdx.x % blocks) * 256 + 64 * wave;
  f32x4 d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int c = 0; c < R; c += 32) {
    const bool in = c + 8 * g < R;  // whole chunks of 8 ranks
    f32x4 h0 = {0.f, 0.f, 0.f, 0.f}, h1 = h0;
    if (in && row >= 0) {
      const float *hm = h + (int64_t)row * R + c + 8 * g;
      h0 = *reinterpret_cast<const f32x4 *>(hm);
      h1 = *reinterpret_cast<const f32x4 *>(hm + 4);
    }
    bf16x8 w[4];
    if constexpr (KMAJOR) {  // column n0 + 4 r + j
      i32x2 v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = i32x2{0, 0};
        if (in && n0 + 4 * r < N)  // whole chunks: N is a multiple of 16
          v[e] = *reinterpret_cast<const i32x2 *>(W + ((int64_t)a * R + c + 8 * g + e) * N + n0 +
                                                  4 * r);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        i32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = j & 1 ? pack_hi(v[2 * e][j >> 1], v[2 * e + 1][j >> 1])
                       : pack_lo(v[2 * e][j >> 1], v[2 * e + 1][j >> 1]);
        w[j] = __builtin_bit_cast(bf16x8, o);
      }
    } else {  // column n0 + 16 j + r
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + 16 * j + r;
        i32x4 o = {0, 0, 0, 0};
        if (in && n < N) o = *reinterpret_cast<const i32x4 *>(W + ((int64_t)a * N + n) * R + c + 8 * g);
        w[j] = __builtin_bit_cast(bf16x8, o);
      }
    }
    const float v[8] = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
    bf16x8 hi, lo;
    split_bf16(v, hi, lo);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, w[j], d[j], 0, 0, 0);
      d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, w[j], d[j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (out[v] < 0) continue;
    float *t = T + (int64_t)out[v] * N + n0;
    if constexpr (KMAJOR) {
      if (n0 + 4 * r < N)
        *reinterpret_cast<f32x4 *>(t + 4 * r) = f32x4{d[0][v], d[1][v], d[2][v], d[3][v]};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + 16 * j + r < N) t[16 * j + r] = d[j][v];
    }
  }
}

// One launch (NT = 1) for a contraction of at most two steps a wave on a grid of
// at most one workgroup a CU (M = 500, K = 4096, R = 64: 9.9 us, 13.7 in ranges with
// their second launch); else ranges of one step a wave while that keeps the grid
// within two workgroups a CU (M = 2048, N = 14336, R = 16: 20.7 us, 26.6 whole).
bool shrink_whole(int64_t M, int64_t C, int64_t L, int64_t R) {
  return C <= 2 * 16 * kStep && lora_plan_layout(M, L).tiles * ((R + 15) / 16) <= 256;
}

int shrink_ranges(int64_t M, int64_t C, int64_t L, int64_t R) {
  if (shrink_whole(M, C, L, R)) return 1;
  const int64_t blocks = (lora_plan_layout(M, L).tiles + 3) / 4 * ((R + 15) / 16);
  const int64_t most = (C + 4 * kStep - 1) / (4 * kStep);
  int64_t z = 512 / blocks;
  z = z > most ? most : z;
  return z < 1 ? 1 : (int)z;
}

template <bool KMAJOR, class SC>
hipError_t go_shrink(const uint16_t *x, int64_t M, int64_t C, const uint16_t *A,
                     const float *alpha, int64_t L, int64_t R, const int32_t *plan, float *h,
                     float *part, const SC &sc, hipStream_t st) {
  const LoraPlanLayout p = lora_plan_layout(M, L);
  const int ranks = (int)((R + 15) / 16);
  if (shrink_whole(M, C, L, R)) {
    const int tiles = (int)p.tiles, blocks = tiles * ranks;
    hipLaunchKernelGGL((k_lora_shrink<1, 16, KMAJOR, SC>),
                       dim3((unsigned)(blocks + (SC::on ? (M + 3) / 4 : 0))), dim3(1024), 0, st, x,
                       C, A, alpha, (int)R, M, L, plan, h, (float *)nullptr, C, tiles, ranks,
                       blocks, sc);
    return hipGetLastError();
  }
  int z = shrink_ranges(M, C, L, R);
  const int64_t range = (C + (int64_t)z * kStep - 1) / ((int64_t)z * kStep) * kStep;
  if (z > 1) z = (int)((C + range - 1) / range);
  const int tiles = (int)((p.tiles + 3) / 4), blocks = tiles * ranks * z;
  hipLaunchKernelGGL((k_lora_shrink<4, 4, KMAJOR, SC>),
                     dim3((unsigned)(blocks + (SC::on ? M : 0))), dim3(256), 0, st, x, C, A, alpha,
                     (int)R, M, L, plan, h, z > 1 ? part : nullptr, range, tiles, ranks, blocks,
                     sc);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || z <= 1) return e;
  const int64_t n = p.tiles * kLoraTile * (R / 4);
  hipLaunchKernelGGL(k_lora_shrink_sum, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, part,
                     z, alpha, (int)R, M, L, plan, h);
  return hipGetLastError();
}

constexpr int kWgradWaves = 2800;

template <int W, int RT>
hipError_t go_wgrad(const LoraWgradArgs &a, hipStream_t st) {
  constexpr int bytes = W / 2 * RT * 8 * 64 * 16;
  static_assert(bytes <= 65536, "what any launch may have of LDS");
  const int tb = a.dB ? (int)((a.N + 63) / 64) : 0, ta = a.dA ? (int)((a.K + 127) / 128) : 0;
  const dim3 grid((unsigned)(tb + ta), (unsigned)a.L, (unsigned)((a.R + 16 * RT - 1) / (16 * RT)));
  hipLaunchKernelGGL((k_lora_wgrad<W, RT>), grid, dim3(64 * W), bytes, st, a, tb);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_plan(const int32_t *idx, int64_t M, int64_t L, int32_t *plan,
                            hipStream_t st) {
  hipLaunchKernelGGL(k_lora_plan, dim3(1), dim3(1024), 0, st, idx, M, L, plan);
  return hipGetLastError();
}

// Z ranges over T tiles take Z T 64 R bytes. Z is at most one range for each step of
// the waves, and it is 512 / (ceil(T / 4) ranks) at most (else 1, without partial
// sums), so Z T <= 2048 / ranks; both bounds grow with M where Z T itself does not.
size_t lora_shrink_most_bytes(int64_t M, int64_t C, int64_t L, int64_t R) {
  if (shrink_whole(M, C, L, R)) return 0;  // and so is every smaller batch
  const int64_t ranks = (R + 15) / 16, most = (C + 4 * kStep - 1) / (4 * kStep);
  const int64_t steps = most * lora_plan_layout(M, L).tiles, places = 2048 / ranks;
  if (most <= 1) return 0;
  return (size_t)(steps < places ? steps : places) * kLoraTile * (size_t)R * 4;
}

hipError_t launch_lora_shrink(const uint16_t *x, int64_t M, int64_t K, const uint16_t *A,
                              const float *alpha, int64_t L, int64_t R, const int32_t *plan,
                              float *h, float *part, hipStream_t st) {
  if (M >= kLoraTiledMinM) return go_shrink<false>(x, M, K, A, alpha, L, R, plan, h, part, NoScale{}, st);
  const int32_t *idx = plan + lora_plan_layout(M, L).idx;
  // a rank a workgroup while those are few; from 8 a CU on x is better read once for 4
  // (calls with N = K = 4096: M = 1, R = 8 7.1 us, 7.7 with 4; M = 32, R = 32 17.3, 17.4;
  // M = 16, R = 128 23.0, 22.9; M = 63, R = 64 31.7, 30.4)
  if (M * R < 2048)
    hipLaunchKernelGGL(k_lora_shrink_rows<1>, dim3((unsigned)R, (unsigned)M), dim3(256), 0, st, x,
                       K, A, alpha, (int)R, idx, h);
  else
    hipLaunchKernelGGL(k_lora_shrink_rows<4>, dim3((unsigned)(R / 4), (unsigned)M), dim3(256), 0,
                       st, x, K, A, alpha, (int)R, idx, h);
  return hipGetLastError();
}

hipError_t launch_lora_shrink_t(const uint16_t *dy, int64_t M, int64_t N, const uint16_t *B,
                                const float *alpha, int64_t L, int64_t R, const int32_t *plan,
                                float *u, float *part, const DgradScale *sc, hipStream_t st) {
  if (!sc) return go_shrink<true>(dy, M, N, B, alpha, L, R, plan, u, part, NoScale{}, st);
  if (sc->NP <= 4096)
    return go_shrink<true>(dy, M, N, B, alpha, L, R, plan, u, part, WithScale<2>{*sc}, st);
  if (sc->NP <= 16384)
    return go_shrink<true>(dy, M, N, B, alpha, L, R, plan, u, part, WithScale<8>{*sc}, st);
  return go_shrink<true>(dy, M, N, B, alpha, L, R, plan, u, part, WithScale<0>{*sc}, st);
}

hipError_t launch_lora_products(const float *h, const uint16_t *W, bool kmajor, int64_t M,
                                int64_t N, int64_t L, int64_t R, const int32_t *plan,
                                const int32_t *mixed, float *T, hipStream_t st) {
  const int64_t tiles = lora_plan_layout(M, L).tiles, blocks = (N + 255) / 256;
  // grids of at most 2^31 threads (one of 2^32 or more would run in part): 1089 tiles of
  // 2^22 channels take three, ordinary batches one
  const int64_t slice = (1LL << 31) / 256 / blocks;
  const auto kern = kmajor ? k_lora_products<true> : k_lora_products<false>;
  for (int64_t first = 0; first < tiles; first += slice) {
    const int64_t n = tiles - first < slice ? tiles - first : slice;
    hipLaunchKernelGGL(kern, dim3((unsigned)(n * blocks)), dim3(256), 0, st, h, W, M, N, L, (int)R,
                       plan, mixed, (int)first, (int)blocks, T);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Workgroups of the weight gradients, each 64 channels or 128 inputs of an adapter and
// 16 ranks. The rules below go by M / L, the mean of an adapter's rows: how the rows
// lie is known on the device only. A batch that stacks many adapters and names one
// pays for it (M = 2048, N = K = 4096, R = 16, 32 adapters: 49 us with all rows on one of
// them, 10 with 64 each; 17 where that adapter is stacked alone).
static int64_t wgrad_units(const LoraWgradArgs &a) {
  return ((a.dB ? (a.N + 63) / 64 : 0) + (a.dA ? (a.K + 127) / 128 : 0)) * a.L *
         ((a.R + 15) / 16);
}

// For segments of few rows on average. Backward in a graph, with the sum beside and in
// launches each: M = 63, N = 2560, K = 960 19.8 us, 23.7; M = 500, N = K = 4096, R = 128
// 60.5, 64.4; M = 512, one adapter 43.8, 51.5. 64 adapters, R = 16 (6144 workgroups, for
// which 2 waves are enough): 55.6, 49.1.
bool lora_wgrad_beside(const LoraWgradArgs &a) {
  return a.M / a.L <= 512 && wgrad_units(a) < 2048;
}

hipError_t launch_lora_wgrad_reduce(const LoraWgradArgs &a, const DgradParts &parts,
                                    const LoraTerm &lt, hipStream_t st) {
  const int tb = a.dB ? (int)((a.N + 63) / 64) : 0, ta = a.dA ? (int)((a.K + 127) / 128) : 0;
  const int64_t blocks = (int64_t)(tb + ta) * a.L * ((a.R + 15) / 16);
  hipLaunchKernelGGL(k_lora_wgrad_reduce, dim3((unsigned)(blocks + parts.blocks())), dim3(256), 0,
                     st, a, tb, tb + ta, (int)blocks, parts, lt);
  return hipGetLastError();
}

hipError_t launch_lora_wgrad(const LoraWgradArgs &a, hipStream_t st) {
  // long segments and several blocks of ranks: two of them share a read (M = 8192,
  // 4 adapters, R = 64, N = K = 4096: 139 us of backward without dx, 150 apart)
  if (a.R > 16 && a.M / a.L >= 1024) return go_wgrad<8, 2>(a, st);
  // else the fewest waves a workgroup that make about 3 a SIMD in all: more of
  // them only meet (M = 512, 16 adapters, R = 16, N = K = 4096: 15.4 us with 2, 18.2
  // with 4), fewer leave the memory idle (M = 2048, N = 14336, K = 4096, one adapter:
  // 37 us with 16, 45 with 4)
  const int64_t units = wgrad_units(a);
  if (2 * units >= kWgradWaves) return go_wgrad<2, 1>(a, st);
  if (4 * units >= kWgradWaves) return go_wgrad<4, 1>(a, st);
  if (8 * units >= kWgradWaves) return go_wgrad<8, 1>(a, st);
  return go_wgrad<16, 1>(a, st);
}

}  // namespace aql
