// Gradient of the W8A16 linear to its input: dx[m, k] = sum_n dy[m, n] scale[n] q[n, k].
//
// The contraction runs over the output channels, so the channel scale no longer
// factors out of the sum: the weights are widened to bf16(scale[n] q[n, k]), one
// rounding (at most 2^-8 relative) per weight, which is what a bf16 copy of the
// dequantized weight would hold; products and sums are float32.
//
// Tile: 16 TI rows of dy x 32 NWV columns of dx per workgroup of NWV waves side
// by side along K, each 16 TI x 32, over stages of 64 channels. Operands go
// global -> LDS by buffer loads that write LDS directly: dy as rows of 128 B,
// the weights as they lie, 64 channel rows of 32 NWV bytes, and each wave's own
// copy of the stage's 64 scales. q has the contraction as its slow axis; the
// byte-transposing LDS read (8 rows x 16 columns per 16 lanes) hands each lane
// the 8 channels of one column that the matrix instruction wants, so no
// transposed copy of the weights exists anywhere.
// A ring of SG stages keeps loads in flight behind exact vmcnt waits. dy rows
// store their 16-byte chunks XOR-swizzled by (row / 2) mod 8 and weight rows by
// the row (by row / 2 for 128-byte rows), which spreads each half wave's reads
// over all banks.
#include "w8a16_dgrad.h"

namespace aql {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

constexpr int BC = 64;           // channels a stage
constexpr int OOB = 0x40000000;  // past any range: loads give 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// SIZE bytes a lane from offset off into LDS at dst + SIZE lane.
template <int SIZE>
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t rr, uint32_t dst, int off) {
  lds_void *p = (lds_void *)(uintptr_t)__builtin_amdgcn_readfirstlane(dst);
  if constexpr (SIZE == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rr, p, 16, off, 0, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rr, p, 4, off, 0, 0, 0);
}

constexpr int vmcnt_imm(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }

template <int TI, int NWV, int SG>
struct DgradLds {
  static constexpr int BM = 16 * TI, BK = 32 * NWV;
  static constexpr int NX = BM / 8 / NWV;     // dy loads per wave and stage (8 rows x 128 B)
  static constexpr int NL = NX + 2 + 1;       // + weights (1 KB each) + scales
  static constexpr int XS = BM * 128, QS = BC * BK, SS = NWV * 256;
  static constexpr int STAGE = XS + QS + SS;
  static constexpr int RING = SG * STAGE;
  static constexpr int TLD = BK + 8;          // bf16 per staged output row
  static constexpr int TILE = BM * TLD * 2;
  static constexpr int TLDF = BK + 4;         // fp32 per staged partial-sum row
  static constexpr int TILEF = BM * TLDF * 4;
  static constexpr int BYTES = RING > TILE ? RING : TILE;
  static constexpr int BYTES_SPLIT = RING > TILEF ? RING : TILEF;
  static_assert(NX * NWV * 8 == BM, "dy loads split evenly");
};

// Eight codes (rows n .. n + 7 of a column) times their scales, as bf16.
__device__ __forceinline__ bf16x8 widen_scaled(i32x2 w, const float (&s)[8]) {
  bf16x8 b;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    b[e] = (__bf16)((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))) * s[e]);
  return b;
}

// SPLIT: unit (tile, sp) takes the ks stages from sp * ks and writes its fp32
// sums to part[sp][M][K]; k_w8a16_dgrad_reduce adds them.
template <int TI, int NWV, int SG, bool SPLIT, class LT>
__global__ __launch_bounds__(64 * NWV, SG == 2 ? NWV / 2 : NWV / 4) void k_w8a16_dgrad(
    const uint16_t *__restrict__ dy, const int8_t *__restrict__ q,
    const float *__restrict__ scale, uint16_t *__restrict__ dx, int64_t M, int64_t N, int64_t K,
    int tiles_m, int tiles_k, float *__restrict__ part, int ks, LT lt) {
  using L = DgradLds<TI, NWV, SG>;
  constexpr int BM = L::BM, BK = L::BK, NX = L::NX, NL = L::NL;
  constexpr int CH = BK / 16;      // 16-byte chunks of a weight row
  constexpr int RPL = 1024 / BK;   // weight rows a load covers
  extern __shared__ __attribute__((aligned(16))) char smem[];

  const int nt = tiles_m * tiles_k;
  const int nu = (int)gridDim.x;
  const int lin = blockIdx.x;
  int unit = lin;
  if ((nu & 7) == 0) unit = (lin & 7) * (nu >> 3) + (lin >> 3);  // neighbours on one XCD
  const int tile = unit % nt, sp = unit / nt;
  const int tk = tile / tiles_m, tm = tile % tiles_m;
  const int64_t m0 = (int64_t)tm * BM, k0 = (int64_t)tk * BK;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t mval = M - m0 < BM ? M - m0 : BM;
  const __amdgpu_buffer_rsrc_t rx = rsrc(dy + m0 * N, (uint32_t)(mval * N * 2));
  const __amdgpu_buffer_rsrc_t rs = rsrc(scale, (uint32_t)(N * 4));

  uint32_t xoff[NX];
  int xlim[NX];  // stages in which this lane's chunk lies before N
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int row = 8 * (i * NWV + wave) + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
    xoff[i] = (uint32_t)row * (uint32_t)(2 * N) + 16u * c;
    xlim[i] = row < mval ? (int)((N - 8 * c + BC - 1) / BC) : 0;
  }
  auto qswz = [](int row) { return CH == 16 ? row & 15 : (row >> 1) & 7; };
  int qrow[2];
  uint32_t qoff[2];
  bool qin[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    qrow[i] = RPL * (i * NWV + wave) + lane / CH;
    const int c = (lane % CH) ^ qswz(qrow[i]);
    qoff[i] = (uint32_t)qrow[i] * (uint32_t)K + 16u * c;
    qin[i] = k0 + 16 * c < K;
  }
  const uint32_t lds_base = (uint32_t)(uintptr_t)smem;
  auto issue = [&](int kt) {
    const uint32_t st = lds_base + (uint32_t)((kt % SG) * L::STAGE);
#pragma unroll
    for (int i = 0; i < NX; ++i)
      to_lds<16>(rx, st + 1024u * (i * NWV + wave),
                 kt < xlim[i] ? (int)(xoff[i] + 128u * (uint32_t)kt) : OOB);
    const int64_t n0 = (int64_t)BC * kt;
    const __amdgpu_buffer_rsrc_t rq = rsrc(q + n0 * K + k0, 0x3fffffffu);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      to_lds<16>(rq, st + L::XS + 1024u * (i * NWV + wave),
                 qin[i] && n0 + qrow[i] < N ? (int)qoff[i] : OOB);
    const int64_t ns = n0 + lane;
    to_lds<4>(rs, st + L::XS + L::QS + 256u * wave, ns < N ? (int)(4 * ns) : OOB);
  };

  int fxo[2][TI], fqo[2][2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int R = i * 16 + r;
      fxo[kk][i] = R * 128 + 16 * ((4 * kk + g) ^ ((R >> 1) & 7));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // lanes 2 e and 2 e + 1 of 16 address row e's 16 columns
      const int n = 32 * kk + 8 * g + (r >> 1);
      fqo[kk][j] = L::XS + n * BK + 16 * ((2 * wave + j) ^ qswz(n)) + 8 * (r & 1);
    }
  }

  f32x4 acc[TI][2];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](int kt) {
    const char *st = smem + (kt % SG) * L::STAGE;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const float *sl = reinterpret_cast<const float *>(st + L::XS + L::QS + 256 * wave) + 32 * kk +
                        8 * g;
      const f32x4 s0 = *reinterpret_cast<const f32x4 *>(sl);
      const f32x4 s1 = *reinterpret_cast<const f32x4 *>(sl + 4);
      const float s[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
      bf16x8 fa[TI], fb[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        fb[j] = widen_scaled(__builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                 (lds_i32x2 *)(uintptr_t)((uint32_t)(uintptr_t)st + fqo[kk][j])),
                             s);
#pragma unroll
      for (int i = 0; i < TI; ++i) fa[i] = *reinterpret_cast<const bf16x8 *>(st + fxo[kk][i]);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_s_setprio(0);
    }
  };

  const int nk_all = (int)((N + BC - 1) / BC);
  const int kb = SPLIT ? sp * ks : 0;
  const int nk = SPLIT ? (kb + ks < nk_all ? kb + ks : nk_all) : nk_all;
#pragma unroll
  for (int s = 0; s < SG - 1; ++s) issue(kb + s);
  int kt = kb;
  auto step = [&](int k) {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(NL * (SG - 2)));
    __builtin_amdgcn_s_barrier();  // stage k complete everywhere; slot of k - 1 free
    issue(k + SG - 1);
    compute(k);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this stage's fragment reads done
  };
  const int nmain = nk - (SG - 1);
  for (; kt < nmain; ++kt) step(kt);
#pragma unroll
  for (int t = 0; t < SG - 1; ++t) {
    if (kt < nk) {
      if (t == 0) __builtin_amdgcn_s_waitcnt(vmcnt_imm(NL * (SG - 2)));
      else if (t == 1) __builtin_amdgcn_s_waitcnt(vmcnt_imm(SG > 3 ? NL * (SG - 3) : 0));
      else __builtin_amdgcn_s_waitcnt(0x0F70);
      __builtin_amdgcn_s_barrier();
      compute(kt);
      __builtin_amdgcn_s_waitcnt(0xC07F);
    }
    ++kt;
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __syncthreads();

  if constexpr (SPLIT) {
    float *tf = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          tf[(i * 16 + 4 * g + v) * L::TLDF + wave * 32 + j * 16 + r] = acc[i][j][v];
    __syncthreads();
    float *pb = part + (int64_t)sp * M * K;
    for (int u = tid; u < BM * (BK / 4); u += 64 * NWV) {
      const int row = u / (BK / 4), c = u % (BK / 4);
      const int64_t m = m0 + row, k = k0 + 4 * c;
      if (m >= M || k >= K) continue;
      *reinterpret_cast<f32x4 *>(pb + m * K + k) =
          *reinterpret_cast<const f32x4 *>(tf + row * L::TLDF + 4 * c);
    }
    return;
  }
  if constexpr (LT::on) lora_add_tile<true>(acc, lt, m0, M, k0 + 32 * wave);
  uint16_t *tl = reinterpret_cast<uint16_t *>(smem);
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        tl[(i * 16 + 4 * g + v) * L::TLD + wave * 32 + j * 16 + r] = f32_to_bf16_rne(acc[i][j][v]);
  __syncthreads();
  for (int u = tid; u < BM * (BK / 8); u += 64 * NWV) {
    const int row = u / (BK / 8), c = u % (BK / 8);
    const int64_t m = m0 + row, k = k0 + 8 * c;
    if (m >= M || k >= K) continue;  // whole chunks: K is a multiple of 16
    *reinterpret_cast<i32x4 *>(dx + m * K + k) =
        *reinterpret_cast<const i32x4 *>(tl + row * L::TLD + 8 * c);
  }
}

// dx = bf16(part[0] + ... + part[S - 1] + u A), in split order; a thread takes 4
// consecutive columns, so the rows of A are read as whole lines.
template <class LT>
__global__ __launch_bounds__(256) void k_w8a16_dgrad_reduce(const float *__restrict__ part, int S,
                                                            int64_t M, int64_t K,
                                                            uint16_t *__restrict__ dx, LT lt) {
  const int64_t ng = K / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= M * ng) return;
  const int64_t m = i / ng, k = (i - m * ng) * 4;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < S; ++s)
    acc += *reinterpret_cast<const f32x4 *>(part + ((int64_t)s * M + m) * K + k);
  if constexpr (LT::on) {
    const int a = lt.idx[m];
    if (a >= 0) {
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
  *reinterpret_cast<i32x2 *>(dx + m * K + k) = i32x2{(int)lo, (int)hi};
}

template <int TI, int NWV, int SG, class LT>
hipError_t go(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q, const float *scale,
              int64_t K, uint16_t *dx, hipStream_t st, const LT &lt) {
  using L = DgradLds<TI, NWV, SG>;
  void (*kern)(const uint16_t *, const int8_t *, const float *, uint16_t *, int64_t, int64_t, int64_t,
               int, int, float *, int, LT) = k_w8a16_dgrad<TI, NWV, SG, false, LT>;
  (void)hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize,
                            L::BYTES);
  (void)hipGetLastError();
  const int tm = (int)((M + L::BM - 1) / L::BM), tk = (int)((K + L::BK - 1) / L::BK);
  hipLaunchKernelGGL(kern, dim3((unsigned)(tm * tk)), dim3(64 * NWV), L::BYTES, st, dy, q, scale,
                     dx, M, N, K, tm, tk, (float *)nullptr, 0, lt);
  return hipGetLastError();
}

template <int TI, int NWV, int SG, class LT>
hipError_t go_split(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q, const float *scale,
                    int64_t K, uint16_t *dx, float *part, int S, hipStream_t st, const LT &lt) {
  using L = DgradLds<TI, NWV, SG>;
  void (*kern)(const uint16_t *, const int8_t *, const float *, uint16_t *, int64_t, int64_t, int64_t,
               int, int, float *, int, NoLora) = k_w8a16_dgrad<TI, NWV, SG, true, NoLora>;
  (void)hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize,
                            L::BYTES_SPLIT);
  (void)hipGetLastError();
  const int tm = (int)((M + L::BM - 1) / L::BM), tk = (int)((K + L::BK - 1) / L::BK);
  const int nk = (int)((N + BC - 1) / BC);
  const int ks = (nk + S - 1) / S, splits = (nk + ks - 1) / ks;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tm * tk * splits)), dim3(64 * NWV), L::BYTES_SPLIT, st,
                     dy, q, scale, dx, M, N, K, tm, tk, part, ks, NoLora{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t groups = M * (K / 4);
  hipLaunchKernelGGL(k_w8a16_dgrad_reduce<LT>, dim3((unsigned)((groups + 255) / 256)), dim3(256),
                     0, st, part, splits, M, K, dx, lt);
  return hipGetLastError();
}

template <class LT>
hipError_t launch(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q, const float *scale,
                  int64_t K, uint16_t *dx, float *part, size_t part_bytes, hipStream_t st,
                  const LT &lt) {
  const int64_t twide = ((M + 127) / 128) * ((K + 255) / 256);
  if (twide >= 512) return go<8, 8, 2>(dy, M, N, q, scale, K, dx, st, lt);
  if (twide >= 160) return go<8, 8, 4>(dy, M, N, q, scale, K, dx, st, lt);
  const int S = w8a16_dgrad_splits(M, N, K);
  if (S > 1 && part && part_bytes >= w8a16_dgrad_part_bytes(M, N, K))
    return go_split<4, 4, 4>(dy, M, N, q, scale, K, dx, part, S, st, lt);
  return go<4, 4, 4>(dy, M, N, q, scale, K, dx, st, lt);
}

}  // namespace

// 64 x 128 tiles split while the units stay within two a CU and each keeps at
// least 8 stages of 64 channels.
int w8a16_dgrad_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t twide = ((M + 127) / 128) * ((K + 255) / 256);
  if (twide >= 160) return 1;
  const int64_t tiles = ((M + 63) / 64) * ((K + 127) / 128), nk = (N + BC - 1) / BC;
  int S = 1;
  while (S < 32 && tiles * 2 * S <= 512 && nk / (2 * S) >= 8) S *= 2;
  return S;
}

size_t w8a16_dgrad_part_bytes(int64_t M, int64_t N, int64_t K) {
  const int S = w8a16_dgrad_splits(M, N, K);
  return S > 1 ? (size_t)S * (size_t)M * (size_t)K * 4 : 0;
}

hipError_t launch_w8a16_dgrad(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q,
                              const float *scale, int64_t K, uint16_t *dx, float *part,
                              size_t part_bytes, hipStream_t st) {
  return launch(dy, M, N, q, scale, K, dx, part, part_bytes, st, NoLora{});
}

hipError_t launch_w8a16_dgrad(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q,
                              const float *scale, int64_t K, uint16_t *dx, float *part,
                              size_t part_bytes, hipStream_t st, const LoraTerm &lt) {
  return launch(dy, M, N, q, scale, K, dx, part, part_bytes, st, lt);
}

}  // namespace aql
