// Gradient of the W8A16 linear to its input: dx[m, k] = sum_n dy[m, n] scale[n] q[n, k].
//
// The contraction runs over the output channels, so the channel scale no longer
// factors out of the sum: the weights are widened to bf16(scale[n] q[n, k]), one
// rounding (at most 2^-8 relative) per weight, which is what a bf16 copy of the
// dequantized weight would hold; products and sums are float32.
//
// Tile: 16 TI rows of dy x 256 columns of dx per workgroup of 4 waves side by
// side along K, each 16 TI x 64, over stages of 64 channels. Operands go
// global -> LDS by buffer loads that write LDS directly: dy as rows of 128 B,
// the weights as they lie, 64 channel rows of 256 B, and each wave's own copy
// of the stage's 64 scales, one a lane. q has the contraction as its slow axis:
// a lane reads one dword (4 columns) of each of the 8 channel rows it needs, and
// byte j of the eight is its operand for columns 4 r + j, so the matrix
// instructions take the columns in strides of 4 and nothing is transposed,
// neither in memory nor in registers. The scales come to the multiplies by lane
// broadcasts within a row of 16 (DPP), without an LDS read of their own.
// A ring of SG stages keeps loads in flight behind exact vmcnt waits. dy rows
// store their 16-byte chunks XOR-swizzled by (row / 2) mod 8, and weight rows
// theirs by 4 (row / 8 mod 4), which spreads each read over all banks.
#include "w8a16_dgrad.h"

#include <type_traits>

namespace aql {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

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

constexpr int NWV = 4, TJ = 4;  // waves of a workgroup, 16-column blocks of a wave

template <int TI, int SG>
struct DgradLds {
  static constexpr int BM = 16 * TI, BK = 256;
  static constexpr int NX = BM / 8 / NWV;     // dy loads per wave and stage (8 rows x 128 B)
  static constexpr int NQ = BC * BK / 1024 / NWV;  // weight loads (1 KB each)
  static constexpr int NL = NX + NQ + 1;      // + scales
  static constexpr int XS = BM * 128, QS = BC * BK, SS = NWV * 256;
  static constexpr int STAGE = XS + QS + SS;
  static constexpr int RING = SG * STAGE;
  static constexpr int TLD = BK + 8;          // bf16 per staged output row
  static constexpr int TILE = BM * TLD * 2;
  static constexpr int TLDF = BK + 4;         // fp32 per staged partial-sum row
  static constexpr int TILEF = BM * TLDF * 4;
  static constexpr int BYTES = RING > TILE ? RING : TILE;
  static constexpr int BYTES_SPLIT = RING > TILEF ? RING : TILEF;
  static_assert(NX * NWV * 8 == BM && NQ * NWV * 1024 == BC * BK, "loads split evenly");
  static_assert(NL * (SG - 1) < 64, "vmcnt");
};

// The value of lane N of each row of 16 (a DPP operand of the multiply that takes it).
template <int N>
__device__ __forceinline__ float row_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)__float_as_uint(v), 0x150 + N, 0xf, 0xf, false));
}

// Byte J of eight codes (channels n .. n + 7) times their scales, as bf16. Lane t
// of a row of 16 holds the scale of channel 32 (t / 8) + 8 g + t % 8 of the
// stage, so half KK's eight are lanes 8 KK .. 8 KK + 7 of the row.
template <int KK, int J>
__device__ __forceinline__ bf16x8 widen_scaled(const int (&w)[8], float s) {
  bf16x8 b;
  b[0] = (__bf16)((float)(int8_t)(w[0] >> (8 * J)) * row_lane<8 * KK>(s));
  b[1] = (__bf16)((float)(int8_t)(w[1] >> (8 * J)) * row_lane<8 * KK + 1>(s));
  b[2] = (__bf16)((float)(int8_t)(w[2] >> (8 * J)) * row_lane<8 * KK + 2>(s));
  b[3] = (__bf16)((float)(int8_t)(w[3] >> (8 * J)) * row_lane<8 * KK + 3>(s));
  b[4] = (__bf16)((float)(int8_t)(w[4] >> (8 * J)) * row_lane<8 * KK + 4>(s));
  b[5] = (__bf16)((float)(int8_t)(w[5] >> (8 * J)) * row_lane<8 * KK + 5>(s));
  b[6] = (__bf16)((float)(int8_t)(w[6] >> (8 * J)) * row_lane<8 * KK + 6>(s));
  b[7] = (__bf16)((float)(int8_t)(w[7] >> (8 * J)) * row_lane<8 * KK + 7>(s));
  return b;
}

// SPLIT: unit (tile, sp) takes the ks stages from sp * ks and writes its fp32
// sums to part[sp][M][K]; k_w8a16_dgrad_reduce adds them.
template <int TI, int SG, bool SPLIT, class LT>
__global__ __launch_bounds__(64 * NWV, 2) void k_w8a16_dgrad(
    const uint16_t *__restrict__ dy, const int8_t *__restrict__ q,
    const float *__restrict__ scale, uint16_t *__restrict__ dx, int64_t M, int64_t N, int64_t K,
    int tiles_m, int tiles_k, float *__restrict__ part, int ks, LT lt) {
  using L = DgradLds<TI, SG>;
  constexpr int BM = L::BM, BK = L::BK, NX = L::NX, NQ = L::NQ, NL = L::NL;
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
  int qrow[NQ];
  uint32_t qoff[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    qrow[i] = 4 * (i * NWV + wave) + (lane >> 4);
    const int c = (lane & 15) ^ (4 * ((qrow[i] >> 3) & 3));
    qoff[i] = (uint32_t)qrow[i] * (uint32_t)K + 16u * c;
    if (k0 + 16 * c >= K) qrow[i] = OOB;  // a column past K: never loaded
  }
  const int soff = 32 * ((lane >> 3) & 1) + 8 * g + (lane & 7);  // the lane's channel of a stage
  const uint32_t lds_base = (uint32_t)(uintptr_t)smem;
  // stage kt into ring slot `slot`; past N everything reads as zero
  auto issue = [&](int kt, int slot) {
    const uint32_t st = lds_base + (uint32_t)(slot * L::STAGE);
#pragma unroll
    for (int i = 0; i < NX; ++i)
      to_lds<16>(rx, st + 1024u * (i * NWV + wave),
                 kt < xlim[i] ? (int)(xoff[i] + 128u * (uint32_t)kt) : OOB);
    const int64_t n0 = (int64_t)BC * kt;
    const int64_t left = N - n0;
    const int rows = left < BC ? (int)left : BC;  // not positive past the end: none
    const __amdgpu_buffer_rsrc_t rq = rsrc(q + (left > 0 ? n0 : 0) * K + k0, 0x3fffffffu);
#pragma unroll
    for (int i = 0; i < NQ; ++i)
      to_lds<16>(rq, st + L::XS + 1024u * (i * NWV + wave), qrow[i] < rows ? (int)qoff[i] : OOB);
    to_lds<4>(rs, st + L::XS + L::QS + 256u * wave, soff < rows ? (int)(4 * (n0 + soff)) : OOB);
  };

  // fragment offsets within a stage. dy: block i adds 2048 i, half kk flips bit
  // 6 (chunk 4 kk + g under the swizzle); weights: half kk adds 32 rows, channel
  // e of the lane's eight adds e rows
  const int fx = r * 128 + 16 * (g ^ ((r >> 1) & 7));
  const int fq = L::XS + 8 * g * BK + 16 * ((4 * wave + (r >> 2)) ^ (4 * g)) + 4 * (r & 3);
  const int fs = L::XS + L::QS + 256 * wave + 4 * lane;

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Software pipeline over the 32-channel halves of the stages. While the matrix
  // core works on one half, the next half's weights come from LDS and are
  // widened between the matrix instructions, and each block of dy is replaced by
  // the next half's as soon as its products are issued, so only the widened
  // weights are held twice.
  bf16x8 fa[TI], b0[TJ], b1[TJ];
  int raw[8];
  float sv;
  auto read_w = [&](const char *st, auto kk) {
    constexpr int KK = decltype(kk)::value;
    if constexpr (KK == 0) sv = *reinterpret_cast<const float *>(st + fs);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      raw[e] = *reinterpret_cast<const int *>(st + fq + (32 * KK + e) * BK);
  };
  auto read_x = [&](const char *st, auto kk, int i) {
    fa[i] = *reinterpret_cast<const bf16x8 *>(st + (fx ^ (64 * decltype(kk)::value)) + 2048 * i);
  };
  auto widen = [&](auto kk, bf16x8 (&b)[TJ]) {
    constexpr int KK = decltype(kk)::value;
    b[0] = widen_scaled<KK, 0>(raw, sv);
    b[1] = widen_scaled<KK, 1>(raw, sv);
    b[2] = widen_scaled<KK, 2>(raw, sv);
    b[3] = widen_scaled<KK, 3>(raw, sv);
  };
  // the products of the half in fa and b; st and kk: the next half
  auto half = [&](const char *st, auto kk, const bf16x8 (&b)[TJ], bf16x8 (&next)[TJ]) {
    read_w(st, kk);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], b[j], acc[i][j], 0, 0, 0);
      read_x(st, kk, i);
    }
    widen(kk, next);
    __builtin_amdgcn_sched_group_barrier(0x100, 9, 0);  // DS reads: the weights
    __builtin_amdgcn_sched_group_barrier(0x008, TJ, 0);  // MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
    for (int i = 1; i < TI; ++i) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, TI == 8 ? 4 : 8, 0);  // VALU
      }
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  std::integral_constant<int, 0> h0;
  std::integral_constant<int, 1> h1;

  const int nk_all = (int)((N + BC - 1) / BC);
  const int kb = SPLIT ? sp * ks : 0;
  const int nk = (SPLIT ? (kb + ks < nk_all ? kb + ks : nk_all) : nk_all) - kb;  // stages
#pragma unroll
  for (int s = 0; s < SG; ++s) issue(s < nk ? kb + s : nk_all, s);
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(NL * (SG - 1)));
  __builtin_amdgcn_s_barrier();  // stage 0 complete everywhere
  const char *st = smem;
  read_w(st, h0);
#pragma unroll
  for (int i = 0; i < TI; ++i) read_x(st, h0, i);
  widen(h0, b0);
  // Stage t: its second half is read under the first half's products; then its
  // slot is free and takes stage t + SG (zeros past the last), stage t + 1 must
  // have landed, and its first half is read under the second half's products.
  int slot = 0;
  for (int t = 0; t < nk; ++t) {
    half(st, h1, b0, b1);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this wave's reads of the slot are done
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(NL * (SG - 2)));
    __builtin_amdgcn_s_barrier();
    issue(t + SG < nk ? kb + t + SG : nk_all, slot);
    slot = slot + 1 == SG ? 0 : slot + 1;
    st = smem + slot * L::STAGE;
    half(st, h0, b1, b0);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __syncthreads();

  if constexpr (SPLIT) {
    float *tf = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<f32x4 *>(tf + (i * 16 + 4 * g + v) * L::TLDF + 64 * wave + 4 * r) =
            f32x4{acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
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
  // acc[i][j] lane (r, g): rows 16 i + 4 g + v, column 64 wave + 4 r + j
  if constexpr (LT::on) lora_add_tile<true>(acc, lt, m0, M, k0 + 64 * wave);
  uint16_t *tl = reinterpret_cast<uint16_t *>(smem);
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint32_t lo = f32_to_bf16_rne(acc[i][0][v]) | ((uint32_t)f32_to_bf16_rne(acc[i][1][v]) << 16);
      const uint32_t hi = f32_to_bf16_rne(acc[i][2][v]) | ((uint32_t)f32_to_bf16_rne(acc[i][3][v]) << 16);
      *reinterpret_cast<i32x2 *>(tl + (i * 16 + 4 * g + v) * L::TLD + 64 * wave + 4 * r) =
          i32x2{(int)lo, (int)hi};
    }
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

template <int TI, int SG, class LT>
hipError_t go(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q, const float *scale,
              int64_t K, uint16_t *dx, hipStream_t st, const LT &lt) {
  using L = DgradLds<TI, SG>;
  void (*kern)(const uint16_t *, const int8_t *, const float *, uint16_t *, int64_t, int64_t, int64_t,
               int, int, float *, int, LT) = k_w8a16_dgrad<TI, SG, false, LT>;
  (void)hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize,
                            L::BYTES);
  (void)hipGetLastError();
  const int tm = (int)((M + L::BM - 1) / L::BM), tk = (int)((K + L::BK - 1) / L::BK);
  hipLaunchKernelGGL(kern, dim3((unsigned)(tm * tk)), dim3(64 * NWV), L::BYTES, st, dy, q, scale,
                     dx, M, N, K, tm, tk, (float *)nullptr, 0, lt);
  return hipGetLastError();
}

template <int TI, int SG, class LT>
hipError_t go_split(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q, const float *scale,
                    int64_t K, uint16_t *dx, float *part, int S, hipStream_t st, const LT &lt) {
  using L = DgradLds<TI, SG>;
  void (*kern)(const uint16_t *, const int8_t *, const float *, uint16_t *, int64_t, int64_t, int64_t,
               int, int, float *, int, NoLora) = k_w8a16_dgrad<TI, SG, true, NoLora>;
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
  if (twide >= 160) return go<8, 4>(dy, M, N, q, scale, K, dx, st, lt);
  const int S = w8a16_dgrad_splits(M, N, K);
  if (S > 1 && part && part_bytes >= w8a16_dgrad_part_bytes(M, N, K))
    return go_split<4, 4>(dy, M, N, q, scale, K, dx, part, S, st, lt);
  return go<4, 4>(dy, M, N, q, scale, K, dx, st, lt);
}

}  // namespace

// 64 x 256 tiles split while the units stay within two a CU and each keeps at
// least 8 stages of 64 channels.
int w8a16_dgrad_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t twide = ((M + 127) / 128) * ((K + 255) / 256);
  if (twide >= 160) return 1;
  const int64_t tiles = ((M + 63) / 64) * ((K + 255) / 256), nk = (N + BC - 1) / BC;
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
