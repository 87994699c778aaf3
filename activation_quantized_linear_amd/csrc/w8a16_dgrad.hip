// Gradient of the W8A16 linear to its input: dx[m, k] = sum_n dy[m, n] scale[n] q[n, k].
//
// The contraction runs over the output channels, so the channel scale does not
// factor out of the sum. It goes to dy's side, once per element instead of once
// per use of a weight: a first kernel writes d[m, n] = dy[m, n] scale[n] 2^e[m]
// as float16, the row's exponent e[m] bringing its largest product to
// [2^13, 2^14). float16 holds 11 bits where bf16 holds 8, so this rounding
// (2^-11 at most, and 2^-38 of the row's largest product for the tiny ones that
// become subnormal) vanishes beside the output's, and the int8 codes are exact
// in it. The product then runs on the float16 matrix cores with float32 sums,
// and 2^-e comes back in the epilogue.
//
// Tile: 16 TI rows of d x 256 columns of dx per workgroup of 4 waves side by
// side along K, each 16 TI x 64, over stages of 64 channels. Operands go
// global -> LDS by buffer loads that write LDS directly: d as rows of 128 B, the
// weights as they lie, 64 channel rows of 256 B. q has the contraction as its
// slow axis: a lane reads one dword (4 columns) of each of the 8 channel rows it
// needs, and byte j of the eight is its operand for columns 4 r + j, so the
// matrix instructions take the columns in strides of 4 and nothing is
// transposed, in memory or in registers. d is padded with zeros to whole
// stages, so what the last stage reads past N in q adds nothing.
// Measured at M = 2048, K = 4096, in a run of such calls: N = 11008 in 151 us, 1225
// TFLOP/s, and 20 us for the scaling; N = 14336 in 195 us and 23 (a bf16 library
// product of that shape, on weights of twice the bytes: 251). The first milliseconds of
// a burst run 10 to 20% slower, until the clock has risen. The matrix cores are busy
// for 1024 of a stage's 1550 cycles, and what more they do the clock takes back (1.9
// to 2.0 GHz under this load): the same work on 32x32x16 instructions or with two
// workgroups a CU took as long.
// A ring of SG stages keeps loads in flight behind exact vmcnt waits. d rows
// store their 16-byte chunks XOR-swizzled by (row / 2) mod 8, and weight rows
// theirs by 4 (row / 8 mod 4), which spreads each read over all banks.
#include "w8a16_dgrad.h"

#include <type_traits>

namespace aql {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int BC = kDgradStage;  // channels a stage
constexpr int kCode = 9;         // codes enter the matrix cores as q 2^-9

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// ------------------------------------------------------------- scaling of dy

template <int NI>
__global__ __launch_bounds__(256) void k_dgrad_scale(DgradScale a) {
  __shared__ float red[4];
  dgrad_scale_row<NI>(a, blockIdx.x, threadIdx.x, red);
}

// ------------------------------------------------------------------- product

// 16 bytes a lane from offsets off + soff into LDS at dst + 16 lane.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t rr, uint32_t dst, int off, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rr, (lds_void *)(uintptr_t)__builtin_amdgcn_readfirstlane(dst), 16, off, soff, 0, 0);
}

constexpr int vmcnt_imm(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }

template <int I, int N, class F>
__device__ __forceinline__ void static_for(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}

constexpr int NWV = 4, TJ = 4;  // waves of a workgroup, 16-column blocks of a wave

template <int TI, int SG>
struct DgradLds {
  static constexpr int BM = 16 * TI, BK = 256;
  static constexpr int NX = BM / 8 / NWV;  // d loads per wave and stage (8 rows x 128 B)
  static constexpr int NQ = BC * BK / 1024 / NWV;  // weight loads (1 KB each)
  static constexpr int NL = NX + NQ;
  static constexpr int XS = BM * 128, QS = BC * BK;
  static constexpr int STAGE = XS + QS;
  static constexpr int RING = SG * STAGE;
  static constexpr int TLD = BK + 8;  // bf16 per staged output row
  static constexpr int TILE = BM * TLD * 2;
  static constexpr int TLDF = BK + 4;  // fp32 per staged partial-sum row
  static constexpr int TILEF = BM * TLDF * 4;
  static constexpr int BYTES = RING > TILE ? RING : TILE;
  static constexpr int BYTES_SPLIT = RING > TILEF ? RING : TILEF;
  static_assert(BYTES >= LoraLds<BM, BK, true, 2>::BYTES, "the adapter terms stage in the ring");
  static_assert(NX * NWV * 8 == BM && NQ * NWV * 1024 == BC * BK, "loads split evenly");
  static_assert(NL * (SG - 2) < 64, "vmcnt");
};

// Byte J of two dwords of biased codes u = q + 128 -> the low bytes of a pair of
// 16-bit halves.
template <int J>
__device__ __forceinline__ int byte_pair(int lo, int hi) {
  return (int)__builtin_amdgcn_perm((uint32_t)hi, (uint32_t)lo,
                                    0x0c000c00u | (uint32_t)J | ((uint32_t)(J + 4) << 16));
}

// Such a pair -> float16 q 2^-9, exactly: a byte alone is the subnormal u 2^-24,
// and one packed multiply-add takes it to u 2^-9 - 128 2^-9.
__device__ __forceinline__ int unbias(int u) {
  const f16x2 r = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, u),
                                            f16x2{(_Float16)32768.0f, (_Float16)32768.0f},
                                            f16x2{(_Float16)-0.25f, (_Float16)-0.25f});
  return __builtin_bit_cast(int, r);
}

// SPLIT: unit (tile, sp) takes the ks stages from sp * ks and writes its fp32
// sums to part[sp][M][K]; k_w8a16_dgrad_reduce adds them.
template <int TI, int SG, bool SPLIT, class LT>
__global__ __launch_bounds__(64 * NWV, 2) void k_w8a16_dgrad(
    const uint16_t *__restrict__ d, const int32_t *__restrict__ ex, const int8_t *__restrict__ q,
    uint16_t *__restrict__ dx, int64_t M, int64_t N, int64_t NP, int64_t K, int tiles_m,
    int tiles_k, float *__restrict__ part, int ks, LT lt) {
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
  // rows past M lie past the descriptor's end: they read as zero
  const __amdgpu_buffer_rsrc_t rx = rsrc(d + m0 * NP, (uint32_t)(mval * NP * 2));

  // load i of a wave covers d rows 32 i + 8 wave + lane / 8 and weight rows
  // 16 i + 4 wave + lane / 16; the rows' 32 i and 16 i are scalar offsets (they
  // leave d's swizzle alone and flip bit 3 of the weights' chunk for odd i)
  const int xr = 8 * wave + (lane >> 3), qr = 4 * wave + (lane >> 4);
  const int xoff = xr * (int)(2 * NP) + 16 * ((lane & 7) ^ ((xr >> 1) & 7));
  const int qc = (lane & 15) ^ (4 * (qr >> 3));
  const int qoff[2] = {qr * (int)K + 16 * qc, qr * (int)K + 16 * (qc ^ 8)};
  const int nk_all = (int)(NP / BC);
  const int kb = SPLIT ? sp * ks : 0;
  const int nk = (SPLIT ? (kb + ks < nk_all ? kb + ks : nk_all) : nk_all) - kb;  // stages

  const uint32_t lds_base = (uint32_t)(uintptr_t)smem;
  // Where the next stage to load lies; past the last stage it stays on the last
  // one (loaded again, never computed: the counts of loads in flight stay exact).
  int xs = 128 * kb, left_x = nk - 1, left_w = nk - 1;
  const int8_t *wp = q + (int64_t)BC * kb * K + k0;
  uint64_t wleft = (uint64_t)(N * K - ((int64_t)BC * kb * K + k0));
  auto next_x = [&]() {
    xs += left_x > 0 ? 128 : 0;
    --left_x;
  };
  auto next_w = [&]() {
    const uint32_t step = left_w > 0 ? (uint32_t)BC * (uint32_t)K : 0u;
    wp += step;
    wleft -= step;
    --left_w;
  };
  // columns past K read the next row (or, at the end of q, zero) into columns of
  // the tile that are never stored
  auto weights = [&]() {
    const uint32_t hi = (uint32_t)(wleft >> 32), lo = (uint32_t)wleft;
    return rsrc(wp, hi != 0 || lo > 0x7fffffffu ? 0x7fffffffu : lo);
  };
  // load I of d's NX, of the weights' NQ, into ring slot `slot`
  auto load_x = [&](int slot, auto ii) {
    constexpr int I = decltype(ii)::value;
    to_lds(rx, lds_base + (uint32_t)(slot * L::STAGE) + 1024u * (I * NWV + wave), xoff,
           I * 64 * (int)NP + xs);
  };
  auto load_w = [&](__amdgpu_buffer_rsrc_t rq, int slot, auto ii) {
    constexpr int I = decltype(ii)::value;
    to_lds(rq, lds_base + (uint32_t)(slot * L::STAGE) + L::XS + 1024u * (I * NWV + wave),
           qoff[I & 1], I * 16 * (int)K);
  };

  // fragment offsets within a stage. d: block i adds 2048 i, half kk flips bit
  // 6 (chunk 4 kk + g under the swizzle); weights: half kk adds 32 rows, channel
  // e of the lane's eight adds e rows
  const int fx = r * 128 + 16 * (g ^ ((r >> 1) & 7));
  const int fq = L::XS + 8 * g * BK + 16 * ((4 * wave + (r >> 2)) ^ (4 * g)) + 4 * (r & 3);

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Software pipeline over the 32-channel halves of the stages, written in the
  // order it issues in: one wave a SIMD has nobody to hide behind, so what comes
  // between two matrix instructions has to fit the 16 cycles of one (three other
  // instructions). While the matrix core works on one half, the next half's
  // weights come from LDS and are widened, and block i of d is replaced by the
  // next half's once its products are issued, so only the widened weights are
  // held twice.
  f16x8 fa[TI];
  i32x4 wb[2][TJ];
  int raw[8];
  auto read_w = [&](const char *st, auto kk, int e) {  // rows e and e + 1
    const char *w = st + fq + (32 * decltype(kk)::value + e) * BK;
    raw[e] = *reinterpret_cast<const int *>(w);
    raw[e + 1] = *reinterpret_cast<const int *>(w + BK);
  };
  auto read_x = [&](const char *st, auto kk, int i) {
    fa[i] = *reinterpret_cast<const f16x8 *>(st + (fx ^ (64 * decltype(kk)::value)) + 2048 * i);
  };
  // The widening in 40 single instructions: per pair of rows P the bias of both
  // dwords and block 0's pair (4), then the other blocks' pairs (2 each).
  constexpr int STEPS = 40;
  auto widen = [&](i32x4 (&b)[TJ], auto uu) {
    constexpr int U = decltype(uu)::value;
    constexpr int J = U < 16 ? 0 : 1 + (U - 16) / 8, P = U < 16 ? U / 4 : (U - 16) / 2 % 4;
    constexpr int W = U < 16 ? U % 4 : 2 + U % 2;
    if constexpr (W < 2) raw[2 * P + W] ^= 0x80808080;
    if constexpr (W == 2) b[J][P] = byte_pair<J>(raw[2 * P], raw[2 * P + 1]);
    if constexpr (W == 3) b[J][P] = unbias(b[J][P]);
  };
  auto mma = [&](const i32x4 (&b)[TJ], int i, int j) {
    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
        fa[i], __builtin_bit_cast(f16x8, b[j]), acc[i][j], 0, 0, 0);
  };
  std::integral_constant<int, 0> h0;
  std::integral_constant<int, 1> h1;
  constexpr int SLOTS = TI * TJ;  // matrix instructions in a half
  LoraRows<BM> &adapters = *reinterpret_cast<LoraRows<BM> *>(smem + L::BYTES);

  if (nk > 0) {
#pragma unroll
    for (int s = 0; s < SG - 1; ++s) {
      static_for<0, NX>([&](auto ii) { load_x(s, ii); });
      next_x();
      const __amdgpu_buffer_rsrc_t rq = weights();
      static_for<0, NQ>([&](auto ii) { load_w(rq, s, ii); });
      next_w();
    }
    if constexpr (LT::on) lora_rows<BM, 64 * NWV>(adapters, lt, m0, M);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(NL * (SG - 2)));
    __builtin_amdgcn_s_barrier();  // stage 0 complete everywhere
#pragma unroll
    for (int e = 0; e < 8; e += 2) read_w(smem, h0, e);
#pragma unroll
    for (int i = 0; i < TI; ++i) read_x(smem, h0, i);
    static_for<0, STEPS>([&](auto uu) { widen(wb[0], uu); });
    const __amdgpu_buffer_rsrc_t rq = weights();
    static_for<0, NQ>([&](auto ii) { load_w(rq, SG - 1, ii); });
  }
  int slot = 0;
  for (int t = 0; t < nk; ++t) {
    const char *st = smem + slot * L::STAGE;
    const int prev = slot == 0 ? SG - 1 : slot - 1;
    // First half: its products and the second half's operands.
    static_for<0, SLOTS>([&](auto ss) {
      constexpr int S = decltype(ss)::value, I = S / TJ;
      mma(wb[0], I, S % TJ);
      if constexpr (S < 4) read_w(st, h1, 2 * S);
      constexpr int F = 4;  // first slot of the widening
      constexpr int U0 = S < F ? 0 : (S - F) * STEPS / (SLOTS - F);
      constexpr int U1 = S < F ? 0 : (S - F + 1) * STEPS / (SLOTS - F);
      static_for<U0, U1>([&](auto uu) { widen(wb[1], uu); });
      if constexpr (S % TJ == TJ - 1) read_x(st, h1, I);
      if constexpr (S == 1) next_w();
      __builtin_amdgcn_sched_barrier(0);
    });
    // Second half. Under its first products d's loads of stage t - 1 + SG go into
    // the slot that stage t - 1 left at the last barrier. Then this wave's reads
    // of stage t are done; past the barrier its slot is free, its first loads are
    // the weights of stage t + SG, and stage t + 1 has landed everywhere.
    const int freed = slot;
    slot = slot + 1 == SG ? 0 : slot + 1;
    st = smem + slot * L::STAGE;
    const __amdgpu_buffer_rsrc_t rq = weights();
    constexpr int SB = TI;  // matrix instructions before the barrier: TI / 4 blocks
    static_for<0, SLOTS>([&](auto ss) {
      constexpr int S = decltype(ss)::value, I = S / TJ;
      if constexpr (S == SB) {
        next_x();
        __builtin_amdgcn_s_waitcnt(0xC07F);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(NL * (SG - 2)));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      mma(wb[1], I, S % TJ);
      if constexpr (S < SB) {
        constexpr int L0 = S * NX / SB, L1 = (S + 1) * NX / SB;
        static_for<L0, L1>([&](auto ii) { load_x(prev, ii); });
      } else {
        if constexpr (S < SB + 4) read_w(st, h0, 2 * (S - SB));
        if constexpr (S >= SB + 2 && S < SB + 2 + SB / TJ) read_x(st, h0, S - SB - 2);
        if constexpr (S % TJ == TJ - 1) read_x(st, h0, I);
        constexpr int F = SB + 4;
        constexpr int U0 = S < F ? 0 : (S - F) * STEPS / (SLOTS - F);
        constexpr int U1 = S < F ? 0 : (S - F + 1) * STEPS / (SLOTS - F);
        static_for<U0, U1>([&](auto uu) { widen(wb[0], uu); });
        constexpr int L0 = (S - SB) * NQ / (SLOTS - SB), L1 = (S - SB + 1) * NQ / (SLOTS - SB);
        static_for<L0, L1>([&](auto ii) { load_w(rq, freed, ii); });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __syncthreads();

  // acc[i][j] lane (r, g): rows 16 i + 4 g + v, column 64 wave + 4 r + j; the
  // rows' exponents come off (ex is padded to whole tiles)
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const i32x4 e4 = *reinterpret_cast<const i32x4 *>(ex + m0 + 16 * i + 4 * g);
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][j][v] = ldexpf(acc[i][j][v], kCode - e4[v]);
  }
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
  if constexpr (LT::on) {
    if (nk == 0) lora_rows<BM, 64 * NWV>(adapters, lt, m0, M);
    lora_add_tile<BM, BK, 64 * NWV, true, 2>(smem, adapters, acc, lt, m0, k0, 0, 64 * wave);
  }
  uint16_t *tl = reinterpret_cast<uint16_t *>(smem);
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint32_t lo =
          f32_to_bf16_rne(acc[i][0][v]) | ((uint32_t)f32_to_bf16_rne(acc[i][1][v]) << 16);
      const uint32_t hi =
          f32_to_bf16_rne(acc[i][2][v]) | ((uint32_t)f32_to_bf16_rne(acc[i][3][v]) << 16);
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

template <class LT>
__global__ __launch_bounds__(256) void k_w8a16_dgrad_reduce(DgradParts p, LT lt) {
  dgrad_reduce(p, lt, (int64_t)blockIdx.x * 256 + threadIdx.x);
}

struct Call {
  const uint16_t *d;
  const int32_t *ex;
  const int8_t *q;
  uint16_t *dx;
  int64_t M, N, NP, K;
  float *part;
  hipStream_t st;
};

template <int TI, int SG, class LT>
hipError_t go(const Call &c, const LT &lt) {
  using L = DgradLds<TI, SG>;
  constexpr int bytes = L::BYTES + (LT::on ? sizeof(LoraRows<L::BM>) : 0);
  static bool attr_set = false;
  if (!attr_set) {  // more than 64 KB of dynamic LDS; a launch the limit refuses reports itself
    (void)hipFuncSetAttribute((const void *)k_w8a16_dgrad<TI, SG, false, LT>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    (void)hipGetLastError();
    attr_set = true;
  }
  const int tm = (int)((c.M + L::BM - 1) / L::BM), tk = (int)((c.K + L::BK - 1) / L::BK);
  hipLaunchKernelGGL((k_w8a16_dgrad<TI, SG, false, LT>), dim3((unsigned)(tm * tk)), dim3(64 * NWV),
                     bytes, c.st, c.d, c.ex, c.q, c.dx, c.M, c.N, c.NP, c.K, tm, tk,
                     (float *)nullptr, 0, lt);
  return hipGetLastError();
}

template <int TI, int SG, class LT>
hipError_t go_split(const Call &c, int S, const LT &lt, DgradParts *later) {
  using L = DgradLds<TI, SG>;
  static bool attr_set = false;
  if (!attr_set) {
    (void)hipFuncSetAttribute((const void *)k_w8a16_dgrad<TI, SG, true, NoLora>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, L::BYTES_SPLIT);
    (void)hipGetLastError();
    attr_set = true;
  }
  const int tm = (int)((c.M + L::BM - 1) / L::BM), tk = (int)((c.K + L::BK - 1) / L::BK);
  const int nk = (int)(c.NP / BC);
  const int ks = (nk + S - 1) / S, splits = (nk + ks - 1) / ks;
  hipLaunchKernelGGL((k_w8a16_dgrad<TI, SG, true, NoLora>), dim3((unsigned)(tm * tk * splits)),
                     dim3(64 * NWV), L::BYTES_SPLIT, c.st, c.d, c.ex, c.q, c.dx, c.M, c.N, c.NP,
                     c.K, tm, tk, c.part, ks, NoLora{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const DgradParts p{c.part, splits, c.M, c.K, c.dx};
  if (later) {
    *later = p;
    return e;
  }
  hipLaunchKernelGGL(k_w8a16_dgrad_reduce<LT>, dim3((unsigned)p.blocks()), dim3(256), 0, c.st, p,
                     lt);
  return hipGetLastError();
}

// 64 x 256 tiles split while the units stay within one a CU and each keeps at
// least 8 stages of 64 channels (M = 500, N = K = 4096: 33 us; 39 with two units a
// CU, whose partial sums cost more than the second unit hides, 41 with half a one;
// M = 333, N = 2560, K = 960: 18.7, 19.9 with 5 stages a unit).
int splits_of(int64_t M, int64_t N, int64_t K) {
  const int64_t twide = ((M + 127) / 128) * ((K + 255) / 256);
  if (twide >= 160) return 1;
  const int64_t tiles = ((M + 63) / 64) * ((K + 255) / 256), nk = (N + BC - 1) / BC;
  int S = 1;
  while (tiles * 2 * S <= 256 && nk / (2 * S) >= 8) S *= 2;
  return S;
}

// d [M, NP], the rows' exponents, the partial sums.
struct Layout {
  int64_t NP;
  size_t ex, part, total;
};
Layout layout(int64_t M, int64_t N, int64_t K) {
  Layout l;
  l.NP = (N + BC - 1) / BC * BC;
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  l.ex = up((size_t)M * (size_t)l.NP * 2);
  l.part = l.ex + up((size_t)(M + 127) / 128 * 128 * 4);
  const int S = splits_of(M, N, K);
  l.total = l.part + (S > 1 ? (size_t)S * (size_t)M * (size_t)K * 4 : 0);
  return l;
}

template <int NI>
hipError_t scale(const DgradScale &a, hipStream_t st) {
  hipLaunchKernelGGL(k_dgrad_scale<NI>, dim3((unsigned)a.M), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <class LT>
hipError_t launch(const DgradScale &a, const int8_t *q, int64_t K, uint16_t *dx, void *ws,
                  hipStream_t st, const LT &lt, DgradParts *later) {
  const Layout l = layout(a.M, a.N, K);
  const Call c{a.d, a.ex, q, dx, a.M, a.N, a.NP, K,
               reinterpret_cast<float *>(static_cast<char *>(ws) + l.part), st};
  const int64_t twide = ((a.M + 127) / 128) * ((K + 255) / 256);
  if (twide >= 160) return go<8, 4>(c, lt);
  const int S = splits_of(a.M, a.N, K);
  if (S > 1) return go_split<4, 4>(c, S, lt, later);
  return go<4, 4>(c, lt);
}

}  // namespace

bool w8a16_dgrad_split(int64_t M, int64_t N, int64_t K) { return splits_of(M, N, K) > 1; }

size_t w8a16_dgrad_bytes(int64_t M, int64_t N, int64_t K) { return layout(M, N, K).total; }

DgradScale w8a16_dgrad_scale_args(const uint16_t *dy, const float *scale, int64_t M, int64_t N,
                                  int64_t K, void *ws) {
  const Layout l = layout(M, N, K);
  char *base = static_cast<char *>(ws);
  return DgradScale{dy, scale, M, N, l.NP, reinterpret_cast<uint16_t *>(base),
                    reinterpret_cast<int32_t *>(base + l.ex)};
}

hipError_t launch_w8a16_dgrad(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q,
                              const float *s, int64_t K, uint16_t *dx, void *ws, hipStream_t st) {
  const DgradScale a = w8a16_dgrad_scale_args(dy, s, M, N, K, ws);
  hipError_t e;
  if (a.NP <= 2048) e = scale<1>(a, st);
  else if (a.NP <= 4096) e = scale<2>(a, st);
  else if (a.NP <= 8192) e = scale<4>(a, st);
  else if (a.NP <= 16384) e = scale<8>(a, st);
  else e = scale<0>(a, st);
  if (e != hipSuccess) return e;
  return launch(a, q, K, dx, ws, st, NoLora{}, nullptr);
}

hipError_t launch_w8a16_dgrad_scaled(const DgradScale &a, const int8_t *q, int64_t K, uint16_t *dx,
                                     void *ws, hipStream_t st, const LoraTerm &lt,
                                     DgradParts *later) {
  return launch(a, q, K, dx, ws, st, lt, later);
}

}  // namespace aql
