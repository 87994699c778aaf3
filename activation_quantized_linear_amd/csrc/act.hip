// The gradients of y = act(v) * mul + residual, elementwise:
//   dv = dy * mul * act'(v),   dmul = dy * act(v)      (dresidual = dy)
// with v as the forward pass kept it. Bound by memory, 10 bytes an element with mul. A thread
// takes kIlp times 8 elements, 16 bytes a load, all of them out before the first is used.
#include "act.h"

namespace aql {
namespace {

constexpr int kIlp = 2;

// Elements of one launch: a grid holds fewer than 2^32 threads.
constexpr int64_t kSlice = 1LL << 32;
static_assert(kSlice % (256 * 8 * kIlp) == 0 && kSlice / (8 * kIlp) < (1LL << 32), "one grid");

__device__ __forceinline__ i32x4 load8(const uint16_t *p, int64_t i, int64_t n) {
  if (i + 8 <= n) return *reinterpret_cast<const i32x4 *>(p + i);
  i32x4 d = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) d[e >> 1] |= (int)((uint32_t)p[i + e] << (16 * (e & 1)));
  return d;
}

__device__ __forceinline__ void store8(uint16_t *p, int64_t i, int64_t n, const i32x4 &d) {
  if (i + 8 <= n) {
    *reinterpret_cast<i32x4 *>(p + i) = d;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) p[i + e] = (uint16_t)((uint32_t)d[e >> 1] >> (16 * (e & 1)));
}

__device__ __forceinline__ float half_of(const i32x4 &d, int e) {
  return __uint_as_float(e & 1 ? (uint32_t)d[e >> 1] & 0xffff0000u : (uint32_t)d[e >> 1] << 16);
}

template <int ACT, bool MUL>
__global__ __launch_bounds__(256) void k_act_mul_backward(const uint16_t *dy, const uint16_t *pre,
                                                          const uint16_t *mul, int64_t first,
                                                          int64_t n, uint16_t *dv,
                                                          uint16_t *dmul) {
  const int64_t base = first + (int64_t)blockIdx.x * (256 * 8 * kIlp) + 8 * threadIdx.x;
  i32x4 g[kIlp], z[kIlp], f[kIlp];
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    const int64_t i = base + u * (256 * 8);
    g[u] = load8(dy, i, n);
    z[u] = load8(pre, i, n);
    if constexpr (MUL) f[u] = load8(mul, i, n);
  }
#pragma unroll
  for (int u = 0; u < kIlp; ++u) {
    const int64_t i = base + u * (256 * 8);
    i32x4 o, p;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t ov = 0, pv = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = 2 * w + h;
        float a, d;
        act_value_grad<ACT>(half_of(z[u], e), a, d);
        const float gy = half_of(g[u], e);
        float v = gy * d;
        if constexpr (MUL) {
          v = gy * half_of(f[u], e) * d;
          pv |= (uint32_t)f32_to_bf16_rne(gy * a) << (16 * h);
        }
        ov |= (uint32_t)f32_to_bf16_rne(v) << (16 * h);
      }
      o[w] = (int)ov;
      p[w] = (int)pv;
    }
    store8(dv, i, n, o);
    if constexpr (MUL)
      if (dmul) store8(dmul, i, n, p);
  }
}

template <int ACT>
hipError_t launch(const uint16_t *dy, const uint16_t *pre, const uint16_t *mul, int64_t n,
                  uint16_t *dv, uint16_t *dmul, hipStream_t st) {
  for (int64_t first = 0; first < n; first += kSlice) {
    const int64_t m = n - first < kSlice ? n - first : kSlice;
    const dim3 grid((unsigned)((m + 256 * 8 * kIlp - 1) / (256 * 8 * kIlp)));
    if (mul)
      hipLaunchKernelGGL((k_act_mul_backward<ACT, true>), grid, dim3(256), 0, st, dy, pre, mul,
                         first, n, dv, dmul);
    else
      hipLaunchKernelGGL((k_act_mul_backward<ACT, false>), grid, dim3(256), 0, st, dy, pre, mul,
                         first, n, dv, dmul);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_act_mul_backward(const uint16_t *dy, const uint16_t *pre, int act,
                                   const uint16_t *mul, int64_t n, uint16_t *dv, uint16_t *dmul,
                                   hipStream_t st) {
  switch (act) {
    case kActRelu: return launch<kActRelu>(dy, pre, mul, n, dv, dmul, st);
    case kActGelu: return launch<kActGelu>(dy, pre, mul, n, dv, dmul, st);
    case kActGeluTanh: return launch<kActGeluTanh>(dy, pre, mul, n, dv, dmul, st);
    case kActSilu: return launch<kActSilu>(dy, pre, mul, n, dv, dmul, st);
    default: return launch<kActNone>(dy, pre, mul, n, dv, dmul, st);
  }
}

}  // namespace aql
