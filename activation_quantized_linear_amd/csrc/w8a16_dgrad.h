// Gradient of the W8A16 linear to its input (internal to libaql.so).
#pragma once

#include "common.h"
#include "lora.h"

namespace aql {

// Bytes of the workspace: dy times the scales in float16 [M, N rounded up to 64],
// an exponent a row, and the partial sums of shapes that split the contraction.
size_t w8a16_dgrad_bytes(int64_t M, int64_t N, int64_t K);

// dx[m, k] = bf16(sum_n dy[m, n] scale[n] q[n, k] (+ sum_j u[m, j] A[a][j, k]));
// N % 8 == 0, K % 16 == 0, K <= 2^24, N <= 2^22. ws: as above.
hipError_t launch_w8a16_dgrad(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q,
                              const float *scale, int64_t K, uint16_t *dx, void *ws,
                              hipStream_t st);
// lt: h = u [M, R], W = A [L, R, K], N = K.
hipError_t launch_w8a16_dgrad(const uint16_t *dy, int64_t M, int64_t N, const int8_t *q,
                              const float *scale, int64_t K, uint16_t *dx, void *ws,
                              hipStream_t st, const LoraTerm &lt);

}  // namespace aql
