// Activation checkpoints in 8 bits (internal to libaql.so).
#pragma once

#include "common.h"

namespace aql {

constexpr int kCkptGroup = 128;  // values of a row that share one scale

hipError_t launch_act_checkpoint(const void *x, bool bf16, int64_t M, int64_t K, int8_t *xq,
                                 float *xs, hipStream_t st);
hipError_t launch_act_restore(const int8_t *xq, const float *xs, int64_t M, int64_t K, void *x,
                              bool bf16, hipStream_t st);

}  // namespace aql
