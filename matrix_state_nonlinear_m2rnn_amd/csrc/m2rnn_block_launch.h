// Launchers of block kernels that the recurrence's entry points use (defined in m2rnn_block.hip,
// so that the block kernels are compiled in one translation unit only).
#pragma once

#include <hip/hip_runtime.h>

namespace m2rnn {

// Widest token row (N V features) of the output gate + RMSNorm.
constexpr long kNormMaxFeatures = 8192;

// The block forward's output epilogue over the tokens t0 .. t0 + len - 1 of every batch entry of
// a [B, T] sequence of D features: y from the S readout planes part[S][B*T][D] (+ w_r (.) v when
// w_r is set), then out = RMSNorm(y (.) SiLU(gz)) * gamma.  Returns a hipError_t.
int launch_fwd_finish_norm(const float* part, int S, const void* v, bool v_bf16, const float* w_r, const void* gz,
                           bool gz_bf16, const float* gamma, long B, long T, long t0, long len, int D, float eps,
                           float* out, hipStream_t stream);

// Floats of scratch that sum_rows needs for `parts` rows of M columns.
size_t sum_rows_scratch(long parts, long M);

// Sums `parts` rows of M contiguous floats into one row by a fixed tree (zeros for no rows): columns
// j < M0 to out0[j], the others to out1[j - M0].
void sum_rows(const float* part, long parts, long M, float* out0, long M0, float* out1, float* scratch,
              hipStream_t stream);

}  // namespace m2rnn
