// The two forms of the dense tensor-core products: CTA pairs for many rows
// (dense_gemm_sm100.cu), weights as the 128-row operand for few
// (dense_skinny_sm100.cu).
#pragma once

#include "dense.cuh"

namespace moe {

// CTA pairs the tile rules count on: a constant, so that a choice depends on
// the sizes alone.
constexpr int kDensePairs = 74;

// Reduction steps (64 deep, 256 columns) of the rounds that the pair kernel's
// busiest pair runs, a split's overhead among them.
double dense_fwd_pairs_steps(int64_t T, int K, int N, bool gated);
double dense_dgrad_pairs_steps(int64_t T, int K, int N, int segs);
// CTAs of the pair kernel's input and weight gradients, and the latter's
// estimated time.
int dense_dgrad_pairs_ctas(int64_t T, int K, int N, int segs);
int dense_wgrad_ctas(int64_t T, int K, int N, int problems, bool split);
double dense_wgrad_us(int64_t T, int K, int N, int problems, bool split);
size_t dense_fwd_pairs_part_floats(int64_t T, int K, int N, bool gated);
size_t dense_dgrad_pairs_part_floats(int64_t T, int K, int N, int segs);
cudaError_t launch_dense_fwd_pairs(const void* x, const void* w0, const void* w1, int64_t T, int K, int N,
                                   const DenseOut& o, const DenseWs& ws, cudaStream_t st);
// opens_gate: for a weight gradient that starts beside this kernel.
cudaError_t launch_dense_dgrad_pairs(const void* dz0, const void* dz1, const void* w0, const void* w1, int64_t T,
                                     int K, int N, void* dx, bool opens_gate, const DenseWs& ws, cudaStream_t st);

}  // namespace moe
