// The two forms of the dense tensor-core products: CTA pairs for many rows
// (dense_gemm_sm100.cu), weights as the 128-row operand for few
// (dense_skinny_sm100.cu).
#pragma once

#include "dense.cuh"

namespace moe {

// CTA pairs the tile rules count on: a constant, so that a choice depends on
// the sizes alone.
constexpr int kDensePairs = 74;

cudaError_t launch_dense_fwd_pairs(const void* x, const void* w0, const void* w1, int64_t T, int K, int N,
                                   const DenseOut& o, int32_t* flags, cudaStream_t st);
cudaError_t launch_dense_dgrad_pairs(const void* dz0, const void* dz1, const void* w0, const void* w1, int64_t T,
                                     int K, int N, void* dx, int32_t* flags, cudaStream_t st);

}  // namespace moe
