// Launch arguments of the operators around the routed layer: row norms, the
// gate/up projections and the linear layer (norm.cu, dense_*.cu).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxNormWidth = 16384;  // longest row: 512 threads x 32 elements
// SMs the norms' grid is sized for: a constant, so that the number of
// partial sums, and with it the bits of dw and db, is a function of the sizes
// alone.
constexpr int kNormSms = 148;

struct NormArgs {
    int64_t T;
    int H;
    bool layer;  // false: RMS form
    float eps;
    const void* x;
    const float* w;  // [H] or null (ones)
    const float* b;  // [H] or null (zeros)
    void* y;
    float* mean_out;  // [T] or null
    float* rstd_out;
    // backward
    const void* dy;
    const float* mean;
    const float* rstd;
    const void* d_res;  // [T, H] or null
    void* dx;
    float* part;  // [norm_bwd_blocks][2][H], null when neither dw nor db is wanted
    float* dw_out;
    float* db_out;
};

// CTAs (= partial rows) of the backward norm.
int norm_bwd_blocks(int64_t T);
cudaError_t launch_norm_fwd(const NormArgs& a, bool f32, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs& a, bool f32, bool dy_f32, cudaStream_t st);
// out0[c] = sum over p < P of part[p * stride + c]; out1 (when non-null) the
// same of the values `second` floats further on.
cudaError_t launch_sum_partials(const float* part, int64_t stride, int P, int64_t second, int N, float* out0,
                                float* out1, cudaStream_t st);

struct DenseDzArgs {
    int64_t T;
    int N;
    int64_t rows_per_block;  // set by the launcher
    const bf16* dy;          // [T, N]
    const bf16* z;           // [T, N] pre-activations (gated: g)
    const bf16* u;           // gated
    bf16* dz;                // [T, N] (gated: dg); not written for a linear layer without activation
    bf16* dz1;               // gated: du
    float* part;             // [dense_dz_row_blocks][1 or 2][N]
};

int dense_dz_row_blocks(int64_t T, int64_t N, bool gated);
// dz (dg, du) and, where db0 / db1 are non-null, the bias gradients.
cudaError_t launch_dense_dz(DenseDzArgs a, bool gated, int act, float* db0, float* db1, cudaStream_t st);
// ---- tensor-core products (operands bf16, row-major, float32 accumulators)
struct DenseOut {
    int act;
    const float* bias0;  // [N] or null (gated: gate)
    const float* bias1;  // gated: up
    const bf16* res;     // [T, N] or null, added after the activation
    bf16* y;             // [T, N]
    bf16* z0;            // [T, N] or null: pre-activations (gated: g)
    bf16* z1;            // gated: u
};

// Workspace of one product.
struct DenseWs {
    int32_t* flags;
    uint32_t* counters;  // zero between calls
    uint32_t* gate;      // two words, zero between calls: the backward products' (sm100_dense.cuh)
    float* part;         // the product's ..._part_floats
};
constexpr size_t kDenseCounterBytes = 4864;  // of one product, and the gate
constexpr size_t kDenseGateOffset = kDenseCounterBytes - 128;

// y = act(x W^T + b) + res; gated (w1 non-null): y = act(x W0^T + b0) (x W1^T + b1).
size_t dense_fwd_part_floats(int64_t T, int K, int N, bool gated);
cudaError_t launch_dense_fwd(const void* x, const void* w0, const void* w1, int64_t T, int K, int N,
                             const DenseOut& o, const DenseWs& ws, cudaStream_t st);
// How a weight gradient runs: its last wave's tiles split over the tokens where
// that pays; beside: it may start before the launch_dense_dgrad of the same dz
// just before it on the stream has completed.
struct WgradPlan {
    bool split, beside;
};
// dx [T, K] = dz0 W0 (+ dz1 W1), dz [T, N], W [N, K]; segs = 1 or 2 products.
// with_wgrad: launch_dense_wgrad of the same dz comes next, with *plan.
size_t dense_dgrad_part_floats(int64_t T, int K, int N, int segs);
cudaError_t launch_dense_dgrad(const void* dz0, const void* dz1, const void* w0, const void* w1, int64_t T, int K,
                               int N, void* dx, bool with_wgrad, WgradPlan* plan, const DenseWs& ws,
                               cudaStream_t st);
// dW_p [N, K] = dz_p^T x for one or two dz.  ws has other partial sums and
// counters than the input gradient's.
size_t dense_wgrad_part_floats(int64_t T, int K, int N, int problems);
cudaError_t launch_dense_wgrad(const void* dz0, const void* dz1, const void* x, int64_t T, int K, int N, void* dw0,
                               void* dw1, bool f32, WgradPlan plan, const DenseWs& ws, cudaStream_t st);

}  // namespace moe
