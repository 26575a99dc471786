// Elementwise half of the linear and gate/up backward passes (sm_100a): the
// gradients of the pre-activations and the bias gradients.
//
//   linear: dz = dy act'(z);            db = sum over tokens of dz
//   gated:  dg = dh u act'(g), du = dh act(g);  dbg, dbu their sums
//
// Bound by HBM: each input is read once and dz (dg, du) written once, rounded
// to bf16 because it is an operand of the tensor-core products that follow;
// the bias gradients are summed from the unrounded float32 values.  A thread
// owns 8 columns (one 16-byte access per tensor and row) and walks every 8th
// row of its block's range; the block adds its 8 row lanes in shared memory
// and writes one partial row, which launch_sum_partials adds in order.
#include <algorithm>

#include "act.cuh"
#include "dense.cuh"
#include "sm100_dense.cuh"
#include "tma_host.cuh"

namespace moe {
namespace {

constexpr int kCols = 256;  // columns per block: 32 threads x 8
constexpr int kLanes = 8;   // row lanes per block
// Blocks of an SM at once: the grid is one wave of them (a second, partial wave
// cost a third of the time), each walking as many rows as that takes.
constexpr int kBlocksLinear = 6, kBlocksGated = 4;

__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8]) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// kAct: the activation; kGated: dg and du from dh, g, u.  A linear layer without
// an activation has dy itself for dz: column sums alone.
template <int kAct, bool kGated>
__global__ void __launch_bounds__(32 * kLanes, kGated ? kBlocksGated : kBlocksLinear) dense_dz_kernel(const DenseDzArgs a) {
    __shared__ float red[kLanes][kCols + 4];
    sm100::chain_wait();
    sm100::chain_next();
    const int c = blockIdx.x * kCols + threadIdx.x * 8;
    const int64_t r0 = (int64_t)blockIdx.y * a.rows_per_block;
    const int64_t r1 = min(r0 + a.rows_per_block, (int64_t)a.T);
    float s0[8] = {}, s1[8] = {};
    if (c < a.N) {
        for (int64_t r = r0 + threadIdx.y; r < r1; r += kLanes) {
            const int64_t o = r * a.N + c;
            float d[8], z[8], u[8];
            unpack8(*reinterpret_cast<const uint4*>(a.dy + o), d);
            if (kAct != MOE_ACT_NONE || kGated) unpack8(*reinterpret_cast<const uint4*>(a.z + o), z);
            if (kGated) unpack8(*reinterpret_cast<const uint4*>(a.u + o), u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (kGated) {
                    float v, sl;
                    act_slope<kAct>(z[j], v, sl);
                    z[j] = d[j] * u[j] * sl;
                    d[j] *= v;
                    s0[j] += z[j];
                    s1[j] += d[j];
                } else {
                    if (kAct != MOE_ACT_NONE) {
                        float v, sl;
                        act_slope<kAct>(z[j], v, sl);
                        d[j] *= sl;
                    }
                    s0[j] += d[j];
                }
            }
            if (kGated) {
                *reinterpret_cast<uint4*>(a.dz + o) = pack8(z);
                *reinterpret_cast<uint4*>(a.dz1 + o) = pack8(d);
            } else if (kAct != MOE_ACT_NONE) {
                *reinterpret_cast<uint4*>(a.dz + o) = pack8(d);
            }
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int which = 0; which < (kGated ? 2 : 1); ++which) {
        float* dst = red[threadIdx.y] + threadIdx.x * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = which ? s1[j] : s0[j];
        __syncthreads();
        const int cc = threadIdx.y * 32 + threadIdx.x;  // one column per thread
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kLanes; ++k) v += red[k][cc];
        const int col = blockIdx.x * kCols + cc;
        if (col < a.N) a.part[((int64_t)blockIdx.y * (kGated ? 2 : 1) + which) * a.N + col] = v;
        __syncthreads();
    }
}

}  // namespace

// Row ranges: one wave of blocks, each of at least 8 rows.
int dense_dz_row_blocks(int64_t T, int64_t N, bool gated) {
    const int64_t cb = (N + kCols - 1) / kCols;
    const int64_t want = std::max<int64_t>(1, 148 * (gated ? kBlocksGated : kBlocksLinear) / cb);
    return (int)std::min<int64_t>(want, std::max<int64_t>(1, (T + kLanes - 1) / kLanes));
}

cudaError_t launch_dense_dz(DenseDzArgs a, bool gated, int act, float* db0, float* db1, cudaStream_t st) {
    const int rb = dense_dz_row_blocks(a.T, a.N, gated);
    a.rows_per_block = (a.T + rb - 1) / rb;
    if (!(db0 || db1)) a.part = nullptr;
    const dim3 grid((a.N + kCols - 1) / kCols, rb), block(32, kLanes);
    trace_before(gated ? "gated_dgu" : "linear_dz", st);
    cudaError_t e = cudaSuccess;
    by_act(act, [&](auto k) {
        auto* fn = gated ? dense_dz_kernel<k.value, true> : dense_dz_kernel<k.value, false>;
        e = launch_chained(fn, grid, block, 0, 0, st, a);
    });
    trace_after(st);
    if (e != cudaSuccess || !a.part) return e;
    const int per = gated ? 2 : 1;
    return launch_sum_partials(a.part, (int64_t)per * a.N, rb, a.N, a.N, db0, gated ? db1 : nullptr, st);
}

}  // namespace moe
