// Row norms in front of an FFN layer, forward and backward (sm_100a).
//
// Layer norm of a row x of H elements (the RMS form has mu = 0):
//   mu = mean(x),  r = (mean((x - mu)^2) + eps)^-1/2,  xh = (x - mu) r,
//   y = w xh + b.
// With the upstream gradient dy and a = w dy:
//   dx = r (a - mean(a) - xh mean(a xh))   (RMS form: without mean(a)),
//   dw = sum over rows of dy xh,  db = sum over rows of dy,
// and optionally the residual stream's own gradient is added to dx.
//
// Both directions are bound by HBM: 2 flops or so per byte.  A row is read
// once into registers (H <= 16384: up to four groups of 8 elements per
// thread), so the two reductions of the forward (mean, then the squared
// deviations from it: no cancellation) and the two sums of the backward need
// no second read.  Every sum and statistic is float32; y and dx are rounded
// once, to the layer type.
//
// The weight gradients are sums over all rows.  Each CTA walks rows
// blockIdx, blockIdx + grid, ... and keeps its own column sums in registers
// (its threads own fixed columns), writes one partial row per CTA at the end,
// and a second small kernel adds the partial rows in a fixed order: no
// atomics, the same bits on every run.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "tma_host.cuh"

namespace moe {
namespace {

constexpr int kWarpRowMax = 1024;  // rows up to this long: one warp per row
constexpr int kWarpsPerBlock = 8;  // of the warp-per-row kernels

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum of v over the threads of one row: the warp, or the whole block (every
// thread gets the same bits).  `red` is one of two 32-float buffers used in
// turn, so one barrier per sum is enough.
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if (kWarp) return v;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < (int)(blockDim.x / 32) ? red[lane] : 0.f);
}

template <typename X, int VPT, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpsPerBlock : 512) norm_fwd_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    const int g = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    const int64_t row = kWarp ? (int64_t)blockIdx.x * kWarpsPerBlock + threadIdx.x / 32 : blockIdx.x;
    if (kWarp && row >= a.T) return;
    const X* x = static_cast<const X*>(a.x) + row * a.H;
    float v[VPT][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * g + t) * 8;
        if (c < a.H) {
            load8(x + c, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        }
    }
    const float inv = 1.f / (float)a.H;
    const float mu = a.layer ? row_sum<kWarp>(s, red[0]) * inv : 0.f;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if ((i * g + t) * 8 < a.H) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] -= mu;
                s = fmaf(v[i][j], v[i][j], s);
            }
        }
    const float r = rsqrtf(row_sum<kWarp>(s, red[1]) * inv + a.eps);
    if (t == 0) {
        if (a.mean_out && a.layer) a.mean_out[row] = mu;
        if (a.rstd_out) a.rstd_out[row] = r;
    }
    X* y = static_cast<X*>(a.y) + row * a.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * g + t) * 8;
        if (c < a.H) {
            float w[8], b[8];
            if (a.w) load8(a.w + c, w);
            if (a.b) load8(a.b + c, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = v[i][j] * r;
                v[i][j] = a.w ? (a.b ? fmaf(xh, w[j], b[j]) : xh * w[j]) : (a.b ? xh + b[j] : xh);
            }
            store8(y + c, v[i]);
        }
    }
}

// One partial row of dw (and of db) per CTA: part[blockIdx][0 dw, 1 db][H].
template <typename X, typename G, int VPT, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpsPerBlock : 512) norm_bwd_kernel(const NormArgs a) {
    __shared__ float red[2][2][32];
    __shared__ float cols[kWarp ? kWarpsPerBlock * kWarpRowMax : 1];
    const int g = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    const int warp = threadIdx.x / 32;
    const int64_t first = kWarp ? (int64_t)blockIdx.x * kWarpsPerBlock + warp : blockIdx.x;
    const int64_t step = kWarp ? (int64_t)gridDim.x * kWarpsPerBlock : gridDim.x;
    const float inv = 1.f / (float)a.H;
    float dw[VPT][8] = {}, db[VPT][8] = {};
    int par = 0;
    for (int64_t row = first; row < a.T; row += step, par ^= 1) {
        const X* x = static_cast<const X*>(a.x) + row * a.H;
        const G* dy = static_cast<const G*>(a.dy) + row * a.H;
        const float r = a.rstd[row], mu = a.layer ? a.mean[row] : 0.f;
        float xh[VPT][8], d[VPT][8];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * g + t) * 8;
            if (c < a.H) {
                load8(x + c, xh[i]);
                load8(dy + c, d[i]);
                float w[8];
                if (a.w) load8(a.w + c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[i][j] = (xh[i][j] - mu) * r;
                    dw[i][j] = fmaf(d[i][j], xh[i][j], dw[i][j]);
                    db[i][j] += d[i][j];
                    if (a.w) d[i][j] *= w[j];
                    s1 += d[i][j];
                    s2 = fmaf(d[i][j], xh[i][j], s2);
                }
            }
        }
        s2 = warp_sum(s2);
        if (a.layer) s1 = warp_sum(s1);
        if (!kWarp) {
            const int lane = t % 32;
            if (lane == 0) {
                red[par][0][warp] = s1;
                red[par][1][warp] = s2;
            }
            __syncthreads();
            const bool in = lane < (int)(blockDim.x / 32);
            s2 = warp_sum(in ? red[par][1][lane] : 0.f);
            if (a.layer) s1 = warp_sum(in ? red[par][0][lane] : 0.f);
        }
        const float m1 = a.layer ? s1 * inv : 0.f, m2 = s2 * inv;
        const X* res = a.d_res ? static_cast<const X*>(a.d_res) + row * a.H : nullptr;
        X* dx = static_cast<X*>(a.dx) + row * a.H;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * g + t) * 8;
            if (c < a.H) {
                float o[8];
                if (res) load8(res + c, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = r * (d[i][j] - m1 - xh[i][j] * m2);
                    o[j] = res ? v + o[j] : v;
                }
                store8(dx + c, o);
            }
        }
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
    if (!kWarp) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * g + t) * 8;
            if (c < a.H) {
                store8(part + c, dw[i]);
                store8(part + a.H + c, db[i]);
            }
        }
    } else {
        // the block's warps in warp order, dw then db
#pragma unroll
        for (int which = 0; which < 2; ++which) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * 32 + t) * 8;
                if (c < a.H) store8(cols + warp * kWarpRowMax + c, which ? db[i] : dw[i]);
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
                float s = 0.f;
                for (int k = 0; k < kWarpsPerBlock; ++k) s += cols[k * kWarpRowMax + c];
                part[which * a.H + c] = s;
            }
            __syncthreads();
        }
    }
}

// out[c] = sum over p < P of part[p * stride + c], in a fixed order: 32 rows
// of threads take every 32nd partial each, then a tree over them.
__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* __restrict__ part, int64_t stride, int P,
                                                            int64_t second, int N, float* out0, float* out1) {
    __shared__ float s[32][33];
    float* out = blockIdx.y ? out1 : out0;
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    const float* src = part + (blockIdx.y ? second : 0);
    float v = 0.f;
    if (c < N)
        for (int p = threadIdx.y; p < P; p += 32) v += src[p * stride + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    for (int h = 16; h > 0; h >>= 1) {
        if ((int)threadIdx.y < h) s[threadIdx.y][threadIdx.x] += s[threadIdx.y + h][threadIdx.x];
        __syncthreads();
    }
    if (threadIdx.y == 0 && c < N) out[c] = s[0][threadIdx.x];
}

struct Shape {
    bool warp;
    int vpt, threads;
};

// Rows up to 1024 elements take a warp each; longer rows a block of at most
// 512 threads, with as few groups of 8 elements per thread as that allows.
Shape shape_of(int H) {
    const int g = (H + 7) / 8;
    Shape s;
    s.warp = H <= kWarpRowMax;
    if (s.warp) {
        s.vpt = g <= 32 ? 1 : (g <= 64 ? 2 : 4);
        s.threads = 32 * kWarpsPerBlock;
    } else {
        s.vpt = g <= 256 ? 1 : (g <= 1024 ? 2 : 4);
        const int per = (g + s.vpt - 1) / s.vpt;
        s.threads = (per + 31) / 32 * 32;
    }
    return s;
}

template <typename F>
cudaError_t by_shape(const Shape& s, F f) {
    if (s.warp) {
        if (s.vpt == 1) return f(std::integral_constant<int, 1>(), std::true_type());
        if (s.vpt == 2) return f(std::integral_constant<int, 2>(), std::true_type());
        return f(std::integral_constant<int, 4>(), std::true_type());
    }
    if (s.vpt == 1) return f(std::integral_constant<int, 1>(), std::false_type());
    if (s.vpt == 2) return f(std::integral_constant<int, 2>(), std::false_type());
    return f(std::integral_constant<int, 4>(), std::false_type());
}

}  // namespace

int norm_bwd_blocks(int64_t T, int H) {
    const Shape s = shape_of(H);
    const int64_t rows = s.warp ? (T + kWarpsPerBlock - 1) / kWarpsPerBlock : T;
    const int per_sm = s.warp ? 2 : std::max(1, 1024 / s.threads);
    return (int)std::min<int64_t>(rows, (int64_t)kNormBwdSms * per_sm);
}

cudaError_t launch_sum_partials(const float* part, int64_t stride, int P, int64_t second, int N, float* out0,
                                float* out1, cudaStream_t st) {
    trace_before("sum_partials", st);
    sum_partials_kernel<<<dim3((N + 31) / 32, out1 ? 2 : 1), dim3(32, 32), 0, st>>>(part, stride, P, second, N, out0,
                                                                                   out1);
    trace_after(st);
    return cudaGetLastError();
}

cudaError_t launch_norm_fwd(const NormArgs& a, bool f32, cudaStream_t st) {
    const Shape s = shape_of(a.H);
    const int64_t blocks = s.warp ? (a.T + kWarpsPerBlock - 1) / kWarpsPerBlock : a.T;
    trace_before("norm_fwd", st);
    by_shape(s, [&](auto vpt, auto warp) {
        if (f32)
            norm_fwd_kernel<float, vpt.value, warp.value><<<(unsigned)blocks, s.threads, 0, st>>>(a);
        else
            norm_fwd_kernel<bf16, vpt.value, warp.value><<<(unsigned)blocks, s.threads, 0, st>>>(a);
        return cudaSuccess;
    });
    trace_after(st);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool f32, bool dy_f32, cudaStream_t st) {
    const Shape s = shape_of(a.H);
    const int blocks = norm_bwd_blocks(a.T, a.H);
    trace_before("norm_bwd", st);
    by_shape(s, [&](auto vpt, auto warp) {
        if (f32)
            norm_bwd_kernel<float, float, vpt.value, warp.value><<<blocks, s.threads, 0, st>>>(a);
        else if (dy_f32)
            norm_bwd_kernel<bf16, float, vpt.value, warp.value><<<blocks, s.threads, 0, st>>>(a);
        else
            norm_bwd_kernel<bf16, bf16, vpt.value, warp.value><<<blocks, s.threads, 0, st>>>(a);
        return cudaSuccess;
    });
    trace_after(st);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.part) return e;
    return launch_sum_partials(a.part, 2 * (int64_t)a.H, blocks, a.H, a.H, a.dw_out, a.db_out, st);
}

}  // namespace moe
