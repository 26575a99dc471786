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
// Both directions are bound by HBM (a few flops per byte), so the kernels are
// built around bytes in flight: one CTA per SM, whose 16 warps form groups of
// W warps, one row per group at a time.  Each group has a ring of S row slots
// in shared memory that one thread fills with bulk copies (rows are
// contiguous), so that 64 to 96 KB of an SM's bf16 rows (float32: up to 192;
// backward: up to 200; less where the rows are shorter than 512 elements) are on
// their way whatever the registers hold.
// A row is read from HBM once; its statistics (forward: the mean, then the
// squared deviations from it, so no cancellation; backward: the two sums) are
// warp sums joined through shared memory with one barrier of the group each,
// and that barrier is also what frees the previous row's slot.  Every sum and
// statistic is float32; y and dx are rounded once, to the layer type.
//
// The weight gradients are sums over all rows.  A thread owns fixed columns
// and keeps their sums in registers over all its group's rows; a CTA adds its
// groups in order and writes one partial row, and a second small kernel adds
// the partial rows in a fixed order: no atomics, the same bits on every run.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "sm100_dense.cuh"
#include "tma_host.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRingBytes = 200 * 1024;
// The forward's ring, as far as whole rows fill it (but two per group at least, three
// per group of 8 or 16 warps): 80 KB per SM are what HBM's latency asks for, and reading further ahead of the writes mostly costs (bf16,
// RMS form: 16384 rows of 2880 take 32.5 us with 80 KB and 35.2 with 200, 16384 of
// 4096 42.7 and 47.4; but 65536 of 1024 47.3 and 45.0).
constexpr int kFwdRingBytes = 80 * 1024;
constexpr int kMaxSlots = 8;
constexpr int kMaxVpt = 4;  // groups of 8 elements per thread (or 2)

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

// A thread's columns of a float32 vector, or `other` where there is none.
template <int kVpt>
__device__ __forceinline__ void load_cols(float (&v)[kVpt][8], const float* p, int t, int threads, int H, float other) {
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
        const int c = (i * threads + t) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = other;
        if (p && c < H) load8(p + c, v[i]);
    }
}

// Geometry of a launch: W warps per row, S slots per group.
struct Geo {
    int W, S;
    int slot_bytes;  // one row of every tensor that comes through the ring
};

// One group of W warps (a template argument: strides and the joining of the
// warps' sums become constants, 5% of the forward's time).
template <int W>
struct Group {
    static constexpr int groups = kWarps / W, threads = 32 * W;
    int id, t;                // index in the CTA, thread within
    float (*red)[2][kWarps];  // [2][2][warps]
    __device__ explicit Group(float (*red_)[2][kWarps]) {
        id = threadIdx.x / threads;
        t = threadIdx.x % threads;
        red = red_;
    }
    __device__ void sync() const {
        if (W == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(threads) : "memory");
    }
    // Two warps' sums joined over the group: post, a sync, collect.
    __device__ void post(float a, float b, int par) const {
        const int warp = threadIdx.x / 32;
        if (W > 1 && threadIdx.x % 32 == 0) {
            red[par][0][warp] = a;
            red[par][1][warp] = b;
        }
    }
    // The group's W values of one sum, added.
    __device__ float joined(const float* r) const {
        float v = r[id * W + (threadIdx.x & (W - 1))];
#pragma unroll
        for (int o = W / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    __device__ void collect(float& a, float& b, int par) const {
        if (W > 1) {
            a = joined(red[par][0]);
            b = joined(red[par][1]);
        }
    }
    // a and b summed over the group's threads (the same bits in each); par
    // alternates from call to call, so that one barrier is enough.
    __device__ void sum2(float& a, float& b, int par) const {
        a = warp_sum(a);
        b = warp_sum(b);
        post(a, b, par);
        sync();
        collect(a, b, par);
    }
    __device__ float sum1(float a, int par) const {
        a = warp_sum(a);
        if (W > 1) {
            if (threadIdx.x % 32 == 0) red[par][0][threadIdx.x / 32] = a;
            sync();
            a = joined(red[par][0]);
        } else {
            __syncwarp();
        }
        return a;
    }
};

// Waits (bounded) for a slot's copies.  They are this CTA's own, so the wait
// ends; should it not, the row's results become NaN rather than stale values.
__device__ __forceinline__ float slot_wait(uint64_t* bar, uint32_t parity) {
    return mbar_wait(bar, parity) ? 0.f : __int_as_float(0x7fffffff);
}

template <typename X, int kVpt, int W>
__global__ void __launch_bounds__(kThreads, 1) norm_fwd_kernel(const NormArgs a, const Geo geo) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float red[2][2][kWarps];
    __shared__ uint64_t full[kWarps * kMaxSlots];
    const Group<W> g(red);
    uint8_t* ring = smem + (size_t)g.id * geo.S * geo.slot_bytes;
    uint64_t* bar = full + g.id * geo.S;
    const int64_t first = (int64_t)g.id * gridDim.x + blockIdx.x, step = (int64_t)g.groups * gridDim.x;
    const X* x = static_cast<const X*>(a.x);
    auto issue = [&](int64_t row, int s) {
        mbar_arrive_expect_tx(&bar[s], geo.slot_bytes);
        bulk_load(ring + s * geo.slot_bytes, x + row * a.H, geo.slot_bytes, &bar[s]);
    };
    if (g.t == 0) {
        for (int s = 0; s < geo.S; ++s) mbar_init(&bar[s], 1);
        fence_mbar_init();
        chain_wait();
        for (int s = 0; s < geo.S; ++s)
            if (first + s * step < a.T) issue(first + s * step, s);
    }
    chain_wait();
    chain_next();
    g.sync();
    // the thread's columns of w and b stay in registers over all its rows
    float w[kVpt][8], b[kVpt][8];
    load_cols(w, a.w, g.t, g.threads, a.H, 1.f);
    load_cols(b, a.b, g.t, g.threads, a.H, 0.f);
    const float inv = 1.f / (float)a.H;
    int s = 0, par = 0;
    uint32_t ph = 0;
    for (int64_t row = first; row < a.T; row += step) {
        const float bad = slot_wait(&bar[s], ph);
        const X* src = reinterpret_cast<const X*>(ring + s * geo.slot_bytes);
        float val[kVpt][8];  // the row, then its deviations from the mean
        float sum[2] = {bad, 0.f};
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int c = (i * g.threads + g.t) * 8;
            if (c < a.H) {
                load8(src + c, val[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j & 1] += val[i][j];
            }
        }
        float mu = bad;
        if (a.layer) {
            mu = g.sum1(sum[0] + sum[1], par) * inv;
            par ^= 1;
        }
        sum[0] = sum[1] = 0.f;
#pragma unroll
        for (int i = 0; i < kVpt; ++i)
            if ((i * g.threads + g.t) * 8 < a.H) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = val[i][j] -= mu;
                    sum[j & 1] = fmaf(d, d, sum[j & 1]);
                }
            }
        const float r = rsqrtf(g.sum1(sum[0] + sum[1], par) * inv + a.eps);
        par ^= 1;
        // the sum's barrier: every warp of the group has this row in registers
        if (g.t == 0) {
            if (row + geo.S * step < a.T) issue(row + geo.S * step, s);
            if (a.mean_out && a.layer) a.mean_out[row] = mu;
            if (a.rstd_out) a.rstd_out[row] = r;
        }
        X* y = static_cast<X*>(a.y) + row * a.H;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int c = (i * g.threads + g.t) * 8;
            if (c < a.H) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = fmaf(val[i][j] * r, w[i][j], b[i][j]);
                store8(y + c, v);
            }
        }
        if (++s == geo.S) {
            s = 0;
            ph ^= 1;
        }
    }
}

// One partial row of dw (and of db) per CTA: part[blockIdx][0 dw, 1 db][H].
template <typename X, typename G, int kVpt, int W, bool kDb>
__global__ void __launch_bounds__(kThreads, 1) norm_bwd_kernel(const NormArgs a, const Geo geo) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float red[2][2][kWarps];
    __shared__ uint64_t full[kWarps * kMaxSlots];
    const Group<W> g(red);
    uint8_t* ring = smem + (size_t)g.id * geo.S * geo.slot_bytes;
    uint64_t* bar = full + g.id * geo.S;
    const int64_t first = (int64_t)g.id * gridDim.x + blockIdx.x, step = (int64_t)g.groups * gridDim.x;
    const uint32_t xb = a.H * sizeof(X), gb = a.H * sizeof(G);
    auto issue = [&](int64_t row, int s) {
        uint8_t* dst = ring + s * geo.slot_bytes;
        mbar_arrive_expect_tx(&bar[s], geo.slot_bytes);
        bulk_load(dst, static_cast<const X*>(a.x) + row * a.H, xb, &bar[s]);
        bulk_load(dst + xb, static_cast<const G*>(a.dy) + row * a.H, gb, &bar[s]);
        if (a.d_res) bulk_load(dst + xb + gb, static_cast<const X*>(a.d_res) + row * a.H, xb, &bar[s]);
    };
    if (g.t == 0) {
        for (int s = 0; s < geo.S; ++s) mbar_init(&bar[s], 1);
        fence_mbar_init();
        chain_wait();
        for (int s = 0; s < geo.S; ++s)
            if (first + s * step < a.T) issue(first + s * step, s);
    }
    chain_wait();
    chain_next();
    g.sync();
    const float inv = 1.f / (float)a.H;
    float dw[kVpt][8] = {}, db[kVpt][8] = {};
    int s = 0, par = 0;
    uint32_t ph = 0;
    if constexpr (kVpt <= 2) {
        // a and xh stay in registers from the sums to dx, w over all rows (re-reading
        // them from shared memory, 32768 rows of 2048: 88.7 us instead of 79.4);
        // rows of at most 8192 elements, of which the ring holds two at least
        float w[kVpt][8];
        load_cols(w, a.w, g.t, g.threads, a.H, 1.f);
        float r = first < a.T ? a.rstd[first] : 0.f, mu = first < a.T && a.layer ? a.mean[first] : 0.f;
        int prev = 0;
        for (int64_t row = first; row < a.T; row += step, par ^= 1) {
            const float r0 = r, mu0 = mu + slot_wait(&bar[s], ph);
            if (row + step < a.T) {  // the next row's statistics, ahead of their use
                r = a.rstd[row + step];
                mu = a.layer ? a.mean[row + step] : 0.f;
            }
            const uint8_t* slot = ring + s * geo.slot_bytes;
            float xh[kVpt][8], d[kVpt][8];
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                const int c = (i * g.threads + g.t) * 8;
                if (c < a.H) {
                    load8(reinterpret_cast<const X*>(slot) + c, xh[i]);
                    load8(reinterpret_cast<const G*>(slot + xb) + c, d[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        xh[i][j] = (xh[i][j] - mu0) * r0;
                        dw[i][j] = fmaf(d[i][j], xh[i][j], dw[i][j]);
                        if (kDb) db[i][j] += d[i][j];
                        d[i][j] *= w[i][j];
                        s1 += d[i][j];
                        s2 = fmaf(d[i][j], xh[i][j], s2);
                    }
                }
            }
            s1 = warp_sum(s1);
            s2 = warp_sum(s2);
            g.post(s2, s1, par);
            g.sync();
            g.collect(s2, s1, par);
            // every warp of the group is done with the previous row
            if (g.t == 0 && row != first && row + (geo.S - 1) * step < a.T) issue(row + (geo.S - 1) * step, prev);
            const float m1 = a.layer ? s1 * inv : 0.f, m2 = s2 * inv;
            X* dx = static_cast<X*>(a.dx) + row * a.H;
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                const int c = (i * g.threads + g.t) * 8;
                if (c < a.H) {
                    float v[8] = {};
                    if (a.d_res) load8(reinterpret_cast<const X*>(slot + xb + gb) + c, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += r0 * ((d[i][j] - m1) - xh[i][j] * m2);
                    store8(dx + c, v);
                }
            }
            prev = s;
            if (++s == geo.S) {
                s = 0;
                ph ^= 1;
            }
        }
    } else {
        auto weights = [&](int c, float (&w)[8]) {  // from L1, row by row
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.f;
            if (a.w) load8(a.w + c, w);
        };
        // Row k's two sums, then row k - 1's dx, between two barriers: the second
        // half of the previous row covers the barrier and the warp sums of this one.
        struct Row {
            int s;
            float mu, r, s1, s2;
        };
        auto sums = [&](int64_t row, int s, uint32_t ph, float r, float mu) {
            Row o{s, mu + slot_wait(&bar[s], ph), r, 0.f, 0.f};
            const X* x = reinterpret_cast<const X*>(ring + s * geo.slot_bytes);
            const G* dy = reinterpret_cast<const G*>(ring + s * geo.slot_bytes + xb);
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                const int c = (i * g.threads + g.t) * 8;
                if (c < a.H) {
                    float xh[8], d[8], w[8];
                    load8(x + c, xh);
                    load8(dy + c, d);
                    weights(c, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        xh[j] = (xh[j] - o.mu) * r;
                        dw[i][j] = fmaf(d[j], xh[j], dw[i][j]);
                        if (kDb) db[i][j] += d[j];
                        d[j] *= w[j];
                        o.s1 += d[j];
                        o.s2 = fmaf(d[j], xh[j], o.s2);
                    }
                }
            }
            return o;
        };
        auto finish = [&](int64_t row, const Row& o) {
            const uint8_t* slot = ring + o.s * geo.slot_bytes;
            const X* x = reinterpret_cast<const X*>(slot);
            const G* dy = reinterpret_cast<const G*>(slot + xb);
            const X* res = reinterpret_cast<const X*>(slot + xb + gb);
            const float m1 = a.layer ? o.s1 * inv : 0.f, m2 = o.s2 * inv;
            X* dx = static_cast<X*>(a.dx) + row * a.H;
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                const int c = (i * g.threads + g.t) * 8;
                if (c < a.H) {
                    float xh[8], d[8], w[8], v[8] = {};
                    load8(x + c, xh);
                    load8(dy + c, d);
                    weights(c, w);
                    if (a.d_res) load8(res + c, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        xh[j] = (xh[j] - o.mu) * o.r;
                        v[j] += o.r * (fmaf(d[j], w[j], -m1) - xh[j] * m2);
                    }
                    store8(dx + c, v);
                }
            }
        };
        if (geo.S == 1) {
            for (int64_t row = first; row < a.T; row += step, ph ^= 1, par ^= 1) {
                Row o = sums(row, 0, ph, a.rstd[row], a.layer ? a.mean[row] : 0.f);
                g.sum2(o.s2, o.s1, par);
                finish(row, o);
                g.sync();
                if (g.t == 0 && row + step < a.T) issue(row + step, 0);
            }
        } else if (first < a.T) {
            Row last;
            float r = a.rstd[first], mu = a.layer ? a.mean[first] : 0.f;
            int64_t row = first;
            for (; row < a.T; row += step, par ^= 1) {
                const float r0 = r, mu0 = mu;
                if (row + step < a.T) {  // the next row's statistics, ahead of their use
                    r = a.rstd[row + step];
                    mu = a.layer ? a.mean[row + step] : 0.f;
                }
                Row o = sums(row, s, ph, r0, mu0);
                o.s1 = warp_sum(o.s1);
                o.s2 = warp_sum(o.s2);
                g.post(o.s2, o.s1, par);
                if (row != first) finish(row - step, last);
                g.sync();
                g.collect(o.s2, o.s1, par);
                // every warp of the group is done with the previous row
                if (g.t == 0 && row != first && row + (geo.S - 1) * step < a.T)
                    issue(row + (geo.S - 1) * step, last.s);
                last = o;
                if (++s == geo.S) {
                    s = 0;
                    ph ^= 1;
                }
            }
            finish(row - step, last);
        }
    }
    if (!a.part) return;
    // the CTA's groups, in order, through shared memory (the rings are empty)
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
    float* cols = reinterpret_cast<float*>(smem);
    __syncthreads();
#pragma unroll
    for (int which = 0; which < (kDb ? 2 : 1); ++which) {
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int c = (i * g.threads + g.t) * 8;
            if (c < a.H) store8(cols + (size_t)g.id * a.H + c, which ? db[i] : dw[i]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += kThreads) {
            float v = 0.f;
            for (int k = 0; k < g.groups; ++k) v += cols[(size_t)k * a.H + c];
            part[which * a.H + c] = v;
        }
        __syncthreads();
    }
}

// out[c] = sum over p < P of part[p * stride + c], in a fixed order: 32 rows
// of threads take every 32nd partial each, then a tree over them.
__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* part, int64_t stride, int P,
                                                            int64_t second, int N, float* out0, float* out1) {
    __shared__ float s[32][33];
    chain_wait();
    chain_next();
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

// Warps per row: as few as hold the row in `vpt` groups of 8 elements per
// thread, so that a CTA has several independent rows in flight; more when
// `least` slots for every group would not fit.  Slots as the ring of `bytes`
// holds, `least` of them at any rate.
Geo geo_of(int H, int slot_bytes, int vpt, int bytes, int least) {
    Geo g;
    g.slot_bytes = slot_bytes;
    g.W = 1;
    while (g.W * 32 * 8 * vpt < H) g.W *= 2;
    auto slots = [&](int ring) { return ring / (kWarps / g.W) / slot_bytes; };
    while (g.W < kWarps && slots(kRingBytes) < least) g.W *= 2;
    if (g.W >= 8) least = std::max(least, 3);
    g.S = std::max(1, std::min({kMaxSlots, slots(kRingBytes), std::max(least, slots(bytes))}));
    return g;
}

int blocks_of(int64_t T) { return (int)std::min<int64_t>(T, kNormSms); }

// Ring, or the float32 column sums of the CTA's groups at the end.
size_t smem_of(const Geo& g, int H) {
    const size_t groups = kWarps / g.W;
    return std::max(groups * g.S * g.slot_bytes, groups * H * sizeof(float));
}

template <typename Kernel>
cudaError_t launch(Kernel k, const NormArgs& a, const Geo& g, const char* name, cudaStream_t st) {
    const size_t smem = smem_of(g, a.H);
    cudaError_t e = ensure_smem_attr(k, kRingBytes);
    if (e != cudaSuccess) return e;
    trace_before(name, st);
    e = launch_chained(k, blocks_of(a.T), kThreads, smem, 0, st, a, g);
    trace_after(st);
    return e;
}

}  // namespace

int norm_bwd_blocks(int64_t T) { return blocks_of(T); }

cudaError_t launch_sum_partials(const float* part, int64_t stride, int P, int64_t second, int N, float* out0,
                                float* out1, cudaStream_t st) {
    trace_before("sum_partials", st);
    const cudaError_t e = launch_chained(sum_partials_kernel, dim3((N + 31) / 32, out1 ? 2 : 1), dim3(32, 32), 0, 0, st,
                                         part, stride, P, second, N, out0, out1);
    trace_after(st);
    return e;
}

template <typename X, int W>
cudaError_t launch_fwd(const NormArgs& a, const Geo& g, cudaStream_t st) {
    return W * 32 * 8 * 2 >= a.H ? launch(norm_fwd_kernel<X, 2, W>, a, g, "norm_fwd", st)
                                 : launch(norm_fwd_kernel<X, kMaxVpt, W>, a, g, "norm_fwd", st);
}

template <typename X>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t st) {
    const Geo g = geo_of(a.H, a.H * (int)sizeof(X), kMaxVpt, kFwdRingBytes, 2);
    switch (g.W) {
        case 1: return launch_fwd<X, 1>(a, g, st);
        case 2: return launch_fwd<X, 2>(a, g, st);
        case 4: return launch_fwd<X, 4>(a, g, st);
        case 8: return launch_fwd<X, 8>(a, g, st);
        default: return launch_fwd<X, 16>(a, g, st);
    }
}

template <typename X, typename G, bool kDb>
cudaError_t launch_bwd(const NormArgs& a, cudaStream_t st) {
    // two groups of elements per thread up to H = 8192: with four, the sums of
    // both weight gradients alone take half of the registers
    const bool two = a.H <= kWarps * 32 * 8 * 2;
    const Geo g = geo_of(a.H, a.H * (int)(sizeof(X) * (a.d_res ? 2 : 1) + sizeof(G)), two ? 2 : kMaxVpt, kRingBytes, 3);
    const char* name = "norm_bwd";
    if (!two) return launch(norm_bwd_kernel<X, G, kMaxVpt, 16, kDb>, a, g, name, st);
    switch (g.W) {
        case 1: return launch(norm_bwd_kernel<X, G, 2, 1, kDb>, a, g, name, st);
        case 2: return launch(norm_bwd_kernel<X, G, 2, 2, kDb>, a, g, name, st);
        case 4: return launch(norm_bwd_kernel<X, G, 2, 4, kDb>, a, g, name, st);
        case 8: return launch(norm_bwd_kernel<X, G, 2, 8, kDb>, a, g, name, st);
        default: return launch(norm_bwd_kernel<X, G, 2, 16, kDb>, a, g, name, st);
    }
}

cudaError_t launch_norm_fwd(const NormArgs& a, bool f32, cudaStream_t st) {
    return f32 ? launch_fwd<float>(a, st) : launch_fwd<bf16>(a, st);
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool f32, bool dy_f32, cudaStream_t st) {
    cudaError_t e;
    if (a.db_out)
        e = f32 ? launch_bwd<float, float, true>(a, st)
                : (dy_f32 ? launch_bwd<bf16, float, true>(a, st) : launch_bwd<bf16, bf16, true>(a, st));
    else
        e = f32 ? launch_bwd<float, float, false>(a, st)
                : (dy_f32 ? launch_bwd<bf16, float, false>(a, st) : launch_bwd<bf16, bf16, false>(a, st));
    if (e != cudaSuccess || !a.part) return e;
    return launch_sum_partials(a.part, 2 * (int64_t)a.H, norm_bwd_blocks(a.T), a.H, a.H, a.dw_out, a.db_out, st);
}

}  // namespace moe
