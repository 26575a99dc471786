// Matrix products of the linear layer and the gate/up projections for few
// rows (sm_100a): forward and input gradient where the weights' stream from
// HBM is the bound.
//
// The weights take the tensor core's 128-row side and the tokens its column
// side: D[128 output features][tn tokens], so a call of one token wastes 15
// columns of a cheap MMA instead of 255 rows, and every SM spends its time on
// weight bytes.  A CTA owns one tile and one share of the reduction: a cluster
// of S <= 8 CTAs splits the reduction (enough clusters to cover the SMs when
// the output has few feature tiles), and each streams its share through a TMA
// ring of up to 208 KB (weights 16 KB per 64-deep step, read once).  Then CTA r
// of the cluster finishes the r-th share of the tokens: it adds the S partial
// sums, its own and the peers' through distributed shared memory, all S loads
// of an element in flight at once (one at a time they took 4 us of a 9 us call
// of 64 tokens; pushing them instead, by bulk copies or by stores, was slower
// from 128 tokens on).  CTA r starts at its own partial and goes round, so that
// the peers are not all read in the same order; which CTA finishes a token
// depends on the sizes alone, so the bits do not change from run to run.
//
//   forward: A = W rows K-major; gated: two A tiles (gate, up) and two
//            accumulators per step
//   input gradient: A = W read MN-major (features = W's columns), B = dz; the
//            gated pair is one reduction over both (two segments)
//
// Twelve warps: TMA producer, MMA issuer, eight that move the accumulator from
// TMEM to shared memory; then all of them finish the elements (bias,
// activation, residual), which waits on loads and wants many warps.  Waits are
// bounded; no multicast loads.
#include <algorithm>

#include "act.cuh"
#include "dense.cuh"
#include "dense_gemm.cuh"
#include "sm100_dense.cuh"
#include "tma_host.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int kBK = 64;
constexpr int kThreads = 384;
constexpr int kABytes = 128 * kBK * 2;
constexpr int kBox = 64 * kBK * 2;
constexpr int kMaxStages = 12;
constexpr int kRingBytes = 208 * 1024;
// All of an SM's shared memory whatever the sizes: no second CTA that allocates TMEM
// shares the SM, so an allocation never waits for a CTA whose cluster waits for this one.
constexpr size_t kSmem = kRingBytes + 512 + 1024;
constexpr int kRowBytes = 128 * 4;  // one token's 128 features, float32

struct Args {
    int T, N;        // tokens, output features
    int tn;          // tokens per tile (multiple of 16)
    int stages;
    int per;         // reduction steps in a stage: the kernel's kPer
    int seg_steps, steps;
    int splits;      // CTAs per cluster
    int act;
    const float* bias0;
    const float* bias1;
    const bf16* res;
    bf16* y;
    bf16* z0;
    bf16* z1;
    uint32_t tmem_cols;
    int32_t* flags;
    uint32_t* gate;  // to open for a weight gradient beside this kernel, or null
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void store4(bf16* p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <bool kGated, bool kAMN, int kPer>
__global__ void __launch_bounds__(kThreads, 1) dense_skinny_kernel(const __grid_constant__ CUtensorMap mA0,
                                                                   const __grid_constant__ CUtensorMap mA1,
                                                                   const __grid_constant__ CUtensorMap mB0,
                                                                   const __grid_constant__ CUtensorMap mB1,
                                                                   const Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRingBytes);
    uint64_t* empty = full + kMaxStages;
    uint64_t* done = empty + kMaxStages;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // warp: uniform
    const uint32_t rank = a.splits > 1 ? cluster_ctarank() : 0;
    const int n0 = (int)(blockIdx.x / a.splits) * 128, t0 = (int)blockIdx.y * a.tn;
    const int ks0 = (int)((int64_t)a.steps * rank / a.splits), ks1 = (int)((int64_t)a.steps * (rank + 1) / a.splits);
    const int b_bytes = a.tn * kBK * 2;
    const int step_bytes = (kGated ? 2 : 1) * kABytes + b_bytes, stage_bytes = kPer * step_bytes;
    constexpr int kAcc = kGated ? 2 : 1;
    const int tokens = min(a.tn, a.T - t0);
    // tokens CTA r of the cluster finishes
    auto share = [&](int r) { return tokens * r / a.splits; };
    const int tk0 = share((int)rank), tk1 = share((int)rank + 1);
    // steps of the stage that starts at ks: fewer at the end of a segment or of the share
    auto steps_of = [&](int ks) { return kPer == 2 && ks + 1 < ks1 && ks + 1 != a.seg_steps ? 2 : 1; };
    auto load_stage = [&](int ks, int s) {
        const bool seg1 = ks >= a.seg_steps;
        const int n = steps_of(ks);
        mbar_arrive_expect_tx(&full[s], n * step_bytes);
        for (int j = 0; j < n; ++j) {
            const int kc = (seg1 ? ks + j - a.seg_steps : ks + j) * kBK;
            uint8_t* sa = smem + s * stage_bytes + j * step_bytes;
            uint8_t* sb = sa + (kGated ? 2 : 1) * kABytes;
            if (kAMN) {
                const CUtensorMap* pA = seg1 ? &mA1 : &mA0;
                tma_load_3d(sa, pA, &full[s], n0, kc, 0);
                tma_load_3d(sa + kBox, pA, &full[s], n0 + 64, kc, 0);
            } else {
                tma_load_3d(sa, &mA0, &full[s], kc, n0, 0);
                if (kGated) tma_load_3d(sa + kABytes, &mA1, &full[s], kc, n0, 0);
            }
            tma_load_3d(sb, seg1 ? &mB1 : &mB0, &full[s], kc, t0, 0);
        }
        return n;
    };
    int it = 0, ks = ks0;  // the producer's: stages and steps issued so far
    if (threadIdx.x == 0) {
        tma_prefetch_map(&mA0);
        tma_prefetch_map(&mB0);
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        chain_wait();
        for (; it < a.stages && ks < ks1; ++it) ks += load_stage(ks, it);  // these need no free slot
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, a.tmem_cols);
        tmem_relinquish();
    }
    chain_wait();
    if (a.gate && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == kThreads - 1) gate_open(a.gate);
    chain_next();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (; ks < ks1; ++it) {
                if (!wait_or_abort(&empty[s], ph, abort_flag, a.flags)) break;
                ks += load_stage(ks, s);
                if (++s == a.stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            // every copy has landed before the ring is reused or released
            for (int j = std::max(0, it - a.stages); j < it; ++j) drain_wait(&full[j % a.stages], (j / a.stages) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (the whole warp, one lane elected)
        const uint32_t idesc = idesc_bf16_major(128, a.tn, kAMN, false);
        const uint32_t base = smem_u32(smem);
        constexpr uint32_t kStepA = (kAMN ? 2048 : 32) >> 4;
        const uint64_t da0 = kAMN ? desc_mnmajor_sw128(base, kBox, 1024) : desc_kmajor_sw128(base);
        const uint64_t db0 = desc_kmajor_sw128(base + (kGated ? 2 : 1) * kABytes);
        const uint32_t stride = stage_bytes >> 4;
        int s = 0;
        uint32_t ph = 0, sum = 0;
        for (int k = ks0, n; k < ks1; k += n) {
            n = steps_of(k);
            if (!wait_or_abort_warp(&full[s], ph, abort_flag, a.flags)) break;
            tc_fence_after();
            uint64_t da = da0 + (uint32_t)s * stride, db = db0 + (uint32_t)s * stride;
            for (int j = 0; j < n; ++j, da += step_bytes >> 4, db += step_bytes >> 4)
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk) {
                    mma_bf16_warp(tmem_base, da + kk * kStepA, db + kk * 2, idesc, sum);
                    if (kGated) mma_bf16_warp(tmem_base + a.tn, da + (kABytes >> 4) + kk * kStepA, db + kk * 2, idesc, sum);
                    sum = 1;
                }
            mma_commit_warp(&empty[s]);
            if (++s == a.stages) {
                s = 0;
                ph ^= 1;
            }
        }
        mma_commit_warp(done);
        drain_wait(done, 0);
    } else if (warp < 10) {
        // ------------------------------------------------ TMEM -> part[accumulator][token][128 features]
        // (in the ring's place: the accumulator is complete, so every step's
        // operands have been read; after a time-out it may not be, and copies may
        // still be landing: then nothing is moved, and the device flag tells of y)
        const int q = warp & 3, half = (warp - 2) >> 2;  // lanes, every second group of 16 columns
        if (wait_sleep_or_abort_warp(done, 0, abort_flag, a.flags)) {
            tc_fence_after();
            float* part = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int p = 0; p < kAcc; ++p)
                for (int c = 16 * half; c < tokens; c += 32) {
                    float v[16];
                    tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + p * a.tn + c, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(p * a.tn + c + i) * 128 + q * 32 + lane] = v[i];
                }
        }
        tc_fence_before();
    }
    __syncwarp();  // the single-lane roles join their warps
    if (a.splits > 1)
        cluster_sync();
    else
        __syncthreads();

    // ---------------------------------------------------- finish: 4 features of a token per thread
    // and token, kItems tokens at once so that their loads are in flight together
    constexpr int kItems = 2;
    const uint32_t part = smem_u32(smem) + lane * 16;
    const int f = lane * 4, n = n0 + f;  // a warp spans the tile's 128 features
    if (n < a.N) {                       // N is a multiple of 8
        float4 bias[kAcc];
#pragma unroll
        for (int p = 0; p < kAcc; ++p) {
            const float* b = p ? a.bias1 : a.bias0;
            bias[p] = b ? *reinterpret_cast<const float4*>(b + n) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int tok0 = tk0 + warp; tok0 < tk1; tok0 += kItems * (kThreads / 32)) {
            uint2 res[kItems];
            float4 s[kItems][kAcc];
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
                const int tok = tok0 + u * (kThreads / 32);
                res[u] = make_uint2(0u, 0u);
                if (a.res && tok < tk1) res[u] = *reinterpret_cast<const uint2*>(a.res + (int64_t)(t0 + tok) * a.N + n);
#pragma unroll
                for (int p = 0; p < kAcc; ++p) s[u][p] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            // four peers' loads at a time
            for (int r0 = 0; r0 < a.splits; r0 += 4) {
                float4 w[4][kItems][kAcc];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    uint32_t peer = rank + r0 + r;
                    if (peer >= (uint32_t)a.splits) peer -= a.splits;
                    const bool in = r0 + r < a.splits;
                    const uint32_t src = a.splits > 1 ? mapa_shared(part, in ? peer : rank) : part;
#pragma unroll
                    for (int u = 0; u < kItems; ++u)
#pragma unroll
                        for (int p = 0; p < kAcc; ++p) {
                            const int tok = min(tok0 + u * (kThreads / 32), tk1 - 1);
                            w[r][u][p] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (in) w[r][u][p] = ld_cluster_f4(src + (p * a.tn + tok) * kRowBytes);
                        }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int u = 0; u < kItems; ++u)
#pragma unroll
                        for (int p = 0; p < kAcc; ++p) {
                            s[u][p].x += w[r][u][p].x, s[u][p].y += w[r][u][p].y;
                            s[u][p].z += w[r][u][p].z, s[u][p].w += w[r][u][p].w;
                        }
            }
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
                const int tok = tok0 + u * (kThreads / 32);
                if (tok >= tk1) break;
                float v[kAcc][4];
#pragma unroll
                for (int p = 0; p < kAcc; ++p) {
                    v[p][0] = s[u][p].x + bias[p].x, v[p][1] = s[u][p].y + bias[p].y;
                    v[p][2] = s[u][p].z + bias[p].z, v[p][3] = s[u][p].w + bias[p].w;
                }
                const int64_t o = (int64_t)(t0 + tok) * a.N + n;
                if (a.z0) store4(a.z0 + o, v[0]);
                if (kGated && a.z1) store4(a.z1 + o, v[kAcc - 1]);
                by_act(a.act, [&](auto k) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[0][j] = act_value<k.value>(v[0][j]);
                });
                if (kGated)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[0][j] *= v[kAcc - 1][j];
                v[0][0] += __uint_as_float(res[u].x << 16), v[0][1] += __uint_as_float(res[u].x & 0xffff0000u);
                v[0][2] += __uint_as_float(res[u].y << 16), v[0][3] += __uint_as_float(res[u].y & 0xffff0000u);
                store4(a.y + o, v[0]);
            }
        }
    }
    __syncwarp();
    if (a.splits > 1) cluster_sync();  // the peers have read this CTA's partial sums
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, a.tmem_cols);
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int step_bytes_of(int acc, int tn) { return acc * kABytes + tn * kBK * 2; }

// Two steps per stage halve the waits and commits between the MMAs (one token:
// 14336 -> 4096 20.7 instead of 21.8 us, 4096 -> 4096 8.8 instead of 9.7), but leave
// fewer stages: with three, 128 tokens, 7168 -> 2048 12.4 instead of 12.0.
int steps_per_stage(int acc, int tn) { return kRingBytes / (2 * step_bytes_of(acc, tn)) >= (acc == 2 ? 3 : 4) ? 2 : 1; }

// One way of laying a product out, and its estimated time in microseconds.
struct Geometry {
    int tn, splits;
    int64_t ctas;
    double us;
};

// Token tiles of tn, the reduction split over the largest cluster whose
// clusters all fit on the GPU at once, with at least 4 steps per CTA.  The
// estimate began as a fit to 220 measured calls (both forward forms, T = 100 ...
// 800, five weight shapes from 1024 x 1024 to 8192 x 2048, tiles of 64 to 256
// tokens); the rates and issue times below came later, from the calls named there.
// Of the layouts that it chooses now, on six shapes from 768 x 2048 to 8192 x 2048,
// its rms error is 9% for 83 forward calls of 100 to 1000 rows, 13% for 48 of fewer
// and 8% for 77 input gradients.  A step is the slowest of issuing it (0.29 us), its
// MMAs and its bytes at the rate that the SMs draw from L2 together; then the partial
// sums that come from peers, and the tile's way out of TMEM and through the epilogue.
// The weights come from HBM at 6.2 TB/s for one token tile, at 5.0 for several
// (gate/up, 64 rows: 14336 -> 4096 takes 42.4 us in one tile and 52.3 in two, but
// 2880 -> 2880, bound by its steps, 13.2 and 12.0).  Issuing a step of a two-step
// stage takes 0.20 us (192 rows, 2880 -> 2880: three tiles of 64, 10.0 us, not one of
// 192, 11.7); for an input gradient, whose form is chosen together with the weight
// gradient's, that figure moved backward passes by 20% both ways, and 0.29 stays.
Geometry geometry(int64_t T, int N, int64_t k, int steps, int acc, int tn, int64_t most_ctas, bool fwd) {
    // clusters of s CTAs with 209 KB of shared memory each that a B200 holds at
    // once (a cluster stays inside a GPC), a little below what it reports
    static const int kFit[9] = {0, 148, 74, 44, 32, 26, 20, 0, 14};
    const int64_t tiles = (int64_t)cdiv(N, 128) * cdiv(T, tn);
    Geometry g{tn, 1, tiles, 0};
    for (int s = 2; s <= 8; ++s)
        if (tiles <= kFit[s] && tiles * s <= most_ctas && steps >= 4 * s) g.splits = s;
    g.ctas = tiles * g.splits;
    const double rate = T <= tn ? 6.2e6 : 5.0e6;  // of the weights, read once or again by each token tile
    const double ctas = (double)g.ctas, rounds = (double)cdiv(g.ctas, 148), cols = tn * acc;
    const double issue = fwd && steps_per_stage(acc, tn) == 2 ? 0.20 : 0.29;
    const double step = std::max({issue, 0.0016 * cols, step_bytes_of(acc, tn) * std::min(ctas, 148.0) / 17.6e6});
    const double stream = std::max(rounds * cdiv(steps, g.splits) * step, acc * (double)N * k * 2 / rate);
    g.us = 2.8 + stream + 0.016 * cols * (g.splits - 1) / g.splits + rounds * cols * (0.0094 + 0.017 / g.splits);
    return g;
}

// The best geometry, over token tiles of at most 256 tokens (gated: 128, two
// accumulators) and down to 32, of at most most_ctas CTAs (tn = 0 when there is
// none).
constexpr int64_t kAnyCtas = INT64_MAX;
Geometry best_geometry(int64_t T, int N, int64_t k, int segs, bool gated, int64_t most_ctas, bool fwd) {
    const int acc = gated ? 2 : 1, steps = cdiv(k, kBK) * segs;
    const int64_t least = cdiv(T, 256 / acc);
    Geometry best{};
    for (int64_t n = least; n < least + 8; ++n) {
        const int tn = cdiv(cdiv(T, n), 16) * 16;
        if (n > least && tn < 32) break;
        const Geometry g = geometry(T, N, k * segs, steps, acc, tn, most_ctas, fwd);
        if (g.ctas <= most_ctas && (best.tn == 0 || g.us < best.us)) best = g;
    }
    return best;
}

void fill(Args& a, const Geometry& g, int64_t T, int N, int64_t k, int segs, bool gated, int32_t* flags) {
    const int acc = gated ? 2 : 1;
    a.T = (int)T;
    a.N = N;
    a.seg_steps = cdiv(k, kBK);
    a.steps = a.seg_steps * segs;
    a.tn = g.tn;
    a.splits = g.splits;
    a.per = steps_per_stage(acc, a.tn);
    a.stages = std::min(kMaxStages, kRingBytes / (a.per * step_bytes_of(acc, a.tn)));
    const uint32_t cols = acc * a.tn;
    a.tmem_cols = 32;
    while (a.tmem_cols < cols) a.tmem_cols *= 2;
    a.flags = flags;
}

template <bool kGated, bool kAMN>
cudaError_t launch(const CUtensorMap& A0, const CUtensorMap& A1, const CUtensorMap& B0, const CUtensorMap& B1,
                   const Args& a, const char* name, cudaStream_t st) {
    auto* fn = a.per == 2 ? dense_skinny_kernel<kGated, kAMN, 2> : dense_skinny_kernel<kGated, kAMN, 1>;
    cudaError_t e = ensure_smem_attr(fn, kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(cdiv(a.N, 128) * a.splits), (unsigned)cdiv(a.T, a.tn), 1);
    trace_before(name, st);
    e = launch_chained(fn, grid, kThreads, kSmem, a.splits, st, A0, A1, B0, B1, a);
    trace_after(st);
    return e;
}

cudaError_t launch_fwd_skinny(const Geometry& g, const void* x, const void* w0, const void* w1, int64_t T, int K, int N,
                              const DenseOut& o, int32_t* flags, cudaStream_t st) {
    Args a{};
    fill(a, g, T, N, K, 1, w1 != nullptr, flags);
    a.act = o.act;
    a.bias0 = o.bias0;
    a.bias1 = o.bias1;
    a.res = o.res;
    a.y = o.y;
    a.z0 = o.z0;
    a.z1 = o.z1;
    CUtensorMap A0, A1, B;
    if (!make_tile_map(&A0, false, w0, K, N, 1, 128) || !make_tile_map(&B, false, x, K, T, 1, a.tn))
        return cudaErrorInvalidValue;
    A1 = A0;
    if (w1 && !make_tile_map(&A1, false, w1, K, N, 1, 128)) return cudaErrorInvalidValue;
    if (w1) return launch<true, false>(A0, A1, B, B, a, "gated_fwd_skinny", st);
    return launch<false, false>(A0, A1, B, B, a, "linear_fwd_skinny", st);
}

cudaError_t launch_dgrad_skinny(const Geometry& g, const void* dz0, const void* dz1, const void* w0, const void* w1,
                                int64_t T, int K, int N, void* dx, bool opens_gate, const DenseWs& ws,
                                cudaStream_t st) {
    Args a{};
    fill(a, g, T, K, N, dz1 ? 2 : 1, false, ws.flags);
    a.gate = opens_gate ? ws.gate : nullptr;
    a.y = static_cast<bf16*>(dx);
    CUtensorMap A0, A1, B0, B1;
    if (!make_tile_map(&A0, false, w0, K, N, 1, 64) || !make_tile_map(&B0, false, dz0, N, T, 1, a.tn))
        return cudaErrorInvalidValue;
    A1 = A0;
    B1 = B0;
    if (dz1 && (!make_tile_map(&A1, false, w1, K, N, 1, 64) || !make_tile_map(&B1, false, dz1, N, T, 1, a.tn)))
        return cudaErrorInvalidValue;
    return launch<false, true>(A0, A1, B0, B1, a, dz1 ? "gated_dgrad_skinny" : "linear_dgrad_skinny", st);
}

// The pair kernel's estimated time for T rows, N outputs and a reduction of k (in
// `segs` segments): 6.5 us and 0.34 per reduction step of the rounds of tiles
// (`steps`), or its operands at 5.2 TB/s.
double pairs_us(int64_t T, int N, int64_t k, int segs, bool gated, double steps) {
    const double bytes = ((gated ? 2 : 1) * (double)N + (double)T) * k * segs * 2;
    return 6.5 + std::max(bytes / 5.2e6, 0.34 * steps);
}

// Which form a product takes: few rows in this geometry, or pairs (few = false).
struct Choice {
    bool few;
    Geometry g;
    int64_t ctas;
    double us;
};

// The form whose estimated time is less.  At T = 128 the few-row form takes 9.0
// against 14.9 us on 2880 -> 2880 (pairs: 23 tiles for 74 pairs); at T = 256 it
// takes 42.8 against 33.5 us on 4096 -> 14336, where 112 feature tiles read the
// tokens 112 times.
Choice choose(int64_t T, int N, int64_t k, int segs, bool gated, double pair_steps, int pair_ctas,
              int64_t most_ctas = kAnyCtas, bool fwd = false) {
    Choice c{false, {}, pair_ctas, pairs_us(T, N, k, segs, gated, pair_steps)};
    if (T > 65535 * 16) return c;  // the grid's second dimension counts token tiles
    const Geometry g = best_geometry(T, N, k, segs, gated, most_ctas, fwd);
    if (g.tn && (g.us < c.us || c.ctas > most_ctas)) c = Choice{true, g, g.ctas, g.us};
    return c;
}

Choice choose_fwd(int64_t T, int K, int N, bool gated) {
    return choose(T, N, K, 1, gated, dense_fwd_pairs_steps(T, K, N, gated), 0, kAnyCtas, true);
}

// The input gradient's form, and how the weight gradient (where one follows)
// runs.  Beside an input gradient that leaves SMs idle the weight gradient starts
// at once; so either each runs in its fastest form, one after the other, or the
// input gradient in the fastest form that leaves the weight gradient (whole or
// split) its SMs, whichever ends sooner: 10 instead of 15 us for the backward pass
// of 512 x 2048 -> 768.  Beside one that fills the GPU it would only take SMs from
// its last wave (4096 x 4096 -> 14336, gate/up: 1454 instead of 1354 us).
struct DgradPlan {
    Choice c;
    WgradPlan w;
};
DgradPlan plan_dgrad(int64_t T, int K, int N, int segs, bool with_wgrad) {
    const int pair_ctas = dense_dgrad_pairs_ctas(T, K, N, segs);
    const double pair_steps = dense_dgrad_pairs_steps(T, K, N, segs);
    const Choice alone = choose(T, K, N, segs, false, pair_steps, pair_ctas);
    DgradPlan best{alone, {true, with_wgrad && alone.ctas <= 140}};
    if (!with_wgrad) return best;
    double best_us = alone.us + dense_wgrad_us(T, K, N, segs, true);
    for (int split = 0; split < 2; ++split) {
        const int64_t room = 148 - dense_wgrad_ctas(T, K, N, segs, split);
        if (room < 16) continue;
        const Choice fit = choose(T, K, N, segs, false, pair_steps, pair_ctas, room);
        const double us = std::max(fit.us, dense_wgrad_us(T, K, N, segs, split)) + 1;
        if (fit.ctas <= room && us < best_us) {
            best = {fit, {split != 0, true}};
            best_us = us;
        }
    }
    return best;
}

}  // namespace

size_t dense_fwd_part_floats(int64_t T, int K, int N, bool gated) {
    return choose_fwd(T, K, N, gated).few ? 0 : dense_fwd_pairs_part_floats(T, K, N, gated);
}
size_t dense_dgrad_part_floats(int64_t T, int K, int N, int segs) {
    const bool pairs = !plan_dgrad(T, K, N, segs, false).c.few || !plan_dgrad(T, K, N, segs, true).c.few;
    return pairs ? dense_dgrad_pairs_part_floats(T, K, N, segs) : 0;
}

cudaError_t launch_dense_fwd(const void* x, const void* w0, const void* w1, int64_t T, int K, int N,
                             const DenseOut& o, const DenseWs& ws, cudaStream_t st) {
    const Choice c = choose_fwd(T, K, N, w1 != nullptr);
    return c.few ? launch_fwd_skinny(c.g, x, w0, w1, T, K, N, o, ws.flags, st)
                 : launch_dense_fwd_pairs(x, w0, w1, T, K, N, o, ws, st);
}

cudaError_t launch_dense_dgrad(const void* dz0, const void* dz1, const void* w0, const void* w1, int64_t T, int K,
                               int N, void* dx, bool with_wgrad, WgradPlan* plan, const DenseWs& ws,
                               cudaStream_t st) {
    const DgradPlan p = plan_dgrad(T, K, N, dz1 ? 2 : 1, with_wgrad);
    *plan = p.w;
    return p.c.few ? launch_dgrad_skinny(p.c.g, dz0, dz1, w0, w1, T, K, N, dx, p.w.beside, ws, st)
                   : launch_dense_dgrad_pairs(dz0, dz1, w0, w1, T, K, N, dx, p.w.beside, ws, st);
}

}  // namespace moe
