// Matrix products of the linear layer and the gate/up projections on the
// 5th-generation tensor cores (tcgen05, sm_100a), for many rows: forward with
// a fused epilogue, input gradient and weight gradient.
//
//   linear forward  y = act(x W^T + b) + res        A = x,  B = W   (both K-major)
//   gated forward   h = act(x Wg^T + bg) (x Wu^T + bu): each tile's MMA covers
//                   128 gate and the 128 matching up columns, so both
//                   pre-activations of an element meet in one epilogue thread
//   input gradient  dx = dz W (+ dz' W')            A = dz K-major, B = W read MN-major;
//                   the gated pair is one reduction over both (two segments)
//   weight gradient dW = dz^T x (two problems for the gated pair): both MN-major
//
// One persistent kernel template on CTA pairs (cta_group::2): a tile is 256
// rows x 256 columns (gated: 128 output columns, 256 accumulator columns; the
// linear forward has 128-column tiles too), each CTA of the pair stages its own
// 128 rows of A and half of B, and the leader issues M = 256 MMAs that read both
// CTAs' shared memory: per CTA and 64-deep reduction step 32 KB arrive for 2 x 128 x 256 x 64 flops, which keeps operand
// traffic below the tensor pipe's time.  A stage of the ring holds two steps:
// each wait for a stage and each commit holds up the issuing warp's MMAs by
// about 120 ns, and with one step per stage they were a fifth of the time.  TMEM
// holds two accumulators, so a tile's epilogue overlaps the next tile's main
// loop.  Bound by the tensor pipe and the power limit at large sizes (gate/up
// forward, 4096 x 4096 -> 14336: 614 us in a short run, 1.57 PFLOP/s, the pipe 93%
// active at 1.46 GHz), by the stores (weight gradients of few tokens) or the
// operands' HBM reads otherwise.
//
// Tiles that do not fill the last wave of pairs are split along the reduction
// (tail_plan): every split writes its float32 sums to the workspace, and the one
// that arrives last at a tile's counter adds them in split order and runs the
// epilogue (for a weight gradient, a second kernel adds them instead).  Nothing
// waits for another CTA, and the order of the sum is fixed.  The counters count
// warps' regions (32 rows x half the columns), so no CTA-wide barrier is needed,
// and return to zero.
//
// Roles (10 warps): warp 0 TMA producer, warp 1 MMA issuer, warps 2-9
// epilogue: warp w drains TMEM lanes 32 (w % 4) and one half of the columns.
// An epilogue warp stages 32 rows x 128 bytes in shared memory (128-byte
// swizzle) and stores it by TMA, which clips the ragged edges; the residual
// arrives by TMA in the same buffer, the first chunk ahead of the accumulator.
// Every wait is bounded; a timeout sets MOE_DEVFLAG_WAIT_TIMEOUT and the CTA
// unwinds.  No multicast loads.
#include <algorithm>

#include "act.cuh"
#include "dense.cuh"
#include "dense_gemm.cuh"
#include "sm100_dense.cuh"
#include "tma_host.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int kBM = 128;  // rows per CTA (256 per pair)
constexpr int kBK = 64;   // reduction step: one 128-byte swizzle row of bf16
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kAccCols = 256;
constexpr int kTmemCols = 2 * kAccCols;
constexpr int kABytes = kBM * kBK * 2;
constexpr int kBox = 64 * kBK * 2;      // a 64 x 64 box of an MN-major operand
constexpr int kEpiBuf = 32 * 128;       // 32 rows x 128 bytes
constexpr int kEpiBytes = kEpiWarps * kEpiBuf;

// What a tile's epilogue does.
enum Mode {
    kLinear,  // bias, activation, residual; bf16, the pre-activations too where wanted
    kGated,   // the same for two projections and their product
    kPlain,   // bf16
    kF32
};

// Tile shape and shared memory of one variant: kBN output columns.
template <int kMode, int kBN>
struct Cfg {
    static constexpr int kBHalf = kMode == kGated ? 128 : kBN / 2;  // B columns each CTA stages
    static constexpr int kMmaN = 2 * kBHalf;
    static constexpr int kBBytes = kBHalf * kBK * 2;
    static constexpr int kStepBytes = kABytes + kBBytes;  // one 64-deep step
    static constexpr int kStageBytes = 2 * kStepBytes;    // a stage holds two
    static constexpr int kStages = kBHalf == 128 ? 3 : 4;
    static constexpr size_t kEpiOff = (size_t)kStages * kStageBytes;
    static constexpr size_t kBarOff = kEpiOff + kEpiBytes;
    static constexpr size_t kSmem = kBarOff + 512 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Args {
    int M, N;        // output rows and columns of one problem
    int mt, nt;      // its tiles
    int gm;          // row tiles per band
    int seg_steps;   // reduction steps of one segment
    int steps;       // reduction steps in all (segments x seg_steps)
    int full;        // tiles done whole
    int splits;      // the others: each in this many units
    int total;       // units: full + splits * (tiles - full)
    int act;
    const float* bias0;
    const float* bias1;
    bool has_res, has_z0, has_z1;
    float* part;         // partial sums of the split tiles
    uint32_t* counters;  // [split tiles][2 CTAs][8 warps]; null: sum_units_kernel adds the splits
    bool late_wait;      // the kernel before this one writes nothing that this one uses, and opens the gate
    uint32_t* gate;      // to wait at (late_wait) or to open, or null
    int32_t* flags;
};

struct Tile {
    int m0, n0, prob;
    int k0, k1;        // reduction steps
    int slot, split;   // slot >= 0: a unit of the slot-th split tile
};

// Unit t.  Tiles of one problem run in bands of gm row tiles, the row tile
// running fastest, so that pairs working side by side share B's columns and a
// band's A rows stay in L2.
template <int kBN>
__device__ __forceinline__ Tile decode(int t, const Args& a) {
    Tile ti;
    ti.slot = -1;
    ti.split = 0;
    ti.k0 = 0;
    ti.k1 = a.steps;
    if (t >= a.full) {
        const int u = t - a.full;
        const int slot = u / a.splits;
        t = a.full + slot;
        if (a.splits > 1) {
            ti.slot = slot;
            ti.split = u - slot * a.splits;
            ti.k0 = (int)((int64_t)a.steps * ti.split / a.splits);
            ti.k1 = (int)((int64_t)a.steps * (ti.split + 1) / a.splits);
        }
    }
    const int per = a.mt * a.nt, local = t % per;
    const int band = local / (a.gm * a.nt), rem = local - band * a.gm * a.nt;
    const int first = band * a.gm, width = min(a.gm, a.mt - first);
    ti.prob = t / per;
    ti.n0 = rem / width * kBN;
    ti.m0 = (first + rem % width) * (2 * kBM);
    return ti;
}

// Steps of the stage that starts at ks: two, or one at the end of a segment or
// of the tile's share of the reduction.
__device__ __forceinline__ int stage_steps(int ks, const Tile& ti, const Args& a) {
    return ks + 1 < ti.k1 && ks + 1 != a.seg_steps ? 2 : 1;
}

__device__ __forceinline__ uint32_t buf_off(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void pack32(const float (&v)[32], uint32_t* o) {
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = pack2(v[2 * i], v[2 * i + 1]);
}

// v[i] += bias[n + i]; the columns past N (a multiple of 8) are not read.
__device__ __forceinline__ void add_bias(float (&v)[32], const float* bias, int n, int N) {
    if (!bias) return;
#pragma unroll
    for (int i = 0; i < 32; i += 4)
        if (n + i < N) {
            const float4 b = __ldg(reinterpret_cast<const float4*>(bias + n + i));
            v[i] += b.x, v[i + 1] += b.y, v[i + 2] += b.z, v[i + 3] += b.w;
        }
}

// 16 packed words into row `lane` of a staging buffer, columns 32 * sub on.
__device__ __forceinline__ void stage16(uint32_t buf, int lane, int sub, const uint32_t* o) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        st_shared_u4(buf + buf_off(lane, 4 * sub + i), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
}

// The warp's staged buffer -> the map's box at (col, row).
__device__ __forceinline__ void store_buf(const CUtensorMap* map, uint32_t buf, int lane, int col, int row) {
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_3d(map, buf, col, row, 0);
        bulk_commit();
    }
}

// The warp's last store has read the staging buffer.
__device__ __forceinline__ void buffer_free(int lane) {
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
}

template <int kMode, bool kAMN, bool kBMN, int kBN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) dense_gemm_kernel(
    const __grid_constant__ CUtensorMap mA0, const __grid_constant__ CUtensorMap mA1,
    const __grid_constant__ CUtensorMap mB0, const __grid_constant__ CUtensorMap mB1,
    const __grid_constant__ CUtensorMap mD0, const __grid_constant__ CUtensorMap mD1,
    const __grid_constant__ CUtensorMap mD2, const __grid_constant__ CUtensorMap mR, const Args a) {
    using C = Cfg<kMode, kBN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // used in the leader
    uint64_t* empty = full + C::kStages;
    uint64_t* tfull = empty + C::kStages;
    uint64_t* tempty = tfull + 2;  // used in the leader: 8 epilogue warps x 2 CTAs
    uint64_t* drain = tempty + 2;
    uint64_t* rbar = drain + 1;  // residual chunks, one barrier per epilogue warp
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(rbar + kEpiWarps);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // warp: uniform
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        for (int i = 0; i < kEpiWarps; ++i) mbar_init(&rbar[i], 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&mA0);
        tma_prefetch_map(&mB0);
        tma_prefetch_map(&mD0);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, kTmemCols);
        tmem_relinquish_pair();
    }
    // beside the kernel before this one: the operands, from who has waited for them
    bool shut = false;
    if (a.late_wait && threadIdx.x == kThreads - 1) shut = !gate_wait(a.gate);
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    if (!a.late_wait) {
        chain_wait();
        if (a.gate && blockIdx.x == 0 && threadIdx.x == kThreads - 1) gate_open(a.gate);
    } else if (threadIdx.x == kThreads - 1) {
        if (shut) {
            *abort_flag = 1;
            atomicOr(a.flags, 0x2);
        } else {
            gate_passed(a.gate);
        }
    }
    chain_next();
    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            if (a.late_wait) fence_async_global();
            uint32_t it = 0;
            for (int t = pair; t < a.total && !*abort_flag; t += npairs) {
                const Tile ti = decode<kBN>(t, a);
                const int arow = ti.m0 + (int)rank * kBM;
                const int brow = kMode == kGated ? ti.n0 : ti.n0 + (int)rank * C::kBHalf;
                for (int ks = ti.k0, n; ks < ti.k1; ks += n, ++it) {
                    n = stage_steps(ks, ti, a);
                    const int s = it % C::kStages;
                    if (!wait_or_abort(&empty[s], ((it / C::kStages) & 1) ^ 1, abort_flag, a.flags)) break;
                    const bool seg1 = ks >= a.seg_steps;
                    const CUtensorMap* pA = seg1 || ti.prob ? &mA1 : &mA0;
                    const CUtensorMap* pB = seg1 || (kMode == kGated && rank) ? &mB1 : &mB0;
                    if (leader) mbar_arrive_expect_tx(&full[s], 2 * n * C::kStepBytes);
                    for (int j = 0; j < n; ++j) {
                        const int kc = (ks + j - (seg1 ? a.seg_steps : 0)) * kBK;
                        uint8_t* sa = smem + s * C::kStageBytes + j * C::kStepBytes;
                        uint8_t* sb = sa + kABytes;
                        if (kAMN) {
                            tma_load_3d_pair(sa, pA, &full[s], arow, kc, 0);
                            tma_load_3d_pair(sa + kBox, pA, &full[s], arow + 64, kc, 0);
                        } else {
                            tma_load_3d_pair(sa, pA, &full[s], kc, arow, 0);
                        }
                        if (kBMN) {
#pragma unroll
                            for (int i = 0; i < C::kBHalf / 64; ++i)
                                tma_load_3d_pair(sb + i * kBox, pB, &full[s], brow + 64 * i, kc, 0);
                        } else {
                            tma_load_3d_pair(sb, pB, &full[s], kc, brow, 0);
                        }
                    }
                }
            }
            // copies of both CTAs complete on the leader's barriers
            if (leader)
                for (uint32_t j = (it > (uint32_t)C::kStages ? it - C::kStages : 0); j < it; ++j)
                    drain_wait(&full[j % C::kStages], (j / C::kStages) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader)
        // (the whole warp, one lane elected).  One warp's instruction stream paces
        // the tensor core, so it is kept short: descriptors by addition, no
        // division.  (Testing the next stage's barrier ahead gains nothing.)
        if (leader) {
            constexpr uint32_t kIdesc = idesc_bf16_major(2 * kBM, C::kMmaN, kAMN, kBMN);
            constexpr uint32_t kStepA = (kAMN ? 2048 : 32) >> 4, kStepB = (kBMN ? 2048 : 32) >> 4;
            const uint32_t base = smem_u32(smem);
            const uint64_t da0 = kAMN ? desc_mnmajor_sw128(base, kBox, 1024) : desc_kmajor_sw128(base);
            const uint64_t db0 = kBMN ? desc_mnmajor_sw128(base + kABytes, kBox, 1024) : desc_kmajor_sw128(base + kABytes);
            uint32_t s = 0, ph = 0, tc = 0;
            for (int t = pair; t < a.total && !aborted_warp(abort_flag); t += npairs, ++tc) {
                const Tile ti = decode<kBN>(t, a);
                const uint32_t acc = tc & 1;
                if (!wait_or_abort_warp(&tempty[acc], ((tc >> 1) & 1) ^ 1, abort_flag, a.flags)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + acc * kAccCols;
                bool ok = true;
                uint32_t sum = 0;
                for (int ks = ti.k0, n; ks < ti.k1; ks += n) {
                    n = stage_steps(ks, ti, a);
                    if (!wait_or_abort_warp(&full[s], ph, abort_flag, a.flags)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t cur = s;
                    if (++s == C::kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                    uint64_t da = da0 + cur * (C::kStageBytes >> 4), db = db0 + cur * (C::kStageBytes >> 4);
                    for (int j = 0; j < n; ++j, da += C::kStepBytes >> 4, db += C::kStepBytes >> 4)
#pragma unroll
                        for (int kk = 0; kk < kBK / 16; ++kk) {
                            mma_bf16_pair_warp(d, da + kk * kStepA, db + kk * kStepB, kIdesc, sum);
                            sum = 1;
                        }
                    mma_commit_pair_warp(&empty[cur], 0x3);  // frees the stage in both CTAs
                }
                if (!ok) break;
                mma_commit_pair_warp(&tfull[acc], 0x3);
            }
            mma_commit_pair_warp(drain, 0x1);
            drain_wait(drain, 0);
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        const int e = warp - 2, q = warp & 3, half = e >> 2;
        uint8_t* buf_ptr = smem + C::kEpiOff + (size_t)e * kEpiBuf;
        const uint32_t buf = smem_u32(buf_ptr);
        constexpr int kHalfCols = kBN / 2;               // output columns of this warp
        constexpr int kChunk = kMode == kF32 ? 32 : 64;  // columns of the staging buffer
        constexpr int kChunks = kHalfCols / kChunk;
        constexpr int kGroups = C::kMmaN / 64;  // this warp's accumulator columns, in groups of 32
        uint32_t tc = 0, rph = 0;
        for (int t = pair; t < a.total; t += npairs, ++tc) {
            const Tile ti = decode<kBN>(t, a);
            const uint32_t acc = tc & 1;
            const int row = ti.m0 + (int)rank * kBM + q * 32;
            const int col0 = ti.n0 + half * kHalfCols;
            const bool in = row < a.M && col0 < a.N;
            const bool whole = ti.slot < 0;
            // chunk j's residual into the staging buffer
            auto fetch_res = [&](int j) {
                buffer_free(lane);
                if (lane == 0) {
                    mbar_arrive_expect_tx(&rbar[e], kEpiBuf);
                    tma_load_3d(buf_ptr, &mR, &rbar[e], col0 + j * kChunk, row, 0);
                }
            };
            const bool res = kMode == kLinear && a.has_res;
            const bool ahead = res && in && whole;
            if (ahead) fetch_res(0);  // ahead of the accumulator
            if (!wait_sleep_or_abort_warp(&tfull[acc], (tc >> 1) & 1, abort_flag, a.flags)) {
                if (ahead) drain_wait(&rbar[e], rph);
                break;
            }
            tc_fence_after();
            const uint32_t tq = tmem_base + acc * kAccCols + ((uint32_t)(q * 32) << 16);
            // accumulator column of group g (gated: two groups of gate, two of up)
            auto acc_col = [&](int g) {
                return kMode == kGated ? (g >> 1) * 128 + half * 64 + (g & 1) * 32 : half * kHalfCols + g * 32;
            };
            auto accumulator_free = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(&tempty[acc], 0);
            };
            if (!in) {
                accumulator_free();
                continue;
            }
            if (!whole) {
                // this split's sums of the warp's region, [group][8][lane]
                // float4; the split that arrives last puts the sum over the
                // splits, in order, back into TMEM and goes on as for a whole tile
                constexpr int kRegion = 4 * 8 * 32, kUnit = 2 * kEpiWarps * kRegion;
                float4* parts = reinterpret_cast<float4*>(a.part) + (int64_t)ti.slot * a.splits * kUnit +
                                (rank * kEpiWarps + e) * kRegion + lane;
#pragma unroll 1
                for (int g = 0; g < kGroups; ++g) {
                    float v[32];
                    tmem_ld32(tq + acc_col(g), v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        __stcg(parts + (int64_t)ti.split * kUnit + (g * 8 + i) * 32,
                               make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                }
                if (!a.counters) {
                    accumulator_free();
                    continue;
                }
                __threadfence();
                __syncwarp();
                uint32_t before = 0;
                uint32_t* counter = a.counters + (ti.slot * 2 + rank) * kEpiWarps + e;
                if (lane == 0) {
                    before = atomicAdd(counter, 1u);
                    if (before == (uint32_t)a.splits - 1) *counter = 0;  // for the next call
                }
                before = __shfl_sync(0xffffffffu, before, 0);
                if (before != (uint32_t)a.splits - 1) {
                    accumulator_free();
                    continue;
                }
                __threadfence();
#pragma unroll 1
                for (int g = 0; g < kGroups; ++g) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
                    for (int s = 0; s < a.splits; s += 2) {  // two splits' loads in flight
                        const float4* p = parts + (int64_t)s * kUnit + g * 8 * 32;
                        const bool two = s + 1 < a.splits;
                        float4 w[2][8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[0][i] = __ldcg(p + i * 32);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[1][i] = two ? __ldcg(p + kUnit + i * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                v[4 * i] += w[h][i].x, v[4 * i + 1] += w[h][i].y;
                                v[4 * i + 2] += w[h][i].z, v[4 * i + 3] += w[h][i].w;
                            }
                    }
                    tmem_st32(tq + acc_col(g), v);
                }
                if (res) fetch_res(0);
            }
            auto sums = [&](int g, float (&v)[32], bool last) {
                tmem_ld32(tq + acc_col(g), v);
                if (last) accumulator_free();
            };
            if (kMode == kF32) {
#pragma unroll 1
                for (int j = 0; j < kChunks; ++j) {
                    float v[32];
                    sums(j, v, j == kChunks - 1);
                    const int col = col0 + j * 32;
                    if (col >= a.N) continue;
                    buffer_free(lane);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_shared_u4(buf + buf_off(lane, i), __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                     __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
                    store_buf(ti.prob ? &mD1 : &mD0, buf, lane, col, row);
                }
            } else if (kMode == kPlain) {
#pragma unroll 1
                for (int j = 0; j < kChunks; ++j) {
                    float v[64];
                    tmem_ld64(tq + acc_col(2 * j), v);
                    if (j == kChunks - 1) accumulator_free();
                    const int col = col0 + j * kChunk;
                    if (col >= a.N) continue;
                    uint32_t o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = pack2(v[2 * i], v[2 * i + 1]);
                    buffer_free(lane);
                    stage16(buf, lane, 0, o);
                    stage16(buf, lane, 1, o + 16);
                    store_buf(ti.prob ? &mD1 : &mD0, buf, lane, col, row);
                }
            } else if (kMode == kGated) {
                // the kept projections first, one at a time through the buffer
#pragma unroll 1
                for (int p = 0; p < 2; ++p) {
                    if (!(p ? a.has_z1 : a.has_z0)) continue;
                    buffer_free(lane);
#pragma unroll
                    for (int sub = 0; sub < 2; ++sub) {
                        float v[32];
                        sums(2 * p + sub, v, false);
                        add_bias(v, p ? a.bias1 : a.bias0, col0 + 32 * sub, a.N);
                        uint32_t o[16];
                        pack32(v, o);
                        stage16(buf, lane, sub, o);
                    }
                    store_buf(p ? &mD2 : &mD1, buf, lane, col0, row);
                }
                uint32_t h[32];
#pragma unroll
                for (int sub = 0; sub < 2; ++sub) {
                    float g[32], u[32];
                    sums(sub, g, false);
                    sums(2 + sub, u, sub == 1);
                    add_bias(g, a.bias0, col0 + 32 * sub, a.N);
                    add_bias(u, a.bias1, col0 + 32 * sub, a.N);
                    by_act(a.act, [&](auto k) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) g[i] = act_value<k.value>(g[i]) * u[i];
                    });
                    pack32(g, h + 16 * sub);
                }
                buffer_free(lane);
                stage16(buf, lane, 0, h);
                stage16(buf, lane, 1, h + 16);
                store_buf(&mD0, buf, lane, col0, row);
            } else {
#pragma unroll 1
                for (int j = 0; j < kChunks; ++j) {
                    const int col = col0 + j * kChunk;
                    const bool live = col < a.N;
                    if (live) {
                        if (!res) {
                            buffer_free(lane);
                        } else {
                            if (j > 0) fetch_res(j);
                            if (!wait_or_abort_warp(&rbar[e], rph, abort_flag, a.flags)) drain_wait(&rbar[e], rph);
                            rph ^= 1;
                        }
                    }
                    uint32_t y[32];
#pragma unroll
                    for (int sub = 0; sub < 2; ++sub) {
                        float v[32];
                        sums(2 * j + sub, v, j == kChunks - 1 && sub == 1);
                        if (!live) continue;
                        add_bias(v, a.bias0, col + 32 * sub, a.N);
                        uint32_t r[16];
                        if (res)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint4 w = ld_shared_u4(buf + buf_off(lane, 4 * sub + i));
                                r[4 * i] = w.x, r[4 * i + 1] = w.y, r[4 * i + 2] = w.z, r[4 * i + 3] = w.w;
                            }
                        if (a.has_z0) {  // in the place of the residual just read
                            uint32_t o[16];
                            pack32(v, o);
                            stage16(buf, lane, sub, o);
                        }
                        by_act(a.act, [&](auto k) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = act_value<k.value>(v[i]);
                        });
                        if (res)
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                v[2 * i] += __uint_as_float(r[i] << 16);
                                v[2 * i + 1] += __uint_as_float(r[i] & 0xffff0000u);
                            }
                        pack32(v, y + 16 * sub);
                    }
                    if (live) {
                        if (a.has_z0) {
                            store_buf(&mD1, buf, lane, col, row);
                            buffer_free(lane);
                        }
                        stage16(buf, lane, 0, y);
                        stage16(buf, lane, 1, y + 16);
                        store_buf(&mD0, buf, lane, col, row);
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_read<0>();  // the stores land before the kernel counts as complete
    }

    __syncwarp();  // the single-lane roles join their warps
    if (*abort_flag && !leader) {
        // aborted: this CTA's copies complete on the leader's barriers; give
        // any still in flight time to land before shared memory is released
        for (int i = 0; i < 2000; ++i) __nanosleep(100);
    }
    // what follows this kernel may count on the one before it having completed
    if (a.late_wait) chain_wait();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

// The split tiles of a weight gradient, their splits added in order: one thread
// per 4 columns of a row, a block per 32 columns of a warp's region, so that many
// splits are added by the whole GPU at once.
template <typename O>
__global__ void __launch_bounds__(256) sum_units_kernel(const Args a, O* out0, O* out1) {
    chain_wait();
    chain_next();
    constexpr int kRegion = 4 * 8 * 32, kUnit = 2 * kEpiWarps * kRegion;  // float4
    const int slot = blockIdx.x, region = blockIdx.y >> 2, g = blockIdx.y & 3;
    const int i = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Tile ti = decode<256>(a.full + slot * a.splits, a);
    const int e = region & 7, warp = e + 2, row = ti.m0 + (region >> 3) * kBM + (warp & 3) * 32 + lane;
    const int col = ti.n0 + (e >> 2) * 128 + g * 32 + i * 4;
    if (row >= a.M || col >= a.N) return;
    const float4* p =
        reinterpret_cast<const float4*>(a.part) + (int64_t)slot * a.splits * kUnit + region * kRegion + (g * 8 + i) * 32 + lane;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float4 w = __ldcg(p + (int64_t)s * kUnit);
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    O* out = (ti.prob ? out1 : out0) + (int64_t)row * a.N + col;
    if constexpr (sizeof(O) == 4)
        *reinterpret_cast<float4*>(out) = v;
    else
        *reinterpret_cast<uint2*>(out) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
}

struct Maps {
    CUtensorMap A0, A1, B0, B1, D0, D1, D2, R;
};

template <int kMode, bool kAMN, bool kBMN, int kBN>
cudaError_t launch(const Maps& m, const Args& a, const char* name, cudaStream_t st) {
    using C = Cfg<kMode, kBN>;
    auto* fn = dense_gemm_kernel<kMode, kAMN, kBMN, kBN>;
    cudaError_t e = ensure_smem_attr(fn, C::kSmem);
    if (e != cudaSuccess) return e;
    const int grid = 2 * std::max(1, std::min(device_sm_count() / 2, a.total));
    trace_before(name, st);
    e = launch_chained(fn, grid, kThreads, C::kSmem, 0, st, m.A0, m.A1, m.B0, m.B1, m.D0, m.D1, m.D2, m.R, a);
    trace_after(st);
    return e;
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Row tiles per band: A rows of about 32 MB.
int band_of(int64_t k) {
    const int64_t g = (32ll << 20) / (2 * kBM * 2 * std::max<int64_t>(k, 1));
    return (int)std::min<int64_t>(std::max<int64_t>(g, 8), 1 << 20);
}

// Which tiles are split, and how.  Whole waves of kDensePairs tiles are done
// whole; the r tiles of the last, partial wave in S units each where that ends
// sooner.  Costs in reduction steps (0.32 us): ceil(r S / pairs) rounds of steps
// / S, and adding the partial sums: by the split that arrives last (its warps wait
// for L2 round trips), or, for a weight gradient, by a kernel of its own on the
// whole GPU.  Measured on weight gradients of 6 to 48 tiles and 16 to 512 steps:
// 6 tiles of 47 steps take 19.3 us whole, 16.8 in 4 splits added in the kernel,
// 11.0 in 8 added by the second one; a second round of units costs more than it
// gives.
enum Split { kWhole, kInKernel, kOwnKernel };
struct TailPlan {
    int full, splits, slots;
    int cost;  // of the last wave, in steps
};
constexpr int kMaxSplitRounds = 3;  // bounds the workspace: 3 x 74 units of 256 KB
TailPlan tail_plan(int64_t tiles, int steps, Split how) {
    const int r = (int)(tiles % kDensePairs);
    TailPlan best{(int)tiles, 1, 0, r ? steps : 0};
    for (int s = 2; how != kWhole && r && s <= (how == kOwnKernel ? 32 : 8) && steps >= 4 * s; ++s) {
        const int rounds = cdiv((int64_t)r * s, kDensePairs);
        if (rounds > kMaxSplitRounds) break;
        const int cost = rounds * cdiv(steps, s) + (rounds - 1) * 25 +
                         (how == kOwnKernel ? 8 + r * s * 2 / 11 : 12 + 4 * s + r * s / 10);
        if (cost < best.cost) best = {(int)tiles - r, s, r, cost};
    }
    // less than a twentieth of the whole is not worth it: with pairs idle in the
    // last wave the others' clock is higher
    if (best.splits > 1 && (steps - best.cost) * 20 < (tiles / kDensePairs + 1) * steps)
        best = {(int)tiles, 1, 0, steps};
    return best;
}

constexpr int64_t kUnitFloats = 256 * 256;
constexpr size_t kCounterBytes = (size_t)kDensePairs * 2 * kEpiWarps * sizeof(uint32_t);
static_assert(kCounterBytes <= kDenseGateOffset, "counters");

// Time of a tile of 128 columns against one of 256.
constexpr double kNarrow = 0.65;
struct Problem {  // M x N outputs over `steps` reduction steps, `problems` times
    int64_t M;
    int N, bn, seg_steps, segs, problems;
    Split split;
    int64_t tiles() const { return (int64_t)cdiv(M, 2 * kBM) * cdiv(N, bn) * problems; }
    TailPlan plan() const { return tail_plan(tiles(), seg_steps * segs, split); }
    // reduction steps of the busiest pair, a split's overhead among them
    double pair_steps() const { return (double)(tiles() / kDensePairs) * seg_steps * segs + plan().cost; }
    size_t part_floats() const {
        const TailPlan p = plan();
        return (size_t)p.slots * p.splits * kUnitFloats;
    }
};
// The linear forward has column tiles of 256, or of 128 where the finer grid ends
// sooner: 512 x 4096 -> 4096 takes 19.8 instead of 21.9 us (64 tiles for 74 pairs,
// not 32), 2048 x 1024 -> 1024 8.6 instead of 10.4; but 4096 x 4096 -> 14336, whose
// waves are full either way, would take 421 instead of 329.  An input gradient shares
// the GPU with the weight gradient, which takes up the idle pairs, and gains nothing
// (2048 x 4096 -> 4096: 112.0 and 112.2 us with and without).
Problem fwd_problem(int64_t T, int K, int N, bool gated) {
    const Problem p{T, N, gated ? 128 : 256, cdiv(K, kBK), 1, 1, kInKernel};
    Problem q = p;
    q.bn = 128;
    return !gated && kNarrow * q.pair_steps() < 0.97 * p.pair_steps() ? q : p;
}
Problem dgrad_problem(int64_t T, int K, int N, int segs) { return {T, K, 256, cdiv(N, kBK), segs, 1, kInKernel}; }
Problem wgrad_problem(int64_t T, int K, int N, int problems, bool split) {
    return {N, K, 256, cdiv(T, kBK), 1, problems, split ? kOwnKernel : kWhole};
}

Args args_of(const Problem& pr, const DenseWs& ws) {
    const TailPlan p = pr.plan();
    Args a{};
    a.M = (int)pr.M;
    a.N = pr.N;
    a.mt = cdiv(pr.M, 2 * kBM);
    a.nt = cdiv(pr.N, pr.bn);
    // no more than there are, so that a band's tiles, gm x nt, are no more than all of
    // them: 1024 row tiles of 2^22 column tiles (one row of 2^30 outputs) would not
    // fit an int
    a.gm = std::min(a.mt, band_of((int64_t)pr.seg_steps * pr.segs * kBK));
    a.seg_steps = pr.seg_steps;
    a.steps = pr.seg_steps * pr.segs;
    a.full = p.full;
    a.splits = p.splits;
    a.total = p.full + p.slots * p.splits;
    a.part = ws.part;
    a.counters = pr.split == kOwnKernel ? nullptr : ws.counters;
    a.flags = ws.flags;
    return a;
}

}  // namespace

double dense_fwd_pairs_steps(int64_t T, int K, int N, bool gated) {
    const Problem p = fwd_problem(T, K, N, gated);
    return p.pair_steps() * (!gated && p.bn == 128 ? kNarrow : 1);
}
double dense_dgrad_pairs_steps(int64_t T, int K, int N, int segs) { return dgrad_problem(T, K, N, segs).pair_steps(); }
static int ctas_of(const Problem& p) {
    const TailPlan t = p.plan();
    return 2 * std::min(kDensePairs, t.full + t.slots * t.splits);
}
int dense_dgrad_pairs_ctas(int64_t T, int K, int N, int segs) { return ctas_of(dgrad_problem(T, K, N, segs)); }
int dense_wgrad_ctas(int64_t T, int K, int N, int problems, bool split) {
    return ctas_of(wgrad_problem(T, K, N, problems, split));
}
double dense_wgrad_us(int64_t T, int K, int N, int problems, bool split) {
    const Problem p = wgrad_problem(T, K, N, problems, split);
    return 4.5 + std::max(0.33 * p.pair_steps(), (double)problems * N * K * 4 / 5.2e6);
}
size_t dense_fwd_pairs_part_floats(int64_t T, int K, int N, bool gated) {
    return fwd_problem(T, K, N, gated).part_floats();
}
size_t dense_dgrad_pairs_part_floats(int64_t T, int K, int N, int segs) {
    return dgrad_problem(T, K, N, segs).part_floats();
}
size_t dense_wgrad_part_floats(int64_t T, int K, int N, int problems) {
    return wgrad_problem(T, K, N, problems, true).part_floats();
}

cudaError_t launch_dense_fwd_pairs(const void* x, const void* w0, const void* w1, int64_t T, int K, int N,
                                   const DenseOut& o, const DenseWs& ws, cudaStream_t st) {
    const bool gated = w1 != nullptr;
    const Problem pr = fwd_problem(T, K, N, gated);
    const int bhalf = gated ? 128 : pr.bn / 2;
    Maps m;
    bool ok = make_tile_map(&m.A0, false, x, K, T, 1, kBM) && make_tile_map(&m.B0, false, w0, K, N, 1, bhalf) &&
              make_tile_map(&m.D0, false, o.y, N, T, 1, 32);
    m.A1 = m.A0;
    m.B1 = m.B0;
    m.D1 = m.D2 = m.R = m.D0;
    if (gated) ok = ok && make_tile_map(&m.B1, false, w1, K, N, 1, bhalf);
    if (o.z0) ok = ok && make_tile_map(&m.D1, false, o.z0, N, T, 1, 32);
    if (o.z1) ok = ok && make_tile_map(&m.D2, false, o.z1, N, T, 1, 32);
    if (o.res) ok = ok && make_tile_map(&m.R, false, o.res, N, T, 1, 32);
    if (!ok) return cudaErrorInvalidValue;
    Args a = args_of(pr, ws);
    a.act = o.act;
    a.bias0 = o.bias0;
    a.bias1 = o.bias1;
    a.has_res = o.res != nullptr;
    a.has_z0 = o.z0 != nullptr;
    a.has_z1 = o.z1 != nullptr;
    if (gated) return launch<kGated, false, false, 128>(m, a, "gated_fwd", st);
    return pr.bn == 128 ? launch<kLinear, false, false, 128>(m, a, "linear_fwd", st)
                        : launch<kLinear, false, false, 256>(m, a, "linear_fwd", st);
}

cudaError_t launch_dense_dgrad_pairs(const void* dz0, const void* dz1, const void* w0, const void* w1, int64_t T,
                                     int K, int N, void* dx, bool opens_gate, const DenseWs& ws, cudaStream_t st) {
    Maps m;
    bool ok = make_tile_map(&m.A0, false, dz0, N, T, 1, kBM) && make_tile_map(&m.B0, false, w0, K, N, 1, 64) &&
              make_tile_map(&m.D0, false, dx, K, T, 1, 32);
    m.A1 = m.A0;
    m.B1 = m.B0;
    m.D1 = m.D2 = m.R = m.D0;
    if (dz1)
        ok = ok && make_tile_map(&m.A1, false, dz1, N, T, 1, kBM) && make_tile_map(&m.B1, false, w1, K, N, 1, 64);
    if (!ok) return cudaErrorInvalidValue;
    Args a = args_of(dgrad_problem(T, K, N, dz1 ? 2 : 1), ws);
    a.gate = opens_gate ? ws.gate : nullptr;
    return launch<kPlain, false, true, 256>(m, a, dz1 ? "gated_dgrad" : "linear_dgrad", st);
}

cudaError_t launch_dense_wgrad(const void* dz0, const void* dz1, const void* x, int64_t T, int K, int N, void* dw0,
                               void* dw1, bool f32, WgradPlan plan, const DenseWs& ws, cudaStream_t st) {
    Maps m;
    bool ok = make_tile_map(&m.A0, false, dz0, N, T, 1, 64) && make_tile_map(&m.B0, false, x, K, T, 1, 64) &&
              make_tile_map(&m.D0, f32, dw0, K, N, 1, 32);
    m.A1 = m.A0;
    m.B1 = m.B0;
    m.D1 = m.D2 = m.R = m.D0;
    if (dz1) ok = ok && make_tile_map(&m.A1, false, dz1, N, T, 1, 64) && make_tile_map(&m.D1, f32, dw1, K, N, 1, 32);
    if (!ok) return cudaErrorInvalidValue;
    Args a = args_of(wgrad_problem(T, K, N, dz1 ? 2 : 1, plan.split), ws);
    a.late_wait = plan.beside;
    a.gate = plan.beside ? ws.gate : nullptr;
    const char* name = dz1 ? "gated_wgrad" : "linear_wgrad";
    const cudaError_t e =
        f32 ? launch<kF32, true, true, 256>(m, a, name, st) : launch<kPlain, true, true, 256>(m, a, name, st);
    if (e != cudaSuccess || a.total == a.full || a.counters) return e;
    const dim3 grid((a.total - a.full) / a.splits, 2 * kEpiWarps * 4);
    trace_before("wgrad_sum", st);
    const cudaError_t e2 =
        f32 ? launch_chained(sum_units_kernel<float>, grid, 256, 0, 0, st, a, (float*)dw0, (float*)dw1)
            : launch_chained(sum_units_kernel<bf16>, grid, 256, 0, 0, st, a, (bf16*)dw0, (bf16*)dw1);
    trace_after(st);
    return e2;
}

}  // namespace moe
