// Further Blackwell (sm_100a) building blocks as inline PTX, on top of
// sm100.cuh: programmatic launches, tensor stores, MMAs issued from a converged
// warp, and smaller TMEM transfers.  Used by the norm, linear and gated kernels.
#pragma once

#include "sm100.cuh"

namespace moe {
namespace sm100 {

// The waits of sm100.cuh for a whole, converged warp that goes on as one: every
// lane gets the same answer, also when a time-out or another role's abort
// reaches only some of them (a warp that split there would never meet again at
// its next collective instruction).
__device__ __forceinline__ bool wait_or_abort_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                   int32_t* flags) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, flags));
}
__device__ __forceinline__ bool wait_sleep_or_abort_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                         int32_t* flags) {
    return __all_sync(0xffffffffu, wait_sleep_or_abort(bar, parity, abort_flag, flags));
}
__device__ __forceinline__ bool aborted_warp(volatile int* abort_flag) {
    return __any_sync(0xffffffffu, *abort_flag != 0);
}

// ------------------------------------------------- programmatic launches
// A kernel launched by launch_chained (tma_host.cuh) may start while the one
// before it on its stream still runs.  It sets itself up (barriers, TMEM,
// tensor maps), then calls chain_wait before its first access to global
// memory: that returns when the kernel before has completed and its writes are
// visible.  chain_next lets the kernel after it start in the same way, once
// every CTA of this one has called it.  Every kernel calls chain_wait first and
// chain_next second: a kernel that has started then knows that the one before
// the one before it has completed.  That one's writes are promised to who called
// chain_wait, though, so a kernel that uses them without waiting for the one
// between takes them over from it through a gate: a thread of the one between
// opens it (release) after its chain_wait, and the other waits for that (acquire).
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A gate: {open, CTAs that have passed}, both zero between calls.
__device__ __forceinline__ void gate_open(uint32_t* gate) {
    asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(gate) : "memory");
}
// One thread per CTA; false if the gate stays shut for a second or more.
constexpr uint32_t kGatePolls = 1u << 21;
__device__ __forceinline__ bool gate_wait(const uint32_t* gate) {
    for (uint32_t i = 0; i < kGatePolls; ++i) {
        uint32_t open;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(open) : "l"(gate) : "memory");
        if (open) return true;
    }
    return false;
}
// After gate_wait, by the same threads: the last of the grid's CTAs shuts it.
__device__ __forceinline__ void gate_passed(uint32_t* gate) {
    if (atomicAdd(gate + 1, 1u) == gridDim.x - 1) {
        gate[1] = 0;
        gate[0] = 0;
    }
}
// Orders what this thread has seen of global memory before its later
// asynchronous copies from there.
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// ------------------------------------------------------------ TMA stores
// Tiled 3-D store of a shared-memory box to (c0, c1, c2); elements outside the
// tensor are not written.  One bulk group per bulk_commit of the thread.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until at most kLeft of this thread's bulk groups still read shared memory.
template <int kLeft>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}
// Orders this thread's shared-memory accesses before later asynchronous copies.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

// -------------------------------------------------------------- tcgen05
// tcgen05.mma and .commit called by a whole, converged warp; one elected
// lane (always the same one) issues them.  Code that the whole warp runs keeps
// descriptors and addresses in uniform registers, which is where the
// instructions want them: a loop run by one lane alone spends about 80 cycles
// per MMA moving them there.
__device__ __forceinline__ void mma_bf16_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync r|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_bf16_pair_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync r|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit_warp(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b32 r;\n\t"
        "elect.sync r|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void mma_commit_pair_warp(uint64_t* bar, uint16_t cta_mask) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b32 r;\n\t"
        "elect.sync r|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"(cta_mask)
        : "memory");
}

// 16 consecutive float32 columns of the thread's TMEM lane, one wait.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Write 32 float32 columns of the thread's TMEM lane (store and its wait in
// one asm statement).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31, %32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])),
        "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])),
        "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
        "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])),
        "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])),
        "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
        : "memory");
}

}  // namespace sm100
}  // namespace moe
