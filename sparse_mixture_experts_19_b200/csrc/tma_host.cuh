// Host-side helpers shared by the tcgen05 kernels: TMA tensor-map encoding
// through the driver entry point (no link-time dependency on libcuda) and the
// SM count of the current device.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>
#include <utility>

namespace moe {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Rank-3 map of a bf16 tensor [depth][rows][inner] (inner contiguous) with
// box {box_inner, box_rows, 1} and the 128-byte swizzle; out-of-range
// elements of a box read as zero.  A map depends only on these arguments, so
// encoded maps are kept in a small process-wide cache.
inline bool make_map_bf16(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows,
                          uint64_t depth, uint32_t box_inner, uint32_t box_rows) {
    struct Entry {
        const void* base;
        uint64_t inner, rows, depth;
        uint32_t box_inner, box_rows;
        CUtensorMap map;
    };
    constexpr int kCache = 64;
    static Entry cache[kCache];
    static int used = 0, next = 0;
    static std::mutex mu;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (int i = 0; i < used; ++i) {
            const Entry& c = cache[i];
            if (c.base == base && c.inner == inner && c.rows == rows && c.depth == depth &&
                c.box_inner == box_inner && c.box_rows == box_rows) {
                *m = c.map;
                return true;
            }
        }
    }
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {inner, rows, depth};
    cuuint64_t strides[2] = {inner * 2, inner * rows * 2};
    cuuint32_t box[3] = {box_inner, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    std::lock_guard<std::mutex> lock(mu);
    Entry& c = cache[next];
    c = Entry{base, inner, rows, depth, box_inner, box_rows, *m};
    next = (next + 1) % kCache;
    if (used < kCache) ++used;
    return true;
}

// Rank-3 map of a contiguous bf16 or float32 tensor [depth][rows][inner] with
// box {128 bytes, box_rows, 1} and the 128-byte swizzle, for loads (elements
// out of range read as zero) and stores (they are not written).  Encoded anew
// for each call: nothing is kept.
inline bool make_tile_map(CUtensorMap* m, bool f32, const void* base, uint64_t inner, uint64_t rows, uint64_t depth,
                          uint32_t box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const uint64_t es = f32 ? 4 : 2;
    cuuint64_t dims[3] = {inner, rows, depth};
    cuuint64_t strides[2] = {inner * es, inner * rows * es};
    cuuint32_t box[3] = {(cuuint32_t)(128 / es), box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rank-3 map of a byte tensor [depth][rows][inner] (inner contiguous, a
// multiple of 16 bytes) with box {box_inner, box_rows, 1}; box_inner = 128
// takes the 128-byte swizzle (16-byte chunk c of box row r at c ^ (r % 8)),
// other widths none (rows box_inner bytes apart).  Out-of-range bytes of a
// box read as zero.  Cached like make_map_bf16.
inline bool make_map_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t depth,
                        uint32_t box_inner, uint32_t box_rows) {
    struct Entry {
        const void* base;
        uint64_t inner, rows, depth;
        uint32_t box_inner, box_rows;
        CUtensorMap map;
    };
    constexpr int kCache = 32;
    static Entry cache[kCache];
    static int used = 0, next = 0;
    static std::mutex mu;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (int i = 0; i < used; ++i) {
            const Entry& c = cache[i];
            if (c.base == base && c.inner == inner && c.rows == rows && c.depth == depth &&
                c.box_inner == box_inner && c.box_rows == box_rows) {
                *m = c.map;
                return true;
            }
        }
    }
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {inner, rows, depth};
    cuuint64_t strides[2] = {inner, inner * rows};
    cuuint32_t box[3] = {box_inner, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, box_inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    std::lock_guard<std::mutex> lock(mu);
    Entry& c = cache[next];
    c = Entry{base, inner, rows, depth, box_inner, box_rows, *m};
    next = (next + 1) % kCache;
    if (used < kCache) ++used;
    return true;
}

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per kernel (by
// address), device and size.  One entry per kernel, however many devices use it:
// the norm kernels alone are 56 of one type, and share this table.
template <typename Kernel>
inline cudaError_t ensure_smem_attr(Kernel kernel, size_t bytes) {
    struct Done {
        const void* fn;
        size_t bytes;   // the most asked for
        uint64_t devs;  // devices (below 64) that have it
    };
    constexpr int kKernels = 64;
    static Done done[kKernels];
    static int n = 0;
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    const void* fn = reinterpret_cast<const void*>(kernel);
    std::lock_guard<std::mutex> lock(mu);
    int i = 0;
    while (i < n && done[i].fn != fn) ++i;
    const bool known = i < n;
    if (known && done[i].bytes >= bytes) {
        if (done[i].devs & bit) return cudaSuccess;
        bytes = done[i].bytes;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    if (!known) {
        if (n == kKernels) return e;
        done[n++] = Done{fn, bytes, 0};
    } else if (bytes > done[i].bytes) {
        done[i] = Done{fn, bytes, 0};
    }
    done[i].devs |= bit;
    return e;
}

// Launches a kernel whose set-up may overlap the end of the kernel before it
// on the stream (programmatic stream serialization; the kernel calls
// chain_wait).  cluster = 0: no cluster attribute (none, or the kernel's own).
template <typename... P, typename... A>
inline cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster,
                                  cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster > 0) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
    return e == cudaSuccess ? e : cudaGetLastError();  // read, so that it is not left to the next caller
}

inline int device_sm_count() {
    static int count[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    if (!count[dev]) cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev);
    return count[dev] > 0 ? count[dev] : 148;
}

}  // namespace moe
