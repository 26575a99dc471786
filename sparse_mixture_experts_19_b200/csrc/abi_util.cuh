// Argument checks and error reporting shared by the files that implement the
// C ABI (moe_abi.cu, dense_abi.cu).
#pragma once

#include "common.cuh"

namespace moe {

// Records the calling thread's last error (moe_last_error) and returns st.
moe_status_t fail(moe_status_t st, const char* fmt, ...);
moe_status_t cuda_fail(cudaError_t e, const char* where);

inline bool aligned16(const void* ptr) { return ((uintptr_t)ptr & 15) == 0; }
inline size_t align_up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }

// The device check flags of a workspace (its first int32): waits for the
// stream, reads and clears them.
moe_status_t read_device_flags(int32_t* flags, cudaStream_t st, int32_t* flags_out);

}  // namespace moe

#define REQUIRE_PTR(ptr)                                                                    \
    do {                                                                                    \
        if (!(ptr)) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #ptr);                   \
        if (!aligned16(ptr)) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #ptr); \
    } while (0)

#define OPTIONAL_PTR(ptr)                                                                   \
    do {                                                                                    \
        if ((ptr) && !aligned16(ptr)) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #ptr); \
    } while (0)

#define CUDA_TRY(expr, where)                           \
    do {                                                \
        cudaError_t e_ = (expr);                        \
        if (e_ != cudaSuccess) return cuda_fail(e_, where); \
    } while (0)
