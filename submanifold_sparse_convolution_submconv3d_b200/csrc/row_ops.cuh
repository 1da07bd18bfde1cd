// Shared by the operators on feature rows (RMS norm, rotary positions, the 4-bit
// linear layer): host-side argument checks and element access in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "common.cuh"

namespace spconv {

inline spconv_status_t row_fail(spconv_status_t s, const char* msg) noexcept {
    try {
        set_last_error(msg);
    } catch (...) {  // no memory for the message: the status still tells
    }
    return s;
}

inline spconv_status_t row_fail_cuda(cudaError_t e, const char* where) noexcept {
    try {
        set_last_error(std::string(where) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
    } catch (...) {
    }
    return e == cudaErrorMemoryAllocation ? SPCONV_ERR_OOM : SPCONV_ERR_CUDA;
}

inline bool is_aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// A null pointer overlaps nothing.
inline bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    if (!a || !b) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)bbytes && y < x + (uintptr_t)abytes;
}

inline bool dtype_ok(spconv_dtype_t t) { return t == SPCONV_F32 || t == SPCONV_BF16; }
inline int dtype_bytes(spconv_dtype_t t) { return t == SPCONV_BF16 ? 2 : 4; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// max that keeps a NaN of either side (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

}  // namespace spconv
