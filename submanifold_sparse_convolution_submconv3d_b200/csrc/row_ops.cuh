// Shared by the operators on feature rows (RMS norm, rotary positions, the 4-bit
// linear layer): host-side argument checks and element access in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
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

// The GPU this library is built for; the launches deal their work by it.
constexpr int kSms = 148;

// Lets a kernel have `bytes` of dynamic shared memory, once a device (the call costs a
// good part of a microsecond, a launch three).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (e == cudaSuccess && (dev > 63 || !(done.load(std::memory_order_acquire) & bit))) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    }
    return e;
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

// VE neighbouring elements, read and written with one access where they are aligned to
// their size, as single elements with a smaller ALIGN.
template <typename T, int VE, int ALIGN = (int)sizeof(T) * VE>
struct alignas(ALIGN) Vec {
    T v[VE];
};
template <typename V, typename T>
__device__ __forceinline__ V load_vec(const T* p) {
    return *reinterpret_cast<const V*>(p);
}
template <typename V, typename T>
__device__ __forceinline__ void store_vec(T* p, const V& v) {
    *reinterpret_cast<V*>(p) = v;
}

// The elements as fp32 and back, bf16 two at a time.
template <typename T, int VE, int A>
__device__ __forceinline__ void unpack(const Vec<T, VE, A>& v, float* f) {
    if constexpr (sizeof(T) == 2 && VE % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
            const uint32_t two = (uint32_t)__bfloat16_as_ushort(v.v[e]) | ((uint32_t)__bfloat16_as_ushort(v.v[e + 1]) << 16);
            f[e] = __uint_as_float(two << 16);
            f[e + 1] = __uint_as_float(two & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = to_f32(v.v[e]);
    }
}
template <typename T, int VE, int A>
__device__ __forceinline__ void pack(const float* f, Vec<T, VE, A>& v) {
    if constexpr (sizeof(T) == 2 && VE % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(f[e], f[e + 1]);
            v.v[e] = two.x;
            v.v[e + 1] = two.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) v.v[e] = from_f32<T>(f[e]);
    }
}

// 4, 8 or 16 bytes from global to shared memory, asynchronously; groups complete in order.
__device__ __forceinline__ uint32_t shared_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// 16 bytes, of which the first `bytes` are read and the others zero
__device__ __forceinline__ void copy_async_part(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// max that keeps a NaN of either side (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

}  // namespace spconv
