// Root-mean-square norm of feature rows with the residual's addition, in the row's
// type or in 8 bits with a scale per row, and its gradient.
//
//   h = x + residual             y = h * rstd * weight,  rstd = (mean(h^2) + eps)^(-1/2)
//   8 bits: s = max(max |y| / 448, 2^-126), q = e4m3(y / s)
//   gradient, with xh = h * rstd and g = dy * weight:
//     dx = rstd * (g - xh * mean(g * xh)) (+ dsum),   dweight = sum over rows of dy * xh
//
// Everything between the loads and the one rounding of each stored value is fp32.
#include <cuda_fp8.h>

#include "row_ops.cuh"

namespace spconv {
namespace {

constexpr int kNormThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: 1 / s stays finite

struct Sum {
    __device__ static float id() { return 0.0f; }
    __device__ static float f(float a, float b) { return a + b; }
};
struct MaxNan {
    __device__ static float id() { return 0.0f; }
    __device__ static float f(float a, float b) { return max_nan(a, b); }
};

template <typename Op>
__device__ float block_reduce(float v) {
    __shared__ float part[kNormThreads / 32];
    for (int d = 16; d > 0; d >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = Op::id();
    for (int w = 0; w < kNormThreads / 32; ++w) v = Op::f(v, part[w]);
    return v;
}

// One CTA a row.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    k_rms_norm(const T* __restrict__ x, const T* res, const T* __restrict__ weight, int c, float eps, T* sum_out,
               T* __restrict__ out, float* __restrict__ rstd_out, uint8_t* __restrict__ q, float* __restrict__ scale) {
    const int64_t base = (int64_t)blockIdx.x * c;
    const T* r = res ? res + base : nullptr;
    float ss = 0.0f;
    for (int j = threadIdx.x; j < c; j += kNormThreads) {
        const float h = to_f32(x[base + j]) + (r ? to_f32(r[j]) : 0.0f);
        ss += h * h;
    }
    const float rstd = rsqrtf(block_reduce<Sum>(ss) / (float)c + eps);
    float s = 1.0f;
    if (q) {
        float m = 0.0f;
        for (int j = threadIdx.x; j < c; j += kNormThreads) {
            const float h = to_f32(x[base + j]) + (r ? to_f32(r[j]) : 0.0f);
            m = max_nan(m, fabsf(h * rstd * (weight ? to_f32(weight[j]) : 1.0f)));
        }
        s = max_nan(block_reduce<MaxNan>(m) / kE4m3Max, kMinScale);
    }
    for (int j = threadIdx.x; j < c; j += kNormThreads) {
        const float h = to_f32(x[base + j]) + (r ? to_f32(r[j]) : 0.0f);
        const float y = h * rstd * (weight ? to_f32(weight[j]) : 1.0f);
        if (q)
            q[base + j] = __nv_cvt_float_to_fp8(y / s, __NV_SATFINITE, __NV_E4M3);
        else
            out[base + j] = from_f32<T>(y);
        if (sum_out) sum_out[base + j] = from_f32<T>(h);
    }
    if (threadIdx.x == 0) {
        if (rstd_out) rstd_out[blockIdx.x] = rstd;
        if (q) scale[blockIdx.x] = s;
    }
}

// One CTA a row: dx.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    k_rms_norm_dx(const T* __restrict__ dy, const T* __restrict__ h, const T* __restrict__ weight,
                  const float* __restrict__ rstd_in, const T* dsum, int c, T* dx) {
    const int64_t base = (int64_t)blockIdx.x * c;
    const float rstd = rstd_in[blockIdx.x];
    float dot = 0.0f;
    for (int j = threadIdx.x; j < c; j += kNormThreads)
        dot += to_f32(dy[base + j]) * (weight ? to_f32(weight[j]) : 1.0f) * to_f32(h[base + j]) * rstd;
    const float mean = block_reduce<Sum>(dot) / (float)c;
    for (int j = threadIdx.x; j < c; j += kNormThreads) {
        const float g = to_f32(dy[base + j]) * (weight ? to_f32(weight[j]) : 1.0f);
        float d = rstd * (g - to_f32(h[base + j]) * rstd * mean);
        if (dsum) d += to_f32(dsum[base + j]);
        dx[base + j] = from_f32<T>(d);
    }
}

constexpr int kMaxParts = 512;
inline int weight_parts(int64_t n) { return (int)(n < kMaxParts ? n : kMaxParts); }

// part[p][j] = sum of dy * h * rstd over the rows p, p + parts, ...
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    k_rms_norm_dw_part(const T* __restrict__ dy, const T* __restrict__ h, const float* __restrict__ rstd, int64_t n,
                       int c, float* __restrict__ part) {
    for (int j = threadIdx.x; j < c; j += kNormThreads) {
        float s = 0.0f;
        for (int64_t i = blockIdx.x; i < n; i += gridDim.x) s += to_f32(dy[i * c + j]) * to_f32(h[i * c + j]) * rstd[i];
        part[(int64_t)blockIdx.x * c + j] = s;
    }
}
__global__ void k_rms_norm_dw(const float* __restrict__ part, int parts, int c, float* __restrict__ dweight) {
    const int j = blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= c) return;
    float s = 0.0f;
    for (int p = 0; p < parts; ++p) s += part[(int64_t)p * c + j];
    dweight[j] = s;
}

spconv_status_t norm_args(spconv_dtype_t dtype, const void* x, const void* residual, const void* weight, int64_t n,
                          int32_t channels, float eps, const void* sum_out) {
    if (!dtype_ok(dtype)) return row_fail(SPCONV_ERR_INVALID_ARG, "dtype must be F32 or BF16");
    if (n < 0 || n >= (int64_t(1) << 31)) return row_fail(SPCONV_ERR_INVALID_ARG, "n must be in [0, 2^31)");
    if (channels < 1 || channels > SPCONV_NORM_MAX_CHANNELS)
        return row_fail(SPCONV_ERR_INVALID_ARG, "channels must be in [1, 65536]");
    if (!(eps >= 0.0f) || eps > 3.0e38f) return row_fail(SPCONV_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (n == 0) return SPCONV_OK;
    if (!x || !is_aligned(x, 16) || !is_aligned(residual, 16) || !is_aligned(weight, 16) || !is_aligned(sum_out, 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "feature pointers must be 16-byte aligned device pointers");
    if (sum_out && !residual) return row_fail(SPCONV_ERR_INVALID_ARG, "sum_out needs a residual");
    const int64_t bytes = n * channels * dtype_bytes(dtype);
    if ((sum_out != x && overlaps(sum_out, bytes, x, bytes)) ||
        (sum_out != residual && overlaps(sum_out, bytes, residual, bytes)) ||
        overlaps(sum_out, bytes, weight, (int64_t)channels * dtype_bytes(dtype)))
        return row_fail(SPCONV_ERR_INVALID_ARG, "sum_out may be x or residual itself and must not overlap them otherwise");
    return SPCONV_OK;
}

bool hits_inputs(const void* p, int64_t pbytes, const void* x, const void* residual, const void* weight,
                 const void* sum_out, int64_t bytes, int64_t wbytes) {
    return overlaps(p, pbytes, x, bytes) || overlaps(p, pbytes, residual, bytes) ||
           overlaps(p, pbytes, weight, wbytes) || overlaps(p, pbytes, sum_out, bytes);
}

template <typename T>
void launch_norm(const void* x, const void* residual, const void* weight, int64_t n, int c, float eps, void* sum_out,
                 void* out, float* rstd, uint8_t* q, float* scale, cudaStream_t st) {
    k_rms_norm<T><<<(unsigned)n, kNormThreads, 0, st>>>(
        static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<const T*>(weight), c, eps,
        static_cast<T*>(sum_out), static_cast<T*>(out), rstd, q, scale);
}

template <typename T>
void launch_norm_backward(const void* dy, const void* h, const void* weight, const float* rstd, const void* dsum,
                          int64_t n, int c, void* dx, float* dweight, float* ws, cudaStream_t st) {
    k_rms_norm_dx<T><<<(unsigned)n, kNormThreads, 0, st>>>(static_cast<const T*>(dy), static_cast<const T*>(h),
                                                           static_cast<const T*>(weight), rstd,
                                                           static_cast<const T*>(dsum), c, static_cast<T*>(dx));
    if (!dweight) return;
    const int parts = weight_parts(n);
    k_rms_norm_dw_part<T><<<parts, kNormThreads, 0, st>>>(static_cast<const T*>(dy), static_cast<const T*>(h), rstd, n,
                                                          c, ws);
    k_rms_norm_dw<<<(c + 255) / 256, 256, 0, st>>>(ws, parts, c, dweight);
}

}  // namespace
}  // namespace spconv

using namespace spconv;

extern "C" {

spconv_status_t spconv_rms_norm(spconv_dtype_t dtype, const void* x, const void* residual, const void* weight,
                                int64_t n, int32_t channels, float eps, void* sum_out, void* out, float* rstd,
                                void* stream) {
    spconv_status_t s = norm_args(dtype, x, residual, weight, n, channels, eps, sum_out);
    if (s != SPCONV_OK || n == 0) return s;
    if (!out || !is_aligned(out, 16) || !is_aligned(rstd, 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "out and rstd must be 16-byte aligned device pointers");
    const int64_t wbytes = (int64_t)channels * dtype_bytes(dtype), bytes = n * wbytes;
    if (hits_inputs(out, bytes, x, residual, weight, sum_out, bytes, wbytes) ||
        hits_inputs(rstd, n * 4, x, residual, weight, sum_out, bytes, wbytes) || overlaps(out, bytes, rstd, n * 4))
        return row_fail(SPCONV_ERR_INVALID_ARG, "out and rstd must not overlap another buffer of the call");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == SPCONV_BF16)
        launch_norm<__nv_bfloat16>(x, residual, weight, n, channels, eps, sum_out, out, rstd, nullptr, nullptr, st);
    else
        launch_norm<float>(x, residual, weight, n, channels, eps, sum_out, out, rstd, nullptr, nullptr, st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_rms_norm");
}

spconv_status_t spconv_rms_norm_q8(spconv_dtype_t dtype, const void* x, const void* residual, const void* weight,
                                   int64_t n, int32_t channels, float eps, void* sum_out, uint8_t* q, float* scale,
                                   void* stream) {
    spconv_status_t s = norm_args(dtype, x, residual, weight, n, channels, eps, sum_out);
    if (s != SPCONV_OK || n == 0) return s;
    if (!q || !scale || !is_aligned(q, 16) || !is_aligned(scale, 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "q and scale must be 16-byte aligned device pointers");
    const int64_t wbytes = (int64_t)channels * dtype_bytes(dtype), bytes = n * wbytes;
    if (hits_inputs(q, n * channels, x, residual, weight, sum_out, bytes, wbytes) ||
        hits_inputs(scale, n * 4, x, residual, weight, sum_out, bytes, wbytes) ||
        overlaps(q, n * channels, scale, n * 4))
        return row_fail(SPCONV_ERR_INVALID_ARG, "q and scale must not overlap another buffer of the call");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == SPCONV_BF16)
        launch_norm<__nv_bfloat16>(x, residual, weight, n, channels, eps, sum_out, nullptr, nullptr, q, scale, st);
    else
        launch_norm<float>(x, residual, weight, n, channels, eps, sum_out, nullptr, nullptr, q, scale, st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_rms_norm_q8");
}

spconv_status_t spconv_rms_norm_workspace(int64_t n, int32_t channels, int64_t* bytes) {
    if (!bytes) return row_fail(SPCONV_ERR_INVALID_ARG, "null bytes");
    if (n < 0 || n >= (int64_t(1) << 31)) return row_fail(SPCONV_ERR_INVALID_ARG, "n must be in [0, 2^31)");
    if (channels < 1 || channels > SPCONV_NORM_MAX_CHANNELS)
        return row_fail(SPCONV_ERR_INVALID_ARG, "channels must be in [1, 65536]");
    *bytes = (int64_t)weight_parts(n) * channels * 4;
    return SPCONV_OK;
}

spconv_status_t spconv_rms_norm_backward(spconv_dtype_t dtype, const void* dy, const void* h, const void* weight,
                                         const float* rstd, const void* dsum, int64_t n, int32_t channels, void* dx,
                                         float* dweight, void* workspace, void* stream) {
    spconv_status_t s = norm_args(dtype, h, nullptr, weight, n, channels, 0.0f, nullptr);
    if (s != SPCONV_OK) return s;
    if (dweight && !is_aligned(dweight, 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "dweight must be a 16-byte aligned device pointer");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n == 0) {
        const cudaError_t e = dweight ? cudaMemsetAsync(dweight, 0, (size_t)channels * 4, st) : cudaSuccess;
        return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_rms_norm_backward");
    }
    if (!dy || !rstd || !dx || !is_aligned(dy, 16) || !is_aligned(rstd, 16) || !is_aligned(dx, 16) ||
        !is_aligned(dsum, 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "dy, rstd, dsum and dx must be 16-byte aligned device pointers");
    if (dweight && (!workspace || !is_aligned(workspace, 16)))
        return row_fail(SPCONV_ERR_INVALID_ARG, "dweight needs a 16-byte aligned workspace");
    const int64_t wbytes = (int64_t)channels * dtype_bytes(dtype), bytes = n * wbytes;
    const int64_t wsbytes = (int64_t)weight_parts(n) * channels * 4, dwbytes = (int64_t)channels * 4;
    const void* ws = dweight ? workspace : nullptr;
    bool bad = dx != dsum && overlaps(dx, bytes, dsum, bytes);
    bad = bad || overlaps(dx, bytes, dy, bytes) || overlaps(dx, bytes, h, bytes) || overlaps(dx, bytes, weight, wbytes) ||
          overlaps(dx, bytes, rstd, n * 4) || overlaps(dx, bytes, dweight, dwbytes) || overlaps(dx, bytes, ws, wsbytes) ||
          overlaps(dweight, dwbytes, ws, wsbytes);
    const void* ins[5] = {dy, h, dsum, weight, rstd};
    const int64_t sizes[5] = {bytes, bytes, bytes, wbytes, n * 4};
    for (int i = 0; i < 5; ++i)
        bad = bad || overlaps(dweight, dwbytes, ins[i], sizes[i]) || overlaps(ws, wsbytes, ins[i], sizes[i]);
    if (bad)
        return row_fail(SPCONV_ERR_INVALID_ARG,
                        "dx may be dsum itself; dx, dweight and workspace must not overlap another buffer of the call");
    if (dtype == SPCONV_BF16)
        launch_norm_backward<__nv_bfloat16>(dy, h, weight, rstd, dsum, n, channels, dx, dweight,
                                            static_cast<float*>(workspace), st);
    else
        launch_norm_backward<float>(dy, h, weight, rstd, dsum, n, channels, dx, dweight, static_cast<float*>(workspace),
                                    st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_rms_norm_backward");
}

}  // extern "C"
