// The per-voxel linear layer (kernel size 1) on 4-bit weights with group scales,
// for few rows: single tokens, modulation vectors, small latent sets.
//
//   w[k, o] = scales[o, g] * q[o, k] + offsets[o, g],  g = k / group,  q in 0 .. 15
//   out[i, o] = bias[o] + x_scale[i] * sum_k w[k, o] x[i, k]
//
// The sums are kept in fp32 and rounded once.
#include <cuda_fp8.h>

#include "row_ops.cuh"

namespace spconv {
namespace {

__device__ __forceinline__ float e4m3_to_f32(uint8_t v) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}
__device__ __forceinline__ float w4_x(const float* x, int64_t i) { return x[i]; }
__device__ __forceinline__ float w4_x(const __nv_bfloat16* x, int64_t i) { return __bfloat162float(x[i]); }
__device__ __forceinline__ float w4_x(const uint8_t* x, int64_t i) { return e4m3_to_f32(x[i]); }

// One warp an output element; a lane takes every 32nd word of 8 weights.
template <typename T, typename X>
__global__ void __launch_bounds__(256)
    k_linear_w4(const X* __restrict__ x, const float* __restrict__ x_scale, int cin, const uint32_t* __restrict__ packed,
                const T* __restrict__ scales, const T* __restrict__ offsets, int group, const T* __restrict__ bias,
                T* __restrict__ out, int cout) {
    const int o = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int64_t i = blockIdx.y;
    if (o >= cout) return;
    const int words = cin / 8, groups = cin / group;
    float s = 0.0f;
    for (int w = lane; w < words; w += 32) {
        const uint32_t v = packed[(int64_t)o * words + w];
        const int64_t g = (int64_t)o * groups + w * 8 / group;
        const float sc = to_f32(scales[g]), of = to_f32(offsets[g]);
        for (int e = 0; e < 8; ++e) s += (sc * (float)((v >> (4 * e)) & 15u) + of) * w4_x(x, i * cin + 8 * w + e);
    }
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) {
        if (x_scale) s *= x_scale[i];
        if (bias) s += to_f32(bias[o]);
        out[i * cout + o] = from_f32<T>(s);
    }
}

// One thread a (group, output): the output index runs fastest, so the reads of w
// are coalesced.  Runs once per weight matrix.
template <typename T>
__global__ void __launch_bounds__(256)
    k_w4_quantize(const T* __restrict__ w, int cin, int cout, int group, uint32_t* __restrict__ packed,
                  T* __restrict__ scales, T* __restrict__ offsets) {
    const int o = blockIdx.x * 256 + threadIdx.x, g = blockIdx.y;
    if (o >= cout) return;
    const int64_t k0 = (int64_t)g * group;
    float lo = to_f32(w[k0 * cout + o]), hi = lo;
    for (int k = 1; k < group; ++k) {
        const float v = to_f32(w[(k0 + k) * cout + o]);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    // the codes are taken against the scale and offset as they are stored
    const T st = from_f32<T>((hi - lo) / 15.0f), zt = from_f32<T>(lo);
    const float s = to_f32(st), z = to_f32(zt);
    const int64_t at = (int64_t)o * (cin / group) + g;
    scales[at] = st;
    offsets[at] = zt;
    for (int m = 0; m < group / 8; ++m) {
        uint32_t v = 0;
        for (int e = 0; e < 8; ++e) {
            const float c = s > 0.0f ? rintf((to_f32(w[(k0 + 8 * m + e) * cout + o]) - z) / s) : 0.0f;
            v |= (uint32_t)fminf(fmaxf(c, 0.0f), 15.0f) << (4 * e);
        }
        packed[(int64_t)o * (cin / 8) + k0 / 8 + m] = v;
    }
}

// A block unpacks 32 outputs x 32 words: the words are read along the input
// channels, the weights written along the output channels.
template <typename T>
__global__ void __launch_bounds__(256)
    k_w4_dequantize(const uint32_t* __restrict__ packed, const T* __restrict__ scales, const T* __restrict__ offsets,
                    int cin, int cout, int group, T* __restrict__ w) {
    __shared__ uint32_t tile[32][33];
    const int words = cin / 8, groups = cin / group;
    const int w0 = blockIdx.x * 32, o0 = blockIdx.y * 32;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    for (int r = ty; r < 32; r += 8)
        if (o0 + r < cout && w0 + tx < words) tile[r][tx] = packed[(int64_t)(o0 + r) * words + w0 + tx];
    __syncthreads();
    const int o = o0 + tx;
    if (o >= cout) return;
    for (int m = ty; m < 32 && w0 + m < words; m += 8) {
        const uint32_t v = tile[tx][m];
        const int64_t k0 = 8 * (int64_t)(w0 + m), g = (int64_t)o * groups + k0 / group;
        const float s = to_f32(scales[g]), z = to_f32(offsets[g]);
        for (int e = 0; e < 8; ++e) w[(k0 + e) * cout + o] = from_f32<T>(fmaf(s, (float)((v >> (4 * e)) & 15u), z));
    }
}

spconv_status_t w4_args(spconv_dtype_t dtype, const void* packed, const void* scales, const void* offsets, int32_t cin,
                        int32_t cout, int32_t group) {
    if (!dtype_ok(dtype)) return row_fail(SPCONV_ERR_INVALID_ARG, "dtype must be F32 or BF16");
    if (group != 32 && group != 64 && group != 128)
        return row_fail(SPCONV_ERR_INVALID_ARG, "group must be 32, 64 or 128");
    if (cin < group || cin % group || cin > (1 << 20))
        return row_fail(SPCONV_ERR_INVALID_ARG, "cin must be a multiple of group, at most 2^20");
    if (cout < 1 || cout > (1 << 20)) return row_fail(SPCONV_ERR_INVALID_ARG, "cout must be in [1, 2^20]");
    if (!packed || !scales || !offsets || !is_aligned(packed, 16) || !is_aligned(scales, 16) || !is_aligned(offsets, 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "packed, scales and offsets must be 16-byte aligned device pointers");
    return SPCONV_OK;
}

template <typename T, typename X>
void launch_linear_w4(const void* x, const float* x_scale, int64_t n, int cin, const void* packed, const void* scales,
                      const void* offsets, int group, const void* bias, void* out, int cout, cudaStream_t st) {
    k_linear_w4<T, X><<<dim3((cout + 7) / 8, (unsigned)n), 256, 0, st>>>(
        static_cast<const X*>(x), x_scale, cin, static_cast<const uint32_t*>(packed), static_cast<const T*>(scales),
        static_cast<const T*>(offsets), group, static_cast<const T*>(bias), static_cast<T*>(out), cout);
}

}  // namespace
}  // namespace spconv

using namespace spconv;

extern "C" {

spconv_status_t spconv_w4_quantize(spconv_dtype_t dtype, const void* w, int32_t cin, int32_t cout, int32_t group,
                                   uint32_t* packed, void* scales, void* offsets, void* stream) {
    spconv_status_t s = w4_args(dtype, packed, scales, offsets, cin, cout, group);
    if (s != SPCONV_OK) return s;
    if (!w || !is_aligned(w, 16)) return row_fail(SPCONV_ERR_INVALID_ARG, "w must be a 16-byte aligned device pointer");
    const int es = dtype_bytes(dtype);
    const int64_t wb = (int64_t)cin * cout * es, pb = (int64_t)cin * cout / 2, gb = (int64_t)cin / group * cout * es;
    if (overlaps(packed, pb, w, wb) || overlaps(scales, gb, w, wb) || overlaps(offsets, gb, w, wb) ||
        overlaps(packed, pb, scales, gb) || overlaps(packed, pb, offsets, gb) || overlaps(scales, gb, offsets, gb))
        return row_fail(SPCONV_ERR_INVALID_ARG, "the buffers of the call must not overlap");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid((cout + 255) / 256, cin / group);
    if (dtype == SPCONV_BF16)
        k_w4_quantize<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(w), cin, cout, group, packed,
                                                           static_cast<__nv_bfloat16*>(scales),
                                                           static_cast<__nv_bfloat16*>(offsets));
    else
        k_w4_quantize<float><<<grid, 256, 0, st>>>(static_cast<const float*>(w), cin, cout, group, packed,
                                                   static_cast<float*>(scales), static_cast<float*>(offsets));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_w4_quantize");
}

spconv_status_t spconv_w4_dequantize(spconv_dtype_t dtype, const uint32_t* packed, const void* scales,
                                     const void* offsets, int32_t cin, int32_t cout, int32_t group, void* w,
                                     void* stream) {
    spconv_status_t s = w4_args(dtype, packed, scales, offsets, cin, cout, group);
    if (s != SPCONV_OK) return s;
    if (!w || !is_aligned(w, 16)) return row_fail(SPCONV_ERR_INVALID_ARG, "w must be a 16-byte aligned device pointer");
    const int es = dtype_bytes(dtype);
    const int64_t wb = (int64_t)cin * cout * es, pb = (int64_t)cin * cout / 2, gb = (int64_t)cin / group * cout * es;
    if (overlaps(w, wb, packed, pb) || overlaps(w, wb, scales, gb) || overlaps(w, wb, offsets, gb))
        return row_fail(SPCONV_ERR_INVALID_ARG, "w must not overlap packed, scales or offsets");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid((cin / 8 + 31) / 32, (cout + 31) / 32);
    if (dtype == SPCONV_BF16)
        k_w4_dequantize<__nv_bfloat16><<<grid, 256, 0, st>>>(packed, static_cast<const __nv_bfloat16*>(scales),
                                                             static_cast<const __nv_bfloat16*>(offsets), cin, cout, group,
                                                             static_cast<__nv_bfloat16*>(w));
    else
        k_w4_dequantize<float><<<grid, 256, 0, st>>>(packed, static_cast<const float*>(scales),
                                                     static_cast<const float*>(offsets), cin, cout, group,
                                                     static_cast<float*>(w));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_w4_dequantize");
}

spconv_status_t spconv_linear_w4(spconv_dtype_t dtype, const void* x, const float* x_scale, int64_t n, int32_t cin,
                                 const uint32_t* packed, const void* scales, const void* offsets, int32_t group,
                                 const void* bias, void* out, int32_t cout, void* stream) {
    spconv_status_t s = w4_args(dtype, packed, scales, offsets, cin, cout, group);
    if (s != SPCONV_OK) return s;
    if (n < 0) return row_fail(SPCONV_ERR_INVALID_ARG, "n must be >= 0");
    if (n > SPCONV_W4_MAX_ROWS)
        return row_fail(SPCONV_ERR_UNSUPPORTED,
                        "at most 32 rows: unpack the weights (spconv_w4_dequantize) and run a map of kernel size 1");
    if (n == 0) return SPCONV_OK;
    if (!x || !out || !is_aligned(x, 16) || !is_aligned(out, 16) || !is_aligned(bias, 16) || !is_aligned(x_scale, 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "x, x_scale, bias and out must be 16-byte aligned device pointers");
    const int es = dtype_bytes(dtype);
    const int64_t ob = n * cout * es, pb = (int64_t)cin * cout / 2, gb = (int64_t)cin / group * cout * es;
    if (overlaps(out, ob, x, n * cin * (x_scale ? 1 : es)) || overlaps(out, ob, x_scale, n * 4) ||
        overlaps(out, ob, packed, pb) || overlaps(out, ob, scales, gb) || overlaps(out, ob, offsets, gb) ||
        overlaps(out, ob, bias, (int64_t)cout * es))
        return row_fail(SPCONV_ERR_INVALID_ARG, "out must not overlap another buffer of the call");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == SPCONV_BF16 && x_scale)
        launch_linear_w4<__nv_bfloat16, uint8_t>(x, x_scale, n, cin, packed, scales, offsets, group, bias, out, cout, st);
    else if (dtype == SPCONV_BF16)
        launch_linear_w4<__nv_bfloat16, __nv_bfloat16>(x, nullptr, n, cin, packed, scales, offsets, group, bias, out,
                                                       cout, st);
    else if (x_scale)
        launch_linear_w4<float, uint8_t>(x, x_scale, n, cin, packed, scales, offsets, group, bias, out, cout, st);
    else
        launch_linear_w4<float, float>(x, nullptr, n, cin, packed, scales, offsets, group, bias, out, cout, st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_linear_w4");
}

}  // extern "C"
