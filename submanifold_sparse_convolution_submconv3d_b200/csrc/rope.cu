// Rotary positions of feature rows from voxel coordinates, with several axes.
//
// Pair j of every head of a voxel turns by the angle freq[j] * coord[axis[j]]:
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),
// the gradient is the turn by -t.  The angle is kept in turns, as a 64-bit fixed
// point fraction: F = freq / (2 pi) mod 1, scaled by 2^64, and F * coord modulo
// 2^64 is the exact fraction of a turn for any 32-bit coordinate (the error is that
// of F, 2^-65 times the coordinate), where an fp32 product would be off by 2^-24 of
// the whole angle: 4e-3 rad at coordinate 65535.
#include <math.h>

#include <new>

#include "row_ops.cuh"

namespace spconv {
namespace {

constexpr int kMaxPairs = SPCONV_ROPE_MAX_HEAD_DIM / 2;

struct RopeTable {
    uint64_t turn[kMaxPairs];  // F of each pair
    int8_t axis[kMaxPairs];    // 0, 1, 2, or -1: the pair does not turn
};

struct RopeArgs {
    const int4* coords;
    int64_t n, x_row, x_head, o_row, o_head;
    int heads, pairs;
    bool halves, inverse;
};

// One thread a pair.
template <typename T>
__global__ void __launch_bounds__(256) k_rope(const __grid_constant__ RopeTable tab, RopeArgs a, const T* x, T* out) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (id >= a.n * a.heads * a.pairs) return;
    const int j = (int)(id % a.pairs);
    const int head = (int)(id / a.pairs % a.heads);
    const int64_t i = id / a.pairs / a.heads;
    const int4 p = a.coords[i];
    const int axis = tab.axis[j];
    const int64_t pos = axis == 0 ? p.y : axis == 1 ? p.z : axis == 2 ? p.w : 0;
    const int32_t frac = (int32_t)((tab.turn[j] * (uint64_t)pos) >> 32);
    float sn, cs;
    sincospif((float)frac * 0x1p-31f, &sn, &cs);
    if (a.inverse) sn = -sn;
    const int lo = a.halves ? j : 2 * j, hi = a.halves ? j + a.pairs : 2 * j + 1;
    const T* xi = x + i * a.x_row + head * a.x_head;
    T* oi = out + i * a.o_row + head * a.o_head;
    const float u = to_f32(xi[lo]), v = to_f32(xi[hi]);
    oi[lo] = from_f32<T>(u * cs - v * sn);
    oi[hi] = from_f32<T>(u * sn + v * cs);
}

}  // namespace
}  // namespace spconv

struct spconv_rope_s {
    int32_t head_dim = 0;
    spconv_rope_layout_t layout = SPCONV_ROPE_INTERLEAVED;
    spconv::RopeTable table = {};
};

using namespace spconv;

extern "C" {

spconv_status_t spconv_rope_create(int32_t head_dim, spconv_rope_layout_t layout, double base, const double* freqs,
                                   const int32_t* axes, spconv_rope_t* out) {
    if (!out) return row_fail(SPCONV_ERR_INVALID_ARG, "null out");
    if (head_dim < 2 || head_dim > SPCONV_ROPE_MAX_HEAD_DIM || head_dim % 2)
        return row_fail(SPCONV_ERR_INVALID_ARG, "head_dim must be even and in [2, 256]");
    if (layout != SPCONV_ROPE_INTERLEAVED && layout != SPCONV_ROPE_HALVES)
        return row_fail(SPCONV_ERR_INVALID_ARG, "layout must be INTERLEAVED or HALVES");
    if ((freqs == nullptr) != (axes == nullptr))
        return row_fail(SPCONV_ERR_INVALID_ARG, "freqs and axes are given together or not at all");
    if (!freqs && !(base > 0.0 && base < 1e300))
        return row_fail(SPCONV_ERR_INVALID_ARG, "base must be positive and finite");
    const int pairs = head_dim / 2, per = pairs / 3;
    if (freqs)
        for (int j = 0; j < pairs; ++j)
            if (!(fabs(freqs[j]) < 1e300) || axes[j] < -1 || axes[j] > 2)
                return row_fail(SPCONV_ERR_INVALID_ARG, "freqs must be finite and axes in [-1, 2]");
    spconv_rope_s* r = new (std::nothrow) spconv_rope_s();
    if (!r) return row_fail(SPCONV_ERR_OOM, "host allocation failed");
    r->head_dim = head_dim;
    r->layout = layout;
    const long double two_pi = 6.283185307179586476925286766559005768L;
    for (int j = 0; j < pairs; ++j) {
        const int axis = freqs ? axes[j] : j < 3 * per ? j / per : -1;
        const double f = axis < 0 ? 0.0 : freqs ? freqs[j] : pow(base, -(double)(j % per) / per);
        long double t = (long double)f / two_pi;
        t = (t - floorl(t)) * 0x1p64L;
        r->table.turn[j] = t >= 0x1p64L ? 0 : (uint64_t)t;
        r->table.axis[j] = (int8_t)axis;
    }
    *out = r;
    return SPCONV_OK;
}

spconv_status_t spconv_rope_free(spconv_rope_t rope) {
    delete rope;
    return SPCONV_OK;
}

spconv_status_t spconv_rope_apply(spconv_rope_t rope, spconv_dtype_t dtype, const int32_t* coords, int64_t n,
                                  const void* x, int32_t heads, int64_t x_row, int64_t x_head, void* out,
                                  int64_t out_row, int64_t out_head, int32_t inverse, void* stream) {
    if (!rope) return row_fail(SPCONV_ERR_INVALID_ARG, "null handle");
    if (!dtype_ok(dtype)) return row_fail(SPCONV_ERR_INVALID_ARG, "dtype must be F32 or BF16");
    if (n < 0 || n >= (int64_t(1) << 31)) return row_fail(SPCONV_ERR_INVALID_ARG, "n must be in [0, 2^31)");
    if (heads < 1 || heads > 65535) return row_fail(SPCONV_ERR_INVALID_ARG, "heads must be in [1, 65535]");
    const int64_t d = rope->head_dim, limit = int64_t(1) << 40;
    // heads and rows of one tensor must not share elements; either may be the outer one
    // (a stride over one element is not used, and taken as head_dim here)
    if (n <= 1) x_row = out_row = d;
    if (heads == 1) x_head = out_head = d;
    if (x_row < d || out_row < d || x_head < d || out_head < d || x_row > limit || out_row > limit || x_head > limit ||
        out_head > limit)
        return row_fail(SPCONV_ERR_INVALID_ARG, "row and head strides must be in [head_dim, 2^40]");
    const int64_t o_in = out_head * (heads - 1) + d, o_rows = out_row * (n > 0 ? n - 1 : 0) + d;
    if (heads > 1 && n > 1 && out_row < o_in && out_head < o_rows)
        return row_fail(SPCONV_ERR_INVALID_ARG, "the strides of out make its rows and heads share elements");
    if (n == 0) return SPCONV_OK;
    if (!coords || !is_aligned(coords, 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "coords must be a 16-byte aligned device pointer");
    const int es = dtype_bytes(dtype);
    if (!x || !out || !is_aligned(x, es) || !is_aligned(out, es))
        return row_fail(SPCONV_ERR_INVALID_ARG, "x and out must be device pointers aligned to the element");
    if (n * (int64_t)heads > (int64_t(1) << 50) / d) return row_fail(SPCONV_ERR_INVALID_ARG, "too many elements");
    const bool same = x == out && x_row == out_row && x_head == out_head;
    const int64_t xspan = (x_row * (n - 1) + x_head * (heads - 1) + d) * es;
    const int64_t ospan = (out_row * (n - 1) + out_head * (heads - 1) + d) * es;
    if ((!same && overlaps(out, ospan, x, xspan)) || overlaps(out, ospan, coords, n * 16))
        return row_fail(SPCONV_ERR_INVALID_ARG, "out may be x itself with x's strides and must not overlap it otherwise");
    RopeArgs a = {reinterpret_cast<const int4*>(coords), n, x_row, x_head, out_row, out_head, heads, (int)(d / 2),
                  rope->layout == SPCONV_ROPE_HALVES, inverse != 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t blocks = (n * heads * a.pairs + 255) / 256;
    if (blocks > 0x7fffffff) return row_fail(SPCONV_ERR_UNSUPPORTED, "too many elements for one launch");
    if (dtype == SPCONV_BF16)
        k_rope<__nv_bfloat16><<<(unsigned)blocks, 256, 0, st>>>(rope->table, a, static_cast<const __nv_bfloat16*>(x),
                                                                static_cast<__nv_bfloat16*>(out));
    else
        k_rope<float><<<(unsigned)blocks, 256, 0, st>>>(rope->table, a, static_cast<const float*>(x),
                                                        static_cast<float*>(out));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_rope_apply");
}

}  // extern "C"
