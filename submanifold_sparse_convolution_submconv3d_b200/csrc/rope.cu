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
    int chunks;         // items a head
    int voxels;         // voxels a unit
    int unit_heads;     // heads a unit (all of them where a unit has several voxels)
    int head_groups;    // units a voxel (1 where a unit has several voxels)
    int64_t units;
    uint32_t by_chunks, by_voxel, by_pairs;  // ceil(2^32 / d), for division by d
    float sign;         // -1: turn back
};

// id / d for id * d < 2^32, with m = ceil(2^32 / d) (d = 1 wraps to 0)
__device__ __forceinline__ int fast_div(int id, uint32_t m) { return m ? (int)__umulhi((uint32_t)id, m) : id; }

// An item's elements: one 16-byte access, or single elements at any address.
template <typename T, int VE>
struct alignas(sizeof(T) * VE == 16 ? 16 : sizeof(T)) Vec {
    T v[VE];
};

constexpr int kRopeWarps = 8;
constexpr int kRopeTable = 512;   // cosines and sines a unit may hold

// Items: VE neighbouring elements of a head (VE / 2 pairs) in the interleaved layout,
// VE elements of either half (VE pairs) in the halves layout.  A warp takes a unit of
// `voxels` voxels x `unit_heads` heads: it starts the loads of its first items, computes
// the unit's cosines and sines once, a pair a lane, into shared memory, and turns the
// items from there, so the sine's cost is shared by all heads of a voxel.
template <typename T, int VE, bool HALVES>
__global__ void __launch_bounds__(32 * kRopeWarps)
    k_rope(const __grid_constant__ RopeTable tab, const __grid_constant__ RopeArgs a, const T* x, T* out) {
    constexpr int kPairs = HALVES ? VE : VE / 2;  // pairs an item
    constexpr int kInFlight = HALVES ? 2 : 4;
    using V = Vec<T, VE>;
    __shared__ uint64_t turn[kMaxPairs];
    __shared__ int axis[kMaxPairs];
    __shared__ float2 table[kRopeWarps][kRopeTable];
    for (int j = threadIdx.x; j < a.pairs; j += blockDim.x) {
        turn[j] = tab.turn[j];
        axis[j] = tab.axis[j];
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2* cs = table[warp];
    for (int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp; unit < a.units; unit += (int64_t)gridDim.x * kRopeWarps) {
        const int64_t vb = a.head_groups == 1 ? unit : unit / a.head_groups;
        const int h0 = (int)(unit - vb * a.head_groups) * a.unit_heads;
        const int64_t i0 = vb * a.voxels;
        const int nv = (int)min((int64_t)a.voxels, a.n - i0), nh = min(a.unit_heads, a.heads - h0);
        const int items = nv * nh * a.chunks;
        for (int base = lane; base - lane < items; base += 32 * kInFlight) {
            V lo[kInFlight], hi[HALVES ? kInFlight : 1];
            int64_t at[kInFlight];
            int row[kInFlight];
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                const int id = base + 32 * k;
                if (id >= items) continue;
                const int b = a.voxels == 1 ? 0 : fast_div(id, a.by_voxel);
                const int r = id - b * a.heads * a.chunks;
                const int head = fast_div(r, a.by_chunks), chunk = r - head * a.chunks;
                const T* p = x + (i0 + b) * a.x_row + (h0 + head) * a.x_head + chunk * VE;
                lo[k] = *reinterpret_cast<const V*>(p);
                if (HALVES) hi[k] = *reinterpret_cast<const V*>(p + a.pairs);
                at[k] = (i0 + b) * a.o_row + (h0 + head) * a.o_head + chunk * VE;
                row[k] = b * a.pairs + chunk * kPairs;
            }
            if (base == lane) {
                __syncwarp();  // the last unit's readers are done
                for (int e = lane; e < nv * a.pairs; e += 32) {
                    const int b = a.voxels == 1 ? 0 : fast_div(e, a.by_pairs);
                    const int j = e - b * a.pairs;
                    const int ax = axis[j];
                    const int pos = ax < 0 ? 0 : reinterpret_cast<const int*>(a.coords + i0 + b)[1 + ax];
                    const int32_t frac = (int32_t)((turn[j] * (uint64_t)(int64_t)pos) >> 32);
                    float sn, cs_;
                    if (sizeof(T) == 2) {
                        // 2^-21.2 of error on [-pi, pi], against the 2^-9 of the result's rounding
                        const float ang = (float)frac * 1.46291807926715968e-9f;  // 2 pi / 2^32
                        sn = __sinf(ang);
                        cs_ = __cosf(ang);
                    } else {
                        sincospif((float)frac * 0x1p-31f, &sn, &cs_);
                    }
                    cs[e] = make_float2(cs_, sn * a.sign);
                }
                __syncwarp();
            }
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                if (base + 32 * k >= items) continue;
#pragma unroll
                for (int p = 0; p < kPairs; ++p) {
                    const float2 t = cs[row[k] + p];
                    T& ra = HALVES ? lo[k].v[p] : lo[k].v[2 * p];
                    T& rb = HALVES ? hi[HALVES ? k : 0].v[p] : lo[k].v[HALVES ? 0 : 2 * p + 1];
                    const float u = to_f32(ra), v = to_f32(rb);
                    ra = from_f32<T>(u * t.x - v * t.y);
                    rb = from_f32<T>(u * t.y + v * t.x);
                }
                *reinterpret_cast<V*>(out + at[k]) = lo[k];
                if (HALVES) *reinterpret_cast<V*>(out + at[k] + a.pairs) = hi[HALVES ? k : 0];
            }
        }
    }
}

int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 148;
    return sms;
}

uint32_t div_by(int d) { return d == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + d - 1) / d); }

template <typename T, int VE, bool HALVES>
void launch_rope(const RopeTable& tab, RopeArgs a, const void* x, void* out, cudaStream_t st) {
    const int sms = device_sms();
    a.chunks = a.pairs / (HALVES ? VE : VE / 2);
    const int per_voxel = a.heads * a.chunks;  // <= 65535 * 128
    // Items a unit: four loads a lane in flight at once keep the memory busy; where that
    // leaves warps without work, one load a lane spreads a short call over more of them.
    const int full = HALVES ? 64 : 128;
    const int want = a.n * per_voxel >= (int64_t)sms * 32 * full ? full : 32;
    a.voxels = 1;
    a.unit_heads = a.heads;
    if (per_voxel < want) {
        a.voxels = want / per_voxel;
        if (a.voxels * a.pairs > kRopeTable) a.voxels = kRopeTable / a.pairs;
    } else {
        const int groups = (per_voxel + want - 1) / want;
        a.unit_heads = (a.heads + groups - 1) / groups;
    }
    a.head_groups = (a.heads + a.unit_heads - 1) / a.unit_heads;
    a.units = (a.n + a.voxels - 1) / a.voxels * a.head_groups;
    a.by_chunks = div_by(a.chunks);
    a.by_voxel = div_by(per_voxel);
    a.by_pairs = div_by(a.pairs);
    const int64_t blocks = (a.units + kRopeWarps - 1) / kRopeWarps, most = (int64_t)sms * 6;
    k_rope<T, VE, HALVES><<<(unsigned)(blocks < most ? blocks : most), 32 * kRopeWarps, 0, st>>>(
        tab, a, static_cast<const T*>(x), static_cast<T*>(out));
}

// 16-byte items where every head starts on a 16-byte boundary and holds whole items,
// else one pair an item.
template <typename T>
void launch_rope_type(const RopeTable& tab, const RopeArgs& a, bool halves, const void* x, void* out,
                      cudaStream_t st) {
    constexpr int kVe = 16 / (int)sizeof(T);
    const bool wide = is_aligned(x, 16) && is_aligned(out, 16) && a.x_row % kVe == 0 && a.x_head % kVe == 0 &&
                      a.o_row % kVe == 0 && a.o_head % kVe == 0 && a.pairs % (halves ? kVe : kVe / 2) == 0;
    if (halves && wide)
        launch_rope<T, kVe, true>(tab, a, x, out, st);
    else if (halves)
        launch_rope<T, 1, true>(tab, a, x, out, st);
    else if (wide)
        launch_rope<T, kVe, false>(tab, a, x, out, st);
    else
        launch_rope<T, 2, false>(tab, a, x, out, st);
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
    RopeArgs a = {};
    a.coords = reinterpret_cast<const int4*>(coords);
    a.n = n;
    a.x_row = x_row;
    a.x_head = x_head;
    a.o_row = out_row;
    a.o_head = out_head;
    a.heads = heads;
    a.pairs = (int)(d / 2);
    a.sign = inverse ? -1.0f : 1.0f;
    const bool halves = rope->layout == SPCONV_ROPE_HALVES;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == SPCONV_BF16)
        launch_rope_type<__nv_bfloat16>(rope->table, a, halves, x, out, st);
    else
        launch_rope_type<float>(rope->table, a, halves, x, out, st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_rope_apply");
}

}  // extern "C"
