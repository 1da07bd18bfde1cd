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

// The threads of a CTA in groups of TPR, a group a row at a time: 2 to 32 lanes of a
// warp, or the whole CTA.
template <int TPR>
struct Group {
    static constexpr int kThreads = TPR > 128 ? TPR : 128;
    static constexpr int kRows = kThreads / TPR;  // rows a CTA has in work
};

// Joins v over a row's threads; `part` (a warp's share each) is not reused within a row.
template <typename Op, int TPR>
__device__ __forceinline__ float row_reduce(float v, float* part) {
#pragma unroll
    for (int d = (TPR < 32 ? TPR : 32) / 2; d > 0; d >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, d));
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        if (TPR <= 256) {
            v = part[0];
#pragma unroll
            for (int w = 1; w < TPR / 32; ++w) v = Op::f(v, part[w]);
        } else {
            const int lane = threadIdx.x & 31;
            v = lane < TPR / 32 ? part[lane] : Op::id();
#pragma unroll
            for (int d = TPR / 64; d > 0; d >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, d));
            v = __shfl_sync(0xffffffffu, v, 0);
        }
    }
    return v;
}

// y / s rounded once to fp32, for s with the reciprocal `inv`: the product y inv is off by a
// last bit now and then, so that a value next to the middle of two codes falls to the other
// one; the remainder y - s (y inv), exact in one fused operation down to |y| = 2^-102, mends
// it (P. W. Markstein, IBM J. Res. Dev. 34, 1990).  210,354 x 128 bf16 to 8 bits take 19.0 us, with the product alone
// 17.9 and with the division of every value 24.3.  back = -s, or 0 where s is infinite: then
// inv = 0 and the quotients of finite values are 0.
__device__ __forceinline__ float quotient(float y, float back, float inv) {
    const float v = y * inv;
    return fmaf(fmaf(v, back, y), inv, v);
}

// The 8-bit form of a row's values.
template <int VE>
__device__ __forceinline__ void store_e4m3(uint8_t* q, const float* y, float back, float inv) {
    if constexpr (VE == 1) {
        *q = __nv_cvt_float_to_fp8(quotient(y[0], back, inv), __NV_SATFINITE, __NV_E4M3);
    } else {
        Vec<__nv_fp8x2_storage_t, VE / 2> o;
#pragma unroll
        for (int e = 0; e < VE; e += 2)
            o.v[e / 2] = __nv_cvt_float2_to_fp8x2(make_float2(quotient(y[e], back, inv), quotient(y[e + 1], back, inv)),
                                                  __NV_SATFINITE, __NV_E4M3);
        store_vec(q, o);
    }
}

// A row lives in its threads' registers: E elements each, in items of VE, item k of
// thread t at (k * TPR + t) * VE.  One read of x and the residual, one write of each
// result.  Memory bounds it: with the residual 61,463 x 512 bf16 (and rstd) take 39.5 us,
// 6.4 TB/s or 97 % of a plain copy's rate, 61,463 x 1024 to 8 bits 67.3 us (100 %), 20,011 x
// 333 fp32, whose rows start anywhere, 11.5 us (71 %); one row of 1024 channels 2.7 us, most
// of it the launch.  Branches between items cost a third more (they keep the loads apart),
// rows fetched ahead through shared memory as in the gradient are no faster.
template <typename T, int VE, int TPR, int E, bool Q8, bool RES>
__global__ void __launch_bounds__(Group<TPR>::kThreads)
    k_rms_norm(const T* x, const T* res, const T* __restrict__ weight, int64_t n, int c, float eps, T* sum_out,
               T* __restrict__ out, float* __restrict__ rstd_out, uint8_t* __restrict__ q, float* __restrict__ scale) {
    using V = Vec<T, VE>;
    constexpr int kItems = E / VE, kStep = TPR * VE;
    __shared__ float part[2][TPR > 32 ? TPR / 32 : 1];
    const int t = threadIdx.x % TPR;
    const int64_t i = (int64_t)blockIdx.x * Group<TPR>::kRows + threadIdx.x / TPR;
    const bool live = i < n;  // a warp's rows join their sums together, so none leaves early
    const int64_t at = i * c + t * VE;
    const int left = live ? c - t * VE : 0;  // item k is in the row where k * kStep < left
    V vx[kItems], vr[RES ? kItems : 1];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        if (k * kStep >= left) continue;
        vx[k] = load_vec<V>(x + at + k * kStep);
        if (RES) vr[RES ? k : 0] = load_vec<V>(res + at + k * kStep);
    }
    float h[E], ss = 0.0f;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            float v = k * kStep < left ? to_f32(vx[k].v[e]) : 0.0f;
            if (RES) v += k * kStep < left ? to_f32(vr[RES ? k : 0].v[e]) : 0.0f;
            h[k * VE + e] = v;
            ss = fmaf(v, v, ss);
        }
    }
    if (RES && sum_out) {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (k * kStep >= left) continue;
            V o;
            pack(h + k * VE, o);
            store_vec(sum_out + at + k * kStep, o);
        }
    }
    const float rstd = rsqrtf(row_reduce<Sum, TPR>(ss, part[0]) / (float)c + eps);
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] *= rstd;
    if (weight) {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (k * kStep >= left) continue;
            float w[VE];
            unpack(load_vec<V>(weight + t * VE + k * kStep), w);
#pragma unroll
            for (int e = 0; e < VE; ++e) h[k * VE + e] *= w[e];
        }
    }
    if (Q8) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) m = max_nan(m, fabsf(h[e]));
        const float s = max_nan(row_reduce<MaxNan, TPR>(m, part[1]) / kE4m3Max, kMinScale);
        const float inv = 1.0f / s, back = isinf(s) ? 0.0f : -s;
#pragma unroll
        for (int k = 0; k < kItems; ++k)
            if (k * kStep < left) store_e4m3<VE>(q + at + k * kStep, h + k * VE, back, inv);
        if (live && t == 0) scale[i] = s;
    } else {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (k * kStep >= left) continue;
            V o;
            pack(h + k * VE, o);
            store_vec(out + at + k * kStep, o);
        }
    }
    if (rstd_out && live && t == 0) rstd_out[i] = rstd;
}

// Rows longer than 32,768 channels: one CTA a row, read once more for each step.
constexpr int kLongThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    k_rms_norm_long(const T* x, const T* res, const T* __restrict__ weight, int c, float eps, T* sum_out,
                    T* __restrict__ out, float* __restrict__ rstd_out, uint8_t* __restrict__ q,
                    float* __restrict__ scale) {
    __shared__ float part[2][kLongThreads / 32];
    const int64_t base = (int64_t)blockIdx.x * c;
    float ss = 0.0f;
    for (int j = threadIdx.x; j < c; j += kLongThreads) {
        const float h = to_f32(x[base + j]) + (res ? to_f32(res[base + j]) : 0.0f);
        ss += h * h;
    }
    const float rstd = rsqrtf(row_reduce<Sum, kLongThreads>(ss, part[0]) / (float)c + eps);
    float s = 1.0f;
    if (q) {
        float m = 0.0f;
        for (int j = threadIdx.x; j < c; j += kLongThreads) {
            const float h = to_f32(x[base + j]) + (res ? to_f32(res[base + j]) : 0.0f);
            m = max_nan(m, fabsf(h * rstd * (weight ? to_f32(weight[j]) : 1.0f)));
        }
        s = max_nan(row_reduce<MaxNan, kLongThreads>(m, part[1]) / kE4m3Max, kMinScale);
    }
    for (int j = threadIdx.x; j < c; j += kLongThreads) {
        const float h = to_f32(x[base + j]) + (res ? to_f32(res[base + j]) : 0.0f);
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

// CTAs that share the rows of the gradient: a constant, so that the order of the column
// sums depends on the shape alone.  One CTA of 512 threads an SM; more of them add column
// sums to join (8,191 x 4096 bf16: 40.4 us with 148 CTAs, 42.8 with 296).  The longest
// rows, which are read twice, run on two, which cover each other's waits.
constexpr int kParts = kSms, kMaxParts = 2 * kParts;
inline int row_parts(int64_t n, int rows, int most) {
    // Up to four turns of one CTA: its column sums are the result, and the second step's
    // launch (3 us on the host, 2 on the GPU) falls away.
    if (n <= 4 * rows) return 1;
    const int64_t need = (n + rows - 1) / rows;
    return (int)(need < most ? need : most);
}

// Sum of v over the TPR threads of a row group of a CTA that holds several, which wait for
// each other alone.
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float* part, int group) {
#pragma unroll
    for (int d = (TPR < 32 ? TPR : 32) / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
        const float* mine = part + group * kWarps;
        if (kWarps <= 4) {
            v = mine[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v += mine[w];
        } else {
            const int lane = threadIdx.x & 31;
            v = lane < kWarps ? mine[lane] : 0.0f;
#pragma unroll
            for (int d = kWarps / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            v = __shfl_sync(0xffffffffu, v, 0);
        }
    }
    return v;
}

// Rows of the gradient a thread fetches ahead, in shared memory: copies of its own elements,
// so no thread waits for another.
template <typename T, int TPR, int E, bool SUM>  // two rows ahead of the one in work, or one
constexpr int kRowSmem = (SUM ? 3 : 2) * E * (int)sizeof(T) * (TPR > 512 ? TPR : 512);
template <typename T, int TPR, int E, bool SUM>
constexpr int kAhead = 3 * kRowSmem<T, TPR, E, SUM> <= 200 * 1024 ? 2 : 1;
template <typename T, int TPR, int E>
constexpr bool kFetchesAhead = E <= 16 && 2 * kRowSmem<T, TPR, E, true> <= 200 * 1024;

// Dynamic shared memory: the rows on their way, and at the end the column sums of a CTA that
// has one row at a time (with a place left free after every 32).
template <typename T, int TPR, int E, bool SUM>
constexpr int kRingSmem =
    kFetchesAhead<T, TPR, E> ? (kAhead<T, TPR, E, SUM> + 1) * kRowSmem<T, TPR, E, SUM> : 0;
template <typename T, int TPR, int E, bool SUM>
constexpr int kBackwardSmem =
    TPR >= 512 && kRingSmem<T, TPR, E, SUM> < TPR * E / 32 * 33 * 4 ? TPR * E / 32 * 33 * 4 : kRingSmem<T, TPR, E, SUM>;

// Elements [from, to) of an item of 16 bytes, which are not all of it.
__device__ __forceinline__ void store_part(float* p, const Vec<float, 4>& v, int from, int to) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e >= from && e < to) p[e] = v.v[e];
}
__device__ __forceinline__ void store_part(__nv_bfloat16* p, const Vec<__nv_bfloat16, 8>& v, int from, int to) {
    uint32_t w[4];
    memcpy(w, &v, 16);
    if (from > 0 && to < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= from && e < to) p[e] = v.v[e];
    } else if (from > 0) {  // up to a whole word, then two words, then four
        const int word = (from + 1) >> 1;
        const uint32_t first = from >= 4 ? from >= 6 ? w[3] : w[2] : from >= 2 ? w[1] : w[0];
        if (from & 1) reinterpret_cast<uint16_t*>(p)[from] = (uint16_t)(first >> 16);
        if (word & 1) reinterpret_cast<uint32_t*>(p)[word] = word == 1 ? w[1] : w[3];
        if (word <= 2) *reinterpret_cast<uint2*>(p + 4) = make_uint2(w[2], w[3]);
    } else {
        const uint32_t last = to >= 4 ? to >= 6 ? w[3] : w[2] : to >= 2 ? w[1] : w[0];
        if (to & 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        if (to & 2) reinterpret_cast<uint32_t*>(p)[to >= 4 ? 2 : 0] = to >= 4 ? w[2] : w[0];
        if (to & 1) reinterpret_cast<uint16_t*>(p)[to - 1] = (uint16_t)last;
    }
}

// dx of the rows and, in `part`, each CTA's column sums of dy * xh.  A CTA's row groups
// of TPR threads take rows blockIdx.x * kRows + group, and so on by gridDim.x * kRows,
// and wait only within the group; a thread keeps the sums of its columns in registers
// over all its rows, and the groups' sums are joined in shared memory at the end.
//
// SHIFT: rows of c elements where c is no multiple of an item's VE.  The grid makes a group's
// turns a multiple of VE elements apart, so each of its rows starts `shift` elements behind an
// item's start: the items are read whole, the elements of the row before are taken as zero,
// those behind the row are not read, and the two ends are written by elements.  Against rows
// read by one or two elements: 220,147 x 53 bf16 with a dsum 26.5 us, was 77; 24,198 x 379
// 23.2, was 77; 2,214 x 5491 24.1, was 527 (it did not fit the registers).
//
// Memory bounds it as long as the next rows are on their way: without them (loads at
// the top of a turn) 8,191 x 4096 bf16 take 66 us, with them 37.0 us, 5.4 TB/s or 83 % of a
// copy's rate with the sums' second step in it; 209,715 x 128 with a dsum 37.5 us (88 %),
// 3,000 x 6000 fp32 38.6 us (85 %).
template <typename T, int VE, int TPR, int E, bool SUM, bool SHIFT>
__global__ void __launch_bounds__(TPR > 512 ? TPR : 512)
    k_rms_norm_backward(const T* __restrict__ dy, const T* __restrict__ h, const T* __restrict__ weight,
                        const float* __restrict__ rstd_in, const T* dsum, int64_t n, int c, T* dx,
                        float* __restrict__ part) {
    using V = Vec<T, VE>;
    constexpr int kThreads = TPR > 512 ? TPR : 512, kRows = kThreads / TPR, kItems = E / VE;
    constexpr bool kFetch = kFetchesAhead<T, TPR, E>;
    constexpr int kTurns = kAhead<T, TPR, E, SUM>, kStages = kTurns + 1;
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    V* ring = reinterpret_cast<V*>(ring_bytes) + threadIdx.x;  // [stage][dy, h, dsum][item][thread]
    __shared__ float red[2][kThreads / 32];
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    // With a shift the rows of a warp lie 16 apart, so that they all have the same one.
    const int row = SHIFT && TPR < 32 ? threadIdx.x % 32 / TPR * (kThreads / 32) + threadIdx.x / 32 : group;
    const int64_t step = (int64_t)gridDim.x * kRows, stride = step * c;
    int64_t i = (int64_t)blockIdx.x * kRows + row;
    const int shift = SHIFT ? (int)(i * c) & (VE - 1) : 0, end = c + shift;
    const int head = t == 0 ? shift : 0;  // this many elements of item 0 belong to the row before
    const bool edge = head > 0 || (end % VE > 0 && end / VE % TPR == t);  // has an item with some of the row
    int64_t at = i * c - shift + t * VE, at_fetch = at;  // this thread's first element of a row
    float dw[E];
    V w[kItems];
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = 0.0f;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int j = (k * TPR + t) * VE;
#pragma unroll
        for (int e = 0; e < VE; ++e) w[k].v[e] = from_f32<T>(1.0f);
        if (SHIFT) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (weight && j + e >= shift && j + e < end) w[k].v[e] = weight[j + e - shift];
        } else if (weight && j < c) {
            w[k] = load_vec<V>(weight + j);
        }
    }
    const float by_c = 1.0f / (float)c;
    const auto fetch = [&](bool in, int stage) {
        V* to = ring + stage * ((SUM ? 3 : 2) * kItems * kThreads);
        if (in) {
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int j = (k * TPR + t) * VE;
                if (j >= end) continue;
                const int64_t from = at_fetch + k * TPR * VE;
                const auto copy = [&](int array, const T* src) {
                    const uint32_t dst = shared_at(to + (array * kItems + k) * kThreads);
                    // an item is read as far as the row goes; the rest of it is zero
                    if (SHIFT)
                        copy_async_part(dst, src + from, (end - j < VE ? end - j : VE) * (int)sizeof(T));
                    else
                        copy_async<16>(dst, src + from);
                };
                copy(0, dy), copy(1, h);
                if (SUM) copy(2, dsum);
            }
        }
        at_fetch += stride;
        copy_commit();
    };
    if (kFetch) {
#pragma unroll
        for (int a = 0; a < kTurns; ++a) fetch(i + a * step < n, a);
    }
    float rstd_next = i < n ? rstd_in[i] : 0.0f;
    int turn = 0;  // the sums' buffer: a thread may still read the last row's
    int stage = 0;
    for (int64_t i0 = (int64_t)blockIdx.x * kRows; i0 < n; i0 += step, i += step, at += stride, turn ^= 1) {
        const bool live = i < n;
        const float rstd = rstd_next;
        rstd_next = i + step < n ? rstd_in[i + step] : 0.0f;
        V vd[kItems], vh[kItems], vs[kItems];
        const V* from = ring + stage * ((SUM ? 3 : 2) * kItems * kThreads);
        if (kFetch) copy_wait<kTurns - 1>();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int j = (k * TPR + t) * VE;
            if (!live || j >= end) continue;
            if (SHIFT && !kFetch && j + VE > end) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const bool in = j + e < end;
                    vd[k].v[e] = in ? dy[at + k * TPR * VE + e] : from_f32<T>(0.0f);
                    vh[k].v[e] = in ? h[at + k * TPR * VE + e] : from_f32<T>(0.0f);
                    if (SUM) vs[k].v[e] = in ? dsum[at + k * TPR * VE + e] : from_f32<T>(0.0f);
                }
                continue;
            }
            vd[k] = kFetch ? from[k * kThreads] : load_vec<V>(dy + at + k * TPR * VE);
            vh[k] = kFetch ? from[(kItems + k) * kThreads] : load_vec<V>(h + at + k * TPR * VE);
            if (SUM) vs[k] = kFetch ? from[(2 * kItems + k) * kThreads] : load_vec<V>(dsum + at + k * TPR * VE);
        }
        float g[E], xh[E], dot = 0.0f;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (!live || (k * TPR + t) * VE >= end) continue;
            float d[VE], wk[VE];
            unpack(vd[k], d);
            unpack(vh[k], xh + k * VE);
            unpack(w[k], wk);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int o = k * VE + e;
                if (SHIFT && k == 0 && e < head) d[e] = xh[o] = 0.0f;
                xh[o] *= rstd;
                g[o] = d[e] * wk[e];
                dw[o] = fmaf(d[e], xh[o], dw[o]);
                dot = fmaf(g[o], xh[o], dot);
            }
        }
        if (kFetch) {
            // into the stage read in the last turn
            fetch(i + kTurns * step < n, stage == 0 ? kStages - 1 : stage - 1);
            stage = stage == kStages - 1 ? 0 : stage + 1;
        }
        const float mean = group_sum<TPR>(dot, red[turn], group) * by_c;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int j = (k * TPR + t) * VE;
            if (!live || j >= end) continue;
            float o[VE], ds[VE];
            if (SUM) unpack(vs[k], ds);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                o[e] = fmaf(-xh[k * VE + e], mean, g[k * VE + e]);
                o[e] = SUM ? fmaf(rstd, o[e], ds[e]) : rstd * o[e];
            }
            if constexpr (SHIFT) {
                pack(o, vd[k]);
                if (j >= shift && j + VE <= end) store_vec(dx + at + k * TPR * VE, vd[k]);
            } else {
                V packed;
                pack(o, packed);
                store_vec(dx + at + k * TPR * VE, packed);
            }
        }
        if (SHIFT && edge && live) {
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int j = (k * TPR + t) * VE;
                if (j < end && (j < shift || j + VE > end))
                    store_part(dx + at + k * TPR * VE, vd[k], k == 0 ? head : 0, end - j < VE ? end - j : VE);
            }
        }
    }
    cudaTriggerProgrammaticLaunchCompletion();  // the column sums' second step may take its place
    if (!part) return;
    part += (int64_t)blockIdx.x * c;
    if constexpr (kRows == 1) {
        // from a thread's neighbouring columns to neighbouring threads' (written from the
        // registers, 148 x 6688 sums take 8 us)
        __syncthreads();  // the rows' place is free
        float* cols = reinterpret_cast<float*>(ring_bytes);
#pragma unroll
        for (int k = 0; k < kItems; ++k)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int j = (k * TPR + t) * VE + e - shift;
                if (!SHIFT || j >= 0) cols[j + (j >> 5)] = dw[k * VE + e];
            }
        __syncthreads();
        for (int j = threadIdx.x; j < c; j += kThreads) part[j] = cols[j + (j >> 5)];
    } else {
        // a warp's groups first (TPR < 32), then the groups: kShares rows of sums
        constexpr int kShares = TPR < 32 ? kThreads / 32 : kRows;
        __shared__ float cols[kShares][TPR * E];
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int d = TPR; d < 32; d <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], d);
        if (TPR >= 32 || (threadIdx.x & 31) < TPR) {
#pragma unroll
            for (int k = 0; k < kItems; ++k)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const int j = (k * TPR + t) * VE + e - shift;
                    if (!SHIFT || j >= 0) cols[TPR < 32 ? threadIdx.x / 32 : group][j] = dw[k * VE + e];
                }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < c; j += kThreads) {
            float s = cols[0][j];
#pragma unroll
            for (int w = 1; w < kShares; ++w) s += cols[w][j];
            part[j] = s;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    k_rms_norm_backward_long(const T* __restrict__ dy, const T* __restrict__ h, const T* __restrict__ weight,
                             const float* __restrict__ rstd_in, const T* dsum, int64_t n, int c, T* dx,
                             float* __restrict__ part) {
    __shared__ float red[2][kLongThreads / 32];
    int turn = 0;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x, turn ^= 1) {
        const int64_t base = i * c;
        const float rstd = rstd_in[i];
        float dot = 0.0f;
        for (int j = threadIdx.x; j < c; j += kLongThreads) {
            const float dxh = to_f32(dy[base + j]) * (to_f32(h[base + j]) * rstd);
            if (part) {
                float* p = part + (int64_t)blockIdx.x * c + j;
                *p = i == blockIdx.x ? dxh : *p + dxh;
            }
            dot += dxh * (weight ? to_f32(weight[j]) : 1.0f);
        }
        const float mean = row_reduce<Sum, kLongThreads>(dot, red[turn]) / (float)c;
        for (int j = threadIdx.x; j < c; j += kLongThreads) {
            const float g = to_f32(dy[base + j]) * (weight ? to_f32(weight[j]) : 1.0f);
            float d = rstd * (g - to_f32(h[base + j]) * rstd * mean);
            if (dsum) d += to_f32(dsum[base + j]);
            dx[base + j] = from_f32<T>(d);
        }
    }
}

// dweight[j] = sum over the parts, in a fixed order: a CTA takes 32 columns, its warps
// every 32nd part, joined by a tree.  Launched to start while the gradient's last
// CTAs still run; it waits for them before it reads.
__global__ void __launch_bounds__(1024) k_rms_norm_dw(const float* __restrict__ part, int parts, int c,
                                                      float* __restrict__ dweight) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    cudaGridDependencySynchronize();
    float s = 0.0f;
    if (j < c) {
#pragma unroll 7
        for (int p = warp; p < parts; p += 32) s += part[(int64_t)p * c + j];
    }
    sum[warp][lane] = s;
    __syncthreads();
    // column `warp`: its 32 shares to one warp
    s = sum[lane][warp];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0 && blockIdx.x * 32 + warp < c) dweight[blockIdx.x * 32 + warp] = s;
}

cudaError_t launch_dw(const float* part, int parts, int c, float* dweight, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((c + 31) / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rms_norm_dw, part, parts, c, dweight);
}

struct NormArgs {
    const void *x, *res, *weight;
    int64_t n;
    int c;
    float eps;
    void *sum_out, *out;
    float* rstd;
    uint8_t* q;
    float* scale;
    // gradient
    const void* dsum;
    const float* rstd_in;
    void* dx;
    float *dweight, *part;
    cudaStream_t stream;
};

template <typename T, int VE, int TPR, int E, bool Q8>
void launch_forward_as(const NormArgs& a) {
    constexpr int kRows = Group<TPR>::kRows, kThreads = Group<TPR>::kThreads;
    const auto kernel = a.res ? k_rms_norm<T, VE, TPR, E, Q8, true> : k_rms_norm<T, VE, TPR, E, Q8, false>;
    kernel<<<(unsigned)((a.n + kRows - 1) / kRows), kThreads, 0, a.stream>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.res), static_cast<const T*>(a.weight), a.n, a.c, a.eps,
        static_cast<T*>(a.sum_out), static_cast<T*>(a.out), a.rstd, a.q, a.scale);
}

// Rows that do not start on 16-byte boundaries: two elements at a time, or one.  Up to 1024
// channels a warp takes the row (61,463 x 513 bf16: 37 us; 46 with 128 threads a row, which
// wait for each other), longer rows have 16 to 32 elements a thread.
template <typename T, int VE, bool Q8>
void launch_forward_narrow(const NormArgs& a) {
    if (a.c <= 32) launch_forward_as<T, VE, 4, 8, Q8>(a);
    else if (a.c <= 64) launch_forward_as<T, VE, 4, 16, Q8>(a);
    else if (a.c <= 128) launch_forward_as<T, VE, 16, 8, Q8>(a);
    else if (a.c <= 256) launch_forward_as<T, VE, 32, 8, Q8>(a);
    else if (a.c <= 512) launch_forward_as<T, VE, 32, 16, Q8>(a);
    else if (a.c <= 1024) launch_forward_as<T, VE, 32, 32, Q8>(a);
    else if (a.c <= 2048) launch_forward_as<T, VE, 128, 16, Q8>(a);
    else if (a.c <= 4096) launch_forward_as<T, VE, 256, 16, Q8>(a);
    else if (a.c <= 8192) launch_forward_as<T, VE, 256, 32, Q8>(a);
    else if (a.c <= 16384) launch_forward_as<T, VE, 512, 32, Q8>(a);
    else launch_forward_as<T, VE, 1024, 32, Q8>(a);
}

// A thread holds up to 32 elements of a row, and few threads take it, so that a row's sums
// cross few threads and the rows in work, one a group, are many: 210,354 x 80 bf16 to 8 bits
// take 14.4 us with 4 threads a row, 19.5 with 8 and 24.6 with 16.  Two lengths have twice the
// threads that hold the row: up to 64 channels (300,000 x 64 bf16 with a residual 24.7 us,
// with 2 threads 27.7; to 8 bits 15.2 and 14.8) and up to 512 (61,463 x 512 with a residual
// 39.2 us, with 16 threads 39.7; to 8 bits 34.9 and 35.8, without a residual 23.1 and 21.6).
// Above a warp a row has the whole CTA of 128 threads or more.  Many rows of up to 1536
// channels to 8 bits, which join their threads twice, stay in a warp of 48 elements a lane:
// 16,862 x 1408 bf16 19.6 us, 24.8 with 128 threads a row; few rows are 1 us slower so.
template <typename T, bool Q8>
void launch_forward(const NormArgs& a) {
    constexpr int kVe = 16 / (int)sizeof(T);
    if (a.c > 32768) {
        k_rms_norm_long<T><<<(unsigned)a.n, kLongThreads, 0, a.stream>>>(
            static_cast<const T*>(a.x), static_cast<const T*>(a.res), static_cast<const T*>(a.weight), a.c, a.eps,
            static_cast<T*>(a.sum_out), static_cast<T*>(a.out), a.rstd, a.q, a.scale);
    } else if (a.c % kVe == 0) {
        constexpr int kFew = sizeof(T) == 2 ? 2 : 4;  // threads of a row of 32 bytes a thread
        if (a.c <= 16) launch_forward_as<T, kVe, 2, 8, Q8>(a);
        else if (a.c <= 32) launch_forward_as<T, kVe, kFew, 32 / kFew, Q8>(a);
        else if (a.c <= 64) launch_forward_as<T, kVe, 4, 16, Q8>(a);
        else if (a.c <= 96) launch_forward_as<T, kVe, 4, 24, Q8>(a);
        else if (a.c <= 128) launch_forward_as<T, kVe, 4, 32, Q8>(a);
        else if (a.c <= 192) launch_forward_as<T, kVe, 8, 24, Q8>(a);
        else if (a.c <= 256) launch_forward_as<T, kVe, 8, 32, Q8>(a);
        else if (a.c <= 384) launch_forward_as<T, kVe, 16, 24, Q8>(a);
        else if (a.c <= 512) launch_forward_as<T, kVe, 32, 16, Q8>(a);
        else if (a.c <= 768) launch_forward_as<T, kVe, 32, 24, Q8>(a);
        else if (a.c <= 1024) launch_forward_as<T, kVe, 32, 32, Q8>(a);
        else if (Q8 && a.c <= 1536 && a.n >= 16 * kSms) launch_forward_as<T, kVe, 32, Q8 ? 48 : 32, Q8>(a);
        else if (a.c <= 2048) launch_forward_as<T, kVe, 128, 16, Q8>(a);
        else if (a.c <= 4096) launch_forward_as<T, kVe, 128, 32, Q8>(a);
        else if (a.c <= 8192) launch_forward_as<T, kVe, 256, 32, Q8>(a);
        else if (a.c <= 16384) launch_forward_as<T, kVe, 512, 32, Q8>(a);
        else launch_forward_as<T, kVe, 1024, 32, Q8>(a);
    } else if (a.c % 2 == 0) {
        launch_forward_narrow<T, 2, Q8>(a);
    } else {
        launch_forward_narrow<T, 1, Q8>(a);
    }
}

template <typename T, int TPR, int E, bool SUM, bool SHIFT>
int launch_backward_kernel(const NormArgs& a) {
    constexpr int kThreads = TPR > 512 ? TPR : 512, kRows = kThreads / TPR, kVe = 16 / (int)sizeof(T);
    constexpr int kSmem = kBackwardSmem<T, TPR, E, SUM>;
    constexpr auto kernel = k_rms_norm_backward<T, kVe, TPR, E, SUM, SHIFT>;
    int parts = row_parts(a.n, kRows, kParts);
    if (SHIFT && (int64_t)parts * kRows < a.n) {
        // A group keeps its shift over its turns: they are a whole number of items apart.
        int whole = 1;
        while ((int64_t)whole * kRows * a.c % kVe) whole *= 2;
        if (parts % whole) parts = parts == 1 ? (int)((a.n + kRows - 1) / kRows) : parts / whole * whole;
    }
    if (kSmem > 0) {
        static std::atomic<uint64_t> done{0};
        if (allow_smem(kernel, kSmem, done) != cudaSuccess) return 0;  // the caller asks why
    }
    kernel<<<parts, kThreads, kSmem, a.stream>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.res), static_cast<const T*>(a.weight), a.rstd_in,
        static_cast<const T*>(a.dsum), a.n, a.c, static_cast<T*>(a.dx), parts == 1 ? a.dweight : a.part);
    return parts;
}

// Returns the CTAs that wrote column sums.
template <typename T, int TPR, int E>
int launch_backward_as(const NormArgs& a) {
    if (a.c % (16 / (int)sizeof(T)) == 0)
        return a.dsum ? launch_backward_kernel<T, TPR, E, true, false>(a) : launch_backward_kernel<T, TPR, E, false, false>(a);
    return a.dsum ? launch_backward_kernel<T, TPR, E, true, true>(a) : launch_backward_kernel<T, TPR, E, false, true>(a);
}

// A row's items from its first element's: a row that does not start at one may touch one more.
template <typename T>
int row_span(int c) {
    constexpr int kVe = 16 / (int)sizeof(T);
    return c % kVe == 0 ? c : c + kVe - 1;
}

// 32 bytes of a row a thread (bf16: 16 elements, fp32: 8), as many threads as that takes; 16
// bytes a thread and twice the threads are a quarter to a half slower.  From 8,193 channels on
// 16 elements for each of 1024 threads do not fit the 64 registers that a thread then has:
// 180 to 850 bytes a thread go through local memory, 900 x 12,000 bf16 take 32 us, 31 % of a
// copy's rate.  Above 16,384 channels the
// columns' sums are in memory: 900 x 20,000 bf16 66 us, 97 with 32 elements a thread.
template <typename T>
int launch_backward(const NormArgs& a) {
    constexpr int kE = 32 / (int)sizeof(T);
    const int span = row_span<T>(a.c);
    if (span <= 2 * kE) return launch_backward_as<T, 2, kE>(a);
    if (span <= 4 * kE) return launch_backward_as<T, 4, kE>(a);
    if (span <= 8 * kE) return launch_backward_as<T, 8, kE>(a);
    if (span <= 16 * kE) return launch_backward_as<T, 16, kE>(a);
    if (span <= 32 * kE) return launch_backward_as<T, 32, kE>(a);
    if (span <= 64 * kE) return launch_backward_as<T, 64, kE>(a);
    if (span <= 128 * kE) return launch_backward_as<T, 128, kE>(a);
    if (span <= 256 * kE) return launch_backward_as<T, 256, kE>(a);
    if (span <= 512 * kE) return launch_backward_as<T, 512, kE>(a);
    if (span <= 8192) return launch_backward_as<T, 512, 16>(a);
    if (span <= 16384) return launch_backward_as<T, 1024, 16>(a);
    const int parts = row_parts(a.n, 1, kMaxParts);
    k_rms_norm_backward_long<T><<<parts, kLongThreads, 0, a.stream>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.res), static_cast<const T*>(a.weight), a.rstd_in,
        static_cast<const T*>(a.dsum), a.n, a.c, static_cast<T*>(a.dx), parts == 1 ? a.dweight : a.part);
    return parts;
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
    NormArgs a = {x, residual, weight, n, channels, eps, sum_out, out, rstd};
    a.stream = static_cast<cudaStream_t>(stream);
    if (dtype == SPCONV_BF16)
        launch_forward<__nv_bfloat16, false>(a);
    else
        launch_forward<float, false>(a);
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
    NormArgs a = {x, residual, weight, n, channels, eps, sum_out, nullptr, nullptr, q, scale};
    a.stream = static_cast<cudaStream_t>(stream);
    if (dtype == SPCONV_BF16)
        launch_forward<__nv_bfloat16, true>(a);
    else
        launch_forward<float, true>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_rms_norm_q8");
}

spconv_status_t spconv_rms_norm_workspace(int64_t n, int32_t channels, int64_t* bytes) {
    if (!bytes) return row_fail(SPCONV_ERR_INVALID_ARG, "null bytes");
    if (n < 0 || n >= (int64_t(1) << 31)) return row_fail(SPCONV_ERR_INVALID_ARG, "n must be in [0, 2^31)");
    if (channels < 1 || channels > SPCONV_NORM_MAX_CHANNELS)
        return row_fail(SPCONV_ERR_INVALID_ARG, "channels must be in [1, 65536]");
    *bytes = (int64_t)(n < kMaxParts ? n : kMaxParts) * channels * 4;
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
    const int64_t wsbytes = (int64_t)(n < kMaxParts ? n : kMaxParts) * channels * 4, dwbytes = (int64_t)channels * 4;
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
    NormArgs a = {};
    a.x = dy;
    a.res = h;
    a.weight = weight;
    a.n = n;
    a.c = channels;
    a.dsum = dsum;
    a.rstd_in = rstd;
    a.dx = dx;
    a.dweight = dweight;
    a.part = dweight ? static_cast<float*>(workspace) : nullptr;
    a.stream = st;
    const int parts = dtype == SPCONV_BF16 ? launch_backward<__nv_bfloat16>(a) : launch_backward<float>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && dweight && parts > 1) e = launch_dw(a.part, parts, channels, dweight, st);
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_rms_norm_backward");
}

}  // extern "C"
