// Rotary positions of feature rows from voxel coordinates, with several axes.
//
// Pair j of every head of a voxel turns by the angle freq[j] * coord[axis[j]]:
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),
// the gradient is the turn by -t.  The angle is kept in turns, as a 64-bit fixed
// point fraction: F = freq / (2 pi) mod 1, scaled by 2^64, and F * coord modulo
// 2^64 is the exact fraction of a turn for any 32-bit coordinate (the error is that
// of F, which is rounded: 2^-65 of a turn times the coordinate), where an fp32 product
// would be off by 2^-24 of the whole angle: 4e-3 rad at coordinate 65535.
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
    int chunk_blocks;   // blocks of 32 items a head
    int lanes_head;     // lanes on a head: the items of a chunk block, at most 32
    int head_slots;     // heads that a warp turns side by side
    int voxel_slots;    // voxels that a warp turns side by side
    int unit_heads;     // heads a warp turns of each of its voxels
    float sign;         // -1: turn back
};

constexpr int kRopeThreads = 256;
constexpr int kRopeAhead = 2;  // voxels a lane fetches ahead, through shared memory

template <typename T, int VE>
constexpr bool kWide = sizeof(T) * VE == 16;
// Heads a lane turns of a voxel, one after the other: 64 bytes on the way a voxel.
template <bool HALVES>
constexpr int kPasses = HALVES ? 2 : 4;
template <typename T, int VE>
constexpr int kRopeSmem = kWide<T, VE> ? (kRopeAhead + 1) * 4 * 16 * kRopeThreads : 0;

// Items: VE neighbouring elements of a head (VE / 2 pairs) in the interleaved layout,
// VE elements of either half (VE pairs) in the halves layout.
//
// A lane owns one item position of the head for the whole launch, so the cosines and
// sines of its pairs are computed once a voxel and used for all of the voxel's heads
// that the warp turns: head_slots heads (and, where a voxel has few heads, voxel_slots
// voxels) side by side, kPasses of them one after the other.  Warps go from voxel to
// voxel with the next coordinates in registers and the items of the next two voxels on
// their way into shared memory; every lane copies and reads its own, so none waits for
// another.  blockIdx.y: the block of items and the group of heads.
//
// Memory bounds it: 273,995 voxels of 12 x 64 in bf16, out of a packed projection, take
// 136 us, 6.2 TB/s or 95 % of a plain copy's rate; 16,934 of 8 x 96 in fp32 halves 20 us
// (80 %: a head's 12 items leave 8 lanes of a warp idle, and fp32 sines are long); one
// voxel 2.3 us.  One pair a thread with a sine each took 1,717 us for the first.  Items of
// one pair, for heads that are no whole number of 16-byte items, are not fetched ahead and wait
// for their loads: 100,000 voxels of 8 x 72 in bf16 halves 167 us (21 %), of 8 x 36
// interleaved 73 us (24 %).
template <typename T, int VE, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads, 4)
    k_rope(const __grid_constant__ RopeTable tab, const __grid_constant__ RopeArgs a, const T* x, T* out) {
    constexpr int kPairs = HALVES ? VE : VE / 2;  // pairs an item
    constexpr int kVecs = HALVES ? 2 : 1;         // accesses an item
    constexpr int kN = kPasses<HALVES>;
    constexpr bool kRing = kWide<T, VE>;
    using V = Vec<T, VE, kRing ? 16 : (int)sizeof(T)>;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ uint64_t turn[kMaxPairs];
    for (int j = threadIdx.x; j < a.pairs; j += kRopeThreads) turn[j] = tab.turn[j];
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int hg = (int)blockIdx.y / a.chunk_blocks, cb = (int)blockIdx.y - hg * a.chunk_blocks;
    const int slot = lane / a.lanes_head, chunk = cb * 32 + lane % a.lanes_head;
    const int vs = slot / a.head_slots;
    if (vs >= a.voxel_slots || chunk >= a.chunks) return;
    const int h0 = hg * a.unit_heads + slot % a.head_slots, h_end = min(a.heads, (hg + 1) * a.unit_heads);
    const int j0 = chunk * kPairs;
    const int64_t i0 = ((int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5)) * a.voxel_slots + vs;
    if (i0 >= a.n || h0 >= h_end) return;
    const int todo = (h_end - h0 + a.head_slots - 1) / a.head_slots;  // passes of this lane, at most kN
    uint32_t axes = 0;  // two bits a pair: 0 does not turn, else the axis + 1
#pragma unroll
    for (int p = 0; p < kPairs; ++p) axes |= (uint32_t)(tab.axis[j0 + p] + 1) << (2 * p);
    const int64_t step = (int64_t)gridDim.x * (kRopeThreads / 32) * a.voxel_slots;
    const int64_t x_pass = a.head_slots * a.x_head, o_pass = a.head_slots * a.o_head;
    const int64_t x_step = step * a.x_row, o_step = step * a.o_row;
    const T* px = x + i0 * a.x_row + h0 * a.x_head + chunk * VE;
    T* po = out + i0 * a.o_row + h0 * a.o_head + chunk * VE;
    V* ring = reinterpret_cast<V*>(smem) + threadIdx.x;  // [stage][pass, half][thread]
    const auto fetch = [&](bool in, int stage) {
        if (in) {
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                if (k >= todo) continue;
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
                    copy_async<16>(shared_at(ring + ((stage * kN + k) * kVecs + v) * kRopeThreads),
                                   px + k * x_pass + v * a.pairs);
            }
        }
        px += x_step;
        copy_commit();
    };
    if (kRing) {
#pragma unroll
        for (int s = 0; s < kRopeAhead; ++s) fetch(i0 + s * step < a.n, s);
    }
    int4 at = a.coords[i0];
    int stage = 0;
    for (int64_t i = i0; i < a.n; i += step) {
        if (kRing) fetch(i + kRopeAhead * step < a.n, stage == 0 ? kRopeAhead : stage - 1);  // read in the last turn
        const int4 pos = at;
        if (i + step < a.n) at = a.coords[i + step];
        float cs[kPairs], sn[kPairs];
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const uint32_t ax = (axes >> (2 * p)) & 3u;
            const int c = ax == 1 ? pos.y : ax == 2 ? pos.z : ax == 3 ? pos.w : 0;
            // the nearest 2^-32 of a turn
            const int32_t frac = (int32_t)((turn[j0 + p] * (uint64_t)(int64_t)c + (uint64_t(1) << 31)) >> 32);
            if (sizeof(T) == 2) {
                // 2^-21.2 of error on [-pi, pi], against the 2^-9 of the result's rounding
                const float ang = (float)frac * 1.46291807926715968e-9f;  // 2 pi / 2^32
                sn[p] = __sinf(ang) * a.sign;
                cs[p] = __cosf(ang);
            } else {
                // the 8 bits that fp32 leaves of the fraction turn the sine and cosine a little further
                const float high = (float)(frac & ~0xff), rest = (float)(frac & 0xff) * 1.46291807926715968e-9f;
                float sh, ch;
                sincospif(high * 0x1p-31f, &sh, &ch);
                sn[p] = fmaf(ch, rest, sh) * a.sign;
                cs[p] = fmaf(-sh, rest, ch);
            }
        }
        if (kRing) copy_wait<kRopeAhead>();
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            if (k >= todo) continue;
            float f[kVecs * VE];
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                unpack(kRing ? ring[((stage * kN + k) * kVecs + v) * kRopeThreads]
                             : load_vec<V>(px + k * x_pass + v * a.pairs),
                       f + v * VE);
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                float& u = HALVES ? f[p] : f[2 * p];
                float& v = HALVES ? f[(kVecs - 1) * VE + p] : f[2 * p + 1 - (HALVES ? 1 : 0)];
                const float turned = u * cs[p] - v * sn[p];
                v = u * sn[p] + v * cs[p];
                u = turned;
            }
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                V o;
                pack(f + v * VE, o);
                store_vec(po + k * o_pass + v * a.pairs, o);
            }
        }
        if (!kRing) px += x_step;
        po += o_step;
        stage = stage == kRopeAhead ? 0 : stage + 1;
    }
}

template <typename T, int VE, bool HALVES>
void launch_rope(const RopeTable& tab, RopeArgs a, const void* x, void* out, cudaStream_t st) {
    constexpr int kN = kPasses<HALVES>, kWarps = kRopeThreads / 32, kSmem = kRopeSmem<T, VE>, kVoxels = 12;
    a.chunks = a.pairs / (HALVES ? VE : VE / 2);
    a.chunk_blocks = (a.chunks + 31) / 32;
    a.lanes_head = a.chunks < 32 ? a.chunks : 32;
    const int slots = 32 / a.lanes_head;
    // Heads side by side: the fewest that leave a lane no more than kPasses of them, so that
    // a voxel's sines serve as many heads as may be; the rest of the warp takes other voxels
    // (200,000 voxels of 3 x 64 in bf16: 58 us with the 3 heads side by side).
    a.head_slots = 1;
    while (a.head_slots < slots && (slots % a.head_slots != 0 || (a.heads + a.head_slots - 1) / a.head_slots > kN))
        ++a.head_slots;
    a.voxel_slots = slots / a.head_slots;
    // Heads a warp: kPasses a lane, so that a voxel's coordinates and sines are used
    // often, dealt evenly; where that leaves warps without work, one.
    const int64_t warps = (a.n + a.voxel_slots - 1) / a.voxel_slots * a.chunk_blocks;
    const int passes = (a.heads + a.head_slots - 1) / a.head_slots;
    int groups = (passes + kN - 1) / kN;
    if (warps * groups < (int64_t)kSms * 2 * kWarps) groups = passes;  // (times 4 blocks of items: a grid takes it)
    const int per = (passes + groups - 1) / groups;
    a.unit_heads = per * a.head_slots;
    groups = (passes + per - 1) / per;
    const int64_t blocks = (a.n + (int64_t)a.voxel_slots * kWarps - 1) / ((int64_t)a.voxel_slots * kWarps);
    // Four CTAs an SM are resident; more of them, of 12 voxels a warp, follow each other
    // closer than fewer with more voxels: 273,995 voxels of 12 x 64 in bf16 take 158 us on
    // 4 CTAs an SM and 137 us on 32 (7 voxels a warp), 16,934 of 8 x 96 in fp32 20.8 us at
    // 7 voxels a warp and 26.8 us at 2.
    const int64_t resident = ((int64_t)kSms * 4 + groups * a.chunk_blocks - 1) / (groups * a.chunk_blocks);
    const int64_t most = blocks / kVoxels > resident ? blocks / kVoxels : resident;
    if (kSmem > 0) {
        static std::atomic<uint64_t> done{0};
        if (allow_smem(k_rope<T, VE, HALVES>, kSmem, done) != cudaSuccess) return;  // the caller asks why
    }
    k_rope<T, VE, HALVES><<<dim3((unsigned)(blocks < most ? blocks : most), groups * a.chunk_blocks), kRopeThreads, kSmem,
                            st>>>(tab, a, static_cast<const T*>(x), static_cast<T*>(out));
}

// |freq| under 2^64 as the nearest fraction of a turn in units of 2^-64, modulo a turn: the
// double's 53 bits times 1 / (2 pi) to 192 bits, in integers, so that no bit of the
// fraction fades as the frequency grows.
constexpr double kMaxFreq = 0x1p64;
uint64_t turn_of(double freq) {
    static const uint64_t inv_two_pi[3] = {0x36d8a5664f10e410, 0x7f09d5f47d4d3770, 0x28be60db9391054a};  // low word first
    int e = 0;
    const uint64_t m = (uint64_t)ldexp(frexp(fabs(freq), &e), 53);
    const int cut = 128 + 53 - e;  // freq / (2 pi) = m inv_two_pi 2^(e - 53 - 192): bits of the product under 2^-64
    uint64_t p[5] = {};
    for (int i = 0; i < 3; ++i) {
        const unsigned __int128 t = (unsigned __int128)m * inv_two_pi[i] + p[i];
        p[i] = (uint64_t)t;
        p[i + 1] = (uint64_t)(t >> 64);
    }
    if (cut > 256) return 0;
    const int word = cut / 64, bit = cut % 64;
    uint64_t v = bit ? (p[word] >> bit) | (p[word + 1] << (64 - bit)) : p[word];
    v += (p[(cut - 1) / 64] >> ((cut - 1) % 64)) & 1;
    return freq < 0.0 ? 0 - v : v;
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
    RopeTable table = {};
    for (int j = 0; j < pairs; ++j) {
        const int axis = freqs ? axes[j] : j < 3 * per ? j / per : -1;
        const double f = freqs ? freqs[j] : axis < 0 ? 0.0 : pow(base, -(double)(j % per) / per);
        if (!(fabs(f) < kMaxFreq) || axis < -1 || axis > 2)
            return row_fail(SPCONV_ERR_INVALID_ARG,
                            freqs ? "freqs must be under 2^64 in magnitude and axes in [-1, 2]"
                                  : "base makes a frequency of 2^64 or more");
        table.turn[j] = axis < 0 ? 0 : turn_of(f);
        table.axis[j] = (int8_t)axis;
    }
    spconv_rope_s* r = new (std::nothrow) spconv_rope_s();
    if (!r) return row_fail(SPCONV_ERR_OOM, "host allocation failed");
    r->head_dim = head_dim;
    r->layout = layout;
    r->table = table;
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
    if (heads < 1 || heads > 4096) return row_fail(SPCONV_ERR_INVALID_ARG, "heads must be in [1, 4096]");
    const int64_t d = rope->head_dim, limit = int64_t(1) << 40;
    // heads and rows of one tensor must not share elements; either may be the outer one
    // (a stride over one element is not used, and taken as head_dim here)
    if (n <= 1) x_row = out_row = d;
    if (heads == 1) x_head = out_head = d;
    if (x_row < d || out_row < d || x_head < d || out_head < d || x_row > limit || out_row > limit || x_head > limit ||
        out_head > limit)
        return row_fail(SPCONV_ERR_INVALID_ARG, "row and head strides must be in [head_dim, 2^40]");
    // (so that none of the spans below leaves 64 bits)
    if (n > 0 && (x_row > (int64_t(1) << 57) / n || out_row > (int64_t(1) << 57) / n))
        return row_fail(SPCONV_ERR_INVALID_ARG, "n rows must span at most 2^57 elements");
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
