// The per-voxel linear layer (kernel size 1) on 4-bit weights with group scales,
// for few rows: single tokens, modulation vectors, small latent sets.
//
//   w[k, o] = scales[o, g] * q[o, k] + offsets[o, g],  g = k / group,  q in 0 .. 15
//   out[i, o] = bias[o] + x_scale[i] * sum_k w[k, o] x[i, k]
//
// The sums are kept in fp32 and rounded once.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "row_ops.cuh"

namespace spconv {
namespace {

// D += A B (FIRST: D = A B) on a 16 x 8 tile over 16 channels, with fp32 accumulation.
template <bool FIRST>
__device__ __forceinline__ void mma_tile(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
    if (FIRST)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool FIRST>
__device__ __forceinline__ void mma_tile(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
    if (FIRST)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The codes i and i + 4 of a word as two 16-bit floats, and how the sums over them are
// read.  With f(q) what a code becomes, a group gives  sum w x = scale sum f(q) x +
// offset sum x.
//
// Rows of e4m3 run in fp16, whose numbers under 2^-14 are spaced evenly: the bits of q
// in the lowest places are q 2^-24, four places up 16 q 2^-24, so a code needs one mask
// (and every other pair a shift); the pairs four places up meet x / 16, which fp16 holds.
// (The same in e4m3's own steps of 32 channels would take fewer masks, but those steps run
// as conversions and two fp16 steps: a tenth slower for 8 rows through 8192 x 16384.)
template <typename X>
struct Codes {
    using Elem = __half;
    static constexpr uint32_t kOne[2] = {0x3c003c00u, 0x4c004c00u};  // 1 and 16
    __device__ static uint32_t part(uint32_t w, int i) {
        return (i < 2 ? w : w >> 8) & (i & 1 ? 0x00f000f0u : 0x000f000fu);
    }
    __device__ static float scale(float s) { return s * 16777216.0f; }
    __device__ static float offset(float, float z) { return z; }
};
// Rows of bf16: q in the low mantissa bits of 128 makes 128 + q.  A group's sums are then
// rounded at 2^-24 of 128 |x| a channel, far under the result's own 2^-8; taking 128 off first
// would be exact and cost four more instructions a word.
template <>
struct Codes<__nv_bfloat16> {
    using Elem = __nv_bfloat16;
    static constexpr uint32_t kOne[2] = {0x3f803f80u, 0x3f803f80u};
    __device__ static uint32_t part(uint32_t w, int i) { return ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u; }
    __device__ static float scale(float s) { return s; }
    __device__ static float offset(float s, float z) { return fmaf(-128.0f, s, z); }
};
// Rows of fp32: 136 taken off, exactly, so the sums run on -8 .. 7.
template <>
struct Codes<float> {
    using Elem = __nv_bfloat16;
    static constexpr uint32_t kOne[2] = {0x3f803f80u, 0x3f803f80u};
    __device__ static uint32_t part(uint32_t w, int i) {
        const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __float2bfloat162_rn(136.0f));
        return *reinterpret_cast<const uint32_t*>(&q);
    }
    __device__ static float scale(float s) { return s; }
    __device__ static float offset(float s, float z) { return fmaf(8.0f, s, z); }
};

// A lane's share of a group of a row of x: W words of 8 neighbouring elements, each word
// as the pairs (x0, x4), (x1, x5), (x2, x6), (x3, x7) that meet the codes of a word, in
// kParts 16-bit floats each whose sum is x.
template <typename X, int W>
struct XShare;
template <int W>
struct XShare<__nv_bfloat16, W> {
    static constexpr int kParts = 1;
    uint4 v[W];
    __device__ void load(const __nv_bfloat16* p, bool in) {
#pragma unroll
        for (int w = 0; w < W; ++w) v[w] = in ? reinterpret_cast<const uint4*>(p)[w] : make_uint4(0, 0, 0, 0);
    }
    __device__ void pair(int w, int i, uint32_t (&to)[1]) const {
        to[0] = __byte_perm(i < 2 ? v[w].x : v[w].y, i < 2 ? v[w].z : v[w].w, i & 1 ? 0x7632 : 0x5410);
    }
};
template <int W>
struct XShare<__nv_fp8_e4m3, W> {
    static constexpr int kParts = 1;
    uint32_t v[2 * W];
    __device__ void load(const __nv_fp8_e4m3* p, bool in) {
        if (W % 2 == 0) {
#pragma unroll
            for (int w = 0; w < W / 2; ++w) {
                const uint4 u = in ? reinterpret_cast<const uint4*>(p)[w] : make_uint4(0, 0, 0, 0);
                v[4 * w] = u.x, v[4 * w + 1] = u.y, v[(4 * w + 2) % (2 * W)] = u.z, v[(4 * w + 3) % (2 * W)] = u.w;
            }
        } else {
            const uint2 u = in ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
            v[0] = u.x, v[1] = u.y;
        }
    }
    __device__ void pair(int w, int i, uint32_t (&to)[1]) const {
        const uint32_t two = __byte_perm(v[2 * w], v[2 * w + 1], i | ((i + 4) << 4));
        uint32_t r;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
        if (i & 1) {  // meets 16 q
            const __half2 v16 = __hmul2(*reinterpret_cast<const __half2*>(&r), __float2half2_rn(0.0625f));
            r = *reinterpret_cast<const uint32_t*>(&v16);
        }
        to[0] = r;
    }
};
template <int W>
struct XShare<float, W> {
    // Three bf16 parts, each the leading 8 bits (cut, so the next is exact): 24 bits in all.
    static constexpr int kParts = 3;
    float v[8 * W];
    __device__ void load(const float* p, bool in) {
#pragma unroll
        for (int w = 0; w < 2 * W; ++w)
            *reinterpret_cast<float4*>(v + 4 * w) =
                in ? reinterpret_cast<const float4*>(p)[w] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    // (an infinity has one part: what it less itself would be is no number)
    __device__ static void split(float x, uint32_t (&part)[3]) {
        const float most = 3.402823466e38f;
        part[0] = __float_as_uint(x);
        const float rest = fabsf(x) <= most ? x - __uint_as_float(part[0] & 0xffff0000u) : 0.0f;
        part[1] = __float_as_uint(rest);
        part[2] = __float_as_uint(rest - __uint_as_float(part[1] & 0xffff0000u));
    }
    __device__ void pair(int w, int i, uint32_t (&to)[3]) const {
        uint32_t a[3], b[3];
        split(v[8 * w + i], a);
        split(v[8 * w + i + 4], b);
#pragma unroll
        for (int p = 0; p < 3; ++p) to[p] = __byte_perm(a[p], b[p], 0x7632);  // the upper halves
    }
};

// A launch's shape.  NT: blocks of 8 rows a CTA holds; then, of the 65,536 registers of
// an SM, kChunk input channels of x, the sums of MT tiles of 16 outputs and the next
// channels of x fit kWarps warps (fp32 rows take three parts each).
template <typename X, int NT>
struct W4Shape {
    static constexpr int kChunk = NT == 4 || sizeof(X) == 4 ? 64 : 128;
    static constexpr int kMostTiles = sizeof(X) == 4 ? 2 : 8;
    static constexpr int kWarps = NT == 1 && sizeof(X) < 4 ? 16 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kSteps = 8;  // steps (a tile of a chunk) whose codes are on the way
    static constexpr int kRingBytes = kSteps * 2 * (kChunk / 8) * kThreads;
};
// Of an output's scales (and offsets) a CTA holds 256 bytes at a time, 16 more apart, so
// that eight outputs' reads fall on different banks.
constexpr int kW4SegBytes = 256, kW4Pitch = kW4SegBytes + 16;

struct W4Params {
    const float* x_scale;
    int n, cin, cout;
    int tiles;        // tiles of 16 outputs a CTA
};

// A CTA multiplies up to MT tiles of 16 outputs by 8 NT rows.  A warp takes every
// kWarps-th chunk of the input channels: it holds the chunk's part of x in registers, as
// the tensor-core operand, and streams the tiles' codes past it; the warps' sums are
// joined in shared memory at the end.  The codes of the next eight steps are on their way
// into shared memory (a lane copies for its own output alone, so no warp waits for
// another) and the next chunk's x into registers.
//
// What bounds it.  8 e4m3 rows through 8192 x 16384, groups of 128, take 16.9 us, 4.2 TB/s
// of codes and scales or 65 % of a plain copy's rate; bf16 rows 22.3 us, with groups of 64
// 24.3 us.  No unit is full: the integer pipe is busiest (49 %, for 16 bf16 rows 50 %), the
// tensor pipe has 28 (32) %, half of the issue slots are used.  One CTA of 16 warps an SM
// spends 21 % of its time before the first step (first scales and codes on their way), 70 %
// in the steps and 8 % in the join (7,100, 23,200 and 2,600 of 33,000 cycles, measured by
// stamps), and in the steps its warps wait for their own chains of them.  For bf16 making
// operands of the codes (7 instructions a word of 8) is 5 us and the scales are 2.4 us,
// measured by leaving them out.  More rows bring more steps and scaled sums a code: 16 bf16
// rows 29.5 us, 32 rows through 4096 x 16384 27.0 us.  One row through 4096 x 4096: 5.7 us,
// 27 % of a CTA's time before the first step, 65 % in four steps a warp, 8 % in the join.  Fewer tiles a
// CTA (two: 43 us for 8 bf16 rows), and a warp that holds codes and reads x anew for every
// tile (44 us), are slower.  The steps are the 16-channel ones that take operands from
// registers.  tcgen05 would take the codes' operands from tensor or shared memory, so that
// the threads that make them would also write them there, at four times the codes' size, and
// it would save the tensor steps' issue alone, which is not what bounds it; and the sums of
// each group would have to be read back from tensor memory before its scales.
//
// Fragments.  In one 16 x 8 x 16 step lane (g, t) = (lane / 4, lane % 4) holds four
// input channels of outputs g and g + 8 and of row g; which four is free as long as both
// operands agree.  A group's scale must be common to the step, so of a part of kSub
// channels (a group, or as much of it as a chunk has) lane t owns the words
// [t W, t W + W), W = kSub / 32, neighbouring in memory, and each word gives two steps.
// Channels behind the last are zeros of x, whatever their codes (all codes are finite).
//
// Scales.  Over a part the sum of f(q) x is the step's accumulator, started at zero for
// each part; the sum of x comes out of the same instruction with ones in place of the
// codes, once for all tiles.  The CTA's scales are brought into shared memory along the
// groups, as they lie in memory; read per lane from global memory, each of them would
// cost a cache line's lookup.
template <typename T, typename X, int NT, int MT, int GROUP>
__global__ void __launch_bounds__(W4Shape<X, NT>::kThreads)
    k_linear_w4(const X* __restrict__ x, const uint32_t* __restrict__ packed, const T* __restrict__ scales,
                const T* __restrict__ offsets, const T* __restrict__ bias, T* __restrict__ out, const W4Params a) {
    using S = W4Shape<X, NT>;
    using C = Codes<X>;
    using Elem = typename C::Elem;
    constexpr int kOps = 4;  // operand registers a word
    constexpr int kChunk = S::kChunk, kSub = GROUP < kChunk ? GROUP : kChunk, kW = kSub / 32, kSubs = kChunk / kSub;
    constexpr int kLane = kChunk / 32;  // words a lane has of an output's chunk
    constexpr int kThreads = S::kThreads, kWarps = S::kWarps, kRounds = S::kSteps / MT, kSeg = kW4SegBytes / (int)sizeof(T);
    using Share = XShare<X, kW>;
    constexpr int kParts = Share::kParts;
    constexpr uint32_t kHalfBytes = kThreads * kLane * 4, kSlotBytes = 2 * kHalfBytes;
    extern __shared__ __align__(16) unsigned char smem[];
    // [slot][output half][warp][output][words], then [scale, offset][output][group of the segment].
    // A lane copies the words [t kLane, ...) of its output's chunk and reads words [t W, ...)
    // of each part; where these differ (groups shorter than the chunk) the lanes of an output
    // read each other's copies, and its 16-byte pieces change places by the output so that
    // eight outputs' reads fall on different banks.
    constexpr bool kShared = kLane == 4 && kW < 4;
    const int turn = !kShared ? 0 : kW == 2 ? ((threadIdx.x >> 3) & 1) * 2 : (threadIdx.x >> 3) & 3;  // (g >> 1)
    unsigned char* ring = smem + (threadIdx.x / 4) * (kLane * 16);  // this lane's output's
    const uint32_t ring_at = shared_at(ring) + ((threadIdx.x & 3) ^ turn) * (kLane * 4);
    unsigned char* table = smem + S::kRingBytes;
    constexpr int kOffsets = MT * 16 * kW4Pitch;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int words = a.cin / 8, groups = a.cin / GROUP, chunks = (a.cin + kChunk - 1) / kChunk;
    const int o0 = blockIdx.x * a.tiles * 16, row0 = blockIdx.y * NT * 8;
    const int tiles = min(a.tiles, (a.cout - o0 + 15) / 16);
    float y[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[m][b][e] = 0.0f;

    // Codes of tile m of a chunk, kRounds rounds before their turn and into the slot that
    // their turn reads.
    const int my_outs = a.cout - o0 - g;
    const int64_t tile_words = 16 * (int64_t)words;
    constexpr int kCopies = kShared ? 1 : kSubs, kCopy = kLane / kCopies;  // copies an output, words a copy
    const uint32_t* next = packed + (int64_t)(o0 + g) * words + warp * (kChunk / 8) + t * kCopy;  // this lane's, tile 0
    int next_word = warp * (kChunk / 8) + t * kCopy;
    const auto fetch = [&](int m, int slot) {
        if (m < tiles) {
            const uint32_t* from = next + m * tile_words;
            const uint32_t to = ring_at + slot * kSlotBytes;
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                if (next_word + j * (kSub / 8) < words) {
                    if (m * 16 < my_outs) copy_async<4 * kCopy>(to + j * (kCopy * 4), from + j * (kSub / 8));
                    if (m * 16 + 8 < my_outs)
                        copy_async<4 * kCopy>(to + kHalfBytes + j * (kCopy * 4), from + 8 * words + j * (kSub / 8));
                }
            }
        }
        copy_commit();
    };
    const auto next_chunk = [&]() {
        next += kWarps * (kChunk / 8);
        next_word += kWarps * (kChunk / 8);
    };
    // A segment's scales: on their way with the codes, in the largest pieces that the rows
    // of the scales start on (single bf16 scales are too small to copy).
    const auto copy_scales = [&](int seg, int held, auto bytes) {
        constexpr int kBytes = decltype(bytes)::value, kElems = kBytes / (int)sizeof(T);
        const int rows = min(tiles * 16, a.cout - o0), pieces = held / kElems;
        for (int o = threadIdx.x / 16; o < rows; o += kThreads / 16) {
            const int64_t from = (int64_t)(o0 + o) * groups + seg;
            const uint32_t to = shared_at(table + o * kW4Pitch);
#pragma unroll 2
            for (int e = threadIdx.x % 16; e < pieces; e += 16) {
                copy_async<kBytes>(to + e * kBytes, scales + from + e * kElems);
                copy_async<kBytes>(to + kOffsets + e * kBytes, offsets + from + e * kElems);
            }
        }
    };
    const auto fetch_scales = [&](int seg, int held) {
        if (groups * (int)sizeof(T) % 16 == 0) {
            copy_scales(seg, held, std::integral_constant<int, 16>());
        } else if (groups * (int)sizeof(T) % 4 == 0) {
            copy_scales(seg, held, std::integral_constant<int, 4>());
        } else {
            const int rows = min(tiles * 16, a.cout - o0);
#pragma unroll 4
            for (int e = threadIdx.x; e < rows * held; e += kThreads) {
                const int o = e / held, k = e - o * held;
                const T s = scales[(int64_t)(o0 + o) * groups + seg + k], z = offsets[(int64_t)(o0 + o) * groups + seg + k];
                reinterpret_cast<T*>(table + o * kW4Pitch)[k] = s;
                reinterpret_cast<T*>(table + kOffsets + o * kW4Pitch)[k] = z;
            }
        }
    };
    // The first scales before the first codes: the work can begin when one step is there.
    fetch_scales(0, min(kSeg, groups));
    copy_commit();
#pragma unroll
    for (int d = 0; d < kRounds; ++d) {
#pragma unroll
        for (int m = 0; m < MT; ++m) fetch(m, d * MT + m);
        next_chunk();
    }
    const auto load_x = [&](Share (&xs)[NT][kSubs], int chunk) {
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int j = 0; j < kSubs; ++j) {
                const int row = row0 + b * 8 + g, k = chunk * kChunk + j * kSub + t * kW * 8;
                xs[b][j].load(x + (int64_t)row * a.cin + k, row < a.n && k < a.cin);
            }
    };
    Share raw[NT][kSubs];
    load_x(raw, warp);

    int base = 0, chunk = warp;  // base: the round's first slot
    for (int seg = 0; seg < groups; seg += kSeg) {
        const int held = min(kSeg, groups - seg);
        if (seg == 0) {
            copy_wait<S::kSteps>();
        } else {
            __syncthreads();
            fetch_scales(seg, held);
            copy_commit();
            copy_wait<0>();
        }
        __syncthreads();
        for (; chunk < chunks && chunk * kChunk < (seg + held) * GROUP; chunk += kWarps) {
            uint32_t pairs[NT][kSubs][kW][kOps][kParts];
            float sum[NT][kSubs][4];
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int j = 0; j < kSubs; ++j) {
                    const uint32_t ones[4] = {C::kOne[0], C::kOne[0], C::kOne[1], C::kOne[1]};
#pragma unroll
                    for (int i = 0; i < kW; ++i) {
#pragma unroll
                        for (int e = 0; e < kOps; ++e) raw[b][j].pair(i, e, pairs[b][j][i][e]);
#pragma unroll
                        for (int p = 0; p < kParts; ++p)
#pragma unroll
                            for (int h = 0; h < kOps; h += 2) {
                                if (i == 0 && p == 0 && h == 0)
                                    mma_tile<true>(sum[b][j], ones, pairs[b][j][i][h][p], pairs[b][j][i][h + 1][p], Elem());
                                else
                                    mma_tile<false>(sum[b][j], ones, pairs[b][j][i][h][p], pairs[b][j][i][h + 1][p], Elem());
                            }
                    }
                }
            if (chunk + kWarps < chunks) load_x(raw, chunk + kWarps);
            const int at = chunk * kChunk / GROUP - seg;  // the chunk's first group in the segment
            const unsigned char* of_chunk = table + g * kW4Pitch + at * (int)sizeof(T);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                copy_wait<S::kSteps - 1>();
                if (m < tiles) {
                    const unsigned char* from_slot = ring + (base + m) * kSlotBytes;
                    Vec<uint32_t, kLane> w[2];
                    if (kShared) __syncwarp();  // the other lanes' copies have come, too
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (kShared) {
#pragma unroll
                            for (int j = 0; j < kSubs; ++j) {
                                // word j kSub / 8 + t W: the piece of 16 bytes that holds it, and its place there
                                const int piece = (j * kW + (t * kW) / 4) ^ turn, in = (t * kW) % 4;
                                const auto v = *reinterpret_cast<const Vec<uint32_t, kW>*>(
                                    from_slot + r * kHalfBytes + piece * 16 + in * 4);
#pragma unroll
                                for (int i = 0; i < kW; ++i) w[r].v[j * kW + i] = v.v[i];
                            }
                        } else {
                            w[r] = *reinterpret_cast<const Vec<uint32_t, kLane>*>(from_slot + r * kHalfBytes + t * (kLane * 4));
                        }
                    }
                    Vec<T, kSubs> sv[2], zv[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const unsigned char* p = of_chunk + (m * 16 + r * 8) * kW4Pitch;
                        sv[r] = *reinterpret_cast<const Vec<T, kSubs>*>(p);
                        zv[r] = *reinterpret_cast<const Vec<T, kSubs>*>(p + kOffsets);
                    }
#pragma unroll
                    for (int j = 0; j < kSubs; ++j) {
                        float d[NT][4];
#pragma unroll
                        for (int i = 0; i < kW; ++i)
#pragma unroll
                            for (int h = 0; h < kOps; h += 2) {
                                const uint32_t w0 = w[0].v[j * kW + i], w1 = w[1].v[j * kW + i];
                                const uint32_t code[4] = {C::part(w0, h), C::part(w1, h), C::part(w0, h + 1), C::part(w1, h + 1)};
#pragma unroll
                                for (int p = 0; p < kParts; ++p)
#pragma unroll
                                    for (int b = 0; b < NT; ++b) {
                                        if (i == 0 && h == 0 && p == 0)
                                            mma_tile<true>(d[b], code, pairs[b][j][i][h][p], pairs[b][j][i][h + 1][p], Elem());
                                        else
                                            mma_tile<false>(d[b], code, pairs[b][j][i][h][p], pairs[b][j][i][h + 1][p], Elem());
                                    }
                            }
                        if (j > 0 && at + j >= held) continue;  // behind the last group
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float s = to_f32(sv[r].v[j]), sc = C::scale(s), of = C::offset(s, to_f32(zv[r].v[j]));
#pragma unroll
                            for (int b = 0; b < NT; ++b)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    float& to = y[m][b][2 * r + e];
                                    to = fmaf(sc, d[b][2 * r + e], fmaf(of, sum[b][j][e], to));
                                }
                        }
                    }
                }
                if (kShared) __syncwarp();
                fetch(m, base + m);  // the slot's codes have been used
            }
            next_chunk();
            base = base + MT == S::kSteps ? 0 : base + MT;
        }
    }
    copy_wait<0>();  // the ring becomes the join's memory
    __syncthreads();
    float (*join)[MT * 16][NT * 8 + 1] = reinterpret_cast<float (*)[MT * 16][NT * 8 + 1]>(smem);
    // accumulator e of lane (g, t): output g + 8 (e / 2), row 2 t + e % 2
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m >= tiles) continue;
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) join[warp][m * 16 + (e >> 1) * 8 + g][b * 8 + 2 * t + (e & 1)] = y[m][b][e];
    }
    __syncthreads();
    const int outs = min(tiles * 16, a.cout - o0), live = min(NT * 8, a.n - row0);
    for (int o = threadIdx.x % (MT * 16); o < outs; o += MT * 16)
        for (int r = threadIdx.x / (MT * 16); r < live; r += kThreads / (MT * 16)) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v += join[k][o][r];
            if (a.x_scale) v *= a.x_scale[row0 + r];
            if (bias) v += to_f32(bias[o0 + o]);
            out[(int64_t)(row0 + r) * a.cout + o0 + o] = from_f32<T>(v);
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

struct W4Args {
    const void *x, *packed, *scales, *offsets, *bias;
    void* out;
    W4Params p;
    cudaStream_t stream;
};

template <typename T, typename X, int NT, int MT, int GROUP>
void launch_w4_tiles(W4Args a, int tiles) {
    using S = W4Shape<X, NT>;
    static_assert(kW4SegBytes / sizeof(T) % (S::kChunk > GROUP ? S::kChunk / GROUP : 1) == 0, "segments hold whole chunks");
    constexpr int join = S::kWarps * MT * 16 * (NT * 8 + 1) * 4, work = S::kRingBytes + 2 * MT * 16 * kW4Pitch;
    constexpr int smem = work > join ? work : join;
    static_assert(smem <= 227 * 1024, "fits an SM");
    static std::atomic<uint64_t> done{0};
    if (allow_smem(k_linear_w4<T, X, NT, MT, GROUP>, smem, done) != cudaSuccess) return;  // the caller asks why
    const dim3 grid((tiles + a.p.tiles - 1) / a.p.tiles, (a.p.n + 8 * NT - 1) / (8 * NT));
    k_linear_w4<T, X, NT, MT, GROUP><<<grid, S::kThreads, smem, a.stream>>>(
        static_cast<const X*>(a.x), static_cast<const uint32_t*>(a.packed), static_cast<const T*>(a.scales),
        static_cast<const T*>(a.offsets), static_cast<const T*>(a.bias), static_cast<T*>(a.out), a.p);
}

// Tiles a CTA: the most that its registers hold, dealt so that the SMs' shares differ by
// one tile at most.  With one or two, the codes of more chunks are on the way.
template <typename T, typename X, int NT, int GROUP>
void launch_w4_rows(W4Args a) {
    constexpr int kMost = W4Shape<X, NT>::kMostTiles;
    const int tiles = (a.p.cout + 15) / 16, waves = (tiles + kSms * kMost - 1) / (kSms * kMost);
    a.p.tiles = (tiles + kSms * waves - 1) / (kSms * waves);
    if constexpr (kMost > 2) {
        if (a.p.tiles > 2) return launch_w4_tiles<T, X, NT, kMost, GROUP>(a, tiles);
    }
    launch_w4_tiles<T, X, NT, 2, GROUP>(a, tiles);
}

// Rows a CTA: all of them, so that the weights are read once; fp32 rows go 8 at a time.
template <typename T, typename X, int GROUP>
void launch_w4_group(const W4Args& a) {
    if constexpr (sizeof(X) == 4) {
        launch_w4_rows<T, X, 1, GROUP>(a);
    } else {
        if (a.p.n <= 8)
            launch_w4_rows<T, X, 1, GROUP>(a);
        else if (a.p.n <= 16)
            launch_w4_rows<T, X, 2, GROUP>(a);
        else
            launch_w4_rows<T, X, 4, GROUP>(a);
    }
}

template <typename T, typename X>
void launch_linear_w4(const W4Args& a, int group) {
    if (group == 32)
        launch_w4_group<T, X, 32>(a);
    else if (group == 64)
        launch_w4_group<T, X, 64>(a);
    else
        launch_w4_group<T, X, 128>(a);
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
    W4Args a = {x, packed, scales, offsets, bias, out, {}, static_cast<cudaStream_t>(stream)};
    a.p.x_scale = x_scale;
    a.p.n = (int)n;
    a.p.cin = cin;
    a.p.cout = cout;
    if (dtype == SPCONV_BF16 && x_scale)
        launch_linear_w4<__nv_bfloat16, __nv_fp8_e4m3>(a, group);
    else if (dtype == SPCONV_BF16)
        launch_linear_w4<__nv_bfloat16, __nv_bfloat16>(a, group);
    else if (x_scale)
        launch_linear_w4<float, __nv_fp8_e4m3>(a, group);
    else
        launch_linear_w4<float, float>(a, group);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPCONV_OK : row_fail_cuda(e, "spconv_linear_w4");
}

}  // extern "C"
