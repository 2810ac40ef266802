// moe_experts.cu -- bf16 products grouped by expert over ragged receive rows
// ("Balancing and Beyond", section 1: the experts between dispatch and
// combine).
//
// One persistent kernel per product, two CTAs (a pair) on one tile of sums.  The
// weights take the 256 rows of the tensor core's product and the receive rows its
// columns, because the columns can be any multiple of 16: an expert's rows are cut
// into equal tiles, and no more than 15 columns of a tile are computed in vain,
// whether an expert has one row or thousands.
//
//   forward             sums[feature][row]   = W rows^T       W, rows along the contraction
//   gradient of rows    sums[column][row]    = W^T dout^T     W across it
//   gradient of weights sums[w][column]      = dout^T rows    both across it (rows are summed)
//
// Eighteen warps a CTA: one feeds a ring of shared-memory stages with tensor copies
// (128 bytes along memory, 128-byte swizzle), one of the pair issues the products,
// four groups of four turn finished sums into results while the next tile is
// computed: tiles take the two ends of tensor memory in turn, and where two do not
// fit beside each other the shared columns are stored first.  A result row runs
// along the lanes of tensor memory, so the store half turns 16 columns at a time
// through shared memory, in fp32: activations see unrounded sums, and a result row
// is written 256 bytes at a time.
//
// With a gated activation the 128 weight rows of a CTA are 64 gate rows and the 64
// up rows of the same features.
//
// Ragged groups.  The host knows only how many rows there are in all; every CTA
// counts the row tiles of each expert from the layout's counts (a scan over at
// most 1024 experts) and the pairs take tiles pair, pair + pairs, ... of that
// list.  Within an expert row tiles go first, so that the pairs that share a piece
// of its weights run at the same time and it comes from HBM once.  Columns of
// neighbours that a copy reaches into only make sums that nobody stores; where
// rows are summed (weights' gradient) they are cleared in shared memory first.
//
// Few tiles and a long contraction: two or four pairs of a cluster share a tile,
// each over its part of the contraction, and its CTAs' store halves add the parts up
// through distributed shared memory, in part order.
//
// What bounds it.  Few rows an expert: HBM (the weights arrive at 7.0 TB/s).  Many rows, forward: the stages, which arrive
// at up to 54 bytes a clock and SM (16 KB of weights and 16 KB of rows against 512 clocks of products for 256
// columns), and then the power limit: 1024 rows of 32 experts, 7168 -> 2048, run at 1800 TFLOP/s in a burst (the
// library's plain bf16 product: 1920) and 1.4 PFLOP/s in a long run (1690).  Over a whole launch of a few rounds of tiles
// the other products are at neither bound: 44 bytes a clock and SM and 67 % of the tensor pipe for the rows' gradient (which
// reads and writes (g, u) besides), 45 and 71 % for the weights' gradient, 31 and 51 % in 4 bits, where a stage of 256
// columns is 35 KB for 512 clocks: a stage in some 740 clocks, and in 620 with a quarter of its products.  What
// holds the stages back was looked for and not found.  It is not L2: two pairs
// that share their rows by multicast, a quarter fewer bytes out of L2, fill their stages no faster (and clusters of four
// CTAs leave 8 SMs idle: 681 -> 705 us at 272 rows of 64 experts).  Nor is it one warp's issuing: a second copying warp
// changed nothing in 4 bits.  Keeping the weights beside the tensor core between the two products of a wide tile did not
// either (in 16 bits 583 -> 573 us at 1040 rows cut at 320, where 256 columns take 554).
// Nor do earlier requests help: prefetching weights into L2 8 to 20 stages ahead took 685 -> 707 us and more, marking
// them as first to leave it 675 -> 696 us, fetching 128 bytes at a time instead of 256 675 -> 702 us.  Taking 4-bit
// scales to tensor memory one stage early, by the same warp (406 us) or by one of its own (368 us), measured slower than
// between the products (333 us then; 32768 rows of 32 experts, 7168 -> 2 x 2048).
//
// 8-bit integers.  The chip multiplies them far slower than fp16, which holds them exactly, so other warps of a CTA widen
// what the copies bring, weights to tensor memory (a lane a row) and rows to shared memory, and the products take A
// from the one and B from the other.  Beside the copying and the multiplying warp a CTA has one group of four that store and
// sixteen that widen, twenty-two warps; where a contraction is short and tiles are wide, three groups and eight, also twenty-two.  Weights in tensor memory, because shared memory would be written and read 32 KB a
// stage more; sums have 384 of its columns then.  A decode reads half the bytes of bf16 weights (16 tokens, top-8 of 128,
// 7168 -> 2 x 2048: 405 us, 6.0 TB/s, and 714 in the same run); a prefill is at the same power limit (4096 tokens, top-8 of
// 32: 1180 us, 1.63 PFLOP/s).  What the steps there measured (decode, prefill; us): 64 x 64 tiles on the CUDA cores 5245,
// 32670; eight widening warps 919, 1860; sixteen, stages in turn 627, 1220; the multiplying warp waiting for a stage, not for
// half of one 517, 1230; one store group, so that a thread has 80 registers and not 72, 424, 1190; four pieces in flight, not
// eight 411, 1185.  The copies alone take 361 and 458, all but the widening 388 and 983.
//
// Every wait is bounded.  A CTA whose wait gives up records a fault, waits for its
// own copies and products, frees its tensor memory and returns.

#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "moe_clusters.cuh"
#include "moe_experts.cuh"
#include "moe_tc.cuh"

namespace moe {
namespace {

__device__ unsigned int g_expert_faults;

constexpr int kForward = 0, kBackRows = 1, kBackWeights = 2, kForward4 = 3, kForward8 = 4, kShort8 = 5;
template <int OP>                      // integers: a long contraction, or one that the store half would not keep up with
constexpr bool kIntegers = OP == kForward8 || OP == kShort8;
template <int OP>
constexpr int kGroups = OP == kForward8 ? 1 : OP == kShort8 ? 3 : 4;  // of four warps that store
template <int OP>
constexpr int kTailWarp = 2 + 4 * kGroups<OP>;
template <int OP>                      // warps that widen integers: four for either half of a stage, or eight, stages in turn
constexpr int kWideners = OP == kForward8 ? 16 : 8;
template <int OP>
constexpr bool kInTurn = kWideners<OP> > 8;
template <int OP>                      // warp 0 copies, warp 1 multiplies; in the weights' gradient one more clears
constexpr int kThreads = 32 * (kTailWarp<OP> + (OP == kBackWeights ? 1 : kIntegers<OP> ? kWideners<OP> : 0));
constexpr int kHalf = 128;             // rows of the sums in one CTA
constexpr int kColumns = 256;          // most columns of one product instruction
constexpr int kFirst = 128;            // a wider tile is two products: this many columns, and the others
template <int OP>
constexpr int kTop = OP == kForward4 ? 448 : kIntegers<OP> ? 384 : 512;  // columns of tensor memory for sums
constexpr int kRowBytes = 128;         // of a stage, along memory
template <int OP>
constexpr int kStep = OP == kForward4 ? 2 * kRowBytes : kIntegers<OP> ? kRowBytes : kRowBytes / 2;  // its contraction
constexpr int kBoxBytes = 64 * kRowBytes;
constexpr int kBytesA = kHalf * kRowBytes;
template <int OP>
constexpr int kRingBytes = (OP == kForward4 ? 176 : OP == kForward8 ? 195 : OP == kShort8 ? 178 : 180) * 1024;
constexpr int kStages = 12;            // most stages in flight
constexpr int kTurn = 16;              // columns turned at a time
constexpr int kTurnPitch = kHalf + 4;  // floats: rows of the turned block start 16 bytes apart in the banks
constexpr int kTurnBytes = 4 * kTurn * kTurnPitch;
template <int OP>                      // 1024: alignment; in 4 bits also the experts' first scale blocks
constexpr int kSmem = kRingBytes<OP> + kGroups<OP> * kTurnBytes + 1024 + (OP == kForward4 ? 4 * (MOE_MAX_EXPERTS + 4) : 0);

// 4-bit stages end with the scales of 256 codes: 1 KB (two scale blocks along a row) of the weights' 128 rows and of
// every 128 receive rows the tile touches (tiles start at multiples of 64 rows: one of up to 256 touches two, of up to
// 384 three); the products take them from tensor memory above the sums.
constexpr int kScaleBlock = 512;
constexpr int scale_bytes(int columns) { return (columns > 256 ? 4 : 3) * 2 * kScaleBlock; }
constexpr uint32_t kScalesA = kTop<kForward4>, kScalesB = kScalesA + 8;

// 8-bit integers are widened to fp16 (exactly) between copy and product, in pieces of 64 of the contraction: a stage holds
// two.  The weights' pieces lie in tensor memory above the sums, the rows' in shared memory behind the stages.
constexpr int kPieces = 4, kPiece = 64, kPieceColumns = kPiece / 2;
static_assert(kTop<kForward8> + kPieces * kPieceColumns == 512 && kPieces % 4 == 0);

struct Shared {
    uint64_t full[kStages], empty[kStages], done[2], free[2], over[2], last, tail[kStages];
    uint64_t ready[4], seen[4];        // of a store group's block, by the parts of a tile
    uint64_t made[kPieces / 2], used[kPieces];  // pieces of widened integers, two made together
    uint32_t tmem;
    int scratch[32];
    int base[MOE_MAX_EXPERTS + 1];
    ExpertRows rows[MOE_MAX_EXPERTS];
};

// How a launch cuts rows and shared memory: a tile has at most `columns` columns,
// and shared memory holds `stages` stages of `bytes` (16 KB of one operand and
// half the columns of the other); `parts` pairs share a tile.
struct Cut {
    int columns, stages, bytes;
    int parts;                         // pairs that share a tile
};

// Where in the ring of stages a thread is.
struct Ring {
    int stage = 0, at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(const Cut& cut) {
        at += cut.bytes;
        if (++stage == cut.stages) {
            stage = at = 0;
            phase ^= 1u;
        }
    }
};

// Receive rows arrive in boxes of 8, 16, 32, 64 and 128 rows (kMaps maps): a tile's share is two boxes at most for
// each of its halves, the largest power of two and the rest rounded up to one.
constexpr int kMaps = 5;
struct Maps {
    CUtensorMap rows[kMaps], weight_scales, row_scales, out;
};
struct Boxes {
    int rows0, rows1;                  // rows1 == 0: one box
    const CUtensorMap *map0, *map1;
    __device__ __forceinline__ int bytes() const { return (rows0 + rows1) * kRowBytes; }
};
__device__ __forceinline__ Boxes boxes_of(const Maps& maps, int rows) {
    Boxes b{0, 0, &maps.rows[0], &maps.rows[0]};
    if (rows == 0) return b;
    const int top = 31 - __clz(rows), rest = rows - (1 << top);
    b.rows0 = 1 << top;
    b.map0 = &maps.rows[top - 3];
    if (rest > 0) {
        const int up = rest <= 8 ? 3 : 32 - __clz(rest - 1);
        b.rows1 = 1 << up;
        b.map1 = &maps.rows[up - 3];
    }
    return b;
}

// A bounded wait of a whole warp: it gives up together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns = kSecond) {
    return __all_sync(0xffffffffu, wait_second(bar, parity, limit_ns)) != 0;
}

// The same for barriers on which other CTAs arrive for memory that they hand over.
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, within(kSecond, [&] { return tc::try_wait_cluster(bar, parity); })) != 0;
}

// One tile of sums.
struct Tile {
    int e;        // expert
    int first;    // its first receive row
    int f0;       // first of the tile's features (result columns; weight rows in the weights' gradient)
    int m0, rows; // its receive rows, inside the expert (columns of the weights' gradient)
    int n;        // rows, rounded up to the tensor core's columns
    int length;   // of the contraction
};

struct Plan {
    int64_t tiles;
    int features;  // in all
    int wide;      // of them in a tile
    int across;    // tiles of features
    int columns;   // most rows of a tile
};

// How long the end of a contraction of so many stages is waited for: the weights' gradient sums over an expert's rows, of
// which there may be so many that this takes seconds (0.23 us a stage; other contractions have 2^14 stages at most).
template <int OP>
__device__ __forceinline__ uint64_t limit_of(int64_t stages) {
    return OP == kBackWeights ? kSecond + 4000ull * stages : kSecond;
}

template <int OP, bool GLU>
__device__ __forceinline__ Plan make_plan(const ExpertArgs& a, const Cut& cut, const int* base) {
    Plan p;
    p.features = OP == kBackWeights ? a.W : OP == kBackRows ? a.K : a.N;
    p.wide = GLU ? kHalf : 2 * kHalf;
    p.across = (p.features + p.wide - 1) / p.wide;
    p.columns = cut.columns;
    p.tiles = (OP == kBackWeights ? (int64_t)a.E * ((a.K + kColumns - 1) / kColumns) : (int64_t)base[a.E]) * p.across;
    return p;
}

template <int OP, bool GLU>
__device__ __forceinline__ Tile tile_at(const ExpertArgs& a, const Plan& p, const Shared& sh, int64_t i) {
    Tile t;
    int down, j, total;
    if (OP == kBackWeights) {
        down = (a.K + kColumns - 1) / kColumns;
        t.e = (int)(i / ((int64_t)down * p.across));
        j = (int)(i - (int64_t)t.e * down * p.across);
    } else {
        t.e = expert_of_block(sh.base, a.E, (int)(i / p.across));
        down = sh.base[t.e + 1] - sh.base[t.e];
        j = (int)(i - (int64_t)sh.base[t.e] * p.across);
    }
    const ExpertRows x = sh.rows[t.e];
    t.first = x.first;
    t.length = OP == kBackWeights ? x.count : OP == kBackRows ? a.W : a.K;
    total = OP == kBackWeights ? a.K : x.count;
    // equal tiles, in sixteens (in 4 bits by half blocks of scales, in the weights' gradient by the blocks it stores)
    constexpr int kUnit = OP == kForward4 ? 64 : OP == kBackWeights ? 32 : 16;
    const int per = min(rows_of_tile(total, down, kUnit), p.columns);  // (more only where the count of tiles has hit its end)
    t.m0 = (j % down) * per;
    t.f0 = (j / down) * p.wide;
    t.rows = min(per, total - t.m0);
    t.n = OP == kBackWeights ? (t.rows + 31) & ~31 : (t.rows + 15) & ~15;
    return t;
}

// ---- the store half ----------------------------------------------------------

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}
// 1 / (1 + exp(-g)); the reciprocal is good to one unit in the last place, small results included.
__device__ __forceinline__ float sigmoid(float g) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-g)));
    return r;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    st_v4(reinterpret_cast<uint4*>(p), make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]),
                                                  pack2(v[6], v[7])));
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 x = ld_stream_v4(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// 8 floats of a turned row; lanes 4 .. 7 of every 8 read their halves the other way round, so that 8 lanes cover all banks.
__device__ __forceinline__ void turned8(const float* p, bool swap, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p + (swap ? 4 : 0));
    const float4 b = *reinterpret_cast<const float4*>(p + (swap ? 0 : 4));
    v[0] = swap ? b.x : a.x; v[1] = swap ? b.y : a.y; v[2] = swap ? b.z : a.z; v[3] = swap ? b.w : a.w;
    v[4] = swap ? a.x : b.x; v[5] = swap ? a.y : b.y; v[6] = swap ? a.z : b.z; v[7] = swap ? a.w : b.w;
}
// 8 sums of integers times their scales; WEIGHTS: times the weights' too, first.
template <bool WEIGHTS>
__device__ __forceinline__ void scale8(float (&v)[8], float row, const float* weights) {
    if (WEIGHTS) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(weights)), b = __ldg(reinterpret_cast<const float4*>(weights) + 1);
        v[0] *= a.x; v[1] *= a.y; v[2] *= a.z; v[3] *= a.w;
        v[4] *= b.x; v[5] *= b.y; v[6] *= b.z; v[7] *= b.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= row;
}

// ---- 8-bit integers to fp16 ------------------------------------------------------

// 4 integers to 4 fp16: a byte under the exponent of 1024 counts in ones, so the integer is that less 1024 + 128 (the method
// of Kim, Henry, Fahim and Hassan Awadalla, "Who Says Elephants Can't Run", 2022, here with signed bytes in order).
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&lo), bias), y = __hsub2(*reinterpret_cast<__half2*>(&hi), bias);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

__device__ __forceinline__ void store_wide(uint4 w, uint32_t lo, uint32_t hi) {
    const uint2 a = widen4(w.x), b = widen4(w.y), c = widen4(w.z), d = widen4(w.w);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(lo), "r"(a.x), "r"(a.y), "r"(b.x), "r"(b.y) : "memory");
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(hi), "r"(c.x), "r"(c.y), "r"(d.x), "r"(d.y) : "memory");
}

// Half `half` of a stage to a piece: of its 128 weight rows a lane takes 64 bytes of one, to tensor memory; of its `rows`
// receive rows 8 lanes take a 16-byte part of 8 rows at a time, to rows of 128 bytes in shared memory.  16-byte parts of a
// row lie swizzled by the row, here and there, so that 8 lanes cover all banks.  The first rows are loaded ahead: with few
// rows only one warp of the four has any, and the others would wait for its second round of latencies.
__device__ __forceinline__ void widen(uint32_t stage, int half, int rows, uint32_t weights, uint32_t piece, int quarter,
                                      int lane) {
    const int row = quarter * 32 + lane, sub = lane & 7, chunk = lane >> 3;
    const uint32_t from = stage + kBytesA + sub * kRowBytes + (((4 * half + chunk) ^ sub) << 4), to = piece + sub * kRowBytes;
    const uint32_t lo = to + (((2 * chunk) ^ sub) << 4), hi = to + (((2 * chunk + 1) ^ sub) << 4);
    const int r1 = 8 * (3 - quarter);
    uint4 ahead = make_uint4(0, 0, 0, 0);
    if (r1 < rows) ahead = lds_v4(from + r1 * kRowBytes);
    uint32_t v[kPieceColumns];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 w = lds_v4(stage + row * kRowBytes + (((4 * half + i) ^ sub) << 4));
        const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint2 x = widen4(b[j]);
            v[8 * i + 2 * j] = x.x;
            v[8 * i + 2 * j + 1] = x.y;
        }
    }
    tc::st32(weights + ((uint32_t)(quarter * 32) << 16), v);
    for (int r0 = r1; r0 < rows; r0 += 32) {
        const uint4 x = ahead;
        if (r0 + 32 < rows) ahead = lds_v4(from + (r0 + 32) * kRowBytes);
        store_wide(x, lo + r0 * kRowBytes, hi + r0 * kRowBytes);
    }
}

// ---- pre-activations kept in 8 bits: e4m3 codes, a power of two (E8M0) for 32 columns ----
//
// Where a result row is written its 32 columns lie on four neighbouring lanes, so a scale takes two exchanges.  Powers of
// two, so that the code's rounding is the only one, 32 columns because that is what one CTA's store half has beside each
// other at any tile, and the least power that saturates nothing: a value is off by half a step however its 32 columns are
// spread.  4096 tokens, top-8 of 32, 7168 -> 2 x 2048: 1238 us in a long run, 1234 with pre in bf16, 1225 without (half the
// bytes of pre, but its arithmetic: 281.7 us for 8192 rows, 258.8 without pre).  Back, 2048 <- 7168: 661 us, 659 from bf16,
// and 681 with the activation made anew, 134 MB (20 us at the copy rate).

// 8 of 32 columns on each of 4 lanes to codes; returns the scale byte: the least power of two with no value over 448 of
// it (448 = 1.75 * 2^8, so a mantissa over 1.75 takes the next).  All lanes of the warp call it.
__device__ __forceinline__ uint32_t keep8(const float (&v)[8], uint2* codes) {
    uint32_t top = 0;                  // magnitudes as integers order as the floats do, infinity and NaN above all
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool bad = top >= 0x7f800000u;
    const uint32_t b = max((top + 0x1fffffu) >> 23, 8u) - 8;
    const float inv = __uint_as_float((254u - min(b, 253u)) << 23);  // 2^(127 - b)
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    *codes = bad ? make_uint2(0u, 0u) : make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    return bad ? 255u : b;
}

// What 8 codes and their scale byte stand for.
__device__ __forceinline__ void kept8(uint2 codes, uint32_t b, float (&v)[8]) {
    const float x = b == 255u ? NAN : __uint_as_float(b == 0u ? 1u << 22 : b << 23);  // 2^(b - 127)
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x * x;
        v[2 * i + 1] = f.y * x;
    }
}

// The 128 threads of a store group (barriers 1 and up).
__device__ __forceinline__ void store_sync(int group) { asm volatile("bar.sync %0, 128;" :: "r"(1 + group) : "memory"); }
// The same, and whether all of them say yes.
__device__ __forceinline__ bool store_all(int group, bool yes) {
    int all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                 "bar.red.and.pred q, %2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                 : "=r"(all) : "r"((int)yes), "r"(1 + group) : "memory");
    return all != 0;
}
// How the store groups of a tile's parts meet, a group with the same one of every other part.
struct Link {
    uint32_t ready, seen;              // barriers of this store group
    uint32_t phase;                    // of both
    int part, parts, cta;
    bool ok;
};
// 8 floats of a turned row, added up over the parts of the tile in their order.
__device__ __forceinline__ void summed8(const float* p, const Link& link, float (&v)[8]) {
    const uint32_t at = smem_u32(p);
    for (int i = 0; i < link.parts; ++i) {
        const uint32_t there = tc::in_rank(at, 2 * i + link.cta);
        const float4 a = tc::load_cluster(there), b = tc::load_cluster(there + 16);
        const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i == 0 ? w[k] : v[k] + w[k];
    }
}

// A finished tile of the weights' gradient: a lane holds a weight row, so that nothing has to be turned.  A store group
// puts 32 columns of its 128 rows into shared memory (64 bytes a row, swizzled so that 8 lanes cover all banks) and a
// tensor copy takes them from there; the result has no ragged side, and the copy leaves out what lies past its ends.
// 16 rows of 64 experts, 1024 x 1024, take 25.1 us; through the turned block and vector stores, as below, they took 36.6
// us, and straight from registers, 32 bytes a lane at the pitch of a row, 51 us.
__device__ __forceinline__ void store_weights(const Plan& p, const Tile& t, const CUtensorMap* map, uint32_t sums,
                                              uint32_t block, int cta, int group, int tid) {
    const int w0 = t.f0 + cta * kHalf;
    const uint32_t row = block + tid * 64, turn = (tid >> 1) & 3;
    for (int c = group * 32; c < t.n; c += kGroups<kBackWeights> * 32) {
        uint32_t lo[16], hi[16];
        tc::ld16(sums + c, lo);
        tc::ld16(sums + c + 16, hi);
        tc::wait_ld();
        if (tid == 0) bulk_wait_read<0>();
        store_sync(group);  // the copy before has read the block
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t* v = i < 2 ? lo + 8 * i : hi + 8 * (i - 2);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (t.length > 0)
                x = make_uint4(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                               pack2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                               pack2(__uint_as_float(v[4]), __uint_as_float(v[5])),
                               pack2(__uint_as_float(v[6]), __uint_as_float(v[7])));
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                         :: "r"(row + ((i ^ turn) << 4)), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
        }
        fence_proxy_async_smem();
        store_sync(group);
        if (tid == 0 && w0 < p.features) {
            tc::store3(map, t.m0 + c, w0, t.e, block);
            bulk_commit();
        }
    }
}

// A finished tile to its results: the store groups take blocks of 16 columns of the sums in turn, each through its own
// block of shared memory, and fetch the next one while they write.  sums: tensor memory of this warp's lanes; cta: which
// half of the features; tid: of 128; link: how the parts of a tile meet (SPLIT).  up: from the first column to the last,
// else the other way; after `shared` blocks (the columns the next tile's sums take over) this warp arrives on the barrier
// `over`.  KEPT: pre is written, or read, as 8-bit codes.
template <int OP, bool GLU, bool SPLIT, bool KEPT>
__device__ __forceinline__ void store_tile(const ExpertArgs& a, const Plan& p, const Tile& t, uint32_t sums, float* turn,
                                           int cta, int group, int tid, bool up, int shared, uint32_t over, Link& link) {
    constexpr int kMine = GLU ? kHalf / 2 : kHalf;      // features of this CTA
    constexpr int kEights = kMine / 8, kAtOnce = 128 / kEights;
    const int f = t.f0 + cta * kMine + (tid % kEights) * 8;
    const bool live = f < p.features;
    const bool swap = (tid & 4) != 0;
    const bool through = OP == kBackRows && (KEPT || a.pre_in != nullptr);
    const int groups = (p.features + 31) >> 5;          // scales of half a kept row
    const int64_t pitch = through ? 2 * (int64_t)p.features : p.features;
    const int64_t r0 = (int64_t)t.first + t.m0;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + r0 * pitch + f;
    const int count = t.n / kTurn;
    constexpr bool k8 = kIntegers<OP>;
    // Sums of integers are scaled where they are turned, by this thread's weight row; parts of a sum are added first, which
    // is exact below 2^24, and scaled where a result row is written.
    float scale = 1.0f;
    if constexpr (k8 && !SPLIT) {
        const int of = t.f0 + cta * kMine + tid % kMine;
        const float* scales = static_cast<const float*>(a.weight_scales) + (int64_t)t.e * a.W;
        if (of < p.features) scale = __ldg(scales + of + tid / kMine * a.N);
    }
    auto column = [&](int i) { return (up ? i : count - 1 - i) * kTurn; };
    bool told = false;
    auto tell = [&] {
        tc::fence_before_sync();
        __syncwarp();
        if ((tid & 31) == 0) tc::arrive_cluster_tmem(over);
        told = true;
    };
    uint32_t v[kTurn];
    if (!k8 && group < count) tc::ld16(sums + column(group), v);
    for (int b = group; b < count; b += kGroups<OP>) {
        const int c = column(b);
        if (!told && b >= shared) tell();
        if (k8) tc::ld16(sums + c, v);  // (here the registers that fetching ahead takes cost more than it gives: 115 and 112 us)
        tc::wait_ld();
        if (SPLIT) {
            // the block before has been read by all parts
            if (tid == 0 && !within(kSecond, [&] { return tc::try_wait_cluster(link.seen, link.phase ^ 1u); })) link.ok = false;
        }
        store_sync(group);  // the block before has been read
#pragma unroll
        for (int i = 0; i < kTurn; ++i)
            turn[i * kTurnPitch + tid] = k8 && !SPLIT ? __uint_as_float(v[i]) * scale : __uint_as_float(v[i]);
        store_sync(group);
        if (SPLIT) {
            if (tid < link.parts)
                tc::arrive_cluster_smem(tc::in_rank(link.ready, 2 * tid + link.cta));
            if (tid == 0 && !within(kSecond, [&] { return tc::try_wait_cluster(link.ready, link.phase); })) link.ok = false;
            link.ok = store_all(group, link.ok);
            if (!link.ok) break;
            link.phase ^= 1u;
        }
        if (!k8 && b + kGroups<OP> < count) tc::ld16(sums + column(b + kGroups<OP>), v);
#pragma unroll
        for (int i = 0; i < kTurn; i += kAtOnce) {
            const int row = i + tid / kEights;
            const bool mine = live && c + row < t.rows && !(SPLIT && row % link.parts != link.part);
            const float* from = turn + row * kTurnPitch + (tid % kEights) * 8;
            float x[8];
            if constexpr (GLU && KEPT) {
                // the lanes of a scale meet, whether they have columns or not
                float u[8] = {};
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = 0.0f;
                if (mine) {
                    if (SPLIT) {
                        summed8(from, link, x);
                        summed8(from + kHalf / 2, link, u);
                    } else {
                        turned8(from, swap, x);
                        turned8(from + kHalf / 2, swap, u);
                    }
                }
                uint2 gate8, up8;
                const uint32_t gate_scale = keep8(x, &gate8), up_scale = keep8(u, &up8);
                if (!mine) continue;
                const int64_t r = r0 + c + row;
                uint8_t* codes = static_cast<uint8_t*>(a.kept) + r * a.W + f;
                *reinterpret_cast<uint2*>(codes) = gate8;
                *reinterpret_cast<uint2*>(codes + a.N) = up8;
                if ((tid & 3) == 0) {
                    uint8_t* scales = static_cast<uint8_t*>(a.kept_scales) + r * 2 * groups + (f >> 5);
                    scales[0] = (uint8_t)gate_scale;
                    scales[groups] = (uint8_t)up_scale;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = x[k] * sigmoid(x[k]) * u[k];
                store8(out + (c + row) * pitch, x);
                continue;
            }
            if (!mine) continue;
            if (SPLIT) summed8(from, link, x);
            else turned8(from, swap, x);
            const int64_t at = (c + row) * pitch;
            const float row_scale = k8 ? __ldg(static_cast<const float*>(a.row_scales) + r0 + c + row) : 1.0f;
            if constexpr (k8) scale8<SPLIT>(x, row_scale, static_cast<const float*>(a.weight_scales) + (int64_t)t.e * a.W + f);
            if (GLU) {
                float u[8];
                if (SPLIT) summed8(from + kHalf / 2, link, u);
                else turned8(from + kHalf / 2, swap, u);
                if constexpr (k8)
                    scale8<SPLIT>(u, row_scale, static_cast<const float*>(a.weight_scales) + (int64_t)t.e * a.W + a.N + f);
                if (a.pre != nullptr) {
                    __nv_bfloat16* pre = static_cast<__nv_bfloat16*>(a.pre) + (r0 + c + row) * a.W + f;
                    store8(pre, x);
                    store8(pre + a.N, u);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = x[k] * sigmoid(x[k]) * u[k];
                store8(out + at, x);
            } else if (through) {
                const int64_t r = r0 + c + row;
                float g[8], u[8];
                if constexpr (KEPT) {
                    const uint8_t* codes = static_cast<const uint8_t*>(a.kept) + r * pitch + f;
                    const uint8_t* scales = static_cast<const uint8_t*>(a.kept_scales) + r * 2 * groups + (f >> 5);
                    kept8(__ldg(reinterpret_cast<const uint2*>(codes)), __ldg(scales), g);
                    kept8(__ldg(reinterpret_cast<const uint2*>(codes + p.features)), __ldg(scales + groups), u);
                    if (a.act != nullptr) {
                        float act[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) act[k] = g[k] * sigmoid(g[k]) * u[k];
                        store8(static_cast<__nv_bfloat16*>(a.act) + r * p.features + f, act);
                    }
                } else {
                    const __nv_bfloat16* pre = static_cast<const __nv_bfloat16*>(a.pre_in) + r * pitch + f;
                    load8(pre, g);
                    load8(pre + p.features, u);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float s = sigmoid(g[k]);
                    u[k] = x[k] * u[k] * s * (1.0f + g[k] * (1.0f - s));
                    x[k] = x[k] * g[k] * s;
                }
                store8(out + at, u);
                store8(out + at + p.features, x);
            } else {
                store8(out + at, x);
            }
        }
        if (SPLIT) {
            store_sync(group);
            if (tid < link.parts) tc::arrive_cluster(tc::in_rank(link.seen, 2 * tid + link.cta));
        }
    }
    if (!told) tell();
}

// ---- the kernel ----------------------------------------------------------------

// Whether the weights' 128 rows of a CTA come in one box.
template <int OP, bool GLU>
constexpr bool kOneBox = (OP == kForward || OP == kForward4 || kIntegers<OP>) && !GLU;

// The weights (dout, in the weights' gradient) come through map_a, the rows through maps.
template <int OP, bool GLU, bool SPLIT, bool KEPT>
__global__ void __launch_bounds__(kThreads<OP>, 1)
pair_kernel(const ExpertArgs a, const Cut cut, const __grid_constant__ CUtensorMap map_a,
            const __grid_constant__ Maps maps) {
    constexpr bool k4 = OP == kForward4, k8 = kIntegers<OP>;
    constexpr bool across_a = OP == kBackRows || OP == kBackWeights, across_b = OP == kBackWeights;
    extern __shared__ uint8_t dynamic[];
    __shared__ Shared sh;
    const uint32_t skip = (1024u - (smem_u32(dynamic) & 1023u)) & 1023u;
    const uint32_t stages = smem_u32(dynamic) + skip;
    float* turn = reinterpret_cast<float*>(dynamic + skip + kRingBytes<OP>);
    int* blocks = reinterpret_cast<int*>(dynamic + skip + kRingBytes<OP> + kGroups<OP> * kTurnBytes);  // [E + 1], in 4 bits
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::rank_in_cluster(), cta = rank & 1, lead = rank & ~1;
    const uint16_t both = (uint16_t)(3u << lead);
    const int parts = SPLIT ? cut.parts : 1, part = SPLIT ? rank >> 1 : 0;
    const uint32_t full = smem_u32(sh.full), empty = smem_u32(sh.empty);  // 8 bytes a stage
    const uint32_t made = smem_u32(sh.made), used = smem_u32(sh.used);    // 8 bytes a piece
    const uint32_t pieces = stages + cut.stages * cut.bytes, piece_bytes = cut.columns / 2 * kRowBytes;

    if (threadIdx.x == 0) {
        for (int i = 0; i < cut.stages; ++i) {
            // both CTAs' copies arrive on the first CTA's; integers are widened by the CTA that copied them
            mbar_init(full + 8 * i, k8 ? 1 : 2);
            mbar_init(empty + 8 * i, k8 ? 8 : 1);
            mbar_init(smem_u32(&sh.tail[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.done[i]), 1);
            mbar_init(smem_u32(&sh.free[i]), 2 * 4 * kGroups<OP>);
            mbar_init(smem_u32(&sh.over[i]), 2 * 4 * kGroups<OP>);
        }
        if (k8)
            for (int i = 0; i < kPieces; ++i) {
                if (i % 2 == 0) mbar_init(made + 4 * i, 16);  // eight warps in either CTA
                mbar_init(used + 8 * i, 1);
            }
        if (SPLIT)
            for (int i = 0; i < kGroups<OP>; ++i) {
                mbar_init(smem_u32(&sh.ready[i]), parts);
                mbar_init(smem_u32(&sh.seen[i]), parts);
            }
        mbar_init(smem_u32(&sh.last), 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane < (across_b ? 1 : kMaps)) tc::prefetch_map(&maps.rows[lane]);
    if (warp == 0 && lane == kMaps) tc::prefetch_map(&map_a);
    if (k4 && warp == 0 && lane >= 8 && lane < 10) tc::prefetch_map(lane == 8 ? &maps.weight_scales : &maps.row_scales);
    if (warp == 1) tc::alloc_pair(smem_u32(&sh.tmem), 512);
    // the kernel before may still be running until here
    pdl_wait();
    scan_row_blocks(a.count, a.offset, a.E, a.R, sh.base, sh.scratch,
                    [&](int rows) { return tiles_of(rows, cut.columns); }, sh.rows);
    if (k4) scan_row_blocks(a.count, a.offset, a.E, a.R, blocks, sh.scratch, blocks_of_128);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const Plan p = make_plan<OP, GLU>(a, cut, sh.base);
    // the pairs (or the parts of a tile together) and the stages of this part
    const int64_t pair = (blockIdx.x >> 1) / parts, pairs = (gridDim.x >> 1) / parts;
    auto begin_of = [&](const Tile& t) {
        return SPLIT ? (int)((int64_t)((t.length + kStep<OP> - 1) / kStep<OP>) * part / parts) * kStep<OP> : 0;
    };
    auto end_of = [&](const Tile& t) {
        if (!SPLIT) return t.length;
        return min(t.length, (int)((int64_t)((t.length + kStep<OP> - 1) / kStep<OP>) * (part + 1) / parts) * kStep<OP>);
    };

    bool ok = true;
    if (warp == 0) {
        const uint32_t full0 = tc::in_rank(full, k8 ? rank : lead);
        Ring ring;
        int flying = 0;                // stages issued, up to all of them
        for (int64_t i = pair; i < p.tiles && ok; i += pairs) {
            const Tile t = tile_at<OP, GLU>(a, p, sh, i);
            const int n0 = t.n > kColumns ? kFirst : t.n;                     // columns of the first product, others
            const int half = n0 / 2, half1 = (t.n - n0) / 2;                  // columns of B in this CTA
            const int fa = t.f0 + cta * (GLU ? kHalf / 2 : kHalf);            // its first feature
            // A in one box of 128 rows (forward without a gate) or two of 64
            const int boxes_a = GLU ? 2 : kOneBox<OP, GLU> ? fa < p.features
                                                           : min(max((p.features - fa + 63) / 64, 0), 2);
            // (across the contraction: boxes of 64 columns of the one map there is)
            const Boxes b = across_b ? Boxes{64, half > 64 ? 64 : 0, &maps.rows[0], &maps.rows[0]} : boxes_of(maps, half);
            const Boxes c = boxes_of(maps, half1);
            uint32_t bytes = boxes_a * (kOneBox<OP, GLU> ? 2 : 1) * kBoxBytes + b.bytes() + c.bytes();
            // scale blocks: rows of 512 bytes, `groups` to a block of rows
            const int groups = (a.K + 127) >> 7, per = GLU ? 64 : 128, wblocks = (a.N + per - 1) / per;
            const int scaled = k4 ? ((t.m0 & 127) + t.n + 127) >> 7 : 0;      // blocks of receive rows
            const int wrow = k4 ? (t.e * wblocks + min(fa / per, wblocks - 1)) * groups : 0;
            const int rrow = k4 ? (blocks[t.e] + (t.m0 >> 7)) * groups : 0;
            if (k4) bytes += (1 + scaled) * 2 * kScaleBlock;
            const int b0 = (OP == kBackWeights ? 0 : t.first) + t.m0 + cta * half;
            const int c0 = t.first + t.m0 + n0 + cta * half1;
            const int end = end_of(t);
            for (int k0 = begin_of(t); k0 < end; k0 += kStep<OP>) {
                if (!warp_wait(empty + 8 * ring.stage, ring.phase ^ 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = stages + ring.at, sb = sa + kBytesA;
                const int left = t.length - k0;
                // rows past the expert's last that would be summed: the tail warp gets the stage first
                const bool clear = OP == kBackWeights && left < kStep<OP> && (left & 15) != 0;
                if (tc::elect_one()) {
                    const uint32_t bar = clear ? smem_u32(&sh.tail[ring.stage]) : full0 + 8 * ring.stage;
                    tc::arrive_expect_cluster(bar, bytes);
                    if (OP == kBackWeights) {
                        if (boxes_a > 0) tc::load2_pair(sa, &map_a, fa, t.first + k0, bar);
                        if (boxes_a > 1) tc::load2_pair(sa + kBoxBytes, &map_a, fa + 64, t.first + k0, bar);
                        tc::load2_pair(sb, b.map0, b0, t.first + k0, bar);
                        if (b.rows1 > 0) tc::load2_pair(sb + kBoxBytes, b.map0, b0 + 64, t.first + k0, bar);
                    } else {
                        const int x = k4 ? k0 / 2 : k0;                       // along memory
                        if (boxes_a > 0) {
                            if (OP == kBackRows) tc::load3_pair(sa, &map_a, fa, k0, t.e, bar);
                            else tc::load3_pair(sa, &map_a, x, fa, t.e, bar);
                        }
                        if (boxes_a > 1) {
                            if (OP == kBackRows) tc::load3_pair(sa + kBoxBytes, &map_a, fa + 64, k0, t.e, bar);
                            else tc::load3_pair(sa + kBoxBytes, &map_a, x, fa + a.N, t.e, bar);
                        }
                        tc::load2_pair(sb, b.map0, x, b0, bar);
                        if (b.rows1 > 0) tc::load2_pair(sb + b.rows0 * kRowBytes, b.map1, x, b0 + b.rows0, bar);
                        if (k4) {
                            const uint32_t ss = sa + kBytesA + cut.columns / 2 * kRowBytes;
                            const int g = k0 >> 7;
                            tc::load2_pair(ss, &maps.weight_scales, 0, wrow + g, bar);
                            tc::load2_pair(ss + 2 * kScaleBlock, &maps.row_scales, 0, rrow + g, bar);
                            if (scaled > 1)
                                tc::load2_pair(ss + 4 * kScaleBlock, &maps.row_scales, 0, rrow + groups + g, bar);
                            if (scaled > 2)
                                tc::load2_pair(ss + 6 * kScaleBlock, &maps.row_scales, 0, rrow + 2 * groups + g, bar);
                        }
                        const uint32_t sc = sb + b.bytes();
                        if (c.rows0 > 0) tc::load2_pair(sc, c.map0, x, c0, bar);
                        if (c.rows1 > 0) tc::load2_pair(sc + c.rows0 * kRowBytes, c.map1, x, c0 + c.rows0, bar);
                    }
                }
                __syncwarp();
                ring.next(cut);
                flying = min(flying + 1, cut.stages);
            }
        }
        // no copy of this pair is in flight when it ends: its readers have waited for them, unless a wait gave up
        if (cta == 0 || k8)
            for (; flying > 0; --flying) {
                if (ring.stage-- == 0) {
                    ring.stage = cut.stages - 1;
                    ring.phase ^= 1u;
                }
                warp_wait(full + 8 * ring.stage, ring.phase);
            }
    } else if (warp == 1 && cta == 0) {
        Ring ring;
        int n = 0, before = 0;         // tiles so far, columns of the one before
        int piece = 0;
        uint32_t piece_phase = 0;
        for (int64_t i = pair; i < p.tiles && ok; i += pairs, ++n) {
            const Tile t = tile_at<OP, GLU>(a, p, sh, i);
            const bool wide = !across_b && t.n > kColumns;
            // tiles take the low and the high end of tensor memory in turn
            const uint32_t sums = tmem + (n & 1 ? kTop<OP> - t.n : 0);
            // the instruction of the tile and, for a wide one, of its other columns
            const int n0 = wide ? kFirst : t.n, n1 = max(t.n - kFirst, 16);
            const uint32_t instr = tc::instruction_pair(n0, across_a, across_b);
            const uint32_t instr1 = tc::instruction_pair(n1, across_a, across_b);
            // this end is free when the tile before the last is stored, and what the last one holds of it when its store
            // half has been there
            ok = warp_wait_cluster(smem_u32(&sh.free[n & 1]), (uint32_t)((n >> 1) & 1) ^ 1u);
            if (ok && before + t.n > kTop<OP>)
                ok = warp_wait_cluster(smem_u32(&sh.over[(n + 1) & 1]), (uint32_t)(((n - 1) >> 1) & 1));
            if (!ok) break;
            before = t.n;
            tc::fence_after_sync();
            const int begin = begin_of(t), end = end_of(t);
            if constexpr (k8) {
                // a stage at a time: both its pieces are waited for at once, and given back one by one
                const uint32_t instr8 = tc::instruction16_pair(t.n);
                for (int k0 = begin; k0 < end; k0 += kStep<OP>) {
                    ok = warp_wait_cluster(made + 4 * piece, piece_phase);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
                        const uint32_t wa = tmem + kTop<OP> + piece * kPieceColumns;
                        const uint64_t rb = tc::at(tc::kAlongK, pieces + piece * piece_bytes), rb1 = rb + (piece_bytes >> 4);
                        if (end - k0 >= kStep<OP>) {       // without tests between the instructions
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::mma_tmem_pair(sums, wa + k * 8, rb + k * 2, instr8, k0 > begin || k > 0);
                            tc::commit_pair(used + 8 * piece, both);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::mma_tmem_pair(sums, wa + kPieceColumns + k * 8, rb1 + k * 2, instr8, true);
                        } else {
                            const int count = (end - k0) / 16;
                            for (int k = 0; k < min(count, 4); ++k)
                                tc::mma_tmem_pair(sums, wa + k * 8, rb + k * 2, instr8, k0 > begin || k > 0);
                            tc::commit_pair(used + 8 * piece, both);
                            for (int k = 4; k < count; ++k)
                                tc::mma_tmem_pair(sums, wa + k * 8, rb1 + (k - 4) * 2, instr8, true);
                        }
                        tc::commit_pair(used + 8 * (piece + 1), both);
                    }
                    __syncwarp();
                    piece += 2;
                    if (piece == kPieces) {
                        piece = 0;
                        piece_phase ^= 1u;
                    }
                }
            } else
            for (int k0 = begin; k0 < end; k0 += kStep<OP>) {
                // a stage that the tail warps of both CTAs have cleared is theirs to hand over, any other the copies'
                const bool cleared = OP == kBackWeights && t.length - k0 < kStep<OP> && (t.length & 15) != 0;
                if (!(cleared ? warp_wait_cluster(full + 8 * ring.stage, ring.phase)
                              : warp_wait(full + 8 * ring.stage, ring.phase))) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t sa = stages + ring.at;
                const uint64_t da = tc::at(across_a ? tc::kAcrossK : tc::kAlongK, sa);
                const uint64_t db = tc::at(across_b ? tc::kAcrossK : tc::kAlongK, sa + kBytesA);
                constexpr int kOne = k4 ? 64 : 16;                            // contraction of an instruction
                const int count = (min(kStep<OP>, t.length - k0) + kOne - 1) / kOne;
                if (k4 && tc::elect_one()) {
                    const uint32_t ss = sa + kBytesA + cut.columns / 2 * kRowBytes;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        tc::copy_scales_pair(tmem + kScalesA + 4 * g, tc::at(tc::kScales, ss + g * kScaleBlock));
                        tc::copy_scales_pair(tmem + kScalesB + 12 * g, tc::at(tc::kScales, ss + (2 + g) * kScaleBlock));
                        if ((t.m0 & 127) + t.n > 128)
                            tc::copy_scales_pair(tmem + kScalesB + 12 * g + 4,
                                                 tc::at(tc::kScales, ss + (4 + g) * kScaleBlock));
                        if ((t.m0 & 127) + t.n > 256)
                            tc::copy_scales_pair(tmem + kScalesB + 12 * g + 8,
                                                 tc::at(tc::kScales, ss + (6 + g) * kScaleBlock));
                    }
                    // a tile that starts in the middle of a scale block starts two columns of 32 rows later
                    const uint32_t sb4 = tmem + kScalesB + ((t.m0 & 127) >> 5);
                    auto products = [&](uint32_t d, uint64_t db, int n, uint32_t sb, int count) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // two to a scale word
                            if (k < count)
                                tc::mma4_pair(d, da + k * 2, db + k * 2, tc::instruction4_pair(n, k & 1),
                                              tmem + kScalesA + 4 * (k >> 1), sb + 12 * (k >> 1), k0 > begin || k > 0);
                    };
                    auto both_products = [&](int count) {
                        products(sums, db, n0, sb4, count);
                        if (wide)
                            products(sums + kFirst, tc::at(tc::kAlongK, sa + kBytesA + kFirst / 2 * kRowBytes), n1,
                                     sb4 + kFirst / 32, count);
                    };
                    if (count == 4) both_products(4);  // without tests between the instructions (384 columns: 329 -> 325 us)
                    else both_products(count);
                    tc::commit_pair(empty + 8 * ring.stage, both);
                } else if (!k4 && tc::elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < count)
                            tc::mma_pair(sums, da + k * (across_a ? 128 : 2), db + k * (across_b ? 128 : 2), instr,
                                         k0 > begin || k > 0);
                    if (wide) {
                        const uint64_t dc = tc::at(tc::kAlongK, sa + kBytesA + kFirst / 2 * kRowBytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < count)
                                tc::mma_pair(sums + kFirst, da + k * (across_a ? 128 : 2), dc + k * 2, instr1,
                                             k0 > begin || k > 0);
                    }
                    tc::commit_pair(empty + 8 * ring.stage, both);
                }
                __syncwarp();
                ring.next(cut);
            }
            if (!ok) break;
            if (tc::elect_one()) tc::commit_pair(smem_u32(&sh.done[n & 1]), both);
            __syncwarp();
        }
        // whatever was issued is done before tensor memory is freed
        if (tc::elect_one()) tc::commit_pair(smem_u32(&sh.last), both);
        __syncwarp();
        ok = warp_wait(smem_u32(&sh.last), 0) && ok;
    } else if (warp >= 2 && warp < kTailWarp<OP>) {
        const int quarter = warp & 3, group = (warp - 2) >> 2;
        float* mine = turn + group * kTurn * kTurnPitch;
        int n = 0;
        Link link{smem_u32(&sh.ready[group]), smem_u32(&sh.seen[group]), 0, part, parts, cta, true};
        Tile t{};
        if (pair < p.tiles) t = tile_at<OP, GLU>(a, p, sh, pair);
        for (int64_t i = pair; i < p.tiles; i += pairs, ++n) {
            // columns that the next tile's sums share with this one's, and with them its first blocks to store
            const Tile next = tile_at<OP, GLU>(a, p, sh, min(i + pairs, p.tiles - 1));
            const int shared = i + pairs < p.tiles ? max(t.n + next.n - kTop<OP>, 0) / kTurn : 0;
            // One warp of a group watches the sums' barrier, the others sleep at the group's own: sixteen watching
            // warps would take issue slots from the two that feed the tensor core.  A group gives up together.
            const bool got = ((warp - 2) & 3) != 0 ||
                             wait_second(smem_u32(&sh.done[n & 1]), (uint32_t)((n >> 1) & 1),
                                         limit_of<OP>(t.length / kStep<OP>));
            if (!store_all(group, got)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            const uint32_t sums = tmem + (n & 1 ? kTop<OP> - t.n : 0) + ((uint32_t)(quarter * 32) << 16);
            if constexpr (OP == kBackWeights) {
                store_weights(p, t, &maps.out, sums, smem_u32(turn) + group * 32 * kHalf * 2, cta, group, quarter * 32 + lane);
            } else {
                store_tile<OP, GLU, SPLIT, KEPT>(a, p, t, sums, mine, cta, group, quarter * 32 + lane, (n & 1) != 0, shared,
                                           tc::in_rank(smem_u32(&sh.over[n & 1]), lead), link);
                if (SPLIT && !link.ok) {
                    ok = false;
                    break;
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::arrive_cluster_tmem(tc::in_rank(smem_u32(&sh.free[n & 1]), lead));
            t = next;
        }
        if (OP == kBackWeights && quarter * 32 + lane == 0) bulk_wait_all();
    }
    if (k8 && warp >= kTailWarp<OP>) {
        // Widens one half of every (other) stage: this CTA's weights to its tensor memory and its rows to its shared memory,
        // and hands the piece to the first CTA, which multiplies it.  A barrier's parity tells one phase from the next
        // alone, so a group must see every phase of the barriers it waits on.  Where two sets of groups take stages in turn
        // the stages are even in number and the pieces a multiple of four, two to every stage, so that each is always the same
        // group's.
        const int group = (warp - kTailWarp<OP>) >> 2, half = group & 1, quarter = warp & 3;
        const uint32_t made0 = tc::in_rank(made, lead);
        Ring ring;
        int piece = half;
        uint32_t phase = 0;
        bool mine = group < 2;
        for (int64_t i = pair; i < p.tiles && ok; i += pairs) {
            const Tile t = tile_at<OP, GLU>(a, p, sh, i);
            const int end = end_of(t);
            for (int k0 = begin_of(t); k0 < end; k0 += kStep<OP>, mine = mine != kInTurn<OP>, ring.next(cut)) {
                if (mine) {
                    ok = warp_wait(full + 8 * ring.stage, ring.phase) && warp_wait(used + 8 * piece, phase ^ 1u);
                    if (!ok) break;
                    if (k0 + half * kPiece < end) {
                        tc::fence_after_sync();
                        const uint32_t sa = stages + ring.at;
                        widen(sa, half, t.n / 2, tmem + kTop<OP> + piece * kPieceColumns, pieces + piece * piece_bytes,
                              quarter, lane);
                        fence_proxy_async_smem();
                        tc::wait_st();
                        tc::fence_before_sync();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        tc::arrive_cluster_smem(made0 + 8 * (piece >> 1));
                        mbar_arrive(empty + 8 * ring.stage);
                    }
                }
                piece += 2;
                if (piece >= kPieces) {
                    piece -= kPieces;
                    phase ^= 1u;
                }
            }
        }
    }
    if (OP == kBackWeights && warp == kTailWarp<OP>) {
        // Clears the rows past an expert's last in its last stage, in this CTA, and hands the stage on.  The copying warp
        // does not wait for it: doing so there cost a memory latency a tile (1024 rows of 32 experts spread by routing,
        // 2048 x 7168: 660 us against 604 us).
        const uint32_t full0 = tc::in_rank(full, lead);
        uint32_t phases = 0;           // of the tail barriers, a bit each
        int stage = 0;
        int64_t since = 0;             // stages after the last one that was waited for here
        for (int64_t i = pair; i < p.tiles; i += pairs) {
            const Tile t = tile_at<OP, GLU>(a, p, sh, i);
            const int steps = (t.length + kStep<OP> - 1) / kStep<OP>;
            since += steps;
            if ((t.length & 15) != 0) {
                const int at = (stage + steps - 1) % cut.stages;
                if (!warp_wait(smem_u32(&sh.tail[at]), (phases >> at) & 1, limit_of<OP>(since))) {
                    ok = false;
                    break;
                }
                phases ^= 1u << at;
                since = 0;
                const int left = t.length - (steps - 1) * kStep<OP>;
                const int from = left * 8, to = ((left + 15) & ~15) * 8;      // 16-byte pieces of a box
                for (int k = 0; k < cut.bytes / kBoxBytes; ++k)
                    for (int j = from + lane; j < to; j += 32)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                                     :: "r"(stages + at * cut.bytes + k * kBoxBytes + j * 16), "r"(0u) : "memory");
                asm volatile("fence.proxy.async;" ::: "memory");              // also for the first CTA's products
                __syncwarp();
                if (lane == 0) tc::arrive_cluster_smem(full0 + 8 * at);
            }
            stage = (stage + steps) % cut.stages;
        }
    }
    if (!ok && lane == 0) atomicOr(&g_expert_faults, MOE_FAULT_WAIT_TIMEOUT);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    // Not before: blocks of the next kernel that came early would crowd on the SMs that this one leaves free (1014 rows
    // quantised and multiplied in 4 bits, 1216 -> 2 x 864: 21.0 us, and 15.7 us this way).
    pdl_launch_dependents();
    // Commits arrive on barriers of both CTAs, and the cluster's meeting does not wait for them: this CTA ends when the last
    // one, behind all others, has arrived here too (the first CTA has waited for its own).
    if (warp == 1 && cta == 1 && !warp_wait(smem_u32(&sh.last), 0) && lane == 0)
        atomicOr(&g_expert_faults, MOE_FAULT_WAIT_TIMEOUT);
    __syncwarp();
    tc::cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tc::dealloc_pair(tmem, 512);
}

// Tiles of this many columns: as many stages as the ring holds, beside the pieces of widened integers.
template <int OP>
constexpr int pieces_bytes(int columns) { return kIntegers<OP> ? kPieces * columns / 2 * kRowBytes : 0; }
template <int OP>
constexpr Cut cut_at(int columns) {
    Cut cut{columns, 0, 0, 1};
    cut.bytes = kBytesA + cut.columns / 2 * kRowBytes + (OP == kForward4 ? scale_bytes(cut.columns) : 0);
    const int ring = kRingBytes<OP> - pieces_bytes<OP>(columns);
    cut.stages = ring / cut.bytes < kStages ? ring / cut.bytes : kStages;
    if (kIntegers<OP> && kInTurn<OP>) cut.stages &= ~1;  // (see the widening warps)
    return cut;
}
// Two stages at least, an even number of them where groups take them in turn, and all of it inside the ring.
template <int OP>
constexpr bool holds(int columns) {
    const Cut cut = cut_at<OP>(columns);
    return cut.stages >= 2 && !(kInTurn<OP> && cut.stages % 2) && cut.stages * cut.bytes + pieces_bytes<OP>(columns) <= kRingBytes<OP>;
}
static_assert(holds<kForward>(64) && holds<kForward>(128) && holds<kForward>(256) && holds<kForward>(320) && holds<kForward>(384));
static_assert(holds<kBackRows>(64) && holds<kBackRows>(128) && holds<kBackRows>(256) && holds<kBackRows>(320) && holds<kBackRows>(384));
static_assert(holds<kForward4>(64) && holds<kForward4>(128) && holds<kForward4>(256) && holds<kForward4>(384));
static_assert(holds<kForward8>(128) && holds<kForward8>(256) && holds<kShort8>(256) && holds<kBackWeights>(kColumns));

// The cut of a launch, from the mean rows of an expert (all the host knows of them); routing spreads an expert's rows by
// about the square root of their mean, and 3.5 of that hold almost all experts.  The bounds above 256 rows were each timed
// on both sides for three to four widths, 8 and 32 experts, even routing and one whose experts' shares fall as rank^-0.4 (in brackets).
//  * A tile that takes all rows of its expert reads the weights once, and the narrower it is the more stages are in
//    flight: 2 rows an expert (64 experts, 7168 -> 2 x 2048) take 528 us with 64 columns, 548 with 256, 588 with 512; but
//    128 rows take 677 us cut at 64 columns and 582 us cut at 256.
//  * Tiles of more than 256 columns win where they save one: 272 rows take 682 us cut at 320 and 858 us cut at 256, 600
//    rows (32 experts) 702 us at 320 and 773 at 256 [747 and 744].
//  * 384 columns win where most experts fit them and not 320 (32 experts, 384 against 320): 305 rows take 399 and 406 us
//    [461 and 447], 312 rows 406 and 433 [444 and 440], 330 rows 429 and 490 [480 and 448], 360 rows 450 and 525 [491 and
//    488], 375 rows 486 and 521 [530 and 512], 400 rows 594 and 540 [537 and 521].  Over all widths they take 0.91 of the
//    time at 312 to 360 rows [1.02], and 1.07 on either side [1.06].
//  * Many tiles an expert waste little of either, and 256 columns issue fewer instructions: 3000 rows (8 experts) take
//    388 us at 256 and 406 at 320; 1040 rows 594 and 600.  Over all widths 320 columns take 0.99 to 1.02 of 256's time at 700 to
//    900 rows [0.97 to 1.03] and 0.99 to 1.06 from 950 up [0.98 to 1.06].
//  * In 4 bits tensor memory also holds scales, so the next tile's sums wait for most of a wide one's store half; 384 columns
//    pay where they take all rows in one tile or in three (7168 -> 2 x 2048, 32 experts, 384 against 256): 260 rows 131 and
//    145 us, 360 rows 150 and 172, 400 rows 178 and 174, 700 rows 253 and 254, 800 rows 281 and 312, 1024 rows 340 and 355,
//    1150 rows 379 and 383, 1300 rows 449 and 447.  Over all widths one tile of 384 takes 0.89 of the time of 256 [0.97],
//    three 0.987 of four or five [1.004], and those between 1.017 [1.018].  170 rows (16 experts) take 129 us cut at 128 and 97 at 256.
//    The stages in flight count: 384 columns take 330 us with four and 353 with three (1024 rows), 256 columns 129 with five
//    and 142 with four (256 rows).
//  * In 8-bit integers a wide tile pays twice, since its weights are widened for all of its rows at once (8 and 32 experts,
//    six widths, 128 against 256 columns): 40 to 90 rows take 0.98 of the time, 120 rows 1.07, 230 to 1024 rows 1.2 to 1.36
//    from 2048 of contraction on, 1.02 at 512 and 1024.  64 columns take 1.00 at 40 rows and 1.19 at 60 (1 row: the same),
//    192, whose sums lie beside the next tile's, 0.98 up to 1424 of contraction and 1.08 from 2048 on.
template <int OP>
Cut make_cut(const ExpertArgs& a) {
    const double mean = (double)a.R / a.E, most = mean + 3.5 * std::sqrt(mean);
    int columns = kColumns;
    if (OP != kBackWeights) {
        columns = most <= 64 && !kIntegers<OP> ? 64 : most <= 128 ? 128 : 256;
        if (OP != kForward4 && !kIntegers<OP> && most > 256 && mean < 900) columns = mean > 310 && mean <= 365 ? 384 : 320;
        if (OP == kForward4 && most > 256 && (mean <= 365 || (mean > 768 && mean <= 1152))) columns = 384;
    }
    return cut_at<OP>(columns);
}

// Pairs that share a tile: the fewest rounds of tiles times stages of a round.  Sharing costs a round about as long as 14
// stages (two meetings of the parts per 16 columns): one row of one expert, 7168 -> 2 x 1024 (8 tiles of 112 stages), takes
// 13.6 us in four parts, 19.1 in two and 28.4 in one, 300 rows 31.1, 36.6 and 42.9.  Contractions of 28 stages and fewer
// are never shared, so that every part has stages of its own (one row of one expert, 28 stages: 9.1 us in four parts and
// 10.9 in one, in 4 bits 12.6 and 15.0: there is something left here).
// *all: the teams of pairs that run at once; left alone where a tile is one pair's (so too where the device cannot say).
constexpr int kLeastShared = 29, kMostParts = 4;
static_assert(kLeastShared >= kMostParts);
int parts_of(const void* split, int threads, int smem, int64_t tiles, int steps, int64_t pairs, int64_t* all) {
    int best = 1;
    int64_t least = (tiles + pairs - 1) / pairs * steps;
    for (int parts = 2; parts <= kMostParts && steps >= kLeastShared; parts *= 2) {
        const int64_t teams = active_clusters(split, threads, smem, 2 * parts);
        if (teams < 1) continue;
        const int64_t cost = (tiles + teams - 1) / teams * ((steps + parts - 1) / parts + 14);
        if (cost < least) {
            least = cost;
            best = parts;
            *all = teams;
        }
    }
    return best;
}

// Launches a pair kernel in clusters of cut.parts pairs, under programmatic dependent launch.
template <int OP, typename K>
cudaError_t start(K* kern, const ExpertArgs& a, const Cut& cut, int64_t tiles, int64_t teams, const CUtensorMap& ma,
                  const Maps& mb, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * cut.parts * (tiles < teams ? tiles : teams)));
    cfg.blockDim = dim3(kThreads<OP>);
    cfg.dynamicSmemBytes = kSmem<OP>;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * cut.parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, cut, ma, mb);
}

template <int OP, bool GLU>
bool make_maps(const ExpertArgs& a, CUtensorMap* ma, Maps* mb) {
    bool ok;
    if (OP == kBackWeights) {
        ok = tc::make_map(ma, a.dout, false, a.W, a.R, 0, 64) && tc::make_map(&mb->rows[0], a.rows, false, a.K, a.R, 0, 64) &&
             tc::make_map(&mb->out, a.out, false, a.K, a.W, a.E, kHalf, 64);
    } else if (OP == kForward4) {
        const int64_t groups = (a.K + 127) / 128, per = GLU ? 64 : 128;
        ok = tc::make_map(ma, a.weights, true, a.K / 2, a.W, a.E, kOneBox<OP, GLU> ? kHalf : 64) &&
             tc::make_scale_map(&mb->weight_scales, a.weight_scales, a.E * ((a.N + per - 1) / per) * groups) &&
             tc::make_scale_map(&mb->row_scales, a.row_scales, (a.R / 128 + a.E) * groups);
        for (int i = 0; i < kMaps; ++i) ok = ok && tc::make_map(&mb->rows[i], a.rows, true, a.K / 2, a.R, 0, 8 << i);
    } else if (kIntegers<OP>) {
        ok = tc::make_map(ma, a.weights, true, a.K, a.W, a.E, kOneBox<OP, GLU> ? kHalf : 64);
        for (int i = 0; i < kMaps; ++i) ok = ok && tc::make_map(&mb->rows[i], a.rows, true, a.K, a.R, 0, 8 << i);
    } else {
        ok = tc::make_map(ma, a.weights, false, a.K, a.W, a.E, kOneBox<OP, GLU> ? kHalf : 64);
        for (int i = 0; i < kMaps; ++i)
            ok = ok && tc::make_map(&mb->rows[i], OP == kForward ? a.rows : a.dout, false, OP == kForward ? a.K : a.W, a.R,
                                    0, 8 << i);
    }
    return ok;
}

// Integers, few stages a tile and many columns: the store half is what a tile takes, and three groups of it with half the
// widening warps are faster (130 to 1024 rows of 8 and 32 or 40 experts: 1024 of contraction takes 0.83 of the time, 1424 0.92,
// 2048 0.93, 2816 0.99, 3584 1.02, 7168 1.04; 32 experts of 1024 rows, 512 -> 1024: 82.5 -> 50 us; four groups take 0.99 to
// 1.04 of three).  With few rows the weights are what counts (16 rows, 1024 -> 2048: 21.0 and 24.8 us).
constexpr int kLeastLong = 3200;

template <int OP, bool GLU, bool KEPT = false>
cudaError_t launch(const ExpertArgs& a, cudaStream_t s) {
    Cut cut = make_cut<OP>(a);
    // no more pairs than there can be tiles
    const int64_t features = OP == kBackWeights ? a.W : OP == kBackRows ? a.K : a.N, wide = GLU ? kHalf : 2 * kHalf;
    const int64_t across = (features + wide - 1) / wide;
    const int64_t tiles = across * (OP == kBackWeights ? (int64_t)a.E * ((a.K + kColumns - 1) / kColumns)
                                                       : a.R / cut.columns + (int64_t)(a.E < a.R ? a.E : a.R));
    const int64_t pairs = device_sm_count() / 2;
    int64_t teams = pairs;
    auto* kern = pair_kernel<OP, GLU, false, KEPT>;
    if constexpr (OP != kBackWeights && OP != kShort8) {
        auto* split = pair_kernel<OP, GLU, true, KEPT>;
        const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(split), kSmem<OP>);
        if (e != cudaSuccess) return e;
        // (a stage of integers is two pieces, each a stage's worth of products)
        constexpr int kWork = kIntegers<OP> ? kPiece : kStep<OP>;
        const int steps = ((OP == kBackRows ? a.W : a.K) + kWork - 1) / kWork;
        cut.parts = parts_of(reinterpret_cast<const void*>(split), kThreads<OP>, kSmem<OP>, tiles, steps, pairs, &teams);
        if (cut.parts > 1) kern = split;
    }
    if constexpr (OP == kForward8)
        if (cut.parts == 1 && a.K < kLeastLong && cut.columns > 128) return launch<kShort8, GLU>(a, s);
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), kSmem<OP>);
    if (e != cudaSuccess) return e;
    CUtensorMap ma;
    Maps mb{};
    if (!make_maps<OP, GLU>(a, &ma, &mb)) return cudaErrorInvalidValue;
    return start<OP>(kern, a, cut, tiles, teams, ma, mb, s);
}

}  // namespace

cudaError_t launch_expert_forward(const ExpertArgs& a, cudaStream_t s) {
    return a.glu ? launch<kForward, true>(a, s) : launch<kForward, false>(a, s);
}
cudaError_t launch_expert_backward_rows(const ExpertArgs& a, cudaStream_t s) { return launch<kBackRows, false>(a, s); }
cudaError_t launch_expert_forward_kept(const ExpertArgs& a, cudaStream_t s) { return launch<kForward, true, true>(a, s); }
cudaError_t launch_expert_backward_kept(const ExpertArgs& a, cudaStream_t s) {
    return launch<kBackRows, false, true>(a, s);
}
cudaError_t launch_expert_backward_weights(const ExpertArgs& a, cudaStream_t s) {
    return launch<kBackWeights, false>(a, s);
}

cudaError_t launch_expert_forward4(const ExpertArgs& a, cudaStream_t s) {
    return a.glu ? launch<kForward4, true>(a, s) : launch<kForward4, false>(a, s);
}

cudaError_t launch_expert_forward8(const ExpertArgs& a, cudaStream_t s) {
    return a.glu ? launch<kForward8, true>(a, s) : launch<kForward8, false>(a, s);
}

cudaError_t read_expert_faults(uint32_t* bits, cudaStream_t stream) {
    unsigned v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_expert_faults, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_expert_faults, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice,
                                                      stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess) *bits = v;
    return e;
}

}  // namespace moe
