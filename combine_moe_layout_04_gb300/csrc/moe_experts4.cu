// moe_experts.cu -- products grouped by expert over ragged receive rows
// ("Balancing and Beyond", section 1: the experts between dispatch and
// combine).
//
// One persistent kernel per product, one CTA an SM.  A tile is 128 rows of a
// result (receive rows of one expert; for the weights' gradient 128 of an
// expert's weight rows) by BN columns, and its sums stay in tensor memory.  Six
// warps: one thread feeds a ring of shared-memory stages with tensor copies,
// one thread issues the tensor-core products, four warps turn finished sums
// into results while the next tile is already being computed (two tiles' sums
// fit in tensor memory, except for 256 columns in 4 bits, whose scales share
// it).
//
// Which operand runs along the contraction in memory decides the descriptor:
//   forward            out  = rows  W^T   both along it
//   gradient of rows   drows = dout W     W across it
//   gradient of weights dW  = dout^T rows both across it (the rows are summed)
// A stage is the same bytes in all three: 128 bytes along memory by 128 and BN
// rows, 128-byte swizzle, fetched in boxes of 64 rows.
//
// Ragged groups.  The host knows only how many rows there are in all; every CTA
// counts the row blocks of each expert from the layout's counts (a scan over at
// most 1024 experts) and takes tiles blockIdx, blockIdx + grid, ... of that
// list.  Within an expert row blocks go first, so that the CTAs that share a
// piece of its weights run at the same time and it comes from HBM once.  Rows of
// the next expert that a tile's box reaches into only make sums that nobody
// stores; where rows are summed (weights' gradient) they are cleared in shared
// memory first.
//
// Every wait is bounded.  A CTA whose wait gives up records a fault, waits for
// its own copies and products, frees its tensor memory and returns.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_experts.cuh"
#include "moe_tc.cuh"

namespace moe {
namespace {

__device__ unsigned int g_expert4_faults;

// A bounded wait of a whole warp: it gives up together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_second(bar, parity)) != 0;
}

constexpr int kForward = 0, kBackRows = 1, kBackWeights = 2, kForward4 = 3;
constexpr int kThreads = 192;          // warp 0 copies, warp 1 multiplies, warps 2 .. 5 store
constexpr int kTileRows = 128;
constexpr int kRowBytes = 128;         // of a stage, along memory
constexpr int kBoxRows = 64;
constexpr int kBoxBytes = kBoxRows * kRowBytes;
constexpr int kScaleBlock = 512;

template <int OP, int BN>
struct Shape {
    static constexpr bool k4 = OP == kForward4;
    static constexpr int kStep = k4 ? 2 * kRowBytes : 64;                 // contraction of a stage
    static constexpr int kBytesA = kTileRows * kRowBytes, kBytesB = BN * kRowBytes;
    static constexpr int kScaleBytes = k4 ? 2 * kScaleBlock * (1 + BN / 128) : 0;
    static constexpr int kStageBytes = kBytesA + kBytesB + kScaleBytes;
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr int kSums = k4 && BN == 256 ? 1 : 2;                 // tiles in tensor memory
    static constexpr int kColumns = k4 ? 512 : 2 * BN;                    // of tensor memory
    static constexpr uint32_t kScaleA = kSums * BN, kScaleB = kScaleA + 8;
    static constexpr int kSmem = kStages * kStageBytes + 1024;            // 1024: alignment
};

struct Shared {
    uint64_t full[8], empty[8], done[2], free[2], last;
    uint32_t tmem;
    int scratch[32];
    int base[MOE_MAX_EXPERTS + 1];
};

// One tile of a result.
struct Tile {
    int e;        // expert
    int first;    // its first receive row
    int m0, n0;   // first row and column of the tile, inside the expert's result
    int rows;     // rows of the tile that exist
    int block;    // row block, counted over the experts
    int steps;    // stages of its contraction
};

struct Plan {
    int64_t tiles;
    int across;   // tiles side by side
    int length;   // contraction (0: the expert's rows)
    int cols;     // columns of a result
};

template <int OP, int BN, bool GLU>
__device__ __forceinline__ Plan make_plan(const ExpertArgs& a, const int* base) {
    Plan p;
    p.cols = OP == kForward || OP == kForward4 ? a.N : a.K;
    const int wide = GLU ? BN / 2 : BN;
    p.across = (p.cols + wide - 1) / wide;
    p.length = OP == kBackWeights ? 0 : OP == kBackRows ? a.W : a.K;
    p.tiles = OP == kBackWeights ? (int64_t)a.E * ((a.W + kTileRows - 1) / kTileRows) * p.across
                                 : (int64_t)base[a.E] * p.across;
    return p;
}

template <int OP, int BN, bool GLU>
__device__ __forceinline__ Tile tile_at(const ExpertArgs& a, const Plan& p, const int* base, int64_t i) {
    constexpr int kStep = Shape<OP, BN>::kStep;
    constexpr int wide = GLU ? BN / 2 : BN;
    Tile t;
    if (OP == kBackWeights) {
        const int down = (a.W + kTileRows - 1) / kTileRows;
        t.e = (int)(i / ((int64_t)down * p.across));
        const int j = (int)(i - (int64_t)t.e * down * p.across);
        const ExpertRows x = expert_rows(a.count, a.offset, t.e, a.R);
        t.first = x.first;
        t.m0 = (j % down) * kTileRows;
        t.n0 = (j / down) * wide;
        t.rows = min(kTileRows, a.W - t.m0);
        t.block = x.count;
        t.steps = (x.count + kStep - 1) / kStep;
        return t;
    }
    t.e = expert_of_block(base, a.E, (int)(i / p.across));
    const int down = base[t.e + 1] - base[t.e];
    const int j = (int)(i - (int64_t)base[t.e] * p.across);
    const ExpertRows x = expert_rows(a.count, a.offset, t.e, a.R);
    t.first = x.first;
    t.m0 = (j % down) * kTileRows;
    t.n0 = (j / down) * wide;
    t.rows = min(kTileRows, x.count - t.m0);
    t.block = base[t.e] + j % down;
    t.steps = (p.length + kStep - 1) / kStep;
    return t;
}

// ---- the store half ----------------------------------------------------------

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + expf(-g)); }

// 32 columns of a row from c, `left` of them inside the result (a multiple of 8).
__device__ __forceinline__ void store32(__nv_bfloat16* row, int left, const float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (8 * i < left)
            st_v4(reinterpret_cast<uint4*>(row) + i,
                  make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]),
                             pack2(v[8 * i + 4], v[8 * i + 5]), pack2(v[8 * i + 6], v[8 * i + 7])));
}
__device__ __forceinline__ void load32(const __nv_bfloat16* row, int left, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (8 * i < left) x = ld_stream_v4(reinterpret_cast<const uint4*>(row) + i);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = low(w[j]);
            v[8 * i + 2 * j + 1] = high(w[j]);
        }
    }
}
__device__ __forceinline__ void sums32(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    tc::ld32(at, r);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// A finished tile to its results; sums: tensor memory of this warp's lanes.
template <int OP, int BN, bool GLU>
__device__ __forceinline__ void store_tile(const ExpertArgs& a, const Plan& p, const Tile& t, uint32_t sums, int row) {
    const bool live = row < t.rows;
    const int64_t r = OP == kBackWeights ? (int64_t)t.e * a.W + t.m0 + row : (int64_t)t.first + t.m0 + row;
    if (GLU) {
        // accumulator columns: 64 of the gate, their 64 of up, and so on
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + r * a.N + t.n0;
        __nv_bfloat16* pre = a.pre == nullptr ? nullptr : static_cast<__nv_bfloat16*>(a.pre) + r * a.W + t.n0;
#pragma unroll 1
        for (int c = 0; c < BN / 2 && t.n0 + c < a.N; c += 32) {
            float g[32], u[32];
            const uint32_t at = sums + (c >> 6) * 128 + (c & 63);
            sums32(at, g);
            sums32(at + 64, u);
            const int left = live ? a.N - t.n0 - c : 0;
            if (pre != nullptr) {
                store32(pre + c, left, g);
                store32(pre + a.N + c, left, u);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) g[i] = g[i] * sigmoid(g[i]) * u[i];
            store32(out + c, left, g);
        }
        return;
    }
    const bool through = OP == kBackRows && a.pre_in != nullptr;
    const int64_t pitch = through ? 2 * (int64_t)p.cols : p.cols;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + r * pitch + t.n0;
    const __nv_bfloat16* pre = through ? static_cast<const __nv_bfloat16*>(a.pre_in) + r * pitch + t.n0 : nullptr;
#pragma unroll 1
    for (int c = 0; c < BN && t.n0 + c < p.cols; c += 32) {
        const int left = live ? p.cols - t.n0 - c : 0;
        float v[32];
        if (OP == kBackWeights && t.steps == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        } else {
            sums32(sums + c, v);
        }
        if (through) {
            float g[32], u[32];
            load32(pre + c, left, g);
            load32(pre + p.cols + c, left, u);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float s = sigmoid(g[i]);
                u[i] = v[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
                v[i] = v[i] * g[i] * s;
            }
            store32(out + c, left, u);
            store32(out + p.cols + c, left, v);
        } else {
            store32(out + c, left, v);
        }
    }
}

// ---- the kernel ----------------------------------------------------------------

template <int OP, int BN, bool GLU>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const ExpertArgs a, const int box_rows, const __grid_constant__ CUtensorMap map_a,
               const __grid_constant__ CUtensorMap map_b) {
    using S = Shape<OP, BN>;
    constexpr bool across_a = OP == kBackWeights, across_b = OP == kBackRows || OP == kBackWeights;
    extern __shared__ uint8_t dynamic[];
    __shared__ Shared sh;
    const uint32_t stages = (smem_u32(dynamic) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full = [&](int s) { return smem_u32(&sh.full[s]); };
    auto empty = [&](int s) { return smem_u32(&sh.empty[s]); };
    auto stage_at = [&](int s) { return stages + (uint32_t)s * S::kStageBytes; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.done[i]), 1);
            mbar_init(smem_u32(&sh.free[i]), 128);
        }
        mbar_init(smem_u32(&sh.last), 1);
        fence_mbar_init();
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b);
    }
    if (warp == 1) tc::alloc(smem_u32(&sh.tmem), S::kColumns);
    if (OP != kBackWeights) scan_row_blocks(a.count, a.offset, a.E, a.R, sh.base, sh.scratch, blocks_of_128);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const Plan p = make_plan<OP, BN, GLU>(a, sh.base);

    bool ok = true;
    int64_t issued = 0;  // stages
    if (warp == 0 && lane == 0) {
        const int groups = (a.K + 127) >> 7;                                  // of scales along a row
        const int per = GLU ? 64 : 128;
        const int wblocks = (a.N + per - 1) / per;
        for (int64_t i = blockIdx.x; i < p.tiles && ok; i += gridDim.x) {
            const Tile t = tile_at<OP, BN, GLU>(a, p, sh.base, i);
            const int boxes_a = across_a ? (t.rows + kBoxRows - 1) / kBoxRows : (t.rows + box_rows - 1) / box_rows;
            const int bytes_a = across_a ? boxes_a * kBoxBytes : boxes_a * box_rows * kRowBytes;
            // boxes of B that hold a column of the result; with a gate every other box is of the up half
            const int pieces = min((p.cols - t.n0 + kBoxRows - 1) / kBoxRows, GLU ? BN / 128 : BN / kBoxRows);
            const int boxes_b = GLU ? 2 * pieces : pieces;
            for (int kb = 0; kb < t.steps; ++kb) {
                const int s = (int)(issued % S::kStages);
                if (!wait_second(empty(s), (uint32_t)((issued / S::kStages) & 1) ^ 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = stage_at(s), sb = sa + S::kBytesA, bar = full(s);
                int bytes_s = 0, pair = 0, wb0 = 0, wbn = 0;
                if (S::k4) {
                    pair = min(2, groups - 2 * kb) * kScaleBlock;
                    wb0 = t.n0 / per;
                    wbn = min(BN / 128, wblocks - wb0);
                    bytes_s = pair * (1 + wbn);
                }
                mbar_arrive_expect_tx(bar, bytes_a + boxes_b * kBoxBytes + bytes_s);
                if (across_a) {
                    for (int j = 0; j < boxes_a; ++j)
                        tc::load2(sa + j * kBoxBytes, &map_a, t.m0 + j * 64, t.first + kb * 64, bar);
                } else {
                    for (int j = 0; j < boxes_a; ++j)
                        tc::load2(sa + j * box_rows * kRowBytes, &map_a, kb * (S::k4 ? kRowBytes : 64),
                                  t.first + t.m0 + j * box_rows, bar);
                }
                for (int j = 0; j < boxes_b; ++j) {
                    if (OP == kBackWeights)
                        tc::load2(sb + j * kBoxBytes, &map_b, t.n0 + j * 64, t.first + kb * 64, bar);
                    else if (OP == kBackRows)
                        tc::load3(sb + j * kBoxBytes, &map_b, t.n0 + j * 64, kb * 64, t.e, bar);
                    else
                        tc::load3(sb + j * kBoxBytes, &map_b, kb * (S::k4 ? kRowBytes : 64),
                                  GLU ? t.n0 + (j >> 1) * 64 + (j & 1) * a.N : t.n0 + j * 64, t.e, bar);
                }
                if (S::k4) {
                    const uint32_t ss = sb + S::kBytesB;
                    const int block = min(t.block, a.R / 128 + a.E - 1);
                    bulk_g2s(ss, static_cast<const uint8_t*>(a.row_scales) +
                                     ((int64_t)block * groups + 2 * kb) * kScaleBlock, pair, bar);
                    for (int j = 0; j < wbn; ++j)
                        bulk_g2s(ss + (1 + j) * 2 * kScaleBlock,
                                 static_cast<const uint8_t*>(a.weight_scales) +
                                     (((int64_t)t.e * wblocks + wb0 + j) * groups + 2 * kb) * kScaleBlock, pair, bar);
                }
                ++issued;
            }
        }
    } else if (warp == 1) {
        int64_t taken = 0;
        int n = 0;
        for (int64_t i = blockIdx.x; i < p.tiles && ok; i += gridDim.x, ++n) {
            const Tile t = tile_at<OP, BN, GLU>(a, p, sh.base, i);
            const int length = OP == kBackWeights ? t.block : p.length;
            const int half = n % S::kSums;
            const uint32_t sums = tmem + half * BN;
            if (!warp_wait(smem_u32(&sh.free[half]), (uint32_t)((n / S::kSums) & 1) ^ 1u)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            for (int kb = 0; kb < t.steps; ++kb) {
                const int s = (int)(taken % S::kStages);
                if (!warp_wait(full(s), (uint32_t)((taken / S::kStages) & 1))) {
                    ok = false;
                    break;
                }
                ++taken;
                tc::fence_after_sync();
                const uint32_t sa = stage_at(s), sb = sa + S::kBytesA;
                constexpr int kMma = S::k4 ? 64 : 16;                         // contraction of an instruction
                const int left = min(S::kStep, length - kb * S::kStep);
                const int count = (left + kMma - 1) / kMma;
                if (OP == kBackWeights && left % kMma != 0) {
                    // rows past the expert's last are another expert's: clear the ones that would be summed
                    const int n0 = left * 8, n1 = count * kMma * 8;           // 16-byte pieces of a box
                    for (int b = 0; b < (S::kBytesA + S::kBytesB) / kBoxBytes; ++b)
                        for (int j = n0 + lane; j < n1; j += 32)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                                         :: "r"(sa + b * kBoxBytes + j * 16), "r"(0u) : "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    if (S::k4) {
                        const uint32_t ss = sb + S::kBytesB;
                        for (int g = 0; 2 * g < count; ++g) {
                            tc::copy_scales(tmem + S::kScaleA + 4 * g, tc::at(tc::kScales, ss + g * kScaleBlock));
#pragma unroll
                            for (int j = 0; j < BN / 128; ++j)
                                tc::copy_scales(tmem + S::kScaleB + g * (BN / 32) + 4 * j,
                                                tc::at(tc::kScales, ss + ((1 + j) * 2 + g) * kScaleBlock));
                        }
                        for (int k = 0; k < count; ++k)
                            tc::mma4(sums, tc::at(tc::kAlongK, sa + k * 32), tc::at(tc::kAlongK, sb + k * 32),
                                     tc::instruction4(BN, k & 1), tmem + S::kScaleA + 4 * (k >> 1),
                                     tmem + S::kScaleB + (k >> 1) * (BN / 32), kb > 0 || k > 0);
                    } else {
                        for (int k = 0; k < count; ++k) {
                            const uint64_t da = across_a ? tc::at(tc::kAcrossK, sa + k * 2048)
                                                         : tc::at(tc::kAlongK, sa + k * 32);
                            const uint64_t db = across_b ? tc::at(tc::kAcrossK, sb + k * 2048)
                                                         : tc::at(tc::kAlongK, sb + k * 32);
                            tc::mma(sums, da, db, tc::instruction(BN, across_a, across_b), kb > 0 || k > 0);
                        }
                    }
                    tc::commit(empty(s));
                }
                __syncwarp();
            }
            if (ok && lane == 0) tc::commit(smem_u32(&sh.done[half]));
            __syncwarp();
        }
        // whatever was issued is done before tensor memory is freed
        if (lane == 0) tc::commit(smem_u32(&sh.last));
        __syncwarp();
        ok = warp_wait(smem_u32(&sh.last), 0) && ok;
    } else if (warp >= 2) {
        const int quarter = warp & 3;
        int n = 0;
        for (int64_t i = blockIdx.x; i < p.tiles; i += gridDim.x, ++n) {
            const Tile t = tile_at<OP, BN, GLU>(a, p, sh.base, i);
            const int half = n % S::kSums;
            if (!warp_wait(smem_u32(&sh.done[half]), (uint32_t)((n / S::kSums) & 1))) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            store_tile<OP, BN, GLU>(a, p, t, tmem + half * BN + ((uint32_t)(quarter * 32) << 16), quarter * 32 + lane);
            tc::fence_before_sync();
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(&sh.free[half])) : "memory");
        }
    }
    if (!ok && lane == 0) atomicOr(&g_expert4_faults, MOE_FAULT_WAIT_TIMEOUT);
    __syncwarp();
    // no copy of this CTA is in flight when it ends (each was waited for by its reader unless a wait gave up)
    if (warp == 0 && lane == 0)
        for (int64_t i = max((int64_t)0, issued - S::kStages); i < issued; ++i)
            wait_second(full((int)(i % S::kStages)), (uint32_t)((i / S::kStages) & 1));
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::dealloc(tmem, S::kColumns);
}

// ---- host side ---------------------------------------------------------------------

template <int OP, int BN, bool GLU>
cudaError_t launch(const ExpertArgs& a, int box_rows, cudaStream_t s) {
    using S = Shape<OP, BN>;
    CUtensorMap ma, mb;
    bool ok;
    if (OP == kForward4)
        ok = tc::make_map(&ma, a.rows, true, a.K / 2, a.R, 0, box_rows) &&
             tc::make_map(&mb, a.weights, true, a.K / 2, a.W, a.E, kBoxRows);
    else if (OP == kBackWeights)
        ok = tc::make_map(&ma, a.dout, false, a.W, a.R, 0, kBoxRows) && tc::make_map(&mb, a.rows, false, a.K, a.R, 0, kBoxRows);
    else
        ok = tc::make_map(&ma, OP == kForward ? a.rows : a.dout, false, OP == kForward ? a.K : a.W, a.R, 0, box_rows) &&
             tc::make_map(&mb, a.weights, false, a.K, a.W, a.E, kBoxRows);
    if (!ok) return cudaErrorInvalidValue;
    auto* kern = product_kernel<OP, BN, GLU>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), S::kSmem);
    if (e != cudaSuccess) return e;
    // no more CTAs than there can be tiles
    const int cols = OP == kForward || OP == kForward4 ? a.N : a.K;
    const int wide = GLU ? BN / 2 : BN;
    const int64_t across = (cols + wide - 1) / wide;
    const int64_t tiles = across * (OP == kBackWeights ? (int64_t)a.E * ((a.W + kTileRows - 1) / kTileRows)
                                                       : a.R / kTileRows + (int64_t)(a.E < a.R ? a.E : a.R));
    const int sms = device_sm_count();
    kern<<<(unsigned)(tiles < sms ? tiles : sms), kThreads, S::kSmem, s>>>(a, box_rows, ma, mb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_forward4(const ExpertArgs& a, cudaStream_t s) {
    return a.glu ? launch<kForward4, 256, true>(a, kBoxRows, s) : launch<kForward4, 256, false>(a, kBoxRows, s);
}

cudaError_t read_expert4_faults(uint32_t* bits, cudaStream_t stream) {
    unsigned v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_expert4_faults, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_expert4_faults, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice,
                                                      stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess) *bits = v;
    return e;
}

}  // namespace moe
