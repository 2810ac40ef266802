// moe_quant4.cu -- bf16 rows to microscaled 4-bit floating point (MXFP4: E2M1
// codes, one E8M0 scale per 32 columns).
//
// A scale is a power of two, so x / X is exact and the code's own rounding (to
// nearest, ties to even, saturated at 6) is the only one.  The exponent is that
// of the block's largest magnitude less 2, the exponent of E2M1's largest
// value: the largest magnitude lands in [4, 8), and what lands above 6 is
// saturated.
//
// HBM-bound: 64 bytes in, 17 out, per 32 columns: 32768 rows of 7168 columns in
// 95 us (6.3 TB/s of 6.8), 128 rows in 6.7 us (4.7 in a run of such calls).  A block takes 128 rows of 1024
// columns: smaller ones (32 rows: 96 us), blocks of 2048 columns (100 us)
// or blocks that stay and take one piece after another (100 us) measured slower.
// Where those would be few, though, and experts have some dozens of rows, four blocks share
// one: 8192 rows of 8 experts take 26 us and not 38, 1840 rows of 16 experts, 2336 columns, 6.6 and not 11.5; with
// one row of 128 experts (one block per expert and piece either way) it would be 10.7 and not 4.7 us, in a run of such calls.
// Two lanes share a scale, 16 columns each (one 32-byte load), so a warp takes 512
// columns of a row: 256 bytes of codes and four 4-byte words of scales.  With four
// lanes a scale and 16-byte loads the warps' shuffles and index arithmetic,
// paid twice as often, bound it (106 us; 112 with magnitudes compared one by one).
// The next row's loads ahead of the current one's arithmetic gave nothing (95 us) and
// cost the blocks of a decode their single wave (128 rows: 8.7 us).

#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_runtime.h>

#include "moe_experts.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

constexpr int kPiece = 1024;  // columns of a row a warp takes: two loads of 512 in flight

// 16 columns at p to w.  wide: p lies on 32 bytes.
__device__ __forceinline__ void load16(uint32_t* w, const uint16_t* p, bool wide) {
    if (wide) {
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = ld_stream_v4(reinterpret_cast<const uint4*>(p) + i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}

// The codes of 8 columns, times inv.
__device__ __forceinline__ uint32_t codes8(const uint32_t* w, float inv) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = make_float2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
        const uint32_t two = __nv_cvt_float2_to_fp4x2(x, __NV_E2M1, cudaRoundNearest);
        out |= two << (8 * i);
    }
    return out;
}

// 512 columns of a row, c0 + 16 lane on this lane (cols: a multiple of 32), already loaded (w; 0 past the end).  Codes go
// to the row's codes, scales to the 4-byte words of the row's place in the scale blocks: word g of the row is at sc + 512 g.
__device__ __forceinline__ void quantise512(const uint32_t* w, uint8_t* codes, uint8_t* sc, int c0, int cols, int lane) {
    const int c = c0 + 16 * lane;
    const bool live = c < cols;
    // magnitudes as integers order as the floats do; bf16 is 16 bits, so two are compared at once
    uint32_t two = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) two = __vmaxs2(two, w[i] & 0x7fff7fffu);
    two = __vmaxs2(two, __shfl_xor_sync(kFull, two, 1));
    const uint32_t exponent = max(two >> 16, two & 0xffffu) >> 7;
    const bool bad = exponent == 255u;
    const uint32_t b = bad ? 255u : (exponent > 2u ? exponent - 2u : 0u);
    const float inv = __uint_as_float((254u - min(b, 253u)) << 23);  // 2^(127 - b)
    const uint2 out = make_uint2(codes8(w, inv), codes8(w + 4, inv));
    if (live) *reinterpret_cast<uint2*>(codes + (c >> 1)) = bad ? make_uint2(0u, 0u) : out;
    // the four scales of 128 columns meet in their first lane (0, 8, 16, 24); past the last column the scale byte is 0
    uint32_t word = live ? b : 0u;
    word |= __shfl_down_sync(kFull, word, 2) << 8;
    word |= __shfl_down_sync(kFull, word, 4) << 16;
    if ((lane & 7) == 0 && live) *reinterpret_cast<uint32_t*>(sc + (int64_t)(c >> 7) * 512) = word;
}

// Columns c0 .. c0 + 1024 of a row (bf16) to its codes and scales.
__device__ __forceinline__ void quantise_piece(const uint16_t* row, bool wide, uint8_t* codes, uint8_t* sc, int c0, int cols,
                                               int lane) {
    uint32_t w[kPiece / 512][8] = {};
#pragma unroll
    for (int i = 0; i < kPiece / 512; ++i) {
        const int c = c0 + 512 * i + 16 * lane;
        if (c < cols) load16(w[i], row + c, wide);
    }
#pragma unroll
    for (int i = 0; i < kPiece / 512; ++i)
        if (c0 + 512 * i < cols) quantise512(w[i], codes, sc, c0 + 512 * i, cols, lane);
}

// Rows are a multiple of 64 bytes, so all lie on 32 bytes where the first does.
__device__ __forceinline__ bool on_32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// One block of the grid per (row block, piece of 1024 columns, share of its rows); the row blocks
// of the experts follow one another, and the grid covers the most there can be.
__global__ void __launch_bounds__(kThreads)
quant4_rows_kernel(ExpertArgs a, uint8_t* codes, uint8_t* scales) {
    __shared__ int base[MOE_MAX_EXPERTS + 1], scratch[32];
    pdl_wait();
    pdl_launch_dependents();
    scan_row_blocks(a.count, a.offset, a.E, a.R, base, scratch, blocks_of_128);
    const int block = blockIdx.x;
    if (block >= base[a.E]) return;
    const int e = expert_of_block(base, a.E, block);
    const ExpertRows x = expert_rows(a.count, a.offset, e, a.R);
    const int i0 = (block - base[e]) * 128;
    const int n = min(128, x.count - i0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (a.K + 127) >> 7;
    uint8_t* sc = scales + (int64_t)block * groups * 512;
    const bool wide = on_32(a.rows);
    const int share = 128 / gridDim.z, from = blockIdx.z * share;
    for (int i = from + warp; i < min(n, from + share); i += kWarps) {
        const int64_t r = x.first + i0 + i;
        quantise_piece(static_cast<const uint16_t*>(a.rows) + r * a.K, wide, codes + r * (a.K / 2), sc + scale_byte(i, 0),
                       blockIdx.y * kPiece, a.K, lane);
    }
}

// One block per (128-row scale block of an expert's weights); with a gated
// activation the scale block holds 64 gate rows and then their 64 up rows.
__global__ void __launch_bounds__(kThreads)
quant4_weights_kernel(ExpertArgs a, uint8_t* codes, uint8_t* scales) {
    pdl_wait();
    pdl_launch_dependents();
    const int per = a.glu ? 64 : 128;
    const int blocks = (a.N + per - 1) / per;
    const int64_t e = blockIdx.x / blocks;
    const int b = blockIdx.x % blocks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (a.K + 127) >> 7;
    uint8_t* sc = scales + (int64_t)blockIdx.x * groups * 512;
    const bool wide = on_32(a.weights);
    for (int i = warp; i < 128; i += kWarps) {
        const int n = b * per + i % per;                 // result column
        if (n >= a.N) continue;
        const int64_t r = e * a.W + n + (i >= per ? a.N : 0);
        quantise_piece(static_cast<const uint16_t*>(a.weights) + r * a.K, wide, codes + r * (a.K / 2), sc + scale_byte(i, 0),
                       blockIdx.y * kPiece, a.K, lane);
    }
}

}  // namespace

cudaError_t launch_quant4_rows(const ExpertArgs& a, void* codes, void* scales, cudaStream_t s) {
    const int64_t blocks = a.R / 128 + min(a.E, a.R), pieces = (a.K + kPiece - 1) / kPiece;
    const bool share = a.R >= 32 * (int64_t)a.E && blocks * pieces <= 8 * device_sm_count();
    const dim3 grid((unsigned)blocks, (unsigned)pieces, share ? 4u : 1u);
    return launch_pdl(quant4_rows_kernel, grid, dim3(kThreads), 0, s, a, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}

cudaError_t launch_quant4_weights(const ExpertArgs& a, void* codes, void* scales, cudaStream_t s) {
    const int per = a.glu ? 64 : 128;
    const dim3 grid((unsigned)((int64_t)a.E * ((a.N + per - 1) / per)), (unsigned)((a.K + kPiece - 1) / kPiece));
    return launch_pdl(quant4_weights_kernel, grid, dim3(kThreads), 0, s, a, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}

}  // namespace moe
