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
// 112 us (5.3 TB/s of 6.8), 128 rows in 6.7 us.  A block takes 128 rows of 1024
// columns: smaller ones (32 rows: 122 us), or blocks that stay and take one piece of
// work after another (32 rows: 128 us), spend more on finding their expert than
// their better balance gives.  Four lanes share a block, 8
// columns each (one 16-byte load), so a warp takes 256 columns of a row: 128
// bytes of codes and two 4-byte words of scales.

#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_runtime.h>

#include "moe_experts.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

constexpr int kPiece = 1024;  // columns of a row a warp takes: four loads of 256 in flight

// 256 columns of a row, c0 + 8 lane on this lane (cols: a multiple of 32), already loaded (v; 0 past the end).  Codes go
// to the row's codes, scales to the 4-byte words of the row's place in the scale blocks: word g of the row is at sc + 512 g.
__device__ __forceinline__ void quantise256(uint4 v, uint32_t* codes, uint8_t* sc, int c0, int cols, int lane) {
    const int c = c0 + 8 * lane;
    const bool live = c < cols;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    // magnitudes as integers order as the floats do; bf16 is the upper half
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    const uint32_t exponent = top >> 7;
    const bool bad = exponent == 255u;
    const uint32_t b = bad ? 255u : (exponent > 2u ? exponent - 2u : 0u);
    const float inv = __uint_as_float((254u - min(b, 253u)) << 23);  // 2^(127 - b)
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = make_float2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
        const uint32_t two = __nv_cvt_float2_to_fp4x2(x, __NV_E2M1, cudaRoundNearest);
        out |= two << (8 * i);
    }
    if (live) codes[c >> 3] = bad ? 0u : out;
    // the four scales of 128 columns meet in their first lane (0 and 16); past the last column the scale byte is 0
    uint32_t word = live ? b : 0u;
    word |= __shfl_down_sync(kFull, word, 4) << 8;
    word |= __shfl_down_sync(kFull, word, 8) << 16;
    const int col = c0 + 8 * (lane & 16);
    if ((lane & 15) == 0 && col < cols) *reinterpret_cast<uint32_t*>(sc + (int64_t)(col >> 7) * 512) = word;
}

// Columns c0 .. c0 + 1024 of a row (bf16) to its codes and scales.
__device__ __forceinline__ void quantise_piece(const void* row, uint8_t* codes, uint8_t* sc, int c0, int cols, int lane) {
    uint4 v[kPiece / 256];
#pragma unroll
    for (int i = 0; i < kPiece / 256; ++i) {
        const int c = c0 + 256 * i + 8 * lane;
        v[i] = c < cols ? ld_stream_v4(static_cast<const uint4*>(row) + (c >> 3)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kPiece / 256; ++i)
        if (c0 + 256 * i < cols) quantise256(v[i], reinterpret_cast<uint32_t*>(codes), sc, c0 + 256 * i, cols, lane);
}

// One block of the grid per (row block, piece of 1024 columns); the row blocks
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
    for (int i = warp; i < n; i += kWarps) {
        const int64_t r = x.first + i0 + i;
        quantise_piece(static_cast<const uint16_t*>(a.rows) + r * a.K, codes + r * (a.K / 2), sc + scale_byte(i, 0),
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
    for (int i = warp; i < 128; i += kWarps) {
        const int n = b * per + i % per;                 // result column
        if (n >= a.N) continue;
        const int64_t r = e * a.W + n + (i >= per ? a.N : 0);
        quantise_piece(static_cast<const uint16_t*>(a.weights) + r * a.K, codes + r * (a.K / 2), sc + scale_byte(i, 0),
                       blockIdx.y * kPiece, a.K, lane);
    }
}

}  // namespace

cudaError_t launch_quant4_rows(const ExpertArgs& a, void* codes, void* scales, cudaStream_t s) {
    const dim3 grid((unsigned)(a.R / 128 + min(a.E, a.R)), (unsigned)((a.K + kPiece - 1) / kPiece));
    return launch_pdl(quant4_rows_kernel, grid, dim3(kThreads), 0, s, a, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}

cudaError_t launch_quant4_weights(const ExpertArgs& a, void* codes, void* scales, cudaStream_t s) {
    const int per = a.glu ? 64 : 128;
    const dim3 grid((unsigned)((int64_t)a.E * ((a.N + per - 1) / per)), (unsigned)((a.K + kPiece - 1) / kPiece));
    return launch_pdl(quant4_weights_kernel, grid, dim3(kThreads), 0, s, a, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}

}  // namespace moe
