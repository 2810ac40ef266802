// moe_quant8.cu -- bf16 rows to 8-bit integers with one fp32 scale a row.
//
//   s = m / 127,  c = x (127 / m) rounded to nearest, ties to even,  m = largest |x| of the row
//
// A block takes a row: its largest magnitude, then its codes.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_experts.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

// Largest magnitude of two packed bf16 each (as integers they order as the floats do).
__device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w) { return __vmaxs2(top, w & 0x7fff7fffu); }

__device__ __forceinline__ uint32_t code(float x, float inv) { return (uint32_t)__float2int_rn(x * inv) & 0xffu; }

// 8 columns to 8 codes.
__device__ __forceinline__ uint2 codes8(uint4 v, float lift, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[2] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(w[i] << 16) * lift, hi = __uint_as_float(w[i] & 0xffff0000u) * lift;
        out[i / 2] |= (code(lo, inv) | code(hi, inv) << 8) << (16 * (i & 1));
    }
    return make_uint2(out[0], out[1]);
}

__global__ void __launch_bounds__(kThreads)
quant8_kernel(const uint4* __restrict__ rows, int nvec, uint2* __restrict__ codes, float* __restrict__ scales) {
    __shared__ uint32_t part[kThreads / 32];
    const int64_t r = blockIdx.x;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    uint32_t top = 0;
    for (int c = tid; c < nvec; c += kThreads) {
        const uint4 v = rows[r * nvec + c];
        top = larger(larger(larger(larger(top, v.x), v.y), v.z), v.w);
    }
    top = __reduce_max_sync(kFull, max(top >> 16, top & 0xffffu));
    if ((tid & 31) == 0) part[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, part[i]);
    const bool bad = top >= 0x7f80u;
    const float m = __uint_as_float(top << 16);
    const float lift = m < 0x1p-100f ? 0x1p100f : 1.0f;   // 127 / m stays finite
    const float inv = bad || m == 0.0f ? 0.0f : 127.0f / (m * lift);
    if (tid == 0) scales[r] = bad ? NAN : m == 0.0f ? 1.0f : m / 127.0f;
    for (int c = tid; c < nvec; c += kThreads)
        codes[r * nvec + c] = bad ? make_uint2(0u, 0u) : codes8(rows[r * nvec + c], lift, inv);
}

}  // namespace

cudaError_t launch_quant8(const void* rows, int64_t count, int cols, int8_t* codes, float* scales, cudaStream_t s) {
    return launch_pdl(quant8_kernel, dim3((unsigned)count), dim3(kThreads), 0, s, static_cast<const uint4*>(rows), cols / 8,
                      reinterpret_cast<uint2*>(codes), scales);
}

}  // namespace moe
