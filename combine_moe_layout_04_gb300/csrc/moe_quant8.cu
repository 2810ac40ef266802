// moe_quant8.cu -- bf16 rows to 8-bit integers with one fp32 scale a row.
//
//   s = m / 127,  c = x (127 / m) rounded to nearest, ties to even,  m = largest |x| of the row
//
// A row is read once: its threads keep it in registers, 16 columns (32 bytes) a lane at a time and up to four times,
// while they find its largest magnitude.  A warp takes rows of up to 2048 columns, a block of 128 threads up to
// 8192, one of 512 up to 32768; longer rows are read twice.
//
// HBM-bound: 2 bytes in and 1 out a column, 32768 rows of 7168 in 99 us (7.1 TB/s; a block of 256 threads reading every row twice,
// the second time out of L2, took 113), 11994 rows of 1424 in 6.9 (14.3), 128 rows of 7168 in 4.9 us of host time.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kTimes = 4;              // units of 16 columns a thread keeps

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

// Largest magnitudes of the two halves (as integers they order as the floats do, infinity and NaN above all).
__device__ __forceinline__ uint32_t larger16(uint32_t top, const uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxs2(top, w[i] & 0x7fff7fffu);
    return top;
}

// The low byte of the result is x * inv rounded to an integer: 1.5 * 2^23 leaves no bits for a fraction.  (The product is
// rounded first, so that a code does not depend on how the two are put together.)
__device__ __forceinline__ uint32_t rounded(float x, float inv) {
    return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
}

// How a row becomes codes.
struct Scale {
    float lift, inv, value;            // x * lift * inv; value: the row's scale
    bool bad;
};
__device__ __forceinline__ Scale scale_of(uint32_t top) {
    Scale s;
    const float m = __uint_as_float(top << 16);
    s.bad = top >= 0x7f80u;
    s.lift = m < 0x1p-100f ? 0x1p100f : 1.0f;             // so that 127 / m stays finite
    s.inv = s.bad || m == 0.0f ? 0.0f : 127.0f / (m * s.lift);
    s.value = s.bad ? NAN : m == 0.0f ? 1.0f : m / 127.0f;
    return s;
}

__device__ __forceinline__ void codes16(const uint32_t* w, const Scale& s, int8_t* codes) {
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            c[2 * j] = rounded(__uint_as_float(w[2 * i + j] << 16) * s.lift, s.inv);
            c[2 * j + 1] = rounded(__uint_as_float(w[2 * i + j] & 0xffff0000u) * s.lift, s.inv);
        }
        out[i] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
    st_v4(reinterpret_cast<uint4*>(codes), s.bad ? make_uint4(0, 0, 0, 0) : make_uint4(out[0], out[1], out[2], out[3]));
}

// A row to THREADS threads (32: blocks of four such rows).  KEEP: the row fits their registers.
constexpr int kRowsOfWarps = 4;
template <int THREADS, bool KEEP>
__global__ void __launch_bounds__(THREADS == 32 ? 32 * kRowsOfWarps : THREADS)
quant8_kernel(const uint16_t* __restrict__ rows, int64_t count, int cols, int8_t* __restrict__ codes, float* __restrict__ scales) {
    constexpr int kWarps = THREADS / 32;
    __shared__ uint32_t part[kWarps];
    const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t r = THREADS == 32 ? (int64_t)blockIdx.x * kRowsOfWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (THREADS == 32 && r >= count) return;
    const uint16_t* row = rows + r * cols;
    const bool wide = (reinterpret_cast<uintptr_t>(rows) & 31) == 0;  // rows are a multiple of 32 bytes
    uint32_t w[KEEP ? kTimes : 1][8] = {}, top = 0;
    if (KEEP) {
#pragma unroll
        for (int i = 0; i < kTimes; ++i)
            if (16 * (tid + i * THREADS) < cols) load16(w[i], row + 16 * (tid + i * THREADS), wide);
#pragma unroll
        for (int i = 0; i < kTimes; ++i) top = larger16(top, w[i]);
    } else {
        for (int c = 16 * tid; c < cols; c += 16 * THREADS) {
            load16(w[0], row + c, wide);
            top = larger16(top, w[0]);
        }
    }
    top = __reduce_max_sync(kFull, max(top >> 16, top & 0xffffu));
    if (THREADS > 32) {
        if ((tid & 31) == 0) part[tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = max(top, part[i]);
    }
    const Scale s = scale_of(top);
    if (tid == 0) scales[r] = s.value;
    int8_t* to = codes + r * cols;
    if (KEEP) {
#pragma unroll
        for (int i = 0; i < kTimes; ++i)
            if (16 * (tid + i * THREADS) < cols) codes16(w[i], s, to + 16 * (tid + i * THREADS));
    } else {
        for (int c = 16 * tid; c < cols; c += 16 * THREADS) {
            load16(w[0], row + c, wide);
            codes16(w[0], s, to + c);
        }
    }
}

template <int THREADS, bool KEEP>
cudaError_t launch(const void* rows, int64_t count, int cols, int8_t* codes, float* scales, cudaStream_t s) {
    const int64_t blocks = THREADS == 32 ? (count + kRowsOfWarps - 1) / kRowsOfWarps : count;
    return launch_pdl(quant8_kernel<THREADS, KEEP>, dim3((unsigned)blocks), dim3(THREADS == 32 ? 32 * kRowsOfWarps : THREADS),
                      0, s, static_cast<const uint16_t*>(rows), count, cols, codes, scales);
}

}  // namespace

cudaError_t launch_quant8(const void* rows, int64_t count, int cols, int8_t* codes, float* scales, cudaStream_t s) {
    const int units = cols / 16;
    if (units <= 32 * kTimes) return launch<32, true>(rows, count, cols, codes, scales, s);
    if (units <= 128 * kTimes) return launch<128, true>(rows, count, cols, codes, scales, s);
    if (units <= 512 * kTimes) return launch<512, true>(rows, count, cols, codes, scales, s);
    return launch<512, false>(rows, count, cols, codes, scales, s);
}

}  // namespace moe
