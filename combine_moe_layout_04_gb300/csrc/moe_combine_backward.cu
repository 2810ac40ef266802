// moe_combine_backward.cu -- the gradient of the gate-weighted sum: expert
// output rows and gates in one pass ("Balancing and Beyond", section 1).
//
//   dy[pos[t, j]] = bf16(w[t, j] dout[t]),  dw[t, j] = <dout[t], y[pos[t, j]]>
//
// HBM-bound: per token it reads one row and k rows and writes k rows, 4 flops
// an element: 16384 tokens, top-8, h = 7168 (4.0 GB) take 588 us, 6.78 TB/s, what a
// plain copy moves.  A block owns a token, so that dout is read once and the dot
// products end in the block, in an order that the sizes and the device's SMs fix: a thread takes
// every THREADS-th group of 8 columns, then come the lanes, then the warps.  Two,
// four or eight slots' loads are issued together, by the least that takes k: registers for slots that are not
// there would leave room for fewer blocks (16384 tokens, h = 7168: top-1 105 us with two slots and 165 with eight, top-2
// 172 and 214, top-4 311 with four and 323 with eight; top-2, h = 2048: 51 and 77).
//
// The block's size, both sides measured (us): with many tokens threads without columns only
// take room from other blocks (4096 tokens: h = 512, top-10, 14.6 with 64 threads and 47.2 with 256; h = 2048, top-8,
// 45.6 with 128 and 55.1 with 256; 16384 tokens, h = 7168: 588 with 128, 608 with 256, 685 with 512).  With few
// tokens a block should have its row in flight at once (131 tokens, h = 7168: 9.5 with 128, 6.8 with 256, 5.8 with 512).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float2 wide2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// SLOTS are taken at a time.
template <int THREADS, int SLOTS>
__global__ void __launch_bounds__(THREADS)
combine_backward_kernel(const int32_t* __restrict__ pos, int k, int nvec, int R, const uint4* __restrict__ dout,
                        const uint4* __restrict__ y, const float* __restrict__ weights, uint4* __restrict__ dy,
                        float* __restrict__ dweights) {
    constexpr int kWarps = THREADS / 32;
    __shared__ float part[kWarps][SLOTS];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch_dependents();
    for (int j0 = 0; j0 < k; j0 += SLOTS) {
        int64_t row[SLOTS];
        float w[SLOTS], acc[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const bool live = j0 + j < k;
            const int r = live ? pos[t * k + j0 + j] : -1;
            row[j] = r >= 0 && r < R ? (int64_t)r * nvec : -1;
            w[j] = live ? weights[t * k + j0 + j] : 0.0f;
            acc[j] = 0.0f;
        }
        for (int c = tid; c < nvec; c += THREADS) {
            const uint4 d = dout[t * nvec + c];
            uint4 v[SLOTS];
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
                if (row[j] >= 0) v[j] = ld_stream_v4(y + row[j] + c);
            const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                if (row[j] < 0) continue;
                const uint32_t yw[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                uint32_t o[4];
                float sum = 0.0f;  // of the group by itself: fewer roundings in a row than one chain over the thread's columns
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 g = wide2(dw[i]), x = wide2(yw[i]);
                    sum = fmaf(g.x, x.x, sum);
                    sum = fmaf(g.y, x.y, sum);
                    const __nv_bfloat162 p = __floats2bfloat162_rn(w[j] * g.x, w[j] * g.y);
                    o[i] = *reinterpret_cast<const uint32_t*>(&p);
                }
                acc[j] += sum;
                st_v4(dy + row[j] + c, make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], s);
            if (lane == 0) part[warp][j] = acc[j];
        }
        __syncthreads();
        if (tid < SLOTS && j0 + tid < k) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) sum += part[i][tid];
            dweights[t * k + j0 + tid] = sum;
        }
        __syncthreads();
    }
}

template <int THREADS, int SLOTS>
cudaError_t launch(const int32_t* pos, int T, int k, int h, const void* dout, const void* y, const float* weights, void* dy,
                   float* dweights, cudaStream_t s) {
    return launch_pdl(combine_backward_kernel<THREADS, SLOTS>, dim3(T), dim3(THREADS), 0, s, pos, k, h / 8, T * k,
                      static_cast<const uint4*>(dout), static_cast<const uint4*>(y), weights, static_cast<uint4*>(dy),
                      dweights);
}
template <int THREADS>
cudaError_t launch(const int32_t* pos, int T, int k, int h, const void* dout, const void* y, const float* weights, void* dy,
                   float* dweights, cudaStream_t s) {
    if (k <= 2) return launch<THREADS, 2>(pos, T, k, h, dout, y, weights, dy, dweights, s);
    if (k <= 4) return launch<THREADS, 4>(pos, T, k, h, dout, y, weights, dy, dweights, s);
    return launch<THREADS, 8>(pos, T, k, h, dout, y, weights, dy, dweights, s);
}

}  // namespace

cudaError_t launch_combine_backward(const int32_t* pos, int T, int k, int h, const void* dout, const void* y,
                                    const float* weights, void* dy, float* dweights, cudaStream_t s) {
    // a thread for every 8 columns, up to 128 threads where the tokens fill the GPU anyway
    const int sms = device_sm_count();
    const int most = T <= sms ? 512 : T <= 4 * sms ? 256 : 128, want = h / 8 < most ? h / 8 : most;
    if (want <= 32) return launch<32>(pos, T, k, h, dout, y, weights, dy, dweights, s);
    if (want <= 64) return launch<64>(pos, T, k, h, dout, y, weights, dy, dweights, s);
    if (want <= 128) return launch<128>(pos, T, k, h, dout, y, weights, dy, dweights, s);
    if (want <= 256) return launch<256>(pos, T, k, h, dout, y, weights, dy, dweights, s);
    return launch<512>(pos, T, k, h, dout, y, weights, dy, dweights, s);
}

}  // namespace moe
