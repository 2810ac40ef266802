// moe_experts.cu -- products grouped by expert over ragged receive rows
// ("Balancing and Beyond", section 1: the experts between dispatch and
// combine).
//
// The plainest form that is right for every case: one 64 x 64 tile of a result
// per block and step, operands staged in shared memory as fp32, 4 x 4 sums a
// thread.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_experts.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;
constexpr int kForward = 0, kBackRows = 1, kBackWeights = 2, kForward4 = 3;

__device__ __forceinline__ float bf(const void* p, int64_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Value of column k of a row of 4-bit codes; scales: the row's place in its scale blocks.
__device__ __forceinline__ float value4(const uint8_t* codes, const uint8_t* scales, int k) {
    const float mag[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
    const int c = (codes[k >> 1] >> (4 * (k & 1))) & 15;
    const uint32_t b = scales[(int64_t)(k >> 7) * 512 + ((k >> 5) & 3)];
    const float x = b == 255u ? NAN : b == 0u ? __uint_as_float(1u << 22) : __uint_as_float(b << 23);
    return (c & 8 ? -mag[c & 7] : mag[c & 7]) * x;
}

// Grid: x over tiles of result columns, y over experts.
template <int MODE, bool GLU>
__global__ void __launch_bounds__(kThreads) plain_kernel(ExpertArgs a) {
    __shared__ float sa[kStep][kTile + 1], sb[GLU ? 2 : 1][kStep][kTile + 1];
    __shared__ int base[MOE_MAX_EXPERTS + 1], scratch[32];
    const int e = blockIdx.y, n0 = blockIdx.x * kTile, tid = threadIdx.x;
    const ExpertRows x = expert_rows(a.count, a.offset, e, a.R);
    if (MODE == kForward4) scan_row_blocks(a.count, a.offset, a.E, a.R, base, scratch);
    const int M = MODE == kBackWeights ? a.W : x.count;
    const int N = MODE == kForward || MODE == kForward4 ? a.N : a.K;
    const int K = MODE == kBackRows ? a.W : MODE == kBackWeights ? x.count : a.K;
    const int64_t groups = (a.K + 127) >> 7;

    auto left = [&](int m, int k) -> float {
        const int64_t r = x.first + (MODE == kBackWeights ? k : m);
        if (MODE == kForward) return bf(a.rows, r * a.K + k);
        if (MODE == kBackRows) return bf(a.dout, r * a.W + k);
        if (MODE == kBackWeights) return bf(a.dout, r * a.W + m);
        const int block = base[e] + (m >> 7);
        if (block >= a.R / 128 + a.E) return 0.0f;
        return value4(static_cast<const uint8_t*>(a.rows) + r * (a.K / 2),
                      static_cast<const uint8_t*>(a.row_scales) + block * groups * 512 + scale_byte(m & 127, 0), k);
    };
    auto right = [&](int n, int k, int half) -> float {
        const int64_t w = (int64_t)e * a.W + (half ? a.N : 0);
        if (MODE == kForward) return bf(a.weights, (w + n) * a.K + k);
        if (MODE == kBackRows) return bf(a.weights, (w + k) * a.K + n);
        if (MODE == kBackWeights) return bf(a.rows, (int64_t)(x.first + k) * a.K + n);
        const int per = GLU ? 64 : 128;
        const int64_t block = (int64_t)e * ((a.N + per - 1) / per) + n / per;
        return value4(static_cast<const uint8_t*>(a.weights) + (w + n) * (a.K / 2),
                      static_cast<const uint8_t*>(a.weight_scales) + block * groups * 512 +
                          scale_byte(n % per + 64 * half, 0), k);
    };

    for (int m0 = 0; m0 < M; m0 += kTile) {
        float acc[GLU ? 2 : 1][4][4] = {};
        for (int k0 = 0; k0 < K; k0 += kStep) {
            for (int i = tid; i < kStep * kTile; i += kThreads) {
                const int k = i % kStep, c = i / kStep;
                const bool in = k0 + k < K;
                sa[k][c] = in && m0 + c < M ? left(m0 + c, k0 + k) : 0.0f;
#pragma unroll
                for (int half = 0; half < (GLU ? 2 : 1); ++half)
                    sb[half][k][c] = in && n0 + c < N ? right(n0 + c, k0 + k, half) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < kStep; ++k)
#pragma unroll
                for (int half = 0; half < (GLU ? 2 : 1); ++half)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[half][i][j] = fmaf(sa[k][(tid / 16) * 4 + i], sb[half][k][(tid % 16) * 4 + j],
                                                   acc[half][i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + (tid / 16) * 4 + i, n = n0 + (tid % 16) * 4 + j;
                if (m >= M || n >= N) continue;
                const int64_t r = x.first + m;
                const float p = acc[0][i][j];
                if (MODE == kBackWeights) {
                    put(a.out, ((int64_t)e * a.W + m) * a.K + n, p);
                } else if (MODE == kBackRows) {
                    if (a.pre_in == nullptr) {
                        put(a.out, r * a.K + n, p);
                    } else {
                        const float g = bf(a.pre_in, r * 2 * a.K + n), u = bf(a.pre_in, r * 2 * a.K + a.K + n);
                        const float s = 1.0f / (1.0f + expf(-g));
                        put(a.out, r * 2 * a.K + n, p * u * s * (1.0f + g * (1.0f - s)));
                        put(a.out, r * 2 * a.K + a.K + n, p * g * s);
                    }
                } else if (GLU) {
                    const float u = acc[GLU ? 1 : 0][i][j];
                    put(a.out, r * a.N + n, p / (1.0f + expf(-p)) * u);
                    if (a.pre != nullptr) {
                        put(a.pre, r * a.W + n, p);
                        put(a.pre, r * a.W + a.N + n, u);
                    }
                } else {
                    put(a.out, r * a.N + n, p);
                }
            }
    }
}

template <int MODE, bool GLU>
cudaError_t launch(const ExpertArgs& a, int N, cudaStream_t s) {
    plain_kernel<MODE, GLU><<<dim3((N + kTile - 1) / kTile, a.E), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_forward(const ExpertArgs& a, cudaStream_t s) {
    return a.glu ? launch<kForward, true>(a, a.N, s) : launch<kForward, false>(a, a.N, s);
}
cudaError_t launch_expert_backward_rows(const ExpertArgs& a, cudaStream_t s) {
    return launch<kBackRows, false>(a, a.K, s);
}
cudaError_t launch_expert_backward_weights(const ExpertArgs& a, cudaStream_t s) {
    return launch<kBackWeights, false>(a, a.K, s);
}
cudaError_t launch_expert_forward4(const ExpertArgs& a, cudaStream_t s) {
    return a.glu ? launch<kForward4, true>(a, a.N, s) : launch<kForward4, false>(a, a.N, s);
}

}  // namespace moe
