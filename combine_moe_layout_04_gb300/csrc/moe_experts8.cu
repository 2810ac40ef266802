// moe_experts8.cu -- products of 8-bit integers grouped by expert over ragged
// receive rows ("Balancing and Beyond", section 1: the experts between dispatch
// and combine).
//
//   p[r][f] = s_row[r] s_weight[f] sum over k of c_row[r][k] c_weight[f][k]
//
// A block computes 64 rows by 64 features of one expert on the CUDA cores.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_experts.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 64, kThreads = 256;

__global__ void __launch_bounds__(kThreads) forward8_kernel(ExpertArgs a) {
    __shared__ int base[MOE_MAX_EXPERTS + 1], scratch[32];
    __shared__ int x[kTile][kStep / 4 + 1], w[2][kTile][kStep / 4 + 1];
    pdl_wait();
    pdl_launch_dependents();
    scan_row_blocks(a.count, a.offset, a.E, a.R, base, scratch, [](int rows) { return tiles_of(rows, kTile); });
    if ((int)blockIdx.x >= base[a.E]) return;
    const int e = expert_of_block(base, a.E, blockIdx.x);
    const ExpertRows own = expert_rows(a.count, a.offset, e, a.R);
    const int m0 = (blockIdx.x - base[e]) * kTile, f0 = blockIdx.y * kTile;
    const int rows = min(kTile, own.count - m0), halves = a.glu ? 2 : 1;
    const int tr = threadIdx.x / 16 * 4, tf = threadIdx.x % 16 * 4;
    float sum[2][4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kStep) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * kStep / 4; i += kThreads) {
            const int r = i / (kStep / 4), c = i % (kStep / 4);
            const bool in = k0 + 4 * c < a.K;
            x[r][c] = in && r < rows ? *reinterpret_cast<const int*>(static_cast<const int8_t*>(a.rows) +
                                                                     (int64_t)(own.first + m0 + r) * a.K + k0 + 4 * c) : 0;
            for (int h = 0; h < halves; ++h)
                w[h][r][c] = in && f0 + r < a.N ? *reinterpret_cast<const int*>(static_cast<const int8_t*>(a.weights) +
                                                      ((int64_t)e * a.W + h * a.N + f0 + r) * a.K + k0 + 4 * c) : 0;
        }
        __syncthreads();
        for (int h = 0; h < halves; ++h)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    int s = 0;                   // 64 products: far inside an int
                    for (int c = 0; c < kStep / 4; ++c) s = __dp4a(x[tr + i][c], w[h][tf + j][c], s);
                    sum[h][i][j] += (float)s;
                }
    }
    for (int i = 0; i < 4 && tr + i < rows; ++i) {
        const int64_t r = own.first + m0 + tr + i;
        const float sr = static_cast<const float*>(a.row_scales)[r];
        for (int j = 0; j < 4 && f0 + tf + j < a.N; ++j) {
            const int f = f0 + tf + j;
            const float* sw = static_cast<const float*>(a.weight_scales) + (int64_t)e * a.W + f;
            float g = sum[0][i][j] * sw[0] * sr;
            if (a.glu) {
                const float u = sum[1][i][j] * sw[a.N] * sr;
                if (a.pre != nullptr) {
                    static_cast<__nv_bfloat16*>(a.pre)[r * a.W + f] = __float2bfloat16_rn(g);
                    static_cast<__nv_bfloat16*>(a.pre)[r * a.W + a.N + f] = __float2bfloat16_rn(u);
                }
                g = g / (1.0f + expf(-g)) * u;
            }
            static_cast<__nv_bfloat16*>(a.out)[r * a.N + f] = __float2bfloat16_rn(g);
        }
    }
}

}  // namespace

cudaError_t launch_expert_forward8(const ExpertArgs& a, cudaStream_t s) {
    const int64_t blocks = a.R / kTile + min(a.E, a.R);
    return launch_pdl(forward8_kernel, dim3((unsigned)blocks, (unsigned)((a.N + kTile - 1) / kTile)), dim3(kThreads), 0, s, a);
}

}  // namespace moe
