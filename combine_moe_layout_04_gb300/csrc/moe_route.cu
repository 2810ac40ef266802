// moe_route.cu -- the router: top-k choice of the experts from their logits,
// the gates, and the gradient of the gates ("Balancing and Beyond", section
// 3.2: k distinct experts a token).
//
// One warp holds a token's E logits in registers (value i of lane l is expert
// 32 i + l, so that a request covers consecutive logits) and finds the k
// largest by k rounds of a warp maximum: over keys first, then over the lowest
// index among the lanes that hold the maximum, which settles ties.  A key is
// the logit as an unsigned integer in the same order, so a round is two
// integer warp reductions.  Lane j keeps choice j, so the gates are one value a
// lane.
//
// Instructions bound it, not the 4 E bytes a token.  Every lane sorts its keys in
// runs once, a round compares the runs' heads and takes the winner's off.  Up to 256
// experts a lane has one run (16384 x 256, top-8: 11.5 us, 11.1 with runs of 4, but one token 2.2 us and
// 2.4), beyond that runs of 4: sorting longer ones costs more than its rounds save, shorter ones leave
// more heads to a round (16384 x 512, top-8: 17.3 us with runs of 4, 19.9 with 8, 21.2 with 2, and 26.3 when the
// winner looks through its unsorted keys again).  16384 x 128, top-8: 7.8 us forward (floor 1.3 us) and
// 4.8 us backward, with renormalised sigmoids 8.1 and 5.0.  Eight lanes a token, four tokens a warp, measured no faster.
//
// Softmax sums, sigmoids and gradients are fp32 throughout; bf16 logits widen
// exactly, and a bf16 gradient is rounded once, when it is stored.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kRouteThreads = 128;
constexpr unsigned kFull = 0xffffffffu;
constexpr unsigned kTaken = 0, kNan = 1;  // below the key of every number, -infinity included

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float* p, float v) { *p = v; }
__device__ __forceinline__ void narrow(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// An unsigned integer that orders as the float does (-0 and +0 alike).
__device__ __forceinline__ unsigned key_of(float v) {
    if (isnan(v)) return kNan;
    const unsigned u = __float_as_uint(v + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

// exp(v - top), with no weight for -infinity (the difference is NaN when top
// is -infinity too).
__device__ __forceinline__ float soft(float v, float top) { return v == -INFINITY ? 0.0f : expf(v - top); }

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// The logits of a token, V a lane; -infinity past E.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, float (&l)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 32 * i + lane;
        l[i] = e < E ? widen(row[e]) : -INFINITY;
    }
}

// A gate's weight before scale, lane j's for choice j, from its logit v; all:
// every logit of the row.  Returns w, and in *rest 1 less the sigmoid: sigmoid(-v), because the
// difference loses every digit that the gradient needs where the sigmoid nears 1 (1 % at a logit of 12, all at 17).
template <int V>
__device__ __forceinline__ float weight_of(const RouteArgs& a, const float (&all)[V], float v, bool on, float* rest) {
    if (a.score == MOE_SCORE_SOFTMAX) {
        float top = on ? v : -INFINITY, sum;
        if (a.renorm) {
            top = warp_max(top);
            sum = warp_sum(on ? soft(v, top) : 0.0f);
        } else {
            float mine = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) top = fmaxf(top, all[i]);
            top = warp_max(top);
#pragma unroll
            for (int i = 0; i < V; ++i) mine += soft(all[i], top);
            sum = warp_sum(mine);
        }
        return on && sum != 0.0f ? soft(v, top) / sum : 0.0f;
    }
    *rest = sigmoid(-v);
    if (!a.renorm) return on ? sigmoid(v) : 0.0f;
    // exp(min(v, 0)) / (1 + exp(-|v|)) is the sigmoid, and a common factor exp(-least) of the chosen ones leaves their
    // shares as they are: with the largest min(v, 0) for `least` the sum never underflows, however low all of them are
    // (magnitudes as integers order as the floats do; a NaN counts as 0 here and then makes the sum NaN)
    const float low = fminf(v, 0.0f);
    const float least = -__uint_as_float(__reduce_min_sync(kFull, on ? __float_as_uint(fabsf(low)) : 0x7f800000u));
    const float s = on ? soft(low, least) / (1.0f + expf(-fabsf(v))) : 0.0f;
    const float sum = warp_sum(s);
    return sum != 0.0f ? s / sum : 0.0f;
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (t >= a.T) return;
    const int E = a.E;
    float l[V];
    load_row<T, V>(static_cast<const T*>(a.logits) + t * a.E, E, lane, l);
    unsigned key[V], id[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        id[i] = 32 * i + lane;
        key[i] = (int)id[i] < E ? key_of(a.bias != nullptr ? l[i] + a.bias[id[i]] : l[i]) : kTaken;
    }
    // runs, each sorted: neighbours change places only when the later one is larger, so equal keys stay in
    // the order of their ids, and so do equal heads of the runs
    constexpr int kRun = V <= 8 ? V : 4;
#pragma unroll
    for (int r = 0; r < V; r += kRun)
#pragma unroll
        for (int n = kRun - 1; n > 0; --n)
#pragma unroll
            for (int i = r; i < r + n; ++i)
                if (key[i + 1] > key[i]) {
                    const unsigned k = key[i], e = id[i];
                    key[i] = key[i + 1];
                    id[i] = id[i + 1];
                    key[i + 1] = k;
                    id[i + 1] = e;
                }
    int chosen = 0;
    for (int j = 0; j < a.k; ++j) {
        unsigned best = key[0], at = id[0];        // of this lane
#pragma unroll
        for (int r = kRun; r < V; r += kRun)
            if (key[r] > best) {
                best = key[r];
                at = id[r];
            }
        const unsigned top = __reduce_max_sync(kFull, best);
        const unsigned won = __reduce_min_sync(kFull, best == top ? at : kFull);
        if (at == won) {
#pragma unroll
            for (int r = 0; r < V; r += kRun)
                if (V == kRun || id[r] == won) {
#pragma unroll
                    for (int i = r; i + 1 < r + kRun; ++i) {
                        key[i] = key[i + 1];
                        id[i] = id[i + 1];
                    }
                    key[r + kRun - 1] = kTaken;
                }
        }
        if (lane == j) chosen = (int)won;
    }
    const float mine = lane < a.k ? widen(static_cast<const T*>(a.logits)[t * a.E + chosen]) : -INFINITY;
    const bool on = lane < a.k;
    float rest;
    const float w = weight_of<V>(a, l, mine, on, &rest);
    if (on) {
        a.ids[t * a.k + lane] = chosen;
        a.gates[t * a.k + lane] = a.scale * w;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (t >= a.T) return;
    const int E = a.E;
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    T* out = static_cast<T*>(a.dlogits) + t * a.E;
    const bool spread = a.score == MOE_SCORE_SOFTMAX && !a.renorm;  // every logit gets a gradient
    float l[V];
    if (spread) load_row<T, V>(row, E, lane, l);
    int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    const bool on = id >= 0 && id < E;
    if (!on) id = -1;
    const float v = on ? widen(row[id]) : -INFINITY;
    const float g = on ? a.scale * a.dgates[t * a.k + lane] : 0.0f;
    float rest = 0.0f;
    const float w = weight_of<V>(a, l, v, on, &rest);
    const float mean = warp_sum(w * g);
    if (!spread) {
        float grad = w * (g - mean);
        if (a.score == MOE_SCORE_SIGMOID) grad = w * rest * (a.renorm ? g - mean : g);
        __syncwarp();  // dlogits may lie over logits: every lane has read
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (32 * i + lane < E) narrow(out + 32 * i + lane, 0.0f);
        __syncwarp();
        if (on) narrow(out + id, grad);
        return;
    }
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
    top = warp_max(top);
#pragma unroll
    for (int i = 0; i < V; ++i) sum += l[i] = soft(l[i], top);
    sum = warp_sum(sum);
    const float share = sum != 0.0f ? mean / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] *= -share;
    for (int j = 0; j < a.k; ++j) {
        const int e = __shfl_sync(kFull, id, j);
        const float x = __shfl_sync(kFull, w * g, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == 32 * i + lane) l[i] += x;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (32 * i + lane < E) narrow(out + 32 * i + lane, l[i]);
}

template <typename T, int V>
cudaError_t launch(const RouteArgs& a, bool back, cudaStream_t s) {
    constexpr int per = kRouteThreads / 32;
    const dim3 grid((unsigned)((a.T + (int64_t)per - 1) / per));
    return launch_pdl(back ? route_backward_kernel<T, V> : route_kernel<T, V>, grid, dim3(kRouteThreads), 0, s, a);
}

// The registers a lane needs grow with E (at most 1024): powers of two keep
// the unused ones below the used ones.
template <typename T>
cudaError_t pick(const RouteArgs& a, bool back, cudaStream_t s) {
    if (a.E <= 32) return launch<T, 1>(a, back, s);
    if (a.E <= 64) return launch<T, 2>(a, back, s);
    if (a.E <= 128) return launch<T, 4>(a, back, s);
    if (a.E <= 256) return launch<T, 8>(a, back, s);
    if (a.E <= 512) return launch<T, 16>(a, back, s);
    return launch<T, 32>(a, back, s);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
    return a.bf16 ? pick<__nv_bfloat16>(a, false, s) : pick<float>(a, false, s);
}

cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t s) {
    return a.bf16 ? pick<__nv_bfloat16>(a, true, s) : pick<float>(a, true, s);
}

}  // namespace moe
