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

// The ids of the k largest keys of the warp's, the j-th on lane j: equal keys by the lower id.  A lane's ids rise with
// their index.
template <int V>
__device__ __forceinline__ int take_largest(unsigned (&key)[V], unsigned (&id)[V], int k, int lane) {
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
                    const unsigned x = key[i], e = id[i];
                    key[i] = key[i + 1];
                    id[i] = id[i + 1];
                    key[i + 1] = x;
                    id[i + 1] = e;
                }
    int chosen = 0;
    for (int j = 0; j < k; ++j) {
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
    return chosen;
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
    const int chosen = take_largest<V>(key, id, a.k, lane);
    const float mine = lane < a.k ? widen(static_cast<const T*>(a.logits)[t * a.E + chosen]) : -INFINITY;
    const bool on = lane < a.k;
    float rest;
    const float w = weight_of<V>(a, l, mine, on, &rest);
    if (on) {
        a.ids[t * a.k + lane] = chosen;
        a.gates[t * a.k + lane] = a.scale * w;
    }
}

// ---- choice limited to groups ---------------------------------------------------------
//
// As above, but lanes divide among the groups: the largest power of two of them that 32 / groups holds to each, so
// that a group's two largest keys meet in a few exchanges.  A warp ranks the groups by comparing every
// group's value with every other's, and takes the k largest keys of those that stay.
//
// Keys are scores, so that a bias moves them on the scale of the scores; they decide, so their value must not hang on an
// order of additions: the softmax's sum is rounded once (sum_once), all else is one fp32 operation after another.
//
// Instructions bound it, as above: 16384 tokens of 256 experts, top-8 of 4 of 8 groups, sigmoid and bias, 15.4 us (floor
// 2.8; moe_route, which needs no score before its choice, 12.6), 128 experts, top-8 of 3 of 8, softmax, 12.0, 160 experts 15.2,
// 512, 4 of 16 groups, 26.1, one token 2.8.  What it cost otherwise: 22 us with the keys of groups that stay left on their own lanes (512
// experts: 38), 17.6 with lanes and groups divided on the device, 16.2 with a load for every logit (512: 35), 19.7 for 160 experts with
// eight values a lane for five.

// key_of without NaN, which counts as -infinity here, and without -0, which no sum of a score and a bias is.
__device__ __forceinline__ unsigned short_key_of(float v) {
    const unsigned u = __float_as_uint(fmaxf(v, -INFINITY));
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
// The float of such a key; -infinity for none.
__device__ __forceinline__ float value_of(unsigned key) {
    return key == kTaken ? -INFINITY : __uint_as_float(key ^ (~(unsigned)((int)key >> 31) | 0x80000000u));
}

// Sum of one value a lane and V each, rounded once: every addition's error (exact by Knuth's sum of two floats, "Seminumerical
// Algorithms", 4.2.2) is kept and added at the end.  Keys are made of it, and with the bias they must not
// depend on an order of additions.
template <int V>
__device__ __forceinline__ float sum_once(const float (&v)[V]) {
    float s = 0.0f, err = 0.0f;
    auto add = [&](float x, float more) {
        const float t = s + x, b = t - s;
        err += (s - (t - b)) + (x - b) + more;
        s = t;
    };
#pragma unroll
    for (int i = 0; i < V; ++i) add(v[i], 0.0f);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float x = __shfl_xor_sync(kFull, s, d), more = __shfl_xor_sync(kFull, err, d);
        add(x, more);
    }
    return s + err;
}

// Which expert of its group is value j of a lane: four neighbours a lane in turn, so that they come in one load, or, where
// the values are no fours, one.
template <int V>
__device__ __forceinline__ int place(int j, int bits, int sub) {
    return V % 4 == 0 ? ((j >> 2) << (bits + 2)) + (sub << 2) + (j & 3) : (j << bits) + sub;
}
__device__ __forceinline__ void load4(const float* p, float* v) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
}

// take_largest among the groups that stay, their keys spread over PARTS times as many lanes, those of groups that go: fewer
// keys a lane to sort and to move.  before: how many groups come before this lane's.
template <int V, int PARTS>
__device__ __forceinline__ int take_spread(const RouteArgs& a, const unsigned (&key)[V], int group, int sub, int before,
                                           int lane) {
    constexpr int kFew = V / PARTS;
    __shared__ int with_rank[kRouteThreads / 32][MOE_MAX_ROUTE_GROUPS];
    int* ranked = with_rank[threadIdx.x >> 5];
    if (sub == 0 && group < a.groups) ranked[before] = group;
    __syncwarp();
    int part = 0;                                            // of the keys of the group with rank before - part * kept
#pragma unroll
    for (int q = 1; q < PARTS; ++q) part += before >= q * a.kept;
    const bool takes = group < a.groups && before < PARTS * a.kept;
    const int from = takes ? ranked[before - part * a.kept] : 0;
    unsigned few[kFew], id[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
        unsigned mine = kTaken;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            // (a lane of a group that stays keeps the first part of its own)
            const unsigned theirs = q == 0 ? key[i] : __shfl_sync(kFull, key[q * kFew + i], (from << a.bits) + sub);
            if (q == part) mine = theirs;
        }
        few[i] = takes ? mine : kTaken;
        id[i] = from * a.size + place<V>(part * kFew + i, a.bits, sub);
    }
    return take_largest<kFew>(few, id, a.k, lane);
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_groups_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (t >= a.T) return;
    const int size = a.size, wide = 1 << a.bits;             // experts and lanes of a group
    const int group = lane >> a.bits, sub = lane & (wide - 1);
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    float l[V], score[V], bias[V];
    unsigned key[V], id[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = place<V>(i, a.bits, sub);
        id[i] = group < a.groups && at < size ? group * size + at : a.E + i;
        l[i] = -INFINITY;
        bias[i] = 0.0f;
    }
    if (V % 4 == 0 && a.fours) {
#pragma unroll
        for (int i = 0; i + 3 < V; i += 4) {
            if ((int)id[i] >= a.E) continue;
            load4(row + id[i], l + i);
            if (a.bias != nullptr) load4(a.bias + id[i], bias + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if ((int)id[i] >= a.E) continue;
            l[i] = widen(row[id[i]]);
            if (a.bias != nullptr) bias[i] = a.bias[id[i]];
        }
    }
    if (a.score == MOE_SCORE_SOFTMAX) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
        top = warp_max(top);
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] = soft(l[i], top);
        const float sum = sum_once<V>(score);
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] = sum != 0.0f ? score[i] / sum : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] = sigmoid(l[i]);
    }
    unsigned first = kTaken, second = kTaken;                // the two largest keys of this lane, then of its group
#pragma unroll
    for (int i = 0; i < V; ++i) {
        key[i] = short_key_of(score[i] == 0.0f ? -INFINITY : score[i] + bias[i]);  // (no bias: + 0 changes no score)
        if ((int)id[i] >= a.E) key[i] = kTaken;
        second = max(second, min(first, key[i]));
        first = max(first, key[i]);
    }
    for (int d = wide >> 1; d > 0; d >>= 1) {
        const unsigned x = __shfl_xor_sync(kFull, first, d), y = __shfl_xor_sync(kFull, second, d);
        second = max(min(first, x), max(second, y));
        first = max(first, x);
    }
    float value = value_of(first);
    if (a.top == 2) {
        const float more = value_of(second);
        if (more != -INFINITY) value += more;
    }
    const unsigned mine = short_key_of(value);
    int before = 0;                                          // groups that come before this one: equal ones by index
#pragma unroll 4
    for (int g = 0; g < a.groups; ++g) before += __shfl_sync(kFull, mine, g << a.bits) + (g < group) > mine;
    int chosen;
    if (V % 4 == 0 && 4 * a.kept <= a.groups) {
        chosen = take_spread<V, V % 4 == 0 ? 4 : 1>(a, key, group, sub, before, lane);
    } else if (V >= 2 && 2 * a.kept <= a.groups) {
        chosen = take_spread<V, V >= 2 ? 2 : 1>(a, key, group, sub, before, lane);
    } else {
        if (before >= a.kept)
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = kTaken;
        chosen = take_largest<V>(key, id, a.k, lane);
    }
    const bool on = lane < a.k;
    const float logit = on ? widen(row[chosen]) : -INFINITY;
    float rest;
    const float w = weight_of<V>(a, l, logit, on, &rest);
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

template <typename T, int V>
cudaError_t launch_grouped(const RouteArgs& a, cudaStream_t s) {
    constexpr int per = kRouteThreads / 32;
    const dim3 grid((unsigned)((a.T + (int64_t)per - 1) / per));
    return launch_pdl(route_groups_kernel<T, V>, grid, dim3(kRouteThreads), 0, s, a);
}

// By the experts of a lane: those of a group over its lanes (up to 60, where a group has one lane).
template <typename T>
cudaError_t pick_grouped(const RouteArgs& a, cudaStream_t s) {
    const int ones = (a.size + (1 << a.bits) - 1) >> a.bits, each = (a.size + (4 << a.bits) - 1) / (4 << a.bits) * 4;
    if (ones <= 1) return launch_grouped<T, 1>(a, s);
    if (ones <= 2) return launch_grouped<T, 2>(a, s);
    if (each <= 4) return launch_grouped<T, 4>(a, s);
    if (ones == 5 || ones == 6) return launch_grouped<T, 6>(a, s);  // (in fours they would be eight)
    if (each <= 8) return launch_grouped<T, 8>(a, s);
    if (each <= 12) return launch_grouped<T, 12>(a, s);
    if (each <= 16) return launch_grouped<T, 16>(a, s);
    if (each <= 32) return launch_grouped<T, 32>(a, s);
    return launch_grouped<T, 64>(a, s);
}

}  // namespace

cudaError_t launch_route_groups(const RouteArgs& args, cudaStream_t s) {
    RouteArgs a = args;
    a.size = a.E / a.groups;
    for (a.bits = 0; (2 << a.bits) * a.groups <= 32;) ++a.bits;
    a.fours = a.size % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % (a.bf16 ? 8 : 16) == 0 &&
              reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    return a.bf16 ? pick_grouped<__nv_bfloat16>(a, s) : pick_grouped<float>(a, s);
}

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
    return a.bf16 ? pick<__nv_bfloat16>(a, false, s) : pick<float>(a, false, s);
}

cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t s) {
    return a.bf16 ? pick<__nv_bfloat16>(a, true, s) : pick<float>(a, true, s);
}

}  // namespace moe
