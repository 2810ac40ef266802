// moe_experts.cuh -- what the experts' products and their 4-bit quantiser
// share: the walk over ragged groups of receive rows.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// Tries until it succeeds, giving up after limit_ns (or somewhat later: the clock
// is read only once in 1024 tries, because reading it costs more than a stage of a
// product lasts).
template <typename F>
__device__ __forceinline__ bool within(uint64_t limit_ns, F attempt) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (attempt()) return true;
        if ((it & 1023u) == 0u) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > limit_ns) return false;
        }
    }
}
constexpr uint64_t kSecond = 1000000000ull;
__device__ __forceinline__ bool wait_second(uint32_t bar, uint32_t parity, uint64_t limit_ns = kSecond) {
    return within(limit_ns, [&] { return mbar_try_wait(bar, parity); });
}

// Rows of one expert, kept inside [0, R) whatever the layout holds.
struct ExpertRows {
    int first, count;
};
__device__ __forceinline__ ExpertRows expert_rows(const int32_t* count, const int32_t* offset, int e, int R) {
    const int first = min(max(offset[e], 0), R);
    return {first, min(max(count[e], 0), R - first)};
}

// Rows and stages are counted in 32 bits, rounded up to whole tiles (of 384 rows at most) and stages: MOE_MAX_EXPERT_ROWS
// keeps these sums inside them.
__host__ __device__ __forceinline__ int blocks_of_128(int rows) { return (rows + 127) >> 7; }

// Row tiles of at most `columns` rows that `rows` rows are cut into, and the rows of each: equal, in multiples of `unit`
// (a divisor of columns).
__host__ __device__ __forceinline__ int tiles_of(int rows, int columns) { return (rows + columns - 1) / columns; }
__host__ __device__ __forceinline__ int rows_of_tile(int rows, int tiles, int unit) {
    const int least = rows / tiles + (rows % tiles != 0);  // rows + tiles may pass 32 bits
    return (least + unit - 1) / unit * unit;
}

// Sum of counts, at most the largest int: a layout whose counts do not fit its rows may have more blocks than that, and
// is walked as far as an int counts.
__host__ __device__ __forceinline__ int sum_of(int a, int b) { return a > INT32_MAX - b ? INT32_MAX : a + b; }

// base[e] = sum over e' < e of blocks(rows of e'), base[E] the total: the row
// blocks of the experts one after another.  All threads of the block call it (a
// multiple of 32, at most 1024 threads); scratch holds 32 ints.  keep: where
// not NULL, receives every expert's rows.
// WRONG: counts may be so wrong that their sums pass an int.
template <bool WRONG, typename F>
__device__ __forceinline__ void scan_row_blocks_as(const int32_t* count, const int32_t* offset, int E, int R, int* base,
                                                int* scratch, F blocks, ExpertRows* keep) {
    const int n = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (E + n - 1) / n;
    auto add = [](int a, int b) { return WRONG ? sum_of(a, b) : a + b; };
    int sum = 0;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) continue;
        const ExpertRows x = expert_rows(count, offset, e, R);
        sum = add(sum, blocks(x.count));
        if (keep != nullptr) keep[e] = x;
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc = add(inc, v);
    }
    if (lane == 31) scratch[warp] = inc;
    int at = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) at = 0;
    __syncthreads();
    for (int i = 0; i < warp; ++i) at = add(at, scratch[i]);
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e < E) {
            base[e] = at;
            at = add(at, blocks(keep != nullptr ? keep[e].count : expert_rows(count, offset, e, R).count));
            if (e == E - 1) base[E] = at;
        }
    }
    __syncthreads();
}

template <typename F>
__device__ __forceinline__ void scan_row_blocks(const int32_t* count, const int32_t* offset, int E, int R, int* base,
                                                int* scratch, F blocks, ExpertRows* keep = nullptr) {
    // an expert has R / 64 + 1 tiles at most: below this many rows no sum of MOE_MAX_EXPERTS counts passes an int, and
    // the checked sums, which cost 0.2 us, can go
    if (R < 1 << 26) scan_row_blocks_as<false>(count, offset, E, R, base, scratch, blocks, keep);
    else scan_row_blocks_as<true>(count, offset, E, R, base, scratch, blocks, keep);
}

// The expert that owns row block b < base[E]: the last e with base[e] <= b.
__device__ __forceinline__ int expert_of_block(const int* base, int E, int b) {
    int lo = 0, hi = E;  // base[lo] <= b < base[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= b) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Byte of the scale of row i (of a block of 128) and group j (of 4).
__host__ __device__ __forceinline__ int scale_byte(int i, int j) { return (i & 31) * 16 + (i >> 5) * 4 + j; }

}  // namespace moe
