// moe_tc.cuh -- the Blackwell tensor-core instructions that the experts'
// products use: tcgen05 matrix products with accumulators in tensor memory
// (TMEM), fed from shared memory by tensor (TMA) copies.
#pragma once

#include <cuda.h>

#include "moe_internal.cuh"

namespace moe {
namespace tc {

// One lane of a converged warp.  The compiler knows that one thread follows, so
// that the instructions below take their operands without a loop over lanes:
// a step of a product by a branch on lane == 0 takes half as long again (102
// against 88 us for 4096 rows, 2048 -> 9728).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// ---- tensor memory ---------------------------------------------------------

__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of this warp's 32 lanes (the lane quarter of warp % 4); wait_ld before use.
__device__ __forceinline__ void ld16(uint32_t at, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at));
}
// 32 columns of this warp's 32 lanes, written; wait_st before another thread is told.
__device__ __forceinline__ void st32(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        :: "r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
           "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
           "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
           "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- operands --------------------------------------------------------------

// Shared-memory matrix descriptor, less its start address: distances in bytes
// between 64-element pieces of the other dimension (lead) and between groups
// of 8 rows (stride); swizzle 2 = 128-byte, 0 = none.
__host__ __device__ constexpr uint64_t descriptor(uint32_t lead, uint32_t stride, uint32_t swizzle) {
    return ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) | (1ull << 46) | ((uint64_t)swizzle << 61);
}
__device__ __forceinline__ uint64_t at(uint64_t desc, uint32_t smem) { return desc | (uint64_t)((smem >> 4) & 0x3fff); }

// Rows of 128 bytes along the contraction (K-major), 128-byte swizzle: groups of 8 rows lie 1 KB apart.
constexpr uint64_t kAlongK = descriptor(16, 1024, 2);
// 64 x 64 boxes of bf16 whose rows run along the result (MN-major): boxes 8 KB apart, 8 contraction steps 1 KB.
constexpr uint64_t kAcrossK = descriptor(8192, 1024, 2);
// 32 rows x 16 bytes of scales, no swizzle: 8 rows are 128 bytes.
constexpr uint64_t kScales = descriptor(0, 128, 0);

// ---- tensor copies ---------------------------------------------------------

// A box from shared memory to its place, in this thread's bulk group; what lies past the end is left out.
__device__ __forceinline__ void store3(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 :: "l"(map), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(map) : "memory");
}

// ---- pairs of CTAs -------------------------------------------------------------
//
// Two CTAs of a cluster work on one product of 256 rows: each holds 128 rows of A
// and half the columns of B in its shared memory and 128 rows of the sums in its
// tensor memory; one thread of the first CTA issues.

// Columns of tensor memory in both CTAs (a power of two, 32 .. 512): a whole warp
// of each calls it, the address arrives at *slot in its own shared memory.
__device__ __forceinline__ void alloc_pair(uint32_t slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t at, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(at), "r"(cols) : "memory");
}
// Arrives on the barrier at this address in both CTAs (a bit of `ctas` each) when every tensor-core operation this thread
// issued before is done.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t ctas) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"(ctas) : "memory");
}
// Instruction descriptor of a bf16 product with fp32 sums: 256 rows, n columns (a multiple of 16).
__host__ __device__ constexpr uint32_t instruction_pair(int n, bool a_across, bool b_across) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_across ? 1u : 0u) << 15) | ((b_across ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((256u >> 4) << 24);
}
// ... of an fp16 product with fp32 sums, both operands along the contraction.
__host__ __device__ constexpr uint32_t instruction16_pair(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((256u >> 4) << 24);
}
// ... of an E2M1 product with E8M0 scales per 32; half: which two of the four scales of a scale word.
__host__ __device__ constexpr uint32_t instruction4_pair(int n, uint32_t half) {
    return ((2 * half) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((256u >> 4) << 24) |
           ((2 * half) << 29);
}
// D (+)= A B^T, 16 contraction steps.
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(instr), "r"((uint32_t)add) : "memory");
}
// The same with A in tensor memory: a lane holds a row of it, a column two contraction steps.
__device__ __forceinline__ void mma_tmem_pair(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(instr), "r"((uint32_t)add) : "memory");
}
// The same over 64 contraction steps of 4-bit codes, scales from tensor memory.
__device__ __forceinline__ void mma4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, uint32_t sa, uint32_t sb,
                                          bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(instr), "r"(sa), "r"(sb), "r"((uint32_t)add) : "memory");
}
// A scale block's 512 bytes of 4 scales x 128 rows to 4 columns of tensor memory, for all four lane quarters; in both
// CTAs, each from its own shared memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t d, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(d), "l"(desc) : "memory");
}
// Copies into this CTA's shared memory that complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void load2_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void load3_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t rank_in_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address in the cluster's CTA `rank` of what lies at `local` in this one.
__device__ __forceinline__ uint32_t in_rank(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 load_cluster(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
// Arrivals on a barrier of any CTA of the cluster, by what they order before what follows the wait below in another CTA.
// All that this thread (and those it has met at a barrier of its CTA) has read or written, other CTAs' shared memory
// among it; it also waits for results on their way to HBM:
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
// this CTA's own shared memory (weights' gradient of 16 rows of 64 experts with that of the rows, 1024 x 1024: 61 us, and
// 69 with the arrival above; parts of 300 rows of one expert, 7168 -> 2 x 1024: 31.0 us, and 32.1):
__device__ __forceinline__ void arrive_cluster_smem(uint32_t bar) {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
// tensor memory, which the fences above order (1416 -> 2568, 11994 rows of 40 experts: 90 us, and 96 with the first):
__device__ __forceinline__ void arrive_cluster_tmem(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Announces the bytes of a copy; hands over no memory of its own, so it needs no scope (one on each stage's doubles the time).
__device__ __forceinline__ void arrive_expect_cluster(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- host side: tensor maps ---------------------------------------------------

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (no link against the driver library).
inline Encode encoder() {
    static const Encode fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<Encode>(p);
    }();
    return fn;
}

// [depth][rows][cols] of bf16 (or of bytes), dense ([rows][cols] when depth is 0), in boxes of box_rows x box_bytes (64 or
// 128) with a swizzle of box_bytes; what a box reaches past the end reads as zeros.
inline bool make_map(CUtensorMap* map, const void* data, bool bytes, int64_t cols, int64_t rows, int64_t depth,
                     int box_rows, int box_bytes = 128) {
    const Encode encode = encoder();
    if (encode == nullptr) return false;
    const cuuint64_t size = bytes ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
    const cuuint64_t pitch[2] = {(cuuint64_t)cols * size, (cuuint64_t)cols * size * (cuuint64_t)rows};
    const cuuint32_t box[3] = {(cuuint32_t)(box_bytes / size), (cuuint32_t)box_rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, depth > 0 ? 3 : 2,
                  const_cast<void*>(data), dims, pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows] of 512 bytes (scale blocks), two rows a box, as they are.
inline bool make_scale_map(CUtensorMap* map, const void* data, int64_t rows) {
    const Encode encode = encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {128, (cuuint64_t)rows}, pitch[1] = {512};
    const cuuint32_t box[2] = {128, 2}, step[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(data), dims, pitch, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace moe
