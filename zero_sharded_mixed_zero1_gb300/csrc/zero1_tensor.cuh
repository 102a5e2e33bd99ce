// zero1_tensor.cuh - what the tensor-core kernels share: tensor memory, pairs of
// CTAs, boxes of the tensor memory accelerator, and their tensor maps
// (library-internal).
#pragma once

#include <cuda.h>

#include "zero1_async.cuh"
#include "zero1_block.cuh"

namespace {

constexpr uint32_t kTmemCols = 512;  // a kernel takes all of an SM's tensor memory

// ------------------------------------------------------------- tcgen05 -----

__device__ __forceinline__ void tc_alloc(uint32_t *slot)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tc_free(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTmemCols));
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrive on this barrier of both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 32 accumulator columns of this thread's lane.
__device__ __forceinline__ void tc_load32(uint32_t addr, uint32_t r[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_load16(uint32_t addr, uint32_t r[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------- clusters ----

__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on the leading CTA's copy of a barrier.
__device__ __forceinline__ void arrive_leader(uint64_t *bar)
{
    asm volatile(
        "{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, 0; mbarrier.arrive.shared::cluster.b64 _, [a]; }" ::"r"(
            smem_u32(bar))
        : "memory");
}

// The same place in the shared memory of the pair's CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(const void *p, uint32_t rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t read_rank(const uint32_t *p, uint32_t rank)
{
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at_rank(p, rank)) : "memory");
    return x;
}

// A bounded wait of a whole warp; one that runs out is noted in both CTAs.
template <class Bars>
__device__ __forceinline__ bool warp_wait(Bars &b, uint64_t *bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, mbar_wait_long(bar, parity))) return true;
    if ((threadIdx.x & 31) < 2)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_rank(&b.failed, threadIdx.x & 31)), "r"(1u) : "memory");
    __syncwarp();
    return false;
}

// The leading CTA's copy of a barrier, as a cluster address.
__device__ __forceinline__ uint32_t leader_addr(uint64_t *bar)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
    return a;
}

// A box into this CTA's shared memory, counted on the leading CTA's barrier.
__device__ __forceinline__ void tma_2d_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// A box from shared memory, added to what is there or written, and a group of
// its own.  (These reductions keep subnormal values, measured.)
__device__ __forceinline__ void box_out(const CUtensorMap *map, int x, int y, bool add, const uint32_t *place)
{
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                     "r"(x), "r"(y), "r"(smem_u32(place))
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                     "r"(y), "r"(smem_u32(place))
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// All boxes that this warp has sent are written.
__device__ __forceinline__ void boxes_written()
{
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
}

// ------------------------------------------------------------- matrices ----

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A [rows, cols] matrix in boxes of box_x columns and box_y rows, for `call`.
int make_map(const char *call, CUtensorMap *m, CUtensorMapDataType type, int es, const void *p, int64_t rows, int64_t cols, int64_t ld,
             int box_x, const char *what, int box_y, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ld * es)};
    const cuuint32_t box[2] = {(cuuint32_t)box_x, (cuuint32_t)box_y}, one[2] = {1, 1};
    const EncodeTiled fn = encode_tiled();
    if (!fn) return z1_fail(ZERO1_ECUDA, "%s: the driver has no tensor maps", call);
    const CUresult r = fn(m, type, 2, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return z1_fail(ZERO1_ECUDA, "%s: tensor map of %s: error %d", call, what, (int)r);
    return ZERO1_OK;
}

// Rows of bf16 that the tensor memory accelerator can address.
bool rows_aligned(const void *p, int64_t ld, int64_t rows)
{
    return (((uintptr_t)p) & 15) == 0 && (rows <= 1 || (ld % 8 == 0 && ld > 0));
}

}  // namespace
