// zero1_async.cuh - mbarriers with bounded waits and bulk copies, shared by the
// kernels that stage data through shared memory (library-internal).
//
// Every wait is bounded (kWaitNs of %globaltimer); a wait that runs out
// records an error in its source's g_zero1_status, which zero1_device_status
// reports, and the kernel waits (again with a limit) for its own copies in
// flight and returns instead of hanging.  The call's results are then wrong.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

// The status word of the weight-gradient kernel's source (a cudaError_t as int),
// part of what zero1_device_status reports.
int z1_weight_grad_status(uint32_t *status, int32_t clear);

namespace {

__device__ uint32_t g_zero1_status;  // bit 0: a bounded wait ran out

constexpr uint64_t kWaitNs = 1000000000ull;  // 1 s

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t *b, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count));
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t *b, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}

// Bytes announced, bytes written off as if they had come, then arrivals.
__device__ __forceinline__ void mbar_make_up(uint64_t *b, uint32_t arrivals, uint32_t announce, uint32_t write_off)
{
    if (announce)
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(announce) : "memory");
    if (write_off)
        asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(write_off)
                     : "memory");
    if (arrivals)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(arrivals) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint64_t *b, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Wait for the phase of the given parity; false (and the status bit set)
// if it has not completed within limit_ns of %globaltimer, or within
// kWaitPolls polls should the timer not advance.
constexpr uint64_t kWaitPolls = 1ull << 24;

// The timer is only read after kWaitFree polls: a read takes about as long as
// a whole stage of a pipeline that is waited on.
constexpr int kWaitFree = 64;

template <class Try>
__device__ __forceinline__ bool bounded_wait(Try &&done, uint64_t limit_ns)
{
    for (int k = 0; k < kWaitFree; ++k)
        if (done()) return true;
    const uint64_t t0 = global_ns();
    for (uint64_t polls = 1; !done(); ++polls) {
        if (global_ns() - t0 > limit_ns || polls >= kWaitPolls) {
            atomicOr(&g_zero1_status, 1u);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ bool mbar_wait(uint64_t *b, uint32_t parity, uint64_t limit_ns = kWaitNs)
{
    return bounded_wait([&] { return mbar_try(b, parity); }, limit_ns);
}

// The same, letting the hardware suspend the thread for up to kSuspendNs per
// poll: for warps that wait long beside others that compute.
constexpr uint32_t kSuspendNs = 20000;

__device__ __forceinline__ bool mbar_wait_long(uint64_t *b, uint32_t parity)
{
    return bounded_wait(
        [&] {
            uint32_t ok;
            asm volatile(
                "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                : "=r"(ok)
                : "r"(smem_u32(b)), "r"(parity), "r"(kSuspendNs)
                : "memory");
            return ok != 0;
        },
        kWaitNs);
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}

// This source's status word, cleared afterwards if `clear` (host).
cudaError_t async_status(uint32_t *status, int32_t clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_zero1_status, sizeof(uint32_t));
    if (e == cudaSuccess && clear) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_zero1_status, &zero, sizeof(uint32_t));
    }
    return e;
}

}  // namespace
