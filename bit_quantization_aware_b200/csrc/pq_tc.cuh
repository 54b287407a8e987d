// Tensor-core, TMA and mbarrier primitives of the matmul kernels (sm_100a):
// shared-memory descriptors, bounded waits with a status the host reads, and
// rings of mbarrier-guarded slots. Every source that includes this file has
// its own status and abort switch, which pq_device_status() and
// pq_debug_abort_waits() combine.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <stdint.h>

#include <mutex>

#include "pq.h"

namespace pqg {

constexpr uint32_t kMaxSpins = 1u << 22;

// nonzero after a bounded wait gave up (read by pq_device_status)
static __device__ int g_status = 0;
// nonzero: every launch raises its abort flag at start, so its waits give up
// as if their cap had been reached (pq_debug_abort_waits; tests the path)
static __device__ int g_force_abort = 0;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// K-major, 128-byte swizzle shared-memory matrix descriptor: start >> 4,
// leading offset 16 B (unused for this layout), stride between 8-row
// groups 1024 B, descriptor version 1, layout type 2 (128B swizzle).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (uint64_t{1} << 16) |
           (uint64_t{1024 >> 4} << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

__device__ __forceinline__ void mma_commit(uint32_t mbar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     mbar)
                 : "memory");
}

__device__ __forceinline__ void mbar_init(uint32_t mbar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(mbar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(mbar) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mbar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity)
        : "memory");
    return done != 0;
}

// Bounded wait for the phase of the given parity (one thread). Gives up
// early when another role raised the abort flag; raises it (and the device
// status) when the spin limit is reached.
// The loop is kept to the barrier try and a periodic abort check: other
// work in it (even a rarely executed load) measurably slowed the pipeline.
__device__ __forceinline__ bool mbar_wait(uint32_t mbar, uint32_t parity, volatile int* abort) {
    for (uint32_t i = 0; i < kMaxSpins; ++i) {
        if (mbar_try(mbar, parity)) return true;
        if ((i & 63u) == 63u && *abort) return false;
    }
    *abort = 1;
    atomicExch(&g_status, 1);
    return false;
}

// The same, taken by lane 0 for the whole warp (the result is warp-uniform,
// so the warp stays converged for the .sync.aligned tensor-memory ops).
__device__ __forceinline__ bool warp_wait(uint32_t mbar, uint32_t parity, volatile int* abort) {
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(mbar, parity, abort) ? 1 : 0;
    return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// Bounded wait that ignores the abort flag (draining on the way out).
__device__ __forceinline__ void mbar_drain(uint32_t mbar, uint32_t parity) {
    for (uint32_t i = 0; i < kMaxSpins; ++i)
        if (mbar_try(mbar, parity)) return;
    atomicExch(&g_status, 1);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t mbar,
                                            int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Position in a ring of N mbarrier-guarded slots: slot index and the parity
// of its current phase. A wait on parity (phase ^ 1) passes at once on a
// fresh barrier, so a producer's first round needs no special case.
template <int N>
struct Ring {
    uint32_t idx = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++idx == N) {
            idx = 0;
            phase ^= 1u;
        }
    }
};

// Bounded wait for the last min(issued, N) loads of a full-barrier ring.
template <int N>
__device__ __forceinline__ void drain_ring(uint32_t bar0, Ring<N> r, uint32_t issued) {
    const uint32_t n = issued < static_cast<uint32_t>(N) ? issued : static_cast<uint32_t>(N);
    for (uint32_t j = 0; j < n; ++j) {
        if (r.idx == 0) {
            r.idx = N;
            r.phase ^= 1u;
        }
        --r.idx;
        mbar_drain(bar0 + 8u * r.idx, r.phase);
    }
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &qr) ==
                cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// This source's status, cleared (PQ_OK, PQ_ERR_TIMEOUT or PQ_ERR_CUDA), and
// its abort switch.
static inline int take_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return PQ_ERR_CUDA;
    if (v) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
        return PQ_ERR_TIMEOUT;
    }
    return PQ_OK;
}
static inline int set_abort_waits(int on) {
    const int v = on ? 1 : 0;
    return cudaMemcpyToSymbol(g_force_abort, &v, sizeof(v)) == cudaSuccess ? PQ_OK : PQ_ERR_CUDA;
}

// The same of pq_fp8_gemm.cu.
int fp8_take_status();
int fp8_set_abort_waits(int on);

}  // namespace pqg
