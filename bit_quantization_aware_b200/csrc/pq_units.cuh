// What the streaming kernels over batches of matrices share: tuning knobs,
// vector memory accesses, the quantizer's forward and backward on a chunk of
// 8 weights, batch descriptors and the host's unit and grid rules.
#pragma once
#include <cuda_runtime.h>

#include <stdint.h>

#include "pq.h"
#include "pq_launches.cuh"
#include "pq_quant.cuh"

// Tuning knobs (compile-time; the defaults are the measured choice):
//   PQ_PREFETCH      1: bulk L2 prefetch of each CTA's next unit
//   PQ_CTAS_PER_SM   persistent CTAs per SM (0: the occupancy limit)
//   PQ_CHUNKS_PER_THREAD  target chunks of 8 weights per thread and row
//                    (PQ_FWD_CHUNKS_PER_THREAD: the forward's target)
//   PQ_FWD_UNROLL, PQ_BWD_UNROLL  chunks whose loads a thread issues
//                    before computing any of them (PQ_PACK_UNROLL: the
//                    forward instance that writes packed codes only)
//   PQ_LD_HINT, PQ_ST_HINT  cache hints of the streaming loads and stores
//                    (loads: 0 evict-first, 1 read-only path, 2 default,
//                    3 evict-first with a 256-byte L2 prefetch, 4 read-only
//                    without L1 allocation with a 256-byte L2 prefetch)
//   PQ_BWD_MIN_CTAS  resident CTAs per SM the backward's registers must allow
//   PQ_FWD_MIN_CTAS  the same for the forward (PQ_PACK_MIN_CTAS: its
//                    packed-codes-only instance; PQ_RED_MIN_CTAS: the
//                    sharded reduce + backward + AdamW)
//   PQ_DEQ_BULK      1: the dequantization stages each unit's bf16 output in
//                    shared memory and writes it with one bulk copy
//   PQ_DEQ_BUF_KB    size of one such staging buffer (two per CTA)
#ifndef PQ_PREFETCH
#define PQ_PREFETCH 0
#endif
#ifndef PQ_CTAS_PER_SM
#define PQ_CTAS_PER_SM 0
#endif
#ifndef PQ_CHUNKS_PER_THREAD
#define PQ_CHUNKS_PER_THREAD 8
#endif
#ifndef PQ_FWD_CHUNKS_PER_THREAD
#define PQ_FWD_CHUNKS_PER_THREAD 16
#endif
#ifndef PQ_FWD_UNROLL
#define PQ_FWD_UNROLL 3
#endif
#ifndef PQ_PACK_UNROLL
#define PQ_PACK_UNROLL 4
#endif
#ifndef PQ_BWD_UNROLL
#define PQ_BWD_UNROLL 2
#endif
#ifndef PQ_LD_HINT
#define PQ_LD_HINT 0
#endif
#ifndef PQ_BWD_MIN_CTAS
#define PQ_BWD_MIN_CTAS 4
#endif
#ifndef PQ_ST_HINT
#define PQ_ST_HINT 0
#endif
#ifndef PQ_FWD_MIN_CTAS
#define PQ_FWD_MIN_CTAS 4
#endif
#ifndef PQ_DEQ_BULK
#define PQ_DEQ_BULK 1
#endif
#ifndef PQ_DEQ_BUF_KB
#define PQ_DEQ_BUF_KB 32
#endif
#ifndef PQ_PACK_MIN_CTAS
#define PQ_PACK_MIN_CTAS 3
#endif
#ifndef PQ_RED_MIN_CTAS
#define PQ_RED_MIN_CTAS 3
#endif

namespace pq {

constexpr int kThreads = 256;
#ifndef PQ_MAX_BATCH
#define PQ_MAX_BATCH 256
#endif
constexpr int kMaxBatch = PQ_MAX_BATCH;  // descriptors per launch

// ------------------------------------------------------------ memory helpers
// Number of valid weights in chunk `ch` (8 except in a ragged last chunk).
__device__ __forceinline__ int tail_n(int64_t cols, int64_t ch) {
    const int64_t r = cols - ch * 8;
    return r < 8 ? static_cast<int>(r) : 8;
}

// Streaming load/store flavours (PQ_LD_HINT: 0 evict-first, 1 read-only
// path, 2 default; PQ_ST_HINT: 0 evict-first, 1 default).
template <typename T>
__device__ __forceinline__ T ld_stream(const T* p) {
#if PQ_LD_HINT == 0
    return __ldcs(p);
#elif PQ_LD_HINT == 1
    return __ldg(p);
#else
    return *p;
#endif
}
template <typename T>
__device__ __forceinline__ void st_stream(T* p, T v) {
#if PQ_ST_HINT == 0
    __stcs(p, v);
#else
    *p = v;
#endif
}

// Eight consecutive fp32 values (32-byte aligned) as one 256-bit access, so
// a warp's access covers 1024 contiguous bytes (two 16-byte accesses per
// lane would each cover only half of every 32-byte sector).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
#if PQ_LD_HINT == 0
    asm("ld.global.cs.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "l"(p));
#elif PQ_LD_HINT == 3
    asm("ld.global.cs.L2::256B.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "l"(p));
#elif PQ_LD_HINT == 4
    asm("ld.global.nc.L1::no_allocate.L2::256B.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "l"(p));
#else
    const float4 a = ld_stream(reinterpret_cast<const float4*>(p));
    const float4 b = ld_stream(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
#endif
}

__device__ __forceinline__ void load8_tail(const float* p, int n, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (i < n) ? p[i] : 0.0f;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
#if PQ_ST_HINT == 0
    asm volatile("st.global.cs.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
#else
    st_stream(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    st_stream(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
#endif
}

__device__ __forceinline__ void store8_tail(float* p, int n, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
}

__device__ __forceinline__ void load_g8(const uint16_t* p, uint32_t (&gw)[4]) {
    const uint4 u = ld_stream(reinterpret_cast<const uint4*>(p));
    gw[0] = u.x; gw[1] = u.y; gw[2] = u.z; gw[3] = u.w;
}

__device__ __forceinline__ void load_g8_tail(const uint16_t* p, int n, uint32_t (&gw)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t lo = (2 * k < n) ? p[2 * k] : 0u;
        const uint32_t hi = (2 * k + 1 < n) ? p[2 * k + 1] : 0u;
        gw[k] = lo | (hi << 16);
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);  // .x -> low half
    return *reinterpret_cast<uint32_t*>(&b);
}

// Bulk prefetch of [p, p + bytes) into L2 (16-byte aligned, multiple of 16).
__device__ __forceinline__ void prefetch_l2(const void* p, int64_t bytes) {
    const char* c = static_cast<const char*>(p);
    while (bytes > 0) {
        const uint32_t n = bytes > (1 << 20) ? (1u << 20) : static_cast<uint32_t>(bytes);
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(c), "r"(n) : "memory");
        c += n;
        bytes -= n;
    }
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Barrier over the `count` threads of one row group (ids 1..8; id 0 is
// __syncthreads). All threads of the group reach it equally often.
__device__ __forceinline__ void group_barrier(int id, int count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// ------------------------------------------------------------- chunk math
// Forward of one chunk of 8 weights: bf16 outputs as 4 words, packed codes
// as one word (bits*8 significant bits).
template <int Q, bool WQ, bool PACK>
__device__ __forceinline__ void fwd_chunk(const float (&v)[8], const RowScale& s,
                                          uint32_t (&h)[4], uint32_t& pk) {
    constexpr int B = Traits<Q>::bits;
    float x[8];
    divide8(v, s, x);
    pk = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const Elem e0 = quantize_x<Q>(x[i]);
        const Elem e1 = quantize_x<Q>(x[i + 1]);
        if constexpr (WQ) {
            h[i / 2] = pack_bf16x2(__fmul_rn(e0.level, s.a), __fmul_rn(e1.level, s.a));
        }
        if constexpr (PACK) {
            pk |= code_field<Q>(e0) << (B * i);
            pk |= code_field<Q>(e1) << (B * (i + 1));
        }
    }
}

template <int Q, bool VEC, bool WQ, bool PACK>
__device__ __forceinline__ void fwd_store(uint16_t* __restrict__ qrow,
                                          uint8_t* __restrict__ prow, int64_t ch,
                                          int n, const uint32_t (&h)[4],
                                          uint32_t pk) {
    constexpr int B = Traits<Q>::bits;
    if constexpr (VEC) {
        if constexpr (WQ)
            st_stream(reinterpret_cast<uint4*>(qrow + ch * 8),
                      make_uint4(h[0], h[1], h[2], h[3]));
        if constexpr (PACK) {
            if constexpr (B == 2)
                st_stream(reinterpret_cast<unsigned short*>(prow + ch * 2),
                          static_cast<unsigned short>(pk));
            else
                st_stream(reinterpret_cast<unsigned int*>(prow + ch * 4), pk);
        }
    } else {
        if constexpr (WQ) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) qrow[ch * 8 + i] = static_cast<uint16_t>(h[i / 2] >> (16 * (i & 1)));
        }
        if constexpr (PACK) {
            constexpr int per_byte = 8 / B;
#pragma unroll
            for (int k = 0; k < B; ++k)  // B bytes per chunk of 8 codes
                if (k * per_byte < n) prow[ch * B + k] = static_cast<uint8_t>(pk >> (8 * k));
        }
    }
}

// Backward of one chunk: dW for 8 weights and their contribution to the
// row's sum_j g_j * (level_j - inside_j * x_j), accumulated in fp64.
template <int Q>
__device__ __forceinline__ double bwd_chunk(const float (&v)[8], const uint32_t (&gw)[4],
                                            const RowScale& s, float (&d)[8], double acc) {
    float x[8];
    divide8(v, s, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Elem e = quantize_x<Q>(x[i]);
        const uint32_t word = gw[i / 2];
        const float g = (i & 1) ? __uint_as_float(word & 0xFFFF0000u)
                                : __uint_as_float(word << 16);
        d[i] = e.inside ? g : 0.0f;
        const float xm = e.inside ? x[i] : 0.0f;
        // level - xm is exact in fp64; the product and the sum round once
        acc = __fma_rn(static_cast<double>(g),
                       __dsub_rn(static_cast<double>(e.level), static_cast<double>(xm)), acc);
    }
    return acc;
}

// Backward of one chunk with an fp32 upstream gradient (already reduced).
template <int Q>
__device__ __forceinline__ double bwd_chunk_f32(const float (&v)[8], const float (&g)[8],
                                                const RowScale& s, float (&d)[8], double acc) {
    float x[8];
    divide8(v, s, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Elem e = quantize_x<Q>(x[i]);
        d[i] = e.inside ? g[i] : 0.0f;
        const float xm = e.inside ? x[i] : 0.0f;
        acc = __fma_rn(static_cast<double>(g[i]),
                       __dsub_rn(static_cast<double>(e.level), static_cast<double>(xm)), acc);
    }
    return acc;
}

// ------------------------------------------------------------ batches
// Device-side descriptor of one matrix of a batch (kernel parameter space).
struct MatDesc {
    const float* w;
    const float* alpha;
    uint16_t* wq;          // forward bf16 output (nullable)
    uint8_t* packed;       // forward packed codes (nullable)
    const uint16_t* g;     // backward upstream gradient
    float* dw;             // backward dW
    float* dalpha;         // backward d(alpha)
    int64_t rows;
    int64_t cols;
    int64_t unit_begin;    // first unit of this matrix in the batch
    float grad_scale;
    int32_t tpr_log2;      // threads per row = 1 << tpr_log2
    int32_t col_splits;    // forward: column segments per row block
    int32_t pad_;
};

// Descriptors of one launch, passed as the kernel's parameter block. A
// launch of at most kSmallBatch matrices uses the small instantiation: its
// parameter block is 24 KB smaller, which shortens the launch (about 2 us
// measured on one small matrix).
constexpr int kSmallBatch = 8;

template <typename D, int CAP = kMaxBatch>
struct BatchT {
    int32_t n;
    int32_t pad_;
    int64_t total_units;
    D m[CAP];
};
using Batch = BatchT<MatDesc>;
template <int CAP>
using MatBatch = BatchT<MatDesc, CAP>;

// Moves `mi` forward to the matrix that owns unit u (units increase).
template <typename D, int CAP>
__device__ __forceinline__ int find_matrix(const BatchT<D, CAP>& p, int mi, int64_t u) {
    while (mi + 1 < p.n && p.m[mi + 1].unit_begin <= u) ++mi;
    return mi;
}

// Bulk L2 prefetch of the inputs of unit u (vector layout only).
template <bool BWD, int CAP>
__device__ __forceinline__ void prefetch_unit(const MatBatch<CAP>& p, int mi, int64_t u) {
    if (u >= p.total_units) return;
    mi = find_matrix(p, mi, u);
    const MatDesc& m = p.m[mi];
    if (m.col_splits != 1) return;
    const int64_t rpb = kThreads >> m.tpr_log2;
    const int64_t r0 = (u - m.unit_begin) * rpb;
    const int64_t nr = (m.rows - r0) < rpb ? (m.rows - r0) : rpb;
    prefetch_l2(m.w + r0 * m.cols, nr * m.cols * 4);
    if constexpr (BWD) prefetch_l2(m.g + r0 * m.cols, nr * m.cols * 2);
}

// --------------------------------------------------------------- host side
inline int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    return dev;
}

inline int sm_count() {
    static int cached[64] = {0};
    const int dev = current_device();
    if (cached[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        cached[dev] = n;
    }
    return cached[dev];
}

inline bool aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline int ilog2_ceil(int64_t v) {
    int l = 0;
    while ((int64_t{1} << l) < v) ++l;
    return l;
}

// Threads per row: a power of two, 1..256, giving each thread about
// PQ_CHUNKS_PER_THREAD chunks of 8 weights of its row.
inline int choose_tpr_log2_for(int64_t nch, int chunks_per_thread) {
    const int l = ilog2_ceil((nch + chunks_per_thread - 1) / chunks_per_thread);
    return l > 8 ? 8 : l;
}

inline int choose_tpr_log2(int64_t cols) {
    return choose_tpr_log2_for((cols + 7) / 8, PQ_CHUNKS_PER_THREAD);
}

// Row groups of the backward kernels (one row per group: a row's d(alpha)
// is reduced inside its CTA). A matrix with too few rows to give every SM
// a unit takes wider groups (up to one thread per chunk of a row), so its
// chunks spread over more CTAs instead of queueing on a few threads.
inline int bwd_tpr_log2(int64_t rows, int64_t cols) {
    const int64_t nch = (cols + 7) / 8;
    int l = choose_tpr_log2(cols);
    const int lmax = choose_tpr_log2_for(nch, 1);
    while (l < lmax && (rows + (kThreads >> l) - 1) / (kThreads >> l) < sm_count()) ++l;
    return l;
}

inline pq_status_t cuda_status(cudaError_t e) {
    if (e != cudaSuccess) {
        pqc::last_cuda_error = static_cast<int>(e);
        return PQ_ERR_CUDA;
    }
    return PQ_OK;
}

inline int code_bits_of(int q) {
    switch (q) {
        case PQ_BINARY: case PQ_TERNARY: case PQ_SEQ2: case PQ_SEQ2_B: case PQ_LSQ2: return 2;
        case PQ_LSQ3: case PQ_LSQ4: return 4;
        default: return 0;
    }
}

// Calls f.template operator()<Q>() for the runtime quantizer q.
template <typename F>
bool dispatch_q(int q, F&& f) {
    switch (q) {
        case PQ_BINARY: f.template operator()<PQ_BINARY>(); return true;
        case PQ_TERNARY: f.template operator()<PQ_TERNARY>(); return true;
        case PQ_SEQ2: f.template operator()<PQ_SEQ2>(); return true;
        case PQ_SEQ2_B: f.template operator()<PQ_SEQ2_B>(); return true;
        case PQ_LSQ2: f.template operator()<PQ_LSQ2>(); return true;
        case PQ_LSQ3: f.template operator()<PQ_LSQ3>(); return true;
        case PQ_LSQ4: f.template operator()<PQ_LSQ4>(); return true;
        default: return false;
    }
}

// Persistent grid size of one kernel, from its occupancy (once per device).
template <typename K>
int64_t persistent_ctas(K kernel, int* cache) {
    const int dev = current_device();
    if (cache[dev] == 0) {
        int per_sm = PQ_CTAS_PER_SM;
        if (per_sm <= 0 &&
            (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0) !=
                 cudaSuccess || per_sm <= 0))
            per_sm = 4;
        cache[dev] = per_sm * sm_count();
    }
    return cache[dev];
}

}  // namespace pq
