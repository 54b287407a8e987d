// Product of two block-quantized e4m3 matrices on tcgen05 (sm_100a).
//
//   Y[m][n] = sum_kb sa(kb, m) sb(kb, n) D_kb[m][n],  D_kb = A_kb B_kb^T
//
// over K blocks of 128. The tensor cores form D_kb (kind::f8f6f4, fp32 in
// TMEM) from 128-byte rows that TMA brings in with the 128B swizzle; its
// scales are arbitrary fp32 numbers, so each D_kb leaves TMEM and is scaled
// and added in registers by the "promote" warps while the tensor cores form
// the next one in the other half of TMEM.
//
// A tile is 128 rows of A (TMEM lanes, one thread each) by NT rows of B
// (TMEM columns). With a row on a thread, the A scale is one register, and a
// tile scale of B another: one paired multiply-add per two elements. Row
// scales of B are per column and come through shared memory.
//
// Few tiles (short m and n) leave most SMs idle, so a tile's K blocks are
// split over a cluster of SPLIT CTAs, which exchange their sums through
// distributed shared memory and add them in rank order: no workspace, no
// atomics, the same bits every time.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, warp 2 TMEM owner and loader
// of B's row scales, warps 4.. promote. Waits are bounded as in pq_gemm.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <stdint.h>

#include "pq.h"
#include "pq_launches.cuh"
#include "pq_tc.cuh"
#include "pq_units.cuh"

namespace pq8 {

using namespace pqg;

constexpr int kBlock = 128;   // K of a scale block, and of one stage
constexpr int kRows = 128;    // A rows of a tile
constexpr int kScaleSlots = 4;  // K blocks of B row scales in flight

struct Params {
    CUtensorMap ta, tb;  // codes [m][k] in boxes of 128 B x a_box rows, [n][k] in boxes of 128 B x NT rows
    const float* sa;     // [kb][m]
    const float* sb;     // [n / 128][kb] (tile) or [kb][n] (row)
    void* y;
    int64_t m, n, ldy;
    int32_t kb;          // K blocks
    int32_t tiles_m, tiles_n;
    int32_t a_bytes;     // bytes of one A box
    int32_t dtype;       // of y
    int32_t vec;         // 16-byte stores of whole rows are aligned
};

template <int NT, int SPLIT>
struct Layout {
    static constexpr int kPromoteWarps = NT == 256 ? 8 : 4;
    static constexpr int kThreads = 128 + 32 * kPromoteWarps;
    static constexpr int kCols = NT / (kPromoteWarps / 4);  // columns of a promote thread
    static constexpr int kABytes = kRows * kBlock, kBBytes = NT * kBlock;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = NT == 256 ? 4 : NT == 128 ? 6 : 4;
    static constexpr uint32_t kTmemCols = 2 * NT;
    static constexpr int kScaleOff = kStages * kStage;
    static constexpr int kBarOff = kScaleOff + kScaleSlots * NT * 4;
    // full, empty [stages]; dfull, dempty [2]; sfull, sempty [scale slots]; drain
    static constexpr int kNumBars = 2 * kStages + 4 + 2 * kScaleSlots + 1;
    static constexpr int kMiscOff = kBarOff + 8 * kNumBars;
    static constexpr int kBytes = kMiscOff + 16 + 1024;  // + alignment slack
    static_assert(SPLIT == 1 || kRows * NT * 4 <= kStages * kStage, "exchange fits the stages");
};

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, e4m3 A and B, both
// K-major, M = 128, N = nt.
__host__ __device__ constexpr uint32_t idesc_e4m3(int nt) {
    return (1u << 4) | (static_cast<uint32_t>(nt >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(acc)
        : "memory");
}

// 32 columns of this warp's 32 TMEM lanes; the values are there after tmem_wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Two fp32 values in a register pair, and the paired operations on them.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}

// Tile t of the launch: groups of 8 row tiles walk the column tiles, so the
// CTAs at work at one time share their A and B rows in L2.
__device__ __forceinline__ void tile_of(const Params& p, int t, int& tm, int& tn) {
    constexpr int kGroup = 8;
    const int per = kGroup * p.tiles_n;
    const int g = t / per, r = t - g * per;
    const int rows = p.tiles_m - g * kGroup < kGroup ? p.tiles_m - g * kGroup : kGroup;
    tm = g * kGroup + r % rows;
    tn = r / rows;
}

// Rounds v[0..N) and writes it to columns col.. of a row, N a multiple of 8.
template <typename T, int N, typename F>
__device__ __forceinline__ void store_row(T* y, int64_t left, bool vec, F&& v) {
#pragma unroll
    for (int c = 0; c < N; c += 8) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v(c + i);
        if (vec && c + 8 <= left) {
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<float4*>(y + c)[0] = make_float4(f[0], f[1], f[2], f[3]);
                reinterpret_cast<float4*>(y + c)[1] = make_float4(f[4], f[5], f[6], f[7]);
            } else {
                T h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = static_cast<T>(f[i]);
                *reinterpret_cast<uint4*>(y + c) = *reinterpret_cast<const uint4*>(h);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < left) y[c + i] = static_cast<T>(f[i]);
        }
    }
}

template <int N, typename F>
__device__ __forceinline__ void store_out(const Params& p, int64_t row, int64_t col, F&& v) {
    const int64_t left = p.n - col;
    const int64_t at = row * p.ldy + col;
    if (p.dtype == PQ_BF16) store_row<__nv_bfloat16, N>(static_cast<__nv_bfloat16*>(p.y) + at, left, p.vec, v);
    else if (p.dtype == PQ_FP16) store_row<__half, N>(static_cast<__half*>(p.y) + at, left, p.vec, v);
    else store_row<float, N>(static_cast<float*>(p.y) + at, left, p.vec, v);
}

template <int NT, bool BROW, int SPLIT>
__global__ void __cluster_dims__(SPLIT, 1, 1) __launch_bounds__(Layout<NT, SPLIT>::kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ Params p) {
    using L = Layout<NT, SPLIT>;
    constexpr int S = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t{1023});
    const uint32_t sbase = smem_u32(smem);
    const uint32_t b_full = sbase + L::kBarOff, b_empty = b_full + 8u * S;
    const uint32_t b_dfull = b_empty + 8u * S, b_dempty = b_dfull + 16u;
    const uint32_t b_sfull = b_dempty + 16u, b_sempty = b_sfull + 8u * kScaleSlots;
    const uint32_t b_drain = b_sempty + 8u * kScaleSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    float* bscale = reinterpret_cast<float*>(smem + L::kScaleOff);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(b_full + 8u * s, 1);
            mbar_init(b_empty + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(b_dfull + 8u * b, 1);
            mbar_init(b_dempty + 8u * b, L::kPromoteWarps);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(b_sfull + 8u * s, 32);
            mbar_init(b_sempty + 8u * s, L::kPromoteWarps);
        }
        mbar_init(b_drain, 1);
        const int forced = *static_cast<volatile int*>(&g_force_abort);
        *abort = forced;
        if (forced) atomicExch(&g_status, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(L::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // this CTA's tiles, and its K blocks of each
    const int tiles = p.tiles_m * p.tiles_n;
    const int rank = SPLIT == 1 ? 0 : static_cast<int>(blockIdx.x % SPLIT);
    const int first = SPLIT == 1 ? blockIdx.x : blockIdx.x / SPLIT;
    const int step = SPLIT == 1 ? gridDim.x : gridDim.x / SPLIT;
    const int k0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / SPLIT);
    const int k1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / SPLIT);

    if (warp == 0) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            Ring<S> r;
            uint32_t issued = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                int tm, tn;
                tile_of(p, t, tm, tn);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait(b_empty + 8u * r.idx, r.phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = b_full + 8u * r.idx, dst = sbase + r.idx * L::kStage;
                    mbar_expect_tx(bar, static_cast<uint32_t>(p.a_bytes) + L::kBBytes);
                    tma_load_2d(dst, &p.ta, bar, kb * kBlock, tm * kRows);
                    tma_load_2d(dst + L::kABytes, &p.tb, bar, kb * kBlock, tn * NT);
                    r.next();
                    ++issued;
                }
            }
            drain_ring(b_full, r, issued);  // loads in flight land before the CTA may exit
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(NT);
            Ring<S> r;
            Ring<2> d;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                for (int kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait(b_dempty + 8u * d.idx, d.phase ^ 1u, abort) ||
                        !mbar_wait(b_full + 8u * r.idx, r.phase, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = sbase + r.idx * L::kStage;
                    const uint64_t a = sw128_desc(at), b = sw128_desc(at + L::kABytes);
#pragma unroll
                    for (int k = 0; k < kBlock / 32; ++k)
                        mma_ss(tmem + NT * d.idx, a + 2u * k, b + 2u * k, idesc, k > 0);
                    mma_commit(b_empty + 8u * r.idx);
                    mma_commit(b_dfull + 8u * d.idx);
                    r.next();
                    d.next();
                }
            }
            mma_commit(b_drain);  // every MMA completes before TMEM is freed
            mbar_drain(b_drain, 0);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------- B's row scales
        if constexpr (BROW) {
            Ring<kScaleSlots> r;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                int tm, tn;
                tile_of(p, t, tm, tn);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!warp_wait(b_sempty + 8u * r.idx, r.phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < NT / 32; ++i) {
                        const int64_t col = static_cast<int64_t>(tn) * NT + 32 * i + lane;
                        const bool in = col < p.n;
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                         smem_u32(bscale + r.idx * NT + 32 * i + lane)),
                                     "l"(p.sb + (in ? kb * p.n + col : 0)), "r"(in ? 4u : 0u)
                                     : "memory");
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(b_sfull + 8u * r.idx)
                                 : "memory");
                    r.next();
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------- promote
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        constexpr int C = L::kCols;
        Ring<2> d;
        Ring<kScaleSlots> sr;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
            int tm, tn;
            tile_of(p, t, tm, tn);
            const int64_t row = static_cast<int64_t>(tm) * kRows + quarter * 32 + lane;
            const int64_t col = static_cast<int64_t>(tn) * NT + half * C;
            const bool live = row < p.m;
            const float* sa = p.sa + (live ? row : 0);
            const float* sb = p.sb + (BROW ? 0 : col / kBlock * p.kb);
            const bool sb_in = !BROW && col < p.n;
            uint64_t acc[C / 2];
#pragma unroll
            for (int i = 0; i < C / 2; ++i) acc[i] = 0;
            // scales two K blocks ahead
            auto scale = [&](int kb) {
                float v = live && kb < k1 ? __ldg(sa + kb * p.m) : 0.0f;
                if (!BROW) v = __fmul_rn(v, sb_in && kb < k1 ? __ldg(sb + kb) : 0.0f);
                return v;
            };
            float s0 = scale(k0), s1 = scale(k0 + 1);
            for (int kb = k0; kb < k1; ++kb) {
                const float s = s0;
                s0 = s1;
                s1 = scale(kb + 2);
                if (BROW && !warp_wait(b_sfull + 8u * sr.idx, sr.phase, abort)) {
                    ok = false;
                    break;
                }
                if (!warp_wait(b_dfull + 8u * d.idx, d.phase, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t s2 = pair(__float_as_uint(s), __float_as_uint(s));
                const float4* bs = reinterpret_cast<const float4*>(bscale + sr.idx * NT + half * C);
#pragma unroll
                for (int c = 0; c < C; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(tmem + lane_addr + NT * d.idx + half * C + c, v);
                    tmem_wait();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        uint64_t f0 = s2, f1 = s2;
                        if constexpr (BROW) {
                            const float4 b = bs[(c + i) / 4];
                            f0 = mul2(s2, pair(__float_as_uint(b.x), __float_as_uint(b.y)));
                            f1 = mul2(s2, pair(__float_as_uint(b.z), __float_as_uint(b.w)));
                        }
                        acc[(c + i) / 2] = fma2(pair(v[i], v[i + 1]), f0, acc[(c + i) / 2]);
                        acc[(c + i) / 2 + 1] = fma2(pair(v[i + 2], v[i + 3]), f1, acc[(c + i) / 2 + 1]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(b_dempty + 8u * d.idx);
                    if (BROW) mbar_arrive(b_sempty + 8u * sr.idx);
                }
                d.next();
                if (BROW) sr.next();
            }
            if (!ok) break;
            if (live)
                store_out<C>(p, row, col, [&](int i) { return i & 1 ? hi_of(acc[i / 2]) : lo_of(acc[i / 2]); });
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmemCols)
                     : "memory");
}

// k == 0: an empty sum
template <typename T>
__global__ void __launch_bounds__(256) zero_kernel(T* y, int64_t m, int64_t n, int64_t ldy) {
    for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < m * n; i += gridDim.x * int64_t{256})
        y[i / n * ldy + i % n] = static_cast<T>(0.0f);
}

// --------------------------------------------------------------- host side
static bool encode(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const uint8_t* p, int64_t rows,
                   int64_t k, int64_t ld, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {kBlock, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t es[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool BROW, int SPLIT>
static cudaError_t launch(const Params& p, cudaStream_t s) {
    using L = Layout<NT, SPLIT>;
    static bool attr_set[64] = {false};
    auto kernel = fp8_gemm_kernel<NT, BROW, SPLIT>;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const int tiles = p.tiles_m * p.tiles_n;
    const int grid = SPLIT > 1 ? tiles * SPLIT : tiles < pq::sm_count() ? tiles : pq::sm_count();
    kernel<<<grid, L::kThreads, L::kBytes, s>>>(p);
    pqc::count_launch();
    return cudaGetLastError();
}

static int bytes_of(int dtype) { return dtype == PQ_FP32 ? 4 : 2; }

}  // namespace pq8

int pqg::fp8_take_status() { return take_status(); }
int pqg::fp8_set_abort_waits(int on) { return set_abort_waits(on); }

extern "C" pq_status_t pq_fp8_gemm(int64_t m, int64_t n, int64_t k, const uint8_t* a, int64_t lda,
                                   const float* a_scale, const uint8_t* b, int64_t ldb, const float* b_scale,
                                   pq_block_t b_block, void* y, pq_dtype_t y_dtype, int64_t ldy, void* stream) {
    using namespace pq8;
    if (b_block != PQ_BLOCK_ROW && b_block != PQ_BLOCK_TILE) return PQ_ERR_INVALID_ARG;
    if (y_dtype != PQ_BF16 && y_dtype != PQ_FP16 && y_dtype != PQ_FP32) return PQ_ERR_INVALID_ARG;
    if (m < 0 || n < 0 || k < 0) return PQ_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return PQ_OK;
    if (!y || ldy < n) return PQ_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(y) % bytes_of(y_dtype)) return PQ_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k == 0) {
        const unsigned grid = 4 * pq::sm_count();
        if (y_dtype == PQ_FP32) zero_kernel<<<grid, 256, 0, s>>>(static_cast<float*>(y), m, n, ldy);
        else zero_kernel<<<grid, 256, 0, s>>>(static_cast<__half*>(y), m, n, ldy);  // a zero in both types
        pqc::count_launch();
        return pq::cuda_status(cudaGetLastError());
    }
    if (!a || !a_scale || !b || !b_scale || (m > 1 && lda < k) || (n > 1 && ldb < k)) return PQ_ERR_INVALID_ARG;
    if (m == 1) lda = (k + 15) / 16 * 16;  // one row has no pitch
    if (n == 1) ldb = (k + 15) / 16 * 16;
    if (m > (int64_t{1} << 30) || n > (int64_t{1} << 30) || k > (int64_t{1} << 30)) return PQ_ERR_UNSUPPORTED;
    if (!pq::aligned(a, 16) || !pq::aligned(b, 16) || lda % 16 || ldb % 16) return PQ_ERR_MISALIGNED;
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return PQ_ERR_CUDA;
    Params p = {};
    p.sa = a_scale;
    p.sb = b_scale;
    p.y = y;
    p.m = m;
    p.n = n;
    p.ldy = ldy;
    p.kb = static_cast<int32_t>((k + kBlock - 1) / kBlock);
    p.dtype = y_dtype;
    p.vec = pq::aligned(y, 16) && ldy * bytes_of(y_dtype) % 16 == 0;
    constexpr int NT = 128;
    const int64_t tiles_m = (m + kRows - 1) / kRows, tiles_n = (n + NT - 1) / NT;
    if (tiles_m * tiles_n > (int64_t{1} << 27)) return PQ_ERR_UNSUPPORTED;
    p.tiles_m = static_cast<int32_t>(tiles_m);
    p.tiles_n = static_cast<int32_t>(tiles_n);
    // a short A fills only the lanes it has: the others' sums are not read
    const int a_rows = m < kRows ? static_cast<int>((m + 7) / 8 * 8) : kRows;
    p.a_bytes = a_rows * kBlock;
    if (!encode(enc, &p.ta, a, m, k, lda, a_rows) || !encode(enc, &p.tb, b, n, k, ldb, NT)) return PQ_ERR_CUDA;
    return pq::cuda_status(b_block == PQ_BLOCK_ROW ? launch<NT, true, 1>(p, s) : launch<NT, false, 1>(p, s));
}
