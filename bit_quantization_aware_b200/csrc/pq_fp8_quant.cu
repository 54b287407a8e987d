// Block quantization to e4m3 (sm_100a): the operands of pq_fp8_gemm.
//
//   amax = max |x| over a block (not below 2^-96)
//   s = fl(amax / 448), code = e4m3(fl(x * fl(448 / amax)))
//
// round to nearest even, saturating at 448 (x * fl(448 / amax) may round one
// step above it). A block is 128 consecutive values of a row, or a 128 x 128
// tile; the transpose can be quantized in the same pass (its row blocks are
// the matrix's columns, 128 rows at a time), so training reads an activation
// once for the forward product and the weight gradient.
//
// Bound: memory, bytes(x) read and one byte written per code. A thread keeps
// an 8 x 8 patch of the tile in registers between the maximum and the
// rounding, so x is read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <stdint.h>

#include "pq.h"
#include "pq_launches.cuh"
#include "pq_units.cuh"

namespace pqf {

constexpr int kThreads = 256;
constexpr int kBlock = 128;
constexpr float kMax = 448.0f;      // largest finite e4m3
constexpr float kTiny = 0x1p-96f;   // smallest maximum a scale is made from: 448 / amax stays finite

// |x| as ordered bits: NaN above Inf above every finite value.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct Scale {
    float s, r;  // what a code is worth, and the factor in front of its rounding
};
__device__ __forceinline__ Scale scale_of(uint32_t amax_bits) {
    const float amax = __uint_as_float(max(amax_bits, __float_as_uint(kTiny)));
    return {__fdiv_rn(amax, kMax), __fdiv_rn(kMax, amax)};
}

// Codes of v[0..3] times r in one word, v[0] in the lowest byte.
__device__ __forceinline__ uint32_t codes4(float v0, float v1, float v2, float v3, float r0, float r1,
                                           float r2, float r3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v0, r0), __fmul_rn(v1, r1)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v2, r2), __fmul_rn(v3, r3)),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Eight consecutive values of a row as floats; `n` of them exist (<= 0: none).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
    if (VEC && n >= 8) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
            const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 f;
                if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                    f.x = __uint_as_float(w[i] << 16);
                    f.y = __uint_as_float(w[i] & 0xFFFF0000u);
                } else {
                    f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                }
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? static_cast<float>(p[i]) : 0.0f;
}

// Eight codes of consecutive places; `n` of them exist.
template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* p, int n, uint32_t w0, uint32_t w1) {
    if (VEC && n >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w0, w1);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? w0 : w1) >> (8 * (i & 3)));
}

struct QuantParams {
    const void* x;
    int64_t rows, cols, ldx;
    uint8_t* q;     // nullable with s
    int64_t ldq;
    float* s;
    uint8_t* qt;    // nullable with st
    int64_t ldqt;
    float* st;
    int64_t row_blocks, col_blocks;
};

// One CTA: one 128 x 128 tile. Thread (rg, cg) = (tid / 16, tid % 16) holds
// rows 8 rg .. 8 rg + 7 and columns 8 cg .. 8 cg + 7 of it. The transposed
// codes go through shared memory, 8-byte chunk rg of column c at chunk
// rg ^ (c / 8), so both sides of the exchange are free of bank conflicts and
// the rows of the transpose are written 128 bytes at a time.
template <typename T, bool TILE, bool ROWS, bool COLS, bool VEC>
__global__ void __launch_bounds__(kThreads) quant_tile_kernel(const __grid_constant__ QuantParams P) {
    __shared__ uint32_t warp_max[kThreads / 32][kBlock];
    __shared__ float col_r[kBlock];
    __shared__ uint2 tile[COLS ? kBlock * 16 : 1];
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15, warp = tid >> 5;
    const int64_t rb = blockIdx.x / P.col_blocks, cb = blockIdx.x % P.col_blocks;
    const int64_t r0 = rb * kBlock, c0 = cb * kBlock;
    const int nr = static_cast<int>(P.rows - r0 < kBlock ? P.rows - r0 : kBlock);
    const int nc = static_cast<int>(P.cols - c0 < kBlock ? P.cols - c0 : kBlock);
    const T* x = static_cast<const T*>(P.x) + (r0 + 8 * rg) * P.ldx + c0 + 8 * cg;

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) load8<T, VEC>(x + i * P.ldx, 8 * rg + i < nr ? nc - 8 * cg : 0, v[i]);

    float r_tile = 0.0f;
    if constexpr (TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, mag(v[i][j]));
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((tid & 31) == 0) warp_max[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) m = max(m, warp_max[k][0]);
        const Scale sc = scale_of(m);
        r_tile = sc.r;
        if (tid == 0) {
            if constexpr (ROWS) P.s[rb * P.col_blocks + cb] = sc.s;
            if constexpr (COLS) P.st[cb * P.row_blocks + rb] = sc.s;
        }
    }
    if constexpr (ROWS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float r = r_tile;
            const int row = 8 * rg + i;
            if constexpr (!TILE) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, mag(v[i][j]));
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
                const Scale sc = scale_of(m);
                r = sc.r;
                if (cg == 0 && row < nr) P.s[cb * P.rows + r0 + row] = sc.s;
            }
            if (row < nr)
                store8<VEC>(P.q + (r0 + row) * P.ldq + c0 + 8 * cg, nc - 8 * cg,
                            codes4(v[i][0], v[i][1], v[i][2], v[i][3], r, r, r, r),
                            codes4(v[i][4], v[i][5], v[i][6], v[i][7], r, r, r, r));
        }
    }
    if constexpr (COLS) {
        float rc[8];
        if constexpr (TILE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) rc[j] = r_tile;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, mag(v[i][j]));
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                if ((tid & 16) == 0) warp_max[warp][8 * cg + j] = m;
            }
            __syncthreads();
            if (tid < kBlock) {
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < kThreads / 32; ++k) m = max(m, warp_max[k][tid]);
                const Scale sc = scale_of(m);
                col_r[tid] = sc.r;
                if (tid < nc) P.st[rb * P.cols + c0 + tid] = sc.s;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) rc[j] = col_r[8 * cg + j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float r = rc[j];
            tile[(8 * cg + j) * 16 + (rg ^ cg)] =
                make_uint2(codes4(v[0][j], v[1][j], v[2][j], v[3][j], r, r, r, r),
                           codes4(v[4][j], v[5][j], v[6][j], v[7][j], r, r, r, r));
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kBlock / 16; ++k) {
            const int col = k * 16 + rg;  // 16 threads a column, 8 rows each
            const uint2 w = tile[col * 16 + (cg ^ (col >> 3))];
            if (col < nc) store8<VEC>(P.qt + (c0 + col) * P.ldqt + r0 + 8 * cg, nr - 8 * cg, w.x, w.y);
        }
    }
}

// Row blocks without the transpose: 16 threads a block, 16 rows and
// kRowBlocks blocks a CTA, every block's loads in flight at once.
constexpr int kRowBlocks = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const __grid_constant__ QuantParams P) {
    const int rg = threadIdx.x >> 4, cg = threadIdx.x & 15;
    const int64_t groups = (P.col_blocks + kRowBlocks - 1) / kRowBlocks;
    const int64_t row = blockIdx.x / groups * 16 + rg;
    const int64_t cb0 = blockIdx.x % groups * kRowBlocks;
    const T* x = static_cast<const T*>(P.x) + row * P.ldx;
    float v[kRowBlocks][8];
    int n[kRowBlocks];
#pragma unroll
    for (int k = 0; k < kRowBlocks; ++k) {
        const int64_t c = (cb0 + k) * kBlock + 8 * cg;
        const int64_t left = row < P.rows ? P.cols - c : 0;
        n[k] = left > 8 ? 8 : static_cast<int>(left < 0 ? 0 : left);
        load8<T, VEC>(x + c, n[k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < kRowBlocks; ++k) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, mag(v[k][j]));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        const Scale sc = scale_of(m);
        const int64_t cb = cb0 + k;
        if (cg == 0 && row < P.rows && cb < P.col_blocks) P.s[cb * P.rows + row] = sc.s;
        if (n[k] > 0)
            store8<VEC>(P.q + row * P.ldq + cb * kBlock + 8 * cg, n[k],
                        codes4(v[k][0], v[k][1], v[k][2], v[k][3], sc.r, sc.r, sc.r, sc.r),
                        codes4(v[k][4], v[k][5], v[k][6], v[k][7], sc.r, sc.r, sc.r, sc.r));
    }
}

// --------------------------------------------------------------- host side
template <typename T, bool VEC>
static void launch(bool tile, const QuantParams& P, cudaStream_t s) {
    if (!tile && !P.qt) {
        const int64_t groups = (P.col_blocks + kRowBlocks - 1) / kRowBlocks;
        const unsigned grid = static_cast<unsigned>((P.rows + 15) / 16 * groups);
        quant_rows_kernel<T, VEC><<<grid, kThreads, 0, s>>>(P);
    } else {
        const unsigned grid = static_cast<unsigned>(P.row_blocks * P.col_blocks);
        auto kernel = tile ? (P.q ? (P.qt ? quant_tile_kernel<T, true, true, true, VEC>
                                          : quant_tile_kernel<T, true, true, false, VEC>)
                                  : quant_tile_kernel<T, true, false, true, VEC>)
                           : (P.q ? quant_tile_kernel<T, false, true, true, VEC>
                                  : quant_tile_kernel<T, false, false, true, VEC>);
        kernel<<<grid, kThreads, 0, s>>>(P);
    }
    pqc::count_launch();
}

template <typename T>
static pq_status_t run(bool tile, const QuantParams& P, cudaStream_t s) {
    // vector accesses: 16-byte loads (8 two-byte or 4 four-byte values) and
    // 8-byte stores of codes; a row's ragged end goes element by element
    const bool vec = pq::aligned(P.x, 16) && P.ldx % (16 / sizeof(T)) == 0 &&
                     (!P.q || (pq::aligned(P.q, 8) && P.ldq % 8 == 0)) &&
                     (!P.qt || (pq::aligned(P.qt, 8) && P.ldqt % 8 == 0));
    if (vec) launch<T, true>(tile, P, s);
    else launch<T, false>(tile, P, s);
    return pq::cuda_status(cudaGetLastError());
}

}  // namespace pqf

extern "C" pq_status_t pq_fp8_quant(pq_block_t block, pq_dtype_t dtype, int64_t rows, int64_t cols,
                                    const void* x, int64_t ldx, uint8_t* q_out, int64_t ldq, float* s_out,
                                    uint8_t* qt_out, int64_t ldqt, float* st_out, void* stream) {
    if (block != PQ_BLOCK_ROW && block != PQ_BLOCK_TILE) return PQ_ERR_INVALID_ARG;
    if (dtype != PQ_BF16 && dtype != PQ_FP16 && dtype != PQ_FP32) return PQ_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0 || (q_out == nullptr) != (s_out == nullptr) ||
        (qt_out == nullptr) != (st_out == nullptr))
        return PQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return PQ_OK;
    if (!x || (!q_out && !qt_out)) return PQ_ERR_INVALID_ARG;
    if (ldx < cols || (q_out && ldq < cols) || (qt_out && ldqt < rows)) return PQ_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(x) % (dtype == PQ_FP32 ? 4 : 2)) return PQ_ERR_MISALIGNED;
    pqf::QuantParams P = {x, rows, cols, ldx, q_out, ldq, s_out, qt_out, ldqt, st_out,
                          (rows + 127) / 128, (cols + 127) / 128};
    // one CTA a tile (or 16 rows x 4 blocks): at most 2^31 - 1 of them
    if ((rows + 15) / 16 > INT32_MAX / P.col_blocks) return PQ_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case PQ_BF16: return pqf::run<__nv_bfloat16>(block == PQ_BLOCK_TILE, P, s);
        case PQ_FP16: return pqf::run<__half>(block == PQ_BLOCK_TILE, P, s);
        default: return pqf::run<float>(block == PQ_BLOCK_TILE, P, s);
    }
}
