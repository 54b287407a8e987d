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
// rounding, so x is read once. Below that bound instructions count: two-byte
// values stay packed and their magnitudes are compared as 16-bit integers two
// at a time (the order of the bits is the order of the magnitudes, NaN above
// Inf), a block's two divisions are made by one lane, and the maxima of eight
// rows are reduced over 16 lanes by halving (8 shuffles in place of 32).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "pq.h"
#include "pq_launches.cuh"
#include "pq_units.cuh"

namespace pqf {

constexpr int kThreads = 256;
constexpr int kBlock = 128;
constexpr float kMax = 448.0f;      // largest finite e4m3
constexpr float kTiny = 0x1p-96f;   // smallest maximum a scale is made from: 448 / amax stays finite

// A word holds one fp32 or two 16-bit values. Magnitudes as ordered bits: NaN
// above Inf above every finite value.
template <typename T>
constexpr int kPerWord = 4 / sizeof(T);
template <typename T>
__device__ __forceinline__ uint32_t mag(uint32_t w) {
    return w & (sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
}
template <typename T>
__device__ __forceinline__ uint32_t vmax(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 2) return __vmaxu2(a, b);
    else return max(a, b);
}
// The bits of the fp32 value of one magnitude of a word.
template <typename T>
__device__ __forceinline__ uint32_t float_bits(uint32_t m) {
    if constexpr (std::is_same_v<T, float>) return m;
    else if constexpr (std::is_same_v<T, __nv_bfloat16>) return m << 16;
    else return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
}
// The larger magnitude in a word, as fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t fold(uint32_t m) {
    if constexpr (sizeof(T) == 2) m = max(m & 0xFFFFu, m >> 16);
    return float_bits<T>(m);
}

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

// Eight consecutive values of a row; `n` of them exist (<= 0: none).
template <typename T>
struct Eight {
    static constexpr int W = 8 / kPerWord<T>;
    uint32_t w[W];
    __device__ __forceinline__ uint32_t max_word() const {
        uint32_t m = mag<T>(w[0]);
#pragma unroll
        for (int i = 1; i < W; ++i) m = vmax<T>(m, mag<T>(w[i]));
        return m;
    }
    __device__ __forceinline__ void floats(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (std::is_same_v<T, float>) {
                v[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, Eight<T>& x) {
    if (VEC && n >= 8) {
#pragma unroll
        for (int i = 0; i < Eight<T>::W; i += 4) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + i / 4);
            x.w[i] = u.x;
            x.w[i + 1] = u.y;
            x.w[i + 2] = u.z;
            x.w[i + 3] = u.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < Eight<T>::W; ++i) {
        if constexpr (sizeof(T) == 4) {
            x.w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
            x.w[i] = (2 * i < n ? h[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(h[2 * i + 1]) << 16 : 0u);
        }
    }
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
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2)
quant_tile_kernel(const __grid_constant__ QuantParams P) {
    constexpr int W = Eight<T>::W;  // words of eight values
    __shared__ uint32_t warp_max[kThreads / 32][16 * W];
    __shared__ __align__(16) float col_r[kBlock];
    __shared__ uint32_t tile[COLS ? kBlock * 32 : 1];
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15, warp = tid >> 5, lane = tid & 31;
    const int64_t rb = blockIdx.x / P.col_blocks, cb = blockIdx.x % P.col_blocks;
    const int64_t r0 = rb * kBlock, c0 = cb * kBlock;
    const int nr = static_cast<int>(P.rows - r0 < kBlock ? P.rows - r0 : kBlock);
    const int nc = static_cast<int>(P.cols - c0 < kBlock ? P.cols - c0 : kBlock);
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const T* x = static_cast<const T*>(P.x) + (r0 + 8 * rg) * P.ldx + c0 + 8 * cg;

    Eight<T> e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) load8<T, VEC>(x + i * P.ldx, 8 * rg + i < nr ? nc - 8 * cg : 0, e[i]);

    float r_tile = 0.0f;  // TILE
    float r_row = 0.0f;   // of row 8 rg + cg / 2
    if constexpr (TILE) {
        uint32_t m = e[0].max_word();
#pragma unroll
        for (int i = 1; i < 8; ++i) m = vmax<T>(m, e[i].max_word());
        m = __reduce_max_sync(0xFFFFFFFFu, fold<T>(m));
        if (lane == 0) warp_max[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) m = max(m, warp_max[k][0]);
        const Scale sc = scale_of(m);
        r_tile = sc.r;
        if (tid == 0) {
            if constexpr (ROWS) P.s[rb * P.col_blocks + cb] = sc.s;
            if constexpr (COLS) P.st[cb * P.row_blocks + rb] = sc.s;
        }
    } else {
        if constexpr (COLS) {
            uint32_t m[W];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                m[k] = mag<T>(e[0].w[k]);
#pragma unroll
                for (int i = 1; i < 8; ++i) m[k] = vmax<T>(m[k], mag<T>(e[i].w[k]));
                m[k] = vmax<T>(m[k], __shfl_xor_sync(0xFFFFFFFFu, m[k], 16));
            }
            if (lane < 16) {
#pragma unroll
                for (int k = 0; k < W; k += 4)
                    *reinterpret_cast<uint4*>(&warp_max[warp][cg * W + k]) =
                        make_uint4(m[k], m[k + 1], m[k + 2], m[k + 3]);
            }
        }
        if constexpr (ROWS) {
            uint32_t m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = e[i].max_word();
            // halving: a lane ends with row cg / 2 of its eight
#pragma unroll
            for (int h = 4; h > 0; h >>= 1) {
                const bool up = (cg & (2 * h)) != 0;
#pragma unroll
                for (int k = 0; k < h; ++k) {
                    const uint32_t send = up ? m[k] : m[k + h], keep = up ? m[k + h] : m[k];
                    m[k] = vmax<T>(keep, __shfl_xor_sync(0xFFFFFFFFu, send, 2 * h));
                }
            }
            m[0] = vmax<T>(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
            const Scale sc = scale_of(fold<T>(m[0]));
            r_row = sc.r;
            const int row = 8 * rg + (cg >> 1);
            if ((cg & 1) == 0 && row < nr) P.s[cb * P.rows + r0 + row] = sc.s;
        }
        if constexpr (COLS) {
            __syncthreads();
            if (tid < kBlock) {
                const int word = tid / kPerWord<T>;
                uint32_t m = warp_max[0][word];
#pragma unroll
                for (int k = 1; k < kThreads / 32; ++k) m = vmax<T>(m, warp_max[k][word]);
                if constexpr (sizeof(T) == 2) m = tid & 1 ? m >> 16 : m & 0xFFFFu;
                const Scale sc = scale_of(float_bits<T>(m));
                col_r[tid] = sc.r;
                if (tid < nc) P.st[rb * P.cols + c0 + tid] = sc.s;
            }
            __syncthreads();
        }
    }
    float rc[8];
    if constexpr (COLS) {
        if constexpr (TILE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) rc[j] = r_tile;
        } else {
            const float4 a = *reinterpret_cast<const float4*>(&col_r[8 * cg]);
            const float4 b = *reinterpret_cast<const float4*>(&col_r[8 * cg + 4]);
            rc[0] = a.x; rc[1] = a.y; rc[2] = a.z; rc[3] = a.w;
            rc[4] = b.x; rc[5] = b.y; rc[6] = b.z; rc[7] = b.w;
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {  // four rows at a time
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[4 * q + i].floats(v[i]);
        if constexpr (ROWS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 8 * rg + 4 * q + i;
                const float r = TILE ? r_tile : __shfl_sync(0xFFFFFFFFu, r_row, (lane & 16) + 2 * (4 * q + i));
                const uint32_t w0 = codes4(v[i][0], v[i][1], v[i][2], v[i][3], r, r, r, r);
                const uint32_t w1 = codes4(v[i][4], v[i][5], v[i][6], v[i][7], r, r, r, r);
                if (row < nr) store8<VEC>(P.q + (r0 + row) * P.ldq + c0 + 8 * cg, nc - 8 * cg, w0, w1);
            }
        }
        if constexpr (COLS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float r = rc[j];
                tile[(8 * cg + j) * 32 + 2 * (rg ^ cg) + q] = codes4(v[0][j], v[1][j], v[2][j], v[3][j], r, r, r, r);
            }
        }
    }
    if constexpr (COLS) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kBlock / 16; ++k) {
            const int col = k * 16 + rg;  // 16 threads a column, 8 rows each
            const uint2 w = *reinterpret_cast<const uint2*>(&tile[col * 32 + 2 * (cg ^ (col >> 3))]);
            if (col < nc) store8<VEC>(P.qt + (c0 + col) * P.ldqt + r0 + 8 * cg, nr - 8 * cg, w.x, w.y);
        }
    }
}

// Row blocks without the transpose: 16 threads a block, 16 rows and
// kRowBlocks blocks a CTA, every block's loads in flight at once.
constexpr int kRowBlocks = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const __grid_constant__ QuantParams P) {
    const int rg = threadIdx.x >> 4, cg = threadIdx.x & 15, lane = threadIdx.x & 31;
    const int64_t groups = (P.col_blocks + kRowBlocks - 1) / kRowBlocks;
    const int64_t row = blockIdx.x / groups * 16 + rg;
    const int64_t cb0 = blockIdx.x % groups * kRowBlocks;
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const T* x = static_cast<const T*>(P.x) + row * P.ldx;
    Eight<T> e[kRowBlocks];
    int n[kRowBlocks];
#pragma unroll
    for (int k = 0; k < kRowBlocks; ++k) {
        const int64_t c = (cb0 + k) * kBlock + 8 * cg;
        const int64_t left = row < P.rows ? P.cols - c : 0;
        n[k] = left > 8 ? 8 : static_cast<int>(left < 0 ? 0 : left);
        load8<T, VEC>(x + c, n[k], e[k]);
    }
    // the four blocks' maxima by halving: a lane ends with block cg / 4
    static_assert(kRowBlocks == 4, "two halvings");
    uint32_t m[kRowBlocks];
#pragma unroll
    for (int k = 0; k < kRowBlocks; ++k) m[k] = e[k].max_word();
#pragma unroll
    for (int h = 2; h > 0; h >>= 1) {
        const bool up = (cg & (4 * h)) != 0;
#pragma unroll
        for (int k = 0; k < h; ++k) {
            const uint32_t send = up ? m[k] : m[k + h], keep = up ? m[k + h] : m[k];
            m[k] = vmax<T>(keep, __shfl_xor_sync(0xFFFFFFFFu, send, 4 * h));
        }
    }
    m[0] = vmax<T>(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 2));
    m[0] = vmax<T>(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
    const Scale sc = scale_of(fold<T>(m[0]));
    const int64_t cb = cb0 + (cg >> 2);
    if ((cg & 3) == 0 && row < P.rows && cb < P.col_blocks) P.s[cb * P.rows + row] = sc.s;
#pragma unroll
    for (int k = 0; k < kRowBlocks; ++k) {
        const float r = __shfl_sync(0xFFFFFFFFu, sc.r, (lane & 16) + 4 * k);
        float v[8];
        e[k].floats(v);
        if (n[k] > 0)
            store8<VEC>(P.q + row * P.ldq + (cb0 + k) * kBlock + 8 * cg, n[k],
                        codes4(v[0], v[1], v[2], v[3], r, r, r, r), codes4(v[4], v[5], v[6], v[7], r, r, r, r));
    }
}

// --------------------------------------------------------------- host side
// Launch whose CTAs may start while the launch before it in the stream drains
// (the kernels wait for its results themselves).
static cudaError_t launch_after(void (*kernel)(QuantParams), unsigned grid, const QuantParams& P, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P);
    if (e == cudaSuccess) pqc::count_launch();
    return e;
}

template <typename T, bool VEC>
static cudaError_t launch(bool tile, const QuantParams& P, cudaStream_t s) {
    if (!tile && !P.qt) {
        const int64_t groups = (P.col_blocks + kRowBlocks - 1) / kRowBlocks;
        const unsigned grid = static_cast<unsigned>((P.rows + 15) / 16 * groups);
        return launch_after(quant_rows_kernel<T, VEC>, grid, P, s);
    } else {
        const unsigned grid = static_cast<unsigned>(P.row_blocks * P.col_blocks);
        auto kernel = tile ? (P.q ? (P.qt ? quant_tile_kernel<T, true, true, true, VEC>
                                          : quant_tile_kernel<T, true, true, false, VEC>)
                                  : quant_tile_kernel<T, true, false, true, VEC>)
                           : (P.q ? quant_tile_kernel<T, false, true, true, VEC>
                                  : quant_tile_kernel<T, false, false, true, VEC>);
        return launch_after(kernel, grid, P, s);
    }
}

template <typename T>
static pq_status_t run(bool tile, const QuantParams& P, cudaStream_t s) {
    // vector accesses: 16-byte loads (8 two-byte or 4 four-byte values) and
    // 8-byte stores of codes; a row's ragged end goes element by element
    const bool vec = pq::aligned(P.x, 16) && P.ldx % (16 / sizeof(T)) == 0 &&
                     (!P.q || (pq::aligned(P.q, 8) && P.ldq % 8 == 0)) &&
                     (!P.qt || (pq::aligned(P.qt, 8) && P.ldqt % 8 == 0));
    return pq::cuda_status(vec ? launch<T, true>(tile, P, s) : launch<T, false>(tile, P, s));
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
    if (!pq::aligned(s_out, 4) || !pq::aligned(st_out, 4)) return PQ_ERR_MISALIGNED;
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
