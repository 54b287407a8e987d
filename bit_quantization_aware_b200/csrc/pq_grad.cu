// Global gradient norm and clipping (sm_100a).
//
//   norm = sqrt(sum g^2) over all gradients of a step
//   coef = min(1, max_norm / (norm + 1e-6)),  g <- g * coef
//
// The gradients are plain tensors (bf16, fp16, fp32), the quantizer's dW and
// d(alpha) formed on the fly from w, alpha and the upstream gradient (6 bytes
// read per weight where writing dW and reading it back would move 14), or the
// same over row shards with the replicas' gradients summed first.
//
// Sums. Squares are taken and added in fp64: fp32 squares of bf16 and fp32
// gradients leave its range (|g| < 1e-19 or > 1.8e19), and the sum of
// billions of them its precision. Each thread adds its own elements, a fixed
// shuffle tree the warp's, one thread the warps', so the same call gives the
// same bits on every run; every CTA leaves one partial sum in the workspace,
// and the kernel that follows adds those in a fixed order (no atomics).
//
// Bound: memory. fp64 itself has the rate for it, the conversion unit has not
// (fp32 to fp64 conversions kept it 76% busy at 5.0 TB/s of bf16 gradients):
// tensors are widened with integer operations instead, see widen, and the
// quantizer's dW, zero or g, is not converted a second time.
// The norm reads each gradient once; scaling reads and writes
// it once more, from the last unit to the first, so what the norm pass left
// in L2 is read there. An in-place scale with coef == 1 touches nothing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "pq.h"
#include "pq_launches.cuh"
#include "pq_quant.cuh"
#include "pq_units.cuh"

namespace pqn {

using namespace pq;

constexpr int kMaxCtas = 1184;     // CTAs, and so partial sums, of one norm launch
constexpr int kVecBytes = 32;      // bytes of one vector access
constexpr int kVecsPerThread = 4;  // vector accesses a thread has in flight
constexpr int kUnitBytes = kThreads * kVecsPerThread * kVecBytes;  // of a tensor's unit

// ----------------------------------------------------------- element types
template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }

// |v| as fp64 times 2^-896, from fp32 bits: the exponent field moves as it is
// (fp64's bias is 896 more), so zeros and subnormals come out right, and 2^896
// times it is |v| exactly. Inf and NaN come out finite; Special keeps them.
__device__ __forceinline__ double widen(uint32_t bits) {
    return __hiloint2double(static_cast<int>((bits & 0x7FFFFFFFu) >> 3), static_cast<int>(bits << 29));
}
constexpr double kWiden = 0x1p896;

__device__ __forceinline__ double add_square(uint32_t bits, double acc) {
    const double e = __dmul_rn(widen(bits), kWiden);
    return __fma_rn(e, e, acc);
}

// The largest magnitude that a thread met, as ordered bits of T (two 16-bit
// values a word): NaN above Inf above every finite value.
template <typename T>
struct Special {
    uint32_t m = 0;
    __device__ __forceinline__ void see(uint32_t word) {
        if constexpr (sizeof(T) == 2) m = __vmaxu2(m, word & 0x7FFF7FFFu);
        else m = max(m, word & 0x7FFFFFFFu);
    }
    // the thread's sum: NaN or Inf if it met one
    __device__ __forceinline__ double close(double acc) const {
        uint32_t v = m, inf = 0x7F800000u;
        if constexpr (sizeof(T) == 2) {
            v = max(v & 0xFFFFu, v >> 16);
            inf = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;
        }
        if (v < inf) return acc;
        return __hiloint2double(v == inf ? 0x7FF00000 : 0x7FFFFFFF, 0);
    }
};

// One 32-byte vector of T (8 or 16 elements).
template <typename T>
struct Vec {
    static constexpr int kN = kVecBytes / sizeof(T);
    union {
        uint32_t w[8];
        T e[kN];
    };
    __device__ __forceinline__ Vec() {}
};

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, Vec<T>& v) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]),
                   "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p));
}

template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& v) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.w[0]),
                 "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
                 "r"(v.w[7])
                 : "memory");
}

// ------------------------------------------------------------- reductions
// Sum over the CTA in a fixed order; the result is thread 0's.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double slot[kThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = __dadd_rn(v, __shfl_down_sync(0xffffffffu, v, off));
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int k = 1; k < kThreads / 32; ++k) v = __dadd_rn(v, slot[k]);
    return v;
}

// Sum of n partial sums by one CTA, in an order that n alone fixes.
__device__ __forceinline__ double sum_partials(const double* p, int n) {
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) v = __dadd_rn(v, p[i]);
    return block_sum(v);
}

// coef = min(1, max_norm / (norm + 1e-6)); NaN stays NaN.
__device__ __forceinline__ float clip_coef(double norm, double max_norm) {
    const double c = max_norm / (norm + 1e-6);
    return c >= 1.0 ? 1.0f : static_cast<float>(c);
}

// The entry that owns unit u, by bisection: a CTA's first unit may lie behind
// hundreds of entries, whose descriptors it would otherwise read one by one
// (98 tensors of 2048 elements: 12.9 us for the norm and the scaling so).
template <typename D, int CAP>
__device__ __forceinline__ int locate(const BatchT<D, CAP>& b, int64_t u) {
    int lo = 0, hi = b.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.m[mid].unit_begin <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ----------------------------------------------------------------- tensors
struct TensorDesc {  // 32 bytes: 256 of them go with a launch
    const void* g;
    void* out;
    int64_t n_vec;    // 2 n + 1 where vector accesses are aligned (32 bytes), else 2 n
    int64_t unit_begin;
    __device__ __forceinline__ int64_t n() const { return n_vec >> 1; }
    __device__ __forceinline__ bool vec() const { return n_vec & 1; }
    __device__ __forceinline__ bool inplace() const { return out == g; }
};

template <typename T, int CAP>
struct NormBatch {
    BatchT<TensorDesc, CAP> b;
    double* partial;  // [gridDim.x]
};

template <typename T, int CAP>
__global__ void __launch_bounds__(kThreads)
norm_tensors_kernel(const __grid_constant__ NormBatch<T, CAP> P) {
    constexpr int kUnit = kUnitBytes / sizeof(T);
    constexpr int V = Vec<T>::kN;
    double acc[2] = {0.0, 0.0};
    Special<T> special;
    int mi = locate(P.b, blockIdx.x);
    for (int64_t u = blockIdx.x; u < P.b.total_units; u += gridDim.x) {
        mi = find_matrix(P.b, mi, u);
        const TensorDesc& t = P.b.m[mi];
        const int64_t base = (u - t.unit_begin) * kUnit;
        const T* g = static_cast<const T*>(t.g) + base;
        const int n = static_cast<int>(t.n() - base < kUnit ? t.n() - base : kUnit);
        int done = 0;
        if (t.vec()) {
            Vec<T> v[kVecsPerThread];
            done = n / V * V;
#pragma unroll
            for (int k = 0; k < kVecsPerThread; ++k) {
                const int at = (k * kThreads + static_cast<int>(threadIdx.x)) * V;
                if (at < done) load_vec(g + at, v[k]);
            }
#pragma unroll
            for (int k = 0; k < kVecsPerThread; ++k) {
                const int at = (k * kThreads + static_cast<int>(threadIdx.x)) * V;
                if (at < done) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t w = v[k].w[i];
                        special.see(w);
                        if constexpr (std::is_same_v<T, float>) {
                            acc[i & 1] = add_square(w, acc[i & 1]);
                        } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                            acc[0] = add_square(w << 16, acc[0]);
                            acc[1] = add_square(w & 0xFFFF0000u, acc[1]);
                        } else {
                            acc[0] = add_square(__float_as_uint(to_float(v[k].e[2 * i])), acc[0]);
                            acc[1] = add_square(__float_as_uint(to_float(v[k].e[2 * i + 1])), acc[1]);
                        }
                    }
                }
            }
        }
        for (int i = done + static_cast<int>(threadIdx.x); i < n; i += kThreads) {
            if constexpr (sizeof(T) == 2) special.see(reinterpret_cast<const uint16_t*>(g)[i]);
            else special.see(reinterpret_cast<const uint32_t*>(g)[i]);
            acc[0] = add_square(__float_as_uint(to_float(g[i])), acc[0]);
        }
    }
    const double sum = block_sum(special.close(__dadd_rn(acc[0], acc[1])));
    if (threadIdx.x == 0) P.partial[blockIdx.x] = sum;
}

// What closes a norm: the partial sums of its launches and where the results go.
struct NormEnd {
    const double* partial;
    int32_t count;
    int32_t pad_;
    double max_norm;
    double* sumsq;  // nullable
    float* norm;    // nullable
    float* coef;    // nullable
};

__device__ __forceinline__ void write_end(const NormEnd& e, double sum) {
    const double norm = sqrt(sum);
    if (e.sumsq) *e.sumsq = sum;
    if (e.norm) *e.norm = static_cast<float>(norm);
    if (e.coef) *e.coef = clip_coef(norm, e.max_norm);
}

__global__ void __launch_bounds__(kThreads) norm_end_kernel(const NormEnd e) {
    cudaGridDependencySynchronize();
    const double sum = sum_partials(e.partial, e.count);
    if (threadIdx.x == 0) write_end(e, sum);
}

// Scaling rounds twice for a 16-bit output: the product to fp32, as the updates
// that take the factor do, and that to the type. One rounding would need the
// product's remainder, a second operation an element, for 2^-24 of the value.
template <typename T, typename O, int CAP>
struct ScaleBatch {
    BatchT<TensorDesc, CAP> b;
    const float* coef;  // the factor, or NULL: it is formed from `end`
    NormEnd end;        // written by CTA 0 when coef is NULL
};

template <typename T, typename O, int CAP>
__global__ void __launch_bounds__(kThreads)
scale_tensors_kernel(const __grid_constant__ ScaleBatch<T, O, CAP> P) {
    constexpr int kUnit = kUnitBytes / sizeof(T);
    constexpr int V = Vec<T>::kN;
    constexpr int kOut = Vec<O>::kN < V ? V / Vec<O>::kN : 1;  // output vectors per input vector
    __shared__ float s_coef;
    cudaGridDependencySynchronize();
    if (P.coef) {
        if (threadIdx.x == 0) s_coef = *P.coef;
    } else {
        const double sum = sum_partials(P.end.partial, P.end.count);
        if (threadIdx.x == 0) {
            s_coef = clip_coef(sqrt(sum), P.end.max_norm);
            if (blockIdx.x == 0) write_end(P.end, sum);
        }
    }
    __syncthreads();
    const float c = s_coef;
    int mi = locate(P.b, P.b.total_units - 1 - blockIdx.x);
    for (int64_t r = blockIdx.x; r < P.b.total_units; r += gridDim.x) {
        const int64_t u = P.b.total_units - 1 - r;
        while (P.b.m[mi].unit_begin > u) --mi;
        const TensorDesc& t = P.b.m[mi];
        if (t.inplace() && c == 1.0f) continue;
        const int64_t base = (u - t.unit_begin) * kUnit;
        const T* g = static_cast<const T*>(t.g) + base;
        O* out = static_cast<O*>(t.out) + base;
        const int n = static_cast<int>(t.n() - base < kUnit ? t.n() - base : kUnit);
        int done = 0;
        if (t.vec()) {
            Vec<T> v[kVecsPerThread];
            done = n / V * V;
#pragma unroll
            for (int k = 0; k < kVecsPerThread; ++k) {
                const int at = (k * kThreads + static_cast<int>(threadIdx.x)) * V;
                if (at < done) load_vec(g + at, v[k]);
            }
#pragma unroll
            for (int k = 0; k < kVecsPerThread; ++k) {
                const int at = (k * kThreads + static_cast<int>(threadIdx.x)) * V;
                if (at < done) {
#pragma unroll
                    for (int j = 0; j < kOut; ++j) {
                        Vec<O> o;
#pragma unroll
                        for (int i = 0; i < V / kOut; ++i)
                            o.e[i] = from_float<O>(__fmul_rn(to_float(v[k].e[j * (V / kOut) + i]), c));
                        store_vec(out + at + j * (V / kOut), o);
                    }
                }
            }
        }
        for (int i = done + static_cast<int>(threadIdx.x); i < n; i += kThreads)
            out[i] = from_float<O>(__fmul_rn(to_float(g[i]), c));
    }
}

// ------------------------------------------------ the quantizer's gradient
// dW = inside ? g : 0 and d(alpha) of pq_fakequant_bwd, squared and summed
// without writing dW; the d(alpha) of a row is rounded to fp32 first, as the
// backward and the optimizer see it. SHARD: g is the sum over the replicas'
// gradients, as in pq_reduce_bwd_adamw.
constexpr int kMaxSources = 16;

// One chunk: the row's d(alpha) sum as bwd_chunk forms it, and the squares of
// dW from the same widened g.
template <int Q>
__device__ __forceinline__ void norm_chunk(const float (&v)[8], const float (&g)[8], const RowScale& s,
                                           double& acc, double& sq) {
    float x[8];
    divide8(v, s, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Elem e = quantize_x<Q>(x[i]);
        const float xm = e.inside ? x[i] : 0.0f;
        const double dg = static_cast<double>(g[i]);
        acc = __fma_rn(dg, __dsub_rn(static_cast<double>(e.level), static_cast<double>(xm)), acc);
        if (e.inside) sq = __fma_rn(dg, dg, sq);
    }
}

struct GradDesc {
    const float* w;
    const float* alpha;
    const uint16_t* g;  // SHARD: unused
    float* dalpha;      // nullable
    int64_t rows;
    int64_t cols;
    int64_t g_offset;   // SHARD
    int64_t unit_begin;
    float grad_scale;
    int32_t tpr_log2;
};

template <int CAP>
struct GradBatch {
    BatchT<GradDesc, CAP> b;
    const uint16_t* src[kMaxSources];
    int32_t n_src;
    float grad_mult;
    double* partial;
};

template <int Q, bool VEC, bool SHARD, int CAP>
__global__ void __launch_bounds__(kThreads, PQ_BWD_MIN_CTAS)
norm_matrices_kernel(const __grid_constant__ GradBatch<CAP> P) {
    __shared__ double warp_sum[2][kThreads / 32];
    double sq = 0.0;
    int mi = locate(P.b, blockIdx.x), prev_mi = mi, parity = 0;
    // block-uniform trip count: every thread reaches every barrier
    for (int64_t u = blockIdx.x; u < P.b.total_units; u += gridDim.x, parity ^= 1) {
        mi = find_matrix(P.b, mi, u);
        // a new matrix may regroup the threads: let every group finish
        // reading the previous slots first
        if (mi != prev_mi) __syncthreads();
        prev_mi = mi;
        const GradDesc& m = P.b.m[mi];
        const int tl = m.tpr_log2;
        const int tpr = 1 << tl;
        const int lane = threadIdx.x & (tpr - 1);
        const int rsub = threadIdx.x >> tl;
        const int64_t row = (u - m.unit_begin) * (kThreads >> tl) + rsub;
        const int64_t nch = (m.cols + 7) >> 3;
        double acc = 0.0;
        if (row < m.rows && nch > 0) {  // without columns the arrays may be NULL
            const RowScale a = row_scale(__ldg(m.alpha + row));
            const float* wr = m.w + row * m.cols;
            const int64_t goff = (SHARD ? m.g_offset : 0) + row * m.cols;
            constexpr int U = SHARD ? 1 : PQ_BWD_UNROLL;
            for (int64_t ch = lane; ch < nch; ch += U * tpr) {
                float v[U][8];
                uint32_t gw[U][4];
                if constexpr (!SHARD) {
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        const int64_t c = ch + k * tpr;
                        if (c < nch) {
                            if constexpr (VEC) {
                                load8(wr + c * 8, v[k]);
                                load_g8(m.g + goff + c * 8, gw[k]);
                            } else {
                                const int n = tail_n(m.cols, c);
                                load8_tail(wr + c * 8, n, v[k]);
                                load_g8_tail(m.g + goff + c * 8, n, gw[k]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int64_t c = ch + k * tpr;
                    if (c >= nch) continue;
                    float gs[8];
                    if constexpr (SHARD) {
                        const int n = tail_n(m.cols, c);
                        if constexpr (VEC) load8(wr + c * 8, v[k]);
                        else load8_tail(wr + c * 8, n, v[k]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) gs[i] = 0.0f;
#pragma unroll 4
                        for (int r = 0; r < P.n_src; ++r) {
                            if constexpr (VEC) load_g8(P.src[r] + goff + c * 8, gw[k]);
                            else load_g8_tail(P.src[r] + goff + c * 8, n, gw[k]);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                gs[i] = __fadd_rn(gs[i], (i & 1) ? __uint_as_float(gw[k][i / 2] & 0xFFFF0000u)
                                                                 : __uint_as_float(gw[k][i / 2] << 16));
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) gs[i] = __fmul_rn(gs[i], P.grad_mult);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            gs[i] = (i & 1) ? __uint_as_float(gw[k][i / 2] & 0xFFFF0000u)
                                            : __uint_as_float(gw[k][i / 2] << 16);
                    }
                    norm_chunk<Q>(v[k], gs, a, acc, sq);
                }
            }
        }
        // reduce the row group's partial sums in a fixed order
        const int seg = tpr < 32 ? tpr : 32;
        for (int off = seg >> 1; off > 0; off >>= 1)
            acc = __dadd_rn(acc, __shfl_down_sync(0xffffffffu, acc, off, seg));
        if (tpr > 32) {
            if ((threadIdx.x & 31) == 0) warp_sum[parity][threadIdx.x >> 5] = acc;
            group_barrier(1 + rsub, tpr);
            if (lane == 0) {
                const int w0 = threadIdx.x >> 5;
                double t = warp_sum[parity][w0];
                for (int k = 1; k < (tpr >> 5); ++k) t = __dadd_rn(t, warp_sum[parity][w0 + k]);
                acc = t;
            }
        }
        if (lane == 0 && row < m.rows) {
            const float da = static_cast<float>(__dmul_rn(acc, static_cast<double>(m.grad_scale)));
            if (m.dalpha) m.dalpha[row] = da;
            sq = __fma_rn(static_cast<double>(da), static_cast<double>(da), sq);
        }
    }
    sq = block_sum(sq);
    if (threadIdx.x == 0) P.partial[blockIdx.x] = sq;
}

// --------------------------------------------------------------- host side
static int dtype_bytes(int dtype) {
    switch (dtype) {
        case PQ_BF16: case PQ_FP16: return 2;
        case PQ_FP32: return 4;
        default: return 0;
    }
}

static pq_status_t check_tensor(const pq_tensor_t& t, bool scale) {
    if (dtype_bytes(t.dtype) == 0 || t.numel < 0) return PQ_ERR_INVALID_ARG;
    if (t.numel == 0) return PQ_OK;
    if (!t.data) return PQ_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(t.data) % dtype_bytes(t.dtype)) return PQ_ERR_MISALIGNED;
    if (scale && t.out) {
        if (t.out_dtype != t.dtype && t.out_dtype != PQ_FP32) return PQ_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(t.out) % dtype_bytes(t.out_dtype)) return PQ_ERR_MISALIGNED;
        // in place, or apart: units are scaled in any order
        const uintptr_t d = reinterpret_cast<uintptr_t>(t.data), o = reinterpret_cast<uintptr_t>(t.out);
        const uintptr_t dn = static_cast<uintptr_t>(t.numel) * dtype_bytes(t.dtype);
        const uintptr_t on = static_cast<uintptr_t>(t.numel) * dtype_bytes(t.out_dtype);
        if (o < d + dn && d < o + on && !(o == d && t.out_dtype == t.dtype)) return PQ_ERR_INVALID_ARG;
    }
    return PQ_OK;
}

static int out_dtype_of(const pq_tensor_t& t) { return t.out ? t.out_dtype : t.dtype; }

// Where a norm's launches put their partial sums.
struct Partials {
    double* at;
    int32_t used;
    int32_t room;
    // slots of a launch of at most `grid` CTAs, or NULL when the workspace is full
    double* take(int grid) {
        if (used + grid > room) return nullptr;
        double* p = at + used;
        used += grid;
        return p;
    }
};

constexpr int64_t kClasses = 3 + 4;  // launches that partly filled batches can add

static int64_t workspace_bytes(int64_t n_tensors, int64_t n_mats) {
    return (n_tensors / kMaxBatch + n_mats / kMaxBatch + kClasses) * kMaxCtas * 8;
}

template <int CAP, int CAP_FROM, typename D>
static void copy_batch(BatchT<D, CAP>& to, const BatchT<D, CAP_FROM>& from) {
    to.n = from.n;
    to.pad_ = 0;
    to.total_units = from.total_units;
    for (int i = 0; i < from.n; ++i) to.m[i] = from.m[i];
}

template <typename K>
static int grid_of(K kernel, int* cache, int64_t units) {
    int64_t g = persistent_ctas(kernel, cache);
    if (g > kMaxCtas) g = kMaxCtas;
    return static_cast<int>(units < g ? units : g);
}

// Launch that may begin while the kernel before it in the stream drains; it
// waits for that kernel's results (cudaGridDependencySynchronize).
template <typename P>
static cudaError_t launch_after(void (*kernel)(P), int grid, const P& prm, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm);
    if (e == cudaSuccess) pqc::count_launch();
    return e;
}

template <typename T, int CAP>
static pq_status_t launch_norm_cap(const BatchT<TensorDesc>& b, Partials& parts, cudaStream_t s) {
    static int cache[64] = {0};
    static thread_local NormBatch<T, CAP> prm;
    copy_batch(prm.b, b);
    const int grid = grid_of(norm_tensors_kernel<T, CAP>, cache, b.total_units);
    prm.partial = parts.take(grid);
    if (!prm.partial) return PQ_ERR_INVALID_ARG;
    norm_tensors_kernel<T, CAP><<<grid, kThreads, 0, s>>>(prm);
    pqc::count_launch();
    return cuda_status(cudaGetLastError());
}

template <typename T>
static pq_status_t launch_norm(const BatchT<TensorDesc>& b, Partials& parts, cudaStream_t s) {
    if (b.n <= kSmallBatch) return launch_norm_cap<T, kSmallBatch>(b, parts, s);
    return launch_norm_cap<T, kMaxBatch>(b, parts, s);
}

template <typename T, typename O, int CAP>
static pq_status_t launch_scale_cap(const BatchT<TensorDesc>& b, const float* coef, const NormEnd& end,
                                    cudaStream_t s) {
    static int cache[64] = {0};
    static thread_local ScaleBatch<T, O, CAP> prm;
    copy_batch(prm.b, b);
    prm.coef = coef;
    prm.end = end;
    const int grid = grid_of(scale_tensors_kernel<T, O, CAP>, cache, b.total_units);
    return cuda_status(launch_after(scale_tensors_kernel<T, O, CAP>, grid, prm, s));
}

template <typename T, typename O>
static pq_status_t launch_scale(const BatchT<TensorDesc>& b, const float* coef, const NormEnd& end,
                                cudaStream_t s) {
    if (b.n <= kSmallBatch) return launch_scale_cap<T, O, kSmallBatch>(b, coef, end, s);
    return launch_scale_cap<T, O, kMaxBatch>(b, coef, end, s);
}

static void tensor_batch_add(BatchT<TensorDesc>& b, const pq_tensor_t& t) {
    TensorDesc& d = b.m[b.n++];
    d.g = t.data;
    d.out = t.out ? t.out : t.data;
    d.n_vec = 2 * t.numel + (aligned(t.data, kVecBytes) && aligned(d.out, kVecBytes));
    d.unit_begin = b.total_units;
    const int64_t unit = kUnitBytes / dtype_bytes(t.dtype);
    b.total_units += (t.numel + unit - 1) / unit;
}

// Partial sums of the tensors, one launch per dtype and 256 tensors.
static pq_status_t norm_tensors(int32_t n, const pq_tensor_t* ts, Partials& parts, cudaStream_t s) {
    static thread_local BatchT<TensorDesc> b;
    uint32_t present = 0;
    for (int32_t i = 0; i < n; ++i)
        if (ts[i].numel) present |= 1u << ts[i].dtype;
    for (int dtype : {PQ_BF16, PQ_FP16, PQ_FP32}) {
        if (!(present >> dtype & 1u)) continue;
        b.n = 0;
        b.total_units = 0;
        auto flush = [&]() -> pq_status_t {
            if (b.n == 0) return PQ_OK;
            const pq_status_t st = dtype == PQ_BF16   ? launch_norm<__nv_bfloat16>(b, parts, s)
                                   : dtype == PQ_FP16 ? launch_norm<__half>(b, parts, s)
                                                      : launch_norm<float>(b, parts, s);
            b.n = 0;
            b.total_units = 0;
            return st;
        };
        for (int32_t i = 0; i < n; ++i) {
            if (ts[i].dtype != dtype || ts[i].numel == 0) continue;
            if (b.n == kMaxBatch) {
                const pq_status_t st = flush();
                if (st != PQ_OK) return st;
            }
            tensor_batch_add(b, ts[i]);
        }
        const pq_status_t st = flush();
        if (st != PQ_OK) return st;
    }
    return PQ_OK;
}

// Scales the tensors, one launch per pair of dtypes and 256 tensors; `scaled`
// tells whether anything was launched.
static pq_status_t scale_tensors(int32_t n, const pq_tensor_t* ts, const float* coef, const NormEnd& end,
                                 bool& scaled, cudaStream_t s) {
    static thread_local BatchT<TensorDesc> b;
    uint32_t present = 0;  // pairs of dtypes
    for (int32_t i = 0; i < n; ++i)
        if (ts[i].numel) present |= 1u << (4 * ts[i].dtype + out_dtype_of(ts[i]));
    for (int cls = 0; cls < 5; ++cls) {
        static constexpr int kIn[5] = {PQ_BF16, PQ_BF16, PQ_FP16, PQ_FP16, PQ_FP32};
        static constexpr int kOut[5] = {PQ_BF16, PQ_FP32, PQ_FP16, PQ_FP32, PQ_FP32};
        if (!(present >> (4 * kIn[cls] + kOut[cls]) & 1u)) continue;
        b.n = 0;
        b.total_units = 0;
        auto flush = [&]() -> pq_status_t {
            if (b.n == 0) return PQ_OK;
            scaled = true;
            pq_status_t st;
            switch (cls) {
                case 0: st = launch_scale<__nv_bfloat16, __nv_bfloat16>(b, coef, end, s); break;
                case 1: st = launch_scale<__nv_bfloat16, float>(b, coef, end, s); break;
                case 2: st = launch_scale<__half, __half>(b, coef, end, s); break;
                case 3: st = launch_scale<__half, float>(b, coef, end, s); break;
                default: st = launch_scale<float, float>(b, coef, end, s); break;
            }
            b.n = 0;
            b.total_units = 0;
            return st;
        };
        for (int32_t i = 0; i < n; ++i) {
            if (ts[i].numel == 0 || ts[i].dtype != kIn[cls] || out_dtype_of(ts[i]) != kOut[cls]) continue;
            if (b.n == kMaxBatch) {
                const pq_status_t st = flush();
                if (st != PQ_OK) return st;
            }
            tensor_batch_add(b, ts[i]);
        }
        const pq_status_t st = flush();
        if (st != PQ_OK) return st;
    }
    return PQ_OK;
}

template <int Q, bool VEC, bool SHARD, int CAP>
static pq_status_t launch_grad_cap(const GradBatch<kMaxBatch>& b, Partials& parts, cudaStream_t s) {
    static int cache[64] = {0};
    static thread_local GradBatch<CAP> prm;
    copy_batch(prm.b, b.b);
    for (int k = 0; k < kMaxSources; ++k) prm.src[k] = b.src[k];
    prm.n_src = b.n_src;
    prm.grad_mult = b.grad_mult;
    auto kernel = norm_matrices_kernel<Q, VEC, SHARD, CAP>;
    const int grid = grid_of(kernel, cache, b.b.total_units);
    prm.partial = parts.take(grid);
    if (!prm.partial) return PQ_ERR_INVALID_ARG;
    kernel<<<grid, kThreads, 0, s>>>(prm);
    pqc::count_launch();
    return cuda_status(cudaGetLastError());
}

template <bool SHARD>
static pq_status_t launch_grad(int q, bool vec, const GradBatch<kMaxBatch>& b, Partials& parts,
                               cudaStream_t s) {
    pq_status_t st = PQ_OK;
    dispatch_q(q, [&]<int Q>() {
        if (b.b.n <= kSmallBatch)
            st = vec ? launch_grad_cap<Q, true, SHARD, kSmallBatch>(b, parts, s)
                     : launch_grad_cap<Q, false, SHARD, kSmallBatch>(b, parts, s);
        else
            st = vec ? launch_grad_cap<Q, true, SHARD, kMaxBatch>(b, parts, s)
                     : launch_grad_cap<Q, false, SHARD, kMaxBatch>(b, parts, s);
    });
    return st;
}

static void grad_batch_add(GradBatch<kMaxBatch>& b, const GradDesc& m) {
    GradDesc& d = b.b.m[b.b.n++];
    d = m;
    d.unit_begin = b.b.total_units;
    d.tpr_log2 = bwd_tpr_log2(m.rows, m.cols);
    b.b.total_units += (m.rows + (kThreads >> d.tpr_log2) - 1) / (kThreads >> d.tpr_log2);
}

// Partial sums of the quantizer's gradient over n matrices (or shards) that
// desc(i) describes and vec(i) classes; sources are set in b.
template <bool SHARD, typename Desc, typename IsVec>
static pq_status_t norm_matrices(int q, int32_t n, GradBatch<kMaxBatch>& b, Desc desc, IsVec is_vec,
                                 Partials& parts, cudaStream_t s) {
    for (int cls = 0; cls < 2; ++cls) {
        const bool vec = cls == 0;
        b.b.n = 0;
        b.b.pad_ = 0;
        b.b.total_units = 0;
        for (int32_t i = 0; i < n; ++i) {
            const GradDesc d = desc(i);
            // rows without columns have d(alpha) = 0, which the element path writes
            if (d.rows == 0 || is_vec(d) != vec) continue;
            if (b.b.n == kMaxBatch) {
                const pq_status_t st = launch_grad<SHARD>(q, vec, b, parts, s);
                if (st != PQ_OK) return st;
                b.b.n = 0;
                b.b.total_units = 0;
            }
            grad_batch_add(b, d);
        }
        if (b.b.n > 0) {
            const pq_status_t st = launch_grad<SHARD>(q, vec, b, parts, s);
            if (st != PQ_OK) return st;
        }
    }
    return PQ_OK;
}

static bool max_norm_ok(double max_norm) { return max_norm >= 0.0; }  // false for NaN

static pq_status_t take_workspace(void* workspace, int64_t bytes, int64_t need, Partials& parts) {
    if (!workspace || bytes < need || !aligned(workspace, 16)) return PQ_ERR_INVALID_ARG;
    parts.at = static_cast<double*>(workspace);
    parts.used = 0;
    parts.room = static_cast<int32_t>(need / 8);
    return PQ_OK;
}

static pq_status_t check_mats(int q, int32_t n, const pq_matrix_t* mats) {
    if (n < 0 || (n > 0 && (!mats || code_bits_of(q) == 0))) return PQ_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        const pq_matrix_t& m = mats[i];
        if (m.rows < 0 || m.cols < 0) return PQ_ERR_INVALID_ARG;
        if (m.rows > 0 && m.cols > 0 && (!m.w || !m.alpha || !m.g_bf16)) return PQ_ERR_INVALID_ARG;
        if (m.rows > 0 &&
            (!aligned(m.w, 4) || !aligned(m.alpha, 4) || !aligned(m.g_bf16, 2) || !aligned(m.dalpha_out, 4)))
            return PQ_ERR_MISALIGNED;
    }
    return PQ_OK;
}

static pq_status_t check_tensors(int32_t n, const pq_tensor_t* ts, bool scale) {
    if (n < 0 || (n > 0 && !ts)) return PQ_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        const pq_status_t st = check_tensor(ts[i], scale);
        if (st != PQ_OK) return st;
    }
    return PQ_OK;
}

// The scalars that a norm writes, each nullable.
static bool scalars_aligned(const double* sumsq, const float* norm, const float* coef) {
    return aligned(sumsq, 8) && aligned(norm, 4) && aligned(coef, 4);
}

static NormEnd norm_end(const Partials& parts, double max_norm, double* sumsq, float* norm, float* coef) {
    NormEnd e = {};
    e.partial = parts.at;
    e.count = parts.used;
    e.max_norm = max_norm;
    e.sumsq = sumsq;
    e.norm = norm;
    e.coef = coef;
    return e;
}

}  // namespace pqn

using namespace pqn;

extern "C" {

int64_t pq_grad_norm_workspace_bytes(int32_t n_tensors, int32_t n_mats) {
    return n_tensors < 0 || n_mats < 0 ? -1 : workspace_bytes(n_tensors, n_mats);
}

pq_status_t pq_grad_norm(int32_t n, const pq_tensor_t* tensors, pq_quant_t q, int32_t n_mats,
                         const pq_matrix_t* mats, double max_norm, double* sumsq_out, float* norm_out,
                         float* coef_out, void* workspace, int64_t workspace_bytes_, void* stream) {
    pq_status_t st = check_tensors(n, tensors, false);
    if (st == PQ_OK) st = check_mats(q, n_mats, mats);
    if (st != PQ_OK) return st;
    if (!max_norm_ok(max_norm) || (!sumsq_out && !norm_out && !coef_out)) return PQ_ERR_INVALID_ARG;
    if (!scalars_aligned(sumsq_out, norm_out, coef_out)) return PQ_ERR_MISALIGNED;
    Partials parts;
    st = take_workspace(workspace, workspace_bytes_, workspace_bytes(n, n_mats), parts);
    if (st != PQ_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = norm_tensors(n, tensors, parts, s);
    if (st != PQ_OK) return st;
    if (n_mats > 0) {
        static thread_local GradBatch<kMaxBatch> b;
        b.n_src = 0;
        b.grad_mult = 1.0f;
        for (int k = 0; k < kMaxSources; ++k) b.src[k] = nullptr;
        st = norm_matrices<false>(
            q, n_mats, b,
            [&](int32_t i) {
                GradDesc d = {};
                d.w = mats[i].w;
                d.alpha = mats[i].alpha;
                d.g = mats[i].g_bf16;
                d.dalpha = mats[i].dalpha_out;
                d.rows = mats[i].rows;
                d.cols = mats[i].cols;
                d.grad_scale = mats[i].grad_scale;
                return d;
            },
            [](const GradDesc& d) {
                return d.cols > 0 && d.cols % 8 == 0 && aligned(d.w, 32) && aligned(d.g, 16);
            },
            parts, s);
        if (st != PQ_OK) return st;
    }
    return cuda_status(launch_after(norm_end_kernel, 1,
                                    norm_end(parts, max_norm, sumsq_out, norm_out, coef_out), s));
}

pq_status_t pq_reduce_grad_norm(pq_quant_t q, int32_t n_src, const uint16_t* const* g_sources,
                                float grad_mult, int32_t n, const pq_shard_t* shards, double max_norm,
                                double* sumsq_out, float* norm_out, float* coef_out, void* workspace,
                                int64_t workspace_bytes_, void* stream) {
    if (code_bits_of(q) == 0 || n < 0 || (n > 0 && !shards)) return PQ_ERR_INVALID_ARG;
    if (n_src < 1 || n_src > kMaxSources || !g_sources) return PQ_ERR_INVALID_ARG;
    if (!max_norm_ok(max_norm) || (!sumsq_out && !norm_out && !coef_out)) return PQ_ERR_INVALID_ARG;
    if (!scalars_aligned(sumsq_out, norm_out, coef_out)) return PQ_ERR_MISALIGNED;
    static thread_local GradBatch<kMaxBatch> b;
    bool src_aligned = true;
    for (int k = 0; k < kMaxSources; ++k) {
        b.src[k] = k < n_src ? g_sources[k] : nullptr;
        if (k < n_src && !g_sources[k]) return PQ_ERR_INVALID_ARG;
        if (!aligned(b.src[k], 2)) return PQ_ERR_MISALIGNED;
        src_aligned = src_aligned && aligned(b.src[k], 16);
    }
    b.n_src = n_src;
    b.grad_mult = grad_mult;
    for (int32_t i = 0; i < n; ++i) {
        const pq_shard_t& m = shards[i];
        if (m.rows < 0 || m.cols < 0 || m.g_offset < 0) return PQ_ERR_INVALID_ARG;
        if (m.rows > 0 && m.cols > 0 && (!m.alpha || !m.w)) return PQ_ERR_INVALID_ARG;
        if (m.rows > 0 && (!aligned(m.w, 4) || !aligned(m.alpha, 4) || !aligned(m.dalpha_out, 4)))
            return PQ_ERR_MISALIGNED;
    }
    Partials parts;
    pq_status_t st = take_workspace(workspace, workspace_bytes_, workspace_bytes(0, n), parts);
    if (st != PQ_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = norm_matrices<true>(
        q, n, b,
        [&](int32_t i) {
            GradDesc d = {};
            d.w = shards[i].w;
            d.alpha = shards[i].alpha;
            d.dalpha = shards[i].dalpha_out;
            d.rows = shards[i].rows;
            d.cols = shards[i].cols;
            d.g_offset = shards[i].g_offset;
            d.grad_scale = shards[i].grad_scale;
            return d;
        },
        [&](const GradDesc& d) {
            return src_aligned && d.cols > 0 && d.cols % 8 == 0 && d.g_offset % 8 == 0 && aligned(d.w, 32);
        },
        parts, s);
    if (st != PQ_OK) return st;
    return cuda_status(launch_after(norm_end_kernel, 1,
                                    norm_end(parts, max_norm, sumsq_out, norm_out, coef_out), s));
}

pq_status_t pq_clip_coef(int32_t count, const double* sumsq, double max_norm, float* norm_out,
                         float* coef_out, void* stream) {
    if (count < 0 || (count > 0 && !sumsq) || !max_norm_ok(max_norm) || (!norm_out && !coef_out))
        return PQ_ERR_INVALID_ARG;
    if (!scalars_aligned(sumsq, norm_out, coef_out)) return PQ_ERR_MISALIGNED;
    Partials parts = {const_cast<double*>(sumsq), count, count};
    return cuda_status(launch_after(norm_end_kernel, 1, norm_end(parts, max_norm, nullptr, norm_out, coef_out),
                                    static_cast<cudaStream_t>(stream)));
}

pq_status_t pq_grad_scale(int32_t n, const pq_tensor_t* tensors, const float* coef, void* stream) {
    const pq_status_t st = check_tensors(n, tensors, true);
    if (st != PQ_OK) return st;
    if (!coef) return PQ_ERR_INVALID_ARG;
    if (!aligned(coef, 4)) return PQ_ERR_MISALIGNED;
    bool scaled = false;
    return scale_tensors(n, tensors, coef, NormEnd{}, scaled, static_cast<cudaStream_t>(stream));
}

pq_status_t pq_grad_clip(int32_t n, const pq_tensor_t* tensors, double max_norm, float* norm_out,
                         float* coef_out, void* workspace, int64_t workspace_bytes_, void* stream) {
    pq_status_t st = check_tensors(n, tensors, true);
    if (st != PQ_OK) return st;
    if (!max_norm_ok(max_norm) || !norm_out) return PQ_ERR_INVALID_ARG;
    if (!scalars_aligned(nullptr, norm_out, coef_out)) return PQ_ERR_MISALIGNED;
    Partials parts;
    st = take_workspace(workspace, workspace_bytes_, workspace_bytes(n, 0), parts);
    if (st != PQ_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = norm_tensors(n, tensors, parts, s);
    if (st != PQ_OK) return st;
    const NormEnd end = norm_end(parts, max_norm, nullptr, norm_out, coef_out);
    bool scaled = false;
    st = scale_tensors(n, tensors, nullptr, end, scaled, s);
    if (st != PQ_OK || scaled) return st;
    return cuda_status(launch_after(norm_end_kernel, 1, end, s));
}

}  // extern "C"
