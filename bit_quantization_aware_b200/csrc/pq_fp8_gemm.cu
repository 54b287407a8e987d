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
// A CTA has 128 rows of A (TMEM lanes, one promote thread each) by some rows
// of B (TMEM columns). With a row on a thread, the A scale is one register,
// and a tile scale of B another: one multiply-add an element. Row scales of B
// are per column and come through shared memory.
//
// Large products: two CTAs (a pair) form 256 x 256 with cta_group::2, each
// with half of B's rows in its shared memory. The columns' two halves have an
// issuer and four promote warps each and two TMEM buffers each, so one half's
// sums leave TMEM while the other's MMAs run: a K block passes issuer, tensor
// cores, promote warps and back in about twice the tensor cores' time, which
// two buffers of half the width cover and two of the whole width did not.
//
// Few tiles (short m and n) leave most SMs idle, so a tile's K blocks are
// split over a cluster of SPLIT CTAs, which exchange their sums through
// distributed shared memory and add them in rank order: no workspace, no
// atomics, the same bits every time.
//
// Roles: warp 0 TMA producer, warps 1 and 3 MMA issuers (3 in pairs), warp 2
// TMEM owner and loader of B's row scales, warps 4.. promote. Waits are
// bounded as in pq_gemm.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <stdint.h>

#include <atomic>

#include "pq.h"
#include "pq_launches.cuh"
#include "pq_tc.cuh"
#include "pq_units.cuh"

namespace pq8 {

using namespace pqg;

constexpr int kBlock = 128;      // K of a scale block, and of one stage
constexpr int kRows = 128;       // A rows of a CTA: TMEM lanes
constexpr int kMaxStages = 16;
constexpr int kScaleSlots = 8;   // K blocks whose B row scales are in shared memory or on their way
constexpr int kSmemSm = 228 * 1024, kSmemCta = 1024;  // of an SM; reserved for each CTA

struct Params {
    CUtensorMap ta, tb;  // codes [m][k] in boxes of 128 B x a_bytes / 128 rows, [n][k] of 128 B x B rows
    CUtensorMap ty;      // y in boxes of 128 B x 32 rows (tma_out)
    const float* sa;     // [kb][m]
    const float* sb;     // [n / 128][kb] (tile) or [kb][n] (row)
    void* y;
    int64_t m, n, ldy;
    int32_t kb;          // K blocks
    int32_t tiles_m, tiles_n;
    int32_t a_bytes;     // of one A box
    int32_t stages;
    int32_t dtype;       // of y
    int32_t quad;        // four elements at a multiple of four columns are aligned
    int32_t tma_out;     // y suits TMA stores
};

// PAIR: two CTAs of a cluster work on one tile of 256 x NT, each with 128
// rows of A and, of each half of the columns, half of B's rows.
template <int NT, bool BROW, int SPLIT, bool PAIR>
struct Layout {
    static constexpr int kCluster = PAIR ? 2 : SPLIT;
    static constexpr int kParts = PAIR ? 2 : 1;           // of the columns, each with its own issuer
    static constexpr int kCols = NT / kParts;             // columns of an MMA, and of a promote thread
    static constexpr int kBufs = PAIR ? 2 : 4;            // TMEM buffers of each part
    static constexpr int kPromoteWarps = 4 * kParts;
    static constexpr int kThreads = 128 + 32 * kPromoteWarps;
    static constexpr int kBRows = kCols / (PAIR ? 2 : 1);  // B rows of a part in a CTA
    static constexpr int kBBytes = kParts * kBRows * kBlock;
    static constexpr uint32_t kTmemCols = kBufs * NT;
    static constexpr int kCtas = NT == 64 ? 2 : 1;        // resident on an SM
    // full, empty [stages]; dfull, dempty [halves x buffers]; sfull, sempty
    // [scale slots]; drain [halves]; TMEM base, abort, and a pair's words: the
    // K blocks that this CTA loaded, its place in the ring of stages (slot and
    // phase), the other CTA's K blocks and abort
    static constexpr int kNumBars = 2 * kMaxStages + 2 * kParts * kBufs + 2 * kScaleSlots + 2;
    static constexpr int kMiscOff = 8 * kNumBars, kPairOff = kMiscOff + 8;
    static constexpr int kScaleOff = 1024;
    static constexpr int kOutOff = kScaleOff + (BROW ? kScaleSlots * NT * 4 : 0);  // 4 KB a promote warp
    static constexpr int kRingOff = kOutOff + (SPLIT == 1 ? kPromoteWarps * 4096 : 0);
    static_assert(kPairOff + 20 <= kScaleOff && kOutOff % 1024 == 0, "shared memory layout");
    // exchange of a split tile: [from rank][row][column of the slice, padded]
    static constexpr int kSlice = NT / SPLIT, kPitch = kSlice + 4;
    static_assert(SPLIT == 1 || (!PAIR && kSlice % 8 == 0), "slices of whole vectors");

    static constexpr int kSmem = kSmemSm / kCtas - kSmemCta - 1024;  // of a CTA, less the alignment slack
    // As many stages as fit. The MMA reads 128 rows of A whatever its box
    // brought (the rows beyond are other stages' bytes, and lanes that are
    // not read), so the B ring behind the A ring covers a short last box.
    static int stages(int a_bytes) {
        const int n = (kSmem - kRingOff) / (a_bytes + kBBytes);
        return n < kMaxStages ? n : kMaxStages;
    }
    static int bytes(int a_bytes, int stages) {
        const int ring = stages * (a_bytes + kBBytes), exchange = SPLIT > 1 ? SPLIT * kRows * kPitch * 4 : 0;
        return kRingOff + (ring > exchange ? ring : exchange) + 1024;
    }
};

// Position in the ring of stages (see Ring; the number of stages depends on
// how many rows A has).
struct StageRing {
    uint32_t n, idx = 0, phase = 0;
    __device__ __forceinline__ explicit StageRing(uint32_t n_) : n(n_) {}
    __device__ __forceinline__ void next() {
        if (++idx == n) {
            idx = 0;
            phase ^= 1u;
        }
    }
    __device__ __forceinline__ void prev() {
        if (idx == 0) {
            idx = n;
            phase ^= 1u;
        }
        --idx;
    }
};

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, e4m3 A and B, both
// K-major, M = m, N = nt.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int nt) {
    return (1u << 4) | (static_cast<uint32_t>(nt >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <bool PAIR>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(a), "l"(b),
            "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(a), "l"(b),
            "r"(idesc), "r"(acc)
            : "memory");
}

// Arrival on a barrier (PAIR: on both CTAs' barriers) when the MMAs issued so
// far are done.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t mbar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                mbar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        mma_commit(mbar);
}

// Arrival where `yes`, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint32_t mbar, bool yes) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}\n" ::"r"(mbar),
        "r"(static_cast<uint32_t>(yes))
        : "memory");
}

// Arrival on a barrier of the cluster, without release (with one, the pairs
// took twice their time): the threads that arrive so have written no memory.
// They have read tensor memory: tcgen05.wait::ld and the fence before the
// arrival, and the fence behind the wait, order those reads before the MMAs
// that follow, as PTX has it for a relaxed barrier between them.
__device__ __forceinline__ void mbar_arrive_cluster_if(uint32_t addr, bool yes) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}\n" ::"r"(addr),
        "r"(static_cast<uint32_t>(yes))
        : "memory");
}

// A pair's loads: each CTA brings its operands into its own shared memory and
// both arrive, and count their bytes, on the issuing CTA's barrier (an address
// of the cluster's shared memory), so the wait of the thread that issues the
// MMAs covers both CTAs' copies. Copies may land before the arrival that
// announces their bytes: the phase lasts until both CTAs have arrived.
__device__ __forceinline__ void mbar_expect_tx_cluster(uint32_t mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(mbar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t mbar, int32_t x,
                                                 int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(x), "r"(y)
        : "memory");
}

// Whom a wait hears from: this CTA; both CTAs' copies (a pair's operands); the
// other CTA's arrivals, which publish no memory (see mbar_arrive_cluster_if).
enum Heard { kCta, kCopies, kRemote };

// Whether the phase is over, for the whole warp alike: once every lane has
// seen it, since a vote orders no memory and each lane acquires for itself.
template <int HEARD>
__device__ __forceinline__ bool mbar_try_warp(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    if constexpr (HEARD == kRemote)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(mbar), "r"(parity)
            : "memory");
    else if constexpr (HEARD == kCopies)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(mbar), "r"(parity)
            : "memory");
    else
        done = mbar_try(mbar, parity);
    return __all_sync(0xFFFFFFFFu, done);
}

// The same asked ahead: the warp does other work while the answer is on its way.
__device__ __forceinline__ uint32_t mbar_test(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity)
        : "memory");
    return done;
}

// Bounded wait of a whole warp, which stays converged and uniform: a round trip
// between two warps was shorter so than with one lane's wait and a shuffle of
// its result.
template <int HEARD = kCta>
__device__ __forceinline__ bool uniform_wait(uint32_t mbar, uint32_t parity, volatile int* abort) {
    for (uint32_t i = 0; i < kMaxSpins; ++i) {
        if (mbar_try_warp<HEARD>(mbar, parity)) return true;
        if ((i & 63u) == 63u && __any_sync(0xFFFFFFFFu, *abort)) return false;
    }
    *abort = 1;
    atomicExch(&g_status, 1);
    return false;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
    return e != 0;
}

// W columns of this warp's 32 TMEM lanes, a lane a thread; the values are
// there after tmem_wait.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15])
                 : "r"(taddr));
}
// 32 columns of 16 TMEM lanes: thread t has lanes t / 4 (registers 4 j and
// 4 j + 1) and t / 4 + 8 (4 j + 2 and 4 j + 3) of columns 8 j + 2 (t % 4) and
// the one beside it.
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15])
                 : "r"(taddr));
}
// Ends this thread's reads of tensor memory; r, one of their targets, may be
// used behind it and not before.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}

// acc += s * (v * b) on pairs of neighbours, b left out where it is 1. Two
// values an instruction: the promote warps' arithmetic fills the issue slots
// that the issuers' instructions wait for (8192 x 14336 x 4096, cold, when this
// came: 476 us with one value an instruction, 446 with two; row scales,
// 4096 x 4096 x 8190: 330 and 255).
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    return pair(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void fma2(float& x, float& y, uint64_t v, uint64_t s) {
    uint64_t a = pair(x, y);
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(v), "l"(s));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t a, float x, float y, float z, float w) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w)
                 : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t a, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.b32 [%0], %1;\n\tst.shared::cluster.b32 [%0 + 4], %2;" ::"r"(a), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}

// Asynchronous copy of src[i] to shared memory, 0 where i >= n.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, int64_t i, int64_t n) {
    const bool in = i < n;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src + (in ? i : 0)),
                 "r"(in ? 4u : 0u)
                 : "memory");
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

// Where a promote thread's C sums are. ROWS false: row `lane` of its warp's
// 32, columns 0..C-1. ROWS true: rows lane / 4 + 8 i for i < 4, columns
// 8 j + 2 (lane % 4) + e for e < 2, at acc[8 j + 2 i + e] (tmem_ld_rows).

// A warp's 32 rows x C columns to y by way of its 4 KB of shared memory, 128
// bytes of each row at a time (the 128B swizzle: 16-byte chunk c of row r at
// chunk c ^ (r % 8), so the writes are free of bank conflicts), and from there
// by the TMA engine, which clips what lies beyond y, or, where y does not suit
// it, row by row. No K block leaves TMEM during the stores, and direct ones of
// each thread's row, whole sectors or (an odd pitch) elements, took longer.
template <typename T, int C, bool ROWS>
__device__ __forceinline__ void store_typed(const Params& p, uint32_t buf, int lane, int64_t row0, int64_t col,
                                            const float (&acc)[C]) {
    constexpr int W = 128 / sizeof(T);  // columns of a round
    constexpr int B = sizeof(T);
#pragma unroll
    for (int c = 0; c < C; c += W) {
        if (p.tma_out && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        union {
            T e[16 / B];
            uint32_t w[4];
        } o;
        if constexpr (ROWS) {
#pragma unroll
            for (int j = 0; j < W / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = lane / 4 + 8 * i, at = (8 * j + 2 * (lane % 4)) * B;
                    const uint32_t dst = buf + row * 128 + (((at >> 4) ^ (row & 7)) << 4) + (at & 15);
                    o.e[0] = static_cast<T>(acc[c + 8 * j + 2 * i]);
                    o.e[1] = static_cast<T>(acc[c + 8 * j + 2 * i + 1]);
                    if constexpr (B == 4)
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(o.w[0]), "r"(o.w[1]) : "memory");
                    else
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(o.w[0]) : "memory");
                }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
#pragma unroll
                for (int i = 0; i < 16 / B; ++i) o.e[i] = static_cast<T>(acc[c + q * (16 / B) + i]);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 buf + lane * 128 + ((q ^ (lane & 7)) << 4)),
                             "r"(o.w[0]), "r"(o.w[1]), "r"(o.w[2]), "r"(o.w[3])
                             : "memory");
            }
        }
        if (p.tma_out) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && row0 < p.m && col + c < p.n) {
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                                 reinterpret_cast<uint64_t>(&p.ty)),
                             "r"(buf), "r"(static_cast<int32_t>(col + c)), "r"(static_cast<int32_t>(row0))
                             : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            continue;
        }
        __syncwarp();
        const int rows = p.m - row0 < 32 ? static_cast<int>(p.m - row0) : 32;  // <= 0: none
        const int at = c + lane * (4 / B);  // this lane's column: 4 bytes of each row
        const int left = p.n - col - at < 2 ? static_cast<int>(p.n - col - at) : 2;
        T* y = static_cast<T*>(p.y) + row0 * p.ldy + col + at;
        for (int r = 0; r < rows; ++r, y += p.ldy) {
            asm volatile("ld.shared.b32 %0, [%1];"
                         : "=r"(o.w[0])
                         : "r"(buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + ((lane & 3) << 2)));
            if constexpr (B == 4) {
                if (left > 0) *y = o.e[0];
            } else if (left == 2 && (reinterpret_cast<uintptr_t>(y) & 3) == 0) {
                *reinterpret_cast<uint32_t*>(y) = o.w[0];
            } else {
                if (left > 0) y[0] = o.e[0];
                if (left > 1) y[1] = o.e[1];
            }
        }
    }
}

template <int C, bool ROWS>
__device__ __forceinline__ void store(const Params& p, uint32_t buf, int lane, int64_t row0, int64_t col,
                                      const float (&acc)[C]) {
    if (p.dtype == PQ_BF16) store_typed<__nv_bfloat16, C, ROWS>(p, buf, lane, row0, col, acc);
    else if (p.dtype == PQ_FP16) store_typed<__half, C, ROWS>(p, buf, lane, row0, col, acc);
    else store_typed<float, C, ROWS>(p, buf, lane, row0, col, acc);
}

// Four consecutive elements of a row of which `left` exist.
template <typename T>
__device__ __forceinline__ void store4(T* y, int64_t left, bool whole, const float4& v) {
    union {
        T e[4];
        uint32_t w[sizeof(T)];
    } o;
    o.e[0] = static_cast<T>(v.x);
    o.e[1] = static_cast<T>(v.y);
    o.e[2] = static_cast<T>(v.z);
    o.e[3] = static_cast<T>(v.w);
    if (whole && left >= 4) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(y) = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
        else *reinterpret_cast<uint2*>(y) = make_uint2(o.w[0], o.w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) y[i] = o.e[i];
    }
}

template <int NT, bool BROW, int SPLIT, bool PAIR>
__global__ void __cluster_dims__(Layout<NT, BROW, SPLIT, PAIR>::kCluster, 1, 1)
    __launch_bounds__(Layout<NT, BROW, SPLIT, PAIR>::kThreads, Layout<NT, BROW, SPLIT, PAIR>::kCtas)
        fp8_gemm_kernel(const __grid_constant__ Params p) {
    using L = Layout<NT, BROW, SPLIT, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t{1023});
    const uint32_t sbase = smem_u32(smem);
    const uint32_t b_full = sbase, b_empty = b_full + 8u * kMaxStages;
    constexpr uint32_t kD = 8u * L::kParts * L::kBufs;
    const uint32_t b_dfull = b_empty + 8u * kMaxStages, b_dempty = b_dfull + kD;
    const uint32_t b_sfull = b_dempty + kD, b_sempty = b_sfull + 8u * kScaleSlots;
    const uint32_t b_drain = b_sempty + 8u * kScaleSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    volatile uint32_t* pair_words = reinterpret_cast<volatile uint32_t*>(smem + L::kPairOff);
    const float* scales = reinterpret_cast<const float*>(smem + L::kScaleOff);
    const uint32_t a_ring = sbase + L::kRingOff, b_ring = a_ring + p.stages * p.a_bytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(b_full + 8u * s, L::kParts);  // PAIR: both CTAs' producers
            mbar_init(b_empty + 8u * s, L::kParts);
        }
        for (int b = 0; b < L::kParts * L::kBufs; ++b) {
            mbar_init(b_dfull + 8u * b, 1);
            mbar_init(b_dempty + 8u * b, PAIR ? 8 : 4);  // the part's promote warps, of both CTAs
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(b_sfull + 8u * s, 32);
            mbar_init(b_sempty + 8u * s, L::kPromoteWarps);
        }
        for (int h = 0; h < L::kParts; ++h) mbar_init(b_drain + 8u * h, 1);
        const int forced = *static_cast<volatile int*>(&g_force_abort);
        *abort = forced;
        if (forced) atomicExch(&g_status, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_slot)),
                         "r"(L::kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_slot)),
                         "r"(L::kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // the other CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // the launch before this one in the stream may still run (its results are
    // read from here on), and the next one may begin its own set-up
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();

    // this CTA's tiles, its K blocks of each, its rows within a tile
    const int tiles = p.tiles_m * p.tiles_n;
    const int rank = L::kCluster == 1 ? 0 : static_cast<int>(blockIdx.x % L::kCluster);
    const int first = blockIdx.x / L::kCluster;
    const int step = gridDim.x / L::kCluster;
    const int k0 = SPLIT == 1 ? 0 : static_cast<int>(static_cast<int64_t>(p.kb) * rank / SPLIT);
    const int k1 = SPLIT == 1 ? p.kb : static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / SPLIT);
    constexpr int kTileRows = PAIR ? 2 * kRows : kRows;
    const int row_off = PAIR ? rank * kRows : 0;

    // A pair's CTA launches with 168 registers a thread (64,512 in all); the
    // promote warps' 128 sums need more: 8 x 32 x 224 + 4 x 32 x 56 = 64,512
    constexpr bool kSplitRegs = PAIR;
    if (warp < 4) {
        if constexpr (kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            // ------------------------------------------------------ producer
            if (lane == 0) {
                StageRing r(p.stages);
                uint32_t loaded = 0;  // K blocks
                const uint32_t full = PAIR ? map_to_rank(b_full, 0) : b_full;  // the issuer's
                bool ok = true;
                for (int t = first; ok && t < tiles; t += step) {
                    int tm, tn;
                    tile_of(p, t, tm, tn);
                    const int ra = tm * kTileRows + row_off, rb = tn * NT + (PAIR ? rank * L::kBRows : 0);
                    static_assert(L::kBBytes % 1024 == 0, "swizzle atoms");
                    for (int kb = k0; kb < k1; ++kb) {
                        if (!mbar_wait(b_empty + 8u * r.idx, r.phase ^ 1u, abort)) {
                            ok = false;
                            break;
                        }
                        const uint32_t bar = full + 8u * r.idx, bytes = static_cast<uint32_t>(p.a_bytes) + L::kBBytes;
                        const uint32_t a = a_ring + r.idx * p.a_bytes, b = b_ring + r.idx * L::kBBytes;
                        if constexpr (PAIR) {
                            mbar_expect_tx_cluster(bar, bytes);
                            tma_load_2d_pair(a, &p.ta, bar, kb * kBlock, ra);
#pragma unroll
                            for (int h = 0; h < L::kParts; ++h)
                                tma_load_2d_pair(b + h * L::kBRows * kBlock, &p.tb, bar, kb * kBlock, rb + h * L::kCols);
                        } else {
                            mbar_expect_tx(bar, bytes);
                            tma_load_2d(a, &p.ta, bar, kb * kBlock, ra);
                            tma_load_2d(b, &p.tb, bar, kb * kBlock, rb);
                        }
                        r.next();
                        ++loaded;
                    }
                }
                // loads in flight land before the CTA may exit (a pair's: see
                // the end of the kernel)
                if constexpr (PAIR) {
                    pair_words[0] = loaded;
                    pair_words[1] = r.idx;
                    pair_words[2] = r.phase;
                } else {
                    for (uint32_t i = min(loaded, r.n); i > 0; --i) {
                        r.prev();
                        mbar_drain(b_full + 8u * r.idx, r.phase);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1 || (L::kParts == 2 && warp == 3 && rank == 0)) {
            if (!PAIR || rank == 0) {
                // ------------------------------------------------ MMA issuer
                // The whole warp walks the loop and one lane issues, which
                // was faster than a branch of one lane around the loop.
                constexpr uint32_t idesc = idesc_e4m3(kTileRows, L::kCols);
                const int h = warp == 3;
                const uint32_t dfull = b_dfull + 8u * L::kBufs * h, dempty = b_dempty + 8u * L::kBufs * h;
                const bool one = elect_one();
                StageRing r(p.stages);
                Ring<L::kBufs> d;
                bool ok = true;
                // The next block's waits are asked for before this one's
                // MMAs (512 x 4096 x 4096, when this came: 15.9 -> 15.2 us). A
                // pair's two issuers have the time: asking ahead cost them 2%.
                constexpr bool kAhead = L::kParts == 1;
                uint32_t ready = 0;
                for (int t = first; ok && t < tiles; t += step) {
                    for (int kb = k0; kb < k1; ++kb) {
                        const uint64_t a = sw128_desc(a_ring + r.idx * p.a_bytes);
                        const uint64_t b = sw128_desc(b_ring + r.idx * L::kBBytes + h * L::kBRows * kBlock);
                        const uint32_t acc = tmem + (d.idx * L::kParts + h) * L::kCols;
                        const uint32_t free_bar = b_empty + 8u * r.idx, full_bar = dfull + 8u * d.idx;
                        if (!(kAhead && __all_sync(0xFFFFFFFFu, ready)) &&
                            (!uniform_wait<PAIR ? kCopies : kCta>(b_full + 8u * r.idx, r.phase, abort) ||
                             !uniform_wait<PAIR ? kRemote : kCta>(dempty + 8u * d.idx, d.phase ^ 1u, abort))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        r.next();
                        d.next();
                        if constexpr (kAhead)
                            ready = mbar_test(b_full + 8u * r.idx, r.phase) &
                                    mbar_test(dempty + 8u * d.idx, d.phase ^ 1u);
                        if (one) {
#pragma unroll
                            for (int k = 0; k < kBlock / 32; ++k)
                                mma_ss<PAIR>(acc, a + 2u * k, b + 2u * k, idesc, k > 0);
                            commit<PAIR>(full_bar);
                            commit<PAIR>(free_bar);
                        }
                        __syncwarp();
                    }
                }
                // every MMA completes before TMEM is freed
                if (one) {
                    commit<PAIR>(b_drain + 8u * h);
                    mbar_drain(b_drain + 8u * h, 0);
                }
            } else {
                // ------- the pair's other CTA: the issuers' last arrivals here
                if (elect_one())
                    for (int h = 0; h < L::kParts; ++h) mbar_drain(b_drain + 8u * h, 0);
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
                        const uint32_t slot = sbase + L::kScaleOff + r.idx * (NT * 4);
                        const int64_t col = static_cast<int64_t>(tn) * NT + lane;
#pragma unroll
                        for (int i = 0; i < NT / 32; ++i)
                            copy4(slot + 4 * (32 * i + lane), p.sb + kb * p.n, col + 32 * i, p.n);
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(b_sfull + 8u * r.idx)
                                     : "memory");
                        r.next();
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
        }
        if constexpr (SPLIT > 1) {  // the promote warps' two barriers
            cluster_sync();
            cluster_sync();
        }
    } else {
        if constexpr (kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ------------------------------------------------------- promote
        const int quarter = warp & 3, part = (warp - 4) >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        constexpr int C = L::kCols;
        const uint32_t dfull = b_dfull + 8u * L::kBufs * part;
        const uint32_t dempty0 = b_dempty + 8u * L::kBufs * part;
        const uint32_t dempty = PAIR ? map_to_rank(dempty0, 0) : dempty0;  // the issuer's
        const uint32_t out_buf = sbase + L::kOutOff + (warp - 4) * 4096;
        Ring<L::kBufs> d;
        Ring<kScaleSlots> sr;
        bool ok = true;
        const bool one = lane == 0;
        auto free_buffer = [&](uint32_t bar) {
            tc_fence_before();
            __syncwarp();
            if constexpr (PAIR) mbar_arrive_cluster_if(bar, one);
            else mbar_arrive_if(bar, one);
        };
        auto buffer = [&]() { return tmem + lane_addr + d.idx * NT + part * C; };
        // The tile's K blocks into acc, tile scales: an element is one
        // multiply-add behind a TMEM read. The reads run one chunk ahead of
        // the arithmetic, across K blocks too; whether the next block is
        // there is asked two chunks before.
        auto sum_blocks_tile = [&](float(&acc)[C], int64_t row, int64_t col) -> bool {
            constexpr int W = NT == 64 ? 16 : 32;  // columns of a read (registers)
            // rows, columns and K blocks beyond the last take the last one's
            // scale: no branch around the loads
            const float* sa = p.sa + (row < p.m ? row : p.m - 1);
            const float* sb = p.sb + (col < p.n ? col / kBlock : (p.n - 1) / kBlock) * p.kb;
            // scales four K blocks at a time, the next four on their way; an
            // operation on a load, a move included, waits for it
            float na[4], nb[4], cur[4];
            auto fetch = [&](int g) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int b = min(g + j, k1 - 1);
                    na[j] = __ldg(sa + b * p.m);
                    nb[j] = __ldg(sb + b);
                }
            };
            if (k0 >= k1) return true;
            fetch(k0);
            uint32_t v[2][W];
            if (!uniform_wait(dfull + 8u * d.idx, d.phase, abort)) return false;
            tc_fence_after();
            tmem_ld(buffer(), v[0]);
            for (int kb = k0; kb < k1; ++kb) {
                const int j = (kb - k0) & 3;
                if (j == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) cur[i] = __fmul_rn(na[i], nb[i]);
                    fetch(kb + 4);
                }
                const float s = j & 2 ? (j & 1 ? cur[3] : cur[2]) : (j & 1 ? cur[1] : cur[0]);
                const uint32_t src = buffer(), free_bar = dempty + 8u * d.idx;
                d.next();
                uint32_t ready = 0;
                auto add = [&](int c) {
#pragma unroll
                    for (int i = 0; i < W; i += 2)
                        fma2(acc[c + i], acc[c + i + 1], pair(v[c / W % 2][i], v[c / W % 2][i + 1]), pair(s, s));
                };
#pragma unroll
                for (int c = 0; c + W < C; c += W) {
                    tmem_wait(v[c / W % 2]);
                    tmem_ld(src + c + W, v[(c / W + 1) % 2]);
                    if (c == (C > 3 * W ? C - 3 * W : 0)) ready = mbar_test(dfull + 8u * d.idx, d.phase);
                    add(c);
                }
                tmem_wait(v[(C / W - 1) % 2]);
                free_buffer(free_bar);  // all read: the issuer may write the buffer again
                if (kb + 1 < k1) {
                    if (__all_sync(0xFFFFFFFFu, ready)) {
                        tc_fence_after();
                        tmem_ld(buffer(), v[0]);
                        add(C - W);
                        continue;
                    }
                    add(C - W);
                    if (!uniform_wait(dfull + 8u * d.idx, d.phase, abort)) return false;
                    tc_fence_after();
                    tmem_ld(buffer(), v[0]);
                } else {
                    add(C - W);
                }
            }
            return true;
        };
        // The same with row scales of B, in shared memory: an element is a
        // multiplication and a multiply-add. With a whole row on a thread,
        // every scale of the K block would pass through every thread (1024
        // cycles of shared memory a block); read 16 lanes x 8 columns at a
        // time, a thread has a quarter of the columns and four rows.
        auto sum_blocks_row = [&](float(&acc)[C], int64_t row0, int64_t) -> bool {
            const float* sa[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = row0 + lane / 4 + 8 * i;
                sa[i] = p.sa + (row < p.m ? row : p.m - 1);
            }
            float a0[4], a1[4], a[4];  // A's scales of the next two K blocks, and of this one
            auto fetch = [&](int kb, float(&to)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) to[i] = __ldg(sa[i] + min(kb, k1 - 1) * p.m);
            };
            if (k0 >= k1) return true;
            fetch(k0, a0);
            fetch(k0 + 1, a1);
            uint32_t ready = 0;
            auto block = [&](int kb, float(&next)[4]) -> bool {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = next[i];
                fetch(kb + 2, next);
                if (!__all_sync(0xFFFFFFFFu, ready) &&
                    (!uniform_wait(b_sfull + 8u * sr.idx, sr.phase, abort) ||
                     !uniform_wait(dfull + 8u * d.idx, d.phase, abort)))
                    return false;
                tc_fence_after();
                const float* bs = scales + sr.idx * NT + part * C + 2 * (lane % 4);
                const uint32_t src = buffer();
                const uint32_t free_bar = dempty + 8u * d.idx, free_scales = b_sempty + 8u * sr.idx;
                d.next();
                sr.next();
                uint32_t v[2][16];  // 32 columns of 16 rows: reads run one ahead
                tmem_ld_rows(src, v[0]);
#pragma unroll
                for (int c = 0; c < C; c += 32) {
                    float2 b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float2*>(bs + c + 8 * j);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        tmem_wait(v[g]);
                        if (g == 0) tmem_ld_rows(src + c + (16u << 16), v[1]);
                        else if (c + 32 < C) tmem_ld_rows(src + c + 32, v[0]);
                        else free_buffer(free_bar);
                        if (g == 1 && c + 64 == C)
                            ready = mbar_test(b_sfull + 8u * sr.idx, sr.phase) &
                                    mbar_test(dfull + 8u * d.idx, d.phase);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int o = c + 8 * j + 2 * (2 * g + h);
                                fma2(acc[o], acc[o + 1],
                                     mul2(pair(v[g][4 * j + 2 * h], v[g][4 * j + 2 * h + 1]), pair(b[j].x, b[j].y)),
                                     pair(a[2 * g + h], a[2 * g + h]));
                            }
                    }
                }
                __syncwarp();
                mbar_arrive_if(free_scales, one);
                return true;
            };
            for (int kb = k0; kb < k1; kb += 2) {
                if (!block(kb, a0)) return false;
                if (kb + 1 < k1 && !block(kb + 1, a1)) return false;
            }
            return true;
        };
        auto sum_blocks = [&](float(&acc)[C], int64_t row, int64_t col) -> bool {
            if constexpr (BROW) return sum_blocks_row(acc, row, col);
            else return sum_blocks_tile(acc, row + lane, col);
        };
        for (int t = first; ok && t < tiles; t += step) {
            int tm, tn;
            tile_of(p, t, tm, tn);
            const int64_t row0 = static_cast<int64_t>(tm) * kTileRows + row_off + quarter * 32;  // the warp's
            const int64_t col = static_cast<int64_t>(tn) * NT + part * C;
            float acc[C];
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = 0.0f;
            ok = sum_blocks(acc, row0, col);
            if constexpr (SPLIT > 1) {
                constexpr int kPart = kRows * L::kPitch * 4;  // bytes of a rank's sums of a slice
                cluster_sync();  // every CTA's stages are free; rank j adds columns j * kSlice..
#pragma unroll
                for (int j = 0; j < SPLIT; ++j) {
                    const uint32_t dst = map_to_rank(a_ring, j) + rank * kPart;
                    if constexpr (BROW) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = lane / 4 + 8 * i;
                            if (row0 + row < p.m)
#pragma unroll
                                for (int c = 0; c < L::kSlice; c += 8)
                                    st_cluster(dst + ((quarter * 32 + row) * L::kPitch + c + 2 * (lane % 4)) * 4,
                                               acc[j * L::kSlice + c + 2 * i], acc[j * L::kSlice + c + 2 * i + 1]);
                        }
                    } else if (row0 + lane < p.m) {
#pragma unroll
                        for (int c = 0; c < L::kSlice; c += 4)
                            st_cluster(dst + ((quarter * 32 + lane) * L::kPitch + c) * 4, acc[j * L::kSlice + c],
                                       acc[j * L::kSlice + c + 1], acc[j * L::kSlice + c + 2],
                                       acc[j * L::kSlice + c + 3]);
                    }
                }
                cluster_sync();
                // four columns a thread, neighbours along the row
                constexpr int kQuads = L::kSlice / 4;
                const int64_t tile_row = static_cast<int64_t>(tm) * kRows;
                const int rows = p.m - tile_row < kRows ? static_cast<int>(p.m - tile_row) : kRows;
                for (int i = tid - 128; ok && i < rows * kQuads; i += 32 * L::kPromoteWarps) {
                    const int row = i / kQuads, c = i % kQuads * 4;
                    const uint8_t* part = smem + L::kRingOff + (row * L::kPitch + c) * 4;
                    float4 sum = *reinterpret_cast<const float4*>(part);
#pragma unroll
                    for (int r = 1; r < SPLIT; ++r) {
                        const float4 q = *reinterpret_cast<const float4*>(part + r * kPart);
                        sum.x = __fadd_rn(sum.x, q.x);
                        sum.y = __fadd_rn(sum.y, q.y);
                        sum.z = __fadd_rn(sum.z, q.z);
                        sum.w = __fadd_rn(sum.w, q.w);
                    }
                    const int64_t cc = col + rank * L::kSlice + c, at = (tile_row + row) * p.ldy + cc;
                    if (p.dtype == PQ_BF16) store4(static_cast<__nv_bfloat16*>(p.y) + at, p.n - cc, p.quad, sum);
                    else if (p.dtype == PQ_FP16) store4(static_cast<__half*>(p.y) + at, p.n - cc, p.quad, sum);
                    else store4(static_cast<float*>(p.y) + at, p.n - cc, p.quad, sum);
                }
                break;  // a cluster has one tile
            } else {
                if (!ok) break;
                store<C, BROW>(p, out_buf, lane, row0, col, acc);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    tc_fence_before();
    __syncthreads();
    // PAIR: neither CTA frees its memory while the other's MMAs, commits and
    // arrivals reach it, or its own loads are in flight. Where no wait gave up,
    // the issuers have waited for every load of both.
    if constexpr (PAIR) {
        if (tid == 0) st_cluster(map_to_rank(sbase + L::kPairOff + 12, rank ^ 1), pair_words[0], *abort);
        cluster_sync();
        if (*abort || pair_words[4]) {
            if (rank == 0 && tid == 0) {
                // One producer may have loaded up to the ring's length of K
                // blocks more than the other: the missing arrivals come from
                // here, and every load has landed when the phases are over.
                StageRing r(p.stages);
                r.idx = pair_words[1];
                r.phase = pair_words[2];
                const uint32_t n0 = pair_words[0], n1 = pair_words[3];
                for (uint32_t i = n0; i < n1; ++i, r.next()) mbar_arrive(b_full + 8u * r.idx);
                StageRing q = r;
                for (uint32_t i = n1; i < n0; ++i) {
                    q.prev();
                    mbar_arrive(b_full + 8u * q.idx);
                }
                for (uint32_t i = min(max(n0, n1), r.n); i > 0; --i) {
                    r.prev();
                    mbar_drain(b_full + 8u * r.idx, r.phase);
                }
            }
            cluster_sync();
        }
    }
    if (warp == 2) {
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmemCols)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmemCols)
                         : "memory");
    }
}

// k == 0: an empty sum
template <typename T>
__global__ void __launch_bounds__(256) zero_kernel(T* y, int64_t m, int64_t n, int64_t ldy) {
    for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < m * n; i += gridDim.x * int64_t{256})
        y[i / n * ldy + i % n] = static_cast<T>(0.0f);
}

// --------------------------------------------------------------- host side
static bool encode(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, CUtensorMapDataType type, int bytes,
                   const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / bytes), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t es[2] = {1, 1};
    return enc(map, type, 2, const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int bytes_of(int dtype) { return dtype == PQ_FP32 ? 4 : 2; }

// Clusters of a split kernel that the GPU holds at a time (a cluster lives in
// one GPC, so 8 CTAs of a whole SM each fit fewer times than SMs / 8).
template <int NT, int SPLIT>
static int64_t clusters_resident() {
    using L = Layout<NT, false, SPLIT, false>;
    static int cached[64] = {0};
    const int dev = pq::current_device();
    if (cached[dev] == 0) {
        auto kernel = fp8_gemm_kernel<NT, false, SPLIT, false>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(SPLIT);
        cfg.blockDim = dim3(L::kThreads);
        cfg.dynamicSmemBytes = L::kSmem + 1024;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem + 1024) !=
                cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
            cudaGetLastError();  // the estimate stands in
            n = L::kCtas * pq::sm_count() / (SPLIT + 1);
        }
        cached[dev] = n;
    }
    return cached[dev];
}

// Tile width and K split of a problem: the least estimated time
//   4 + waves * (K blocks of a CTA * time of one + 1 + exchange) microseconds
// among the kernels. The times of a K block fit what they measured cold when
// they were built, tile scales / row scales: pairs 0.5 / 0.85
// (8192 x 14336 x 4096: 449 us; 4096 x 4096 x 8190 by rows: 209), 128 wide 0.28
// (512 x 4096 x 4096: 14.0, in pairs 19.6; with row scales 0.6, so that 64
// wide, of which two share an SM, is always ahead, and there is no such
// kernel), 64 wide 0.24 / 0.45, or 0.36 / 0.55 where two CTAs share an SM
// (77 x 14336 x 4096: 17.0, 128 wide 14.7). The exchange of a split grows with
// the sums that it moves: 1 x 4096 x 4096 took 13.5 us in one piece, 10.6 by 2
// and 8.0 by 4; 300 x 700 x 2000 (64 wide) 9.7, 8.0 and 7.9. With every kernel
// forced in turn on 27 products of layers' sizes, from one token to training
// batches, the choice was the fastest, or within 1% of it, at 26 and 2% off at
// one (77 x 4096 x 14336).
struct Plan {
    int nt, split;
    bool pair;
};
static Plan plan(int64_t m, int64_t n, int64_t kb, bool brow) {
    const int64_t sms = pq::sm_count();
    const double rows = m < kRows ? static_cast<double>(m) / kRows : 1.0;
    Plan best = {64, 1, false};
    double best_us = 1e30;
    auto consider = [&](Plan pl, int64_t tiles, int64_t resident, double us_kb, double exchange) {
        const int64_t waves = (tiles + resident - 1) / resident;
        const double us = waves * ((kb + pl.split - 1) / pl.split * us_kb + 1.0 + exchange);
        if (us < best_us) {
            best_us = us;
            best = pl;
        }
    };
    consider({256, 1, true}, (m + 255) / 256 * ((n + 255) / 256), sms / 2, brow ? 0.85 : 0.5, 0.0);
    const int64_t tm = (m + kRows - 1) / kRows, t128 = tm * ((n + 127) / 128), t64 = tm * ((n + 63) / 64);
    for (int split = 1; split <= 8 && split <= kb; split *= 2) {
        const int64_t c64 = split == 1   ? 2 * sms
                            : split == 2 ? clusters_resident<64, 2>()
                            : split == 4 ? clusters_resident<64, 4>()
                                         : clusters_resident<64, 8>();
        const double moved = split == 1 ? 0.0 : 0.3 + rows * (split == 2 ? 1.2 : split == 4 ? 2.5 : 5.0);
        if (!brow) {
            const int64_t c128 = split == 1   ? sms
                                 : split == 2 ? clusters_resident<128, 2>()
                                 : split == 4 ? clusters_resident<128, 4>()
                                              : clusters_resident<128, 8>();
            consider({128, split, false}, t128, c128, 0.28, moved);
        }
        const bool shared = t64 * split > sms;
        consider({64, split, false}, t64, c64, brow ? (shared ? 0.55 : 0.45) : (shared ? 0.36 : 0.24), moved / 2);
    }
    return best;
}

// What pq_debug_fp8_force asked for: width << 8 | split, 0 for the estimate.
static std::atomic<int> g_forced{0};

// The kernel of a problem; false where a forced one cannot take it (row scales
// have none of 128, and a split CTA has at least one K block).
static bool choose(int64_t m, int64_t n, int64_t kb, bool brow, Plan& pl) {
    const int forced = g_forced.load(std::memory_order_relaxed);
    if (!forced) {
        pl = plan(m, n, kb, brow);
        return true;
    }
    pl = {forced >> 8, forced & 255, forced >> 8 == 256};
    return !(brow && pl.nt == 128) && pl.split <= kb;
}

// A set-up launch: the box of A, the stages that fit beside it, the maps.
template <int NT, bool BROW, int SPLIT, bool PAIR>
static pq_status_t launch(Params& p, const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, int64_t k,
                          cudaStream_t s) {
    using L = Layout<NT, BROW, SPLIT, PAIR>;
    static bool attr_set[64] = {false};
    auto kernel = fp8_gemm_kernel<NT, BROW, SPLIT, PAIR>;
    const int64_t tile_rows = PAIR ? 2 * kRows : kRows;
    const int64_t tiles_m = (p.m + tile_rows - 1) / tile_rows, tiles_n = (p.n + NT - 1) / NT;
    if (tiles_m * tiles_n > (int64_t{1} << 27)) return PQ_ERR_UNSUPPORTED;
    p.tiles_m = static_cast<int32_t>(tiles_m);
    p.tiles_n = static_cast<int32_t>(tiles_n);
    // a short A brings only the rows it has: the other lanes are not read
    const int a_rows = p.m < kRows ? static_cast<int>((p.m + 7) / 8 * 8) : kRows;
    p.a_bytes = a_rows * kBlock;
    p.stages = L::stages(p.a_bytes);
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    constexpr CUtensorMapDataType kByte = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!enc || !encode(enc, &p.ta, kByte, 1, a, p.m, k, lda, a_rows) ||
        !encode(enc, &p.tb, kByte, 1, b, p.n, k, ldb, L::kBRows))
        return PQ_ERR_CUDA;
    // TMA stores want 16-byte aligned rows, less than 2^40 bytes apart, that end
    // on 16 bytes, too: columns are clipped to a multiple of 16 bytes only (with
    // n = 198 in rows of 200, columns 198 and 199 were written). Deciding it in
    // the kernel, for the last tile alone, cost every large product 10 to 17%:
    // the registers of its sums.
    const int size = bytes_of(p.dtype);
    p.tma_out = SPLIT == 1 && pq::aligned(p.y, 16) && p.ldy < (int64_t{1} << 40) / size && p.ldy * size % 16 == 0 &&
                p.n * size % 16 == 0;
    if (p.tma_out && !encode(enc, &p.ty, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                             size, p.y, p.m, p.n, p.ldy, 32))
        return PQ_ERR_CUDA;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   L::kSmem + 1024);
        if (e != cudaSuccess) return pq::cuda_status(e);
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const int tiles = p.tiles_m * p.tiles_n;
    const int slots = L::kCtas * pq::sm_count() / L::kCluster;
    const int grid = (SPLIT > 1 || tiles < slots ? tiles : slots) * L::kCluster;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(L::bytes(p.a_bytes, p.stages));
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e == cudaSuccess) pqc::count_launch();
    return pq::cuda_status(e);
}

template <bool BROW, typename... Args>
static pq_status_t launch_plan(const Plan& pl, Args&&... args) {
    if (pl.pair) return launch<256, BROW, 1, true>(args...);
    if constexpr (!BROW)
        if (pl.nt == 128) switch (pl.split) {
                case 1: return launch<128, BROW, 1, false>(args...);
                case 2: return launch<128, BROW, 2, false>(args...);
                case 4: return launch<128, BROW, 4, false>(args...);
                default: return launch<128, BROW, 8, false>(args...);
            }
    switch (pl.split) {
        case 1: return launch<64, BROW, 1, false>(args...);
        case 2: return launch<64, BROW, 2, false>(args...);
        case 4: return launch<64, BROW, 4, false>(args...);
        default: return launch<64, BROW, 8, false>(args...);
    }
}

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
    if (!pq::aligned(a_scale, 4) || !pq::aligned(b_scale, 4)) return PQ_ERR_MISALIGNED;
    Params p = {};
    p.sa = a_scale;
    p.sb = b_scale;
    p.y = y;
    p.m = m;
    p.n = n;
    p.ldy = ldy;
    p.kb = static_cast<int32_t>((k + kBlock - 1) / kBlock);
    p.dtype = y_dtype;
    p.quad = pq::aligned(y, 4 * bytes_of(y_dtype)) && ldy % 4 == 0;
    Plan pl;
    if (!choose(m, n, p.kb, b_block == PQ_BLOCK_ROW, pl)) return PQ_ERR_UNSUPPORTED;
    return b_block == PQ_BLOCK_ROW ? launch_plan<true>(pl, p, a, lda, b, ldb, k, s)
                                   : launch_plan<false>(pl, p, a, lda, b, ldb, k, s);
}

extern "C" pq_status_t pq_debug_fp8_force(int width, int split) {
    const bool any = width == 0 && split == 0, one = split == 1 && (width == 64 || width == 128 || width == 256);
    const bool many = (split == 2 || split == 4 || split == 8) && (width == 64 || width == 128);
    if (!any && !one && !many) return PQ_ERR_INVALID_ARG;
    pq8::g_forced.store(width << 8 | split, std::memory_order_relaxed);
    return PQ_OK;
}

extern "C" pq_status_t pq_debug_fp8_choice(int64_t m, int64_t n, int64_t k, pq_block_t b_block, int* width,
                                           int* split) {
    if (m < 1 || n < 1 || k < 1 || (b_block != PQ_BLOCK_ROW && b_block != PQ_BLOCK_TILE) || !width || !split)
        return PQ_ERR_INVALID_ARG;
    pq8::Plan pl;
    if (!pq8::choose(m, n, (k + pq8::kBlock - 1) / pq8::kBlock, b_block == PQ_BLOCK_ROW, pl))
        return PQ_ERR_UNSUPPORTED;
    *width = pl.nt;
    *split = pl.split;
    return PQ_OK;
}
