// fp_matmul_i8: y[n][m] = x_scale[n] w_scale[e][m] sum_k w[e][m][k] x[n][k], e the expert of row n.
//
// The sum is exact in int32 (K <= 2^17 - 1 keeps 2^14 K below 2^31); it is rounded to fp32, where it has more than 24
// bits, and multiplied there by the token's scale, then by the channel's, and the result rounded to y's type.
//
// One kernel on the 5th-generation tensor cores (kind::i8, accumulators in tensor memory). A tile is 128
// channels of one expert (the MMA's M, tensor-memory lanes) by up to BN of its tokens (the MMA's N, set
// to the tile's own count rounded up to 16, so a group of three tokens costs a 16-wide MMA). With the
// weights on the M side a decode step reads every weight once whatever the tokens, and a group's ragged
// end wastes at most 15 columns. Warps split the work and hand stages over on mbarriers:
//   warp 0             TMA: per k-tile (128 bytes of K) the weight box (128 rows) and the tokens' boxes
//                      (XB rows each), 128-byte swizzle: the MMA's K-major layout.
//   warp 1             four K = 32 MMAs per k-tile, committed to the stage; the tile's last k-tile to the
//                      accumulator slot's barrier (two slots: the next tile's MMAs run during the epilogue).
//   warps 2-9          epilogue: tcgen05.ld, both scales, conversion, stores (32 channels of one token a
//                      warp and store).
// PAIR: two blocks (cta_group::2) share a tile of 256 channels by 256 tokens: each loads its 128 channels and
// half of the tokens, one issues the MMAs of both.
// Blocks are persistent, one per SM, and walk the tiles of all experts (channels fastest, so that blocks
// that run together share a group's tokens); the experts' tile counts come from the offsets on the device.
//
// SPLIT: with fewer tiles than SMs the sum over K of a tile is split among the blocks of a cluster. The
// blocks exchange their int32 partial sums through distributed shared memory: block d of the cluster
// finishes the d-th share of the columns. Integer sums have no order, so the split changes no bit.
// The cluster's barrier is awaited only by the warps that write to the others, and no block waits for another to leave
// (4384 x 1600, 16 tokens: 6.5 us, with both waits 7.2).
//
// What bounds it, and what it takes (one B200, inputs that change from pass to pass):
//   many tokens    the tensor cores, and over seconds the board's power: 4096 x 14336 x 4096 takes 160 us in a burst of
//                  5 ms, 3.0 POP/s, the tensor pipe active 92% of the SMs' cycles at 1.56 GHz (under the profiler); calls
//                  one after the other for 2 s take 182 us each at 1.29 of 1.965 GHz, with the power cap the only reason.
//                  A library's int8 product of these sizes, without scales, takes 155-158 us in a burst and 180-182 over
//                  2 s. One block a tile of 128 x 256 took 187 us in the same replays as the pairs' 157: its operands come
//                  to 1.5 times the bytes from L2, of which the pairs take 12 TB/s.
//   few a group    HBM: 128 experts of 8192 x 5120 over 8192 tokens 850-940 us, 5.9-6.5 TB/s; 64 tokens 280-306.
//   one weight     the way in and out: 5120 x 16384 for one token takes 18.7 us, 13 of them its 84 MB at the copy's
//                  rate; about 4 us are launch, first loads and epilogue, and 120 of 148 SMs have a part.
//   small K        the epilogue: 802 x 12944 x 128 15.9 us, 21 MB of y.
// (The ranges are calls and bursts on several boards; the last two are calls, in a graph's replays 18.4 and 15.4 us. The
// figures beside the rules below are of graph replays, both sides in turn.)
// The issuing warps run their loops as whole warps with one elected lane: run by a lane alone the same loops took
// 380 ns a k-tile, more than the loads (29 us for the single token).
//
// Every wait is bounded; one that runs out sets the context's operator error word, and an abort flag that
// ends the other roles' waits.
#include <cuda.h>  // CUtensorMap

#include <algorithm>

#include "fp_ops.cuh"

namespace {

constexpr int MI_BM = 128;                  // channels per tile
constexpr int MI_BK = 128;                  // bytes of K per k-tile
constexpr int MI_W_BYTES = MI_BM * MI_BK;   // the weight box
constexpr int MI_MAX_STAGES = 12;
constexpr int MI_SMEM = 200 * 1024;         // dynamic shared memory of a block that has its SM alone
constexpr int MI_EPI_WARPS = 8;
constexpr int MI_THREADS = 32 * (2 + MI_EPI_WARPS);
constexpr uint32_t MI_WAIT_LIMIT = 1u << 24;  // polls, 4 us each while nothing comes: about a minute

__host__ __device__ constexpr int mi_box_rows(int bn) { return bn >= 256 ? 64 : 32; }  // rows of a token box

struct alignas(64) MiArgs {
    CUtensorMap tw, tx;  // E M rows of K bytes, boxes of 128 rows; N rows of K bytes, boxes of XB rows
    const float* w_scale;
    const float* x_scale;
    const int32_t* offsets;
    void* y;
    int64_t ldy;
    int32_t M, K, N, E;
    int32_t y_type;
    int32_t yvec;            // rows of y hold whole aligned 16 bytes
    int32_t mt;              // channel tiles of an expert
    int32_t nk;              // k-tiles
    int32_t stages;
    int32_t per;             // (SPLIT) columns that a block of the cluster finishes
    volatile uint64_t* err;
};

// (CLASSES) Weights whose pitch is no multiple of 16: the rows whose number is c modulo C, C = 16 / gcd(pitch, 16),
// lie C pitches apart, a multiple of 16, and begin at the same byte s_c of 16. Each such class is a matrix that TMA
// can read, its rows s_c bytes to the right; a tile is of one class and meets tokens shifted as far (C copies of
// the tokens, zeros around them, which also cancel what the class's rows have before and after K).
constexpr int MI_MAX_CLASSES = 16;
struct alignas(64) MiClassArgs : MiArgs {
    CUtensorMap wc[MI_MAX_CLASSES];
    int32_t classes, per_class;  // C; tiles of an expert's rows of one class
    int32_t box;                 // rows of a tile at most
};

__device__ __forceinline__ uint32_t mi_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// K-major operand with the 128-byte swizzle: 8-row x 128-byte atoms 1024 bytes apart. The low word holds
// the address / 16 (and a 1 at bit 16), so that a later stage or K step is an addition to it.
__device__ __forceinline__ uint32_t mi_desc_lo(uint32_t a) { return ((a >> 4) & 0x3FFF) | (1u << 16); }
constexpr uint32_t MI_DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);

// true in one lane of a converged warp, always the same one
__device__ __forceinline__ bool mi_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}

// byte offset of 16-byte chunk kk of row `row` in that layout
__device__ __forceinline__ uint32_t mi_off(int row, int kk) {
    return (row >> 3) * 1024 + (row & 7) * 128 + ((kk ^ (row & 7)) << 4);
}

__device__ __forceinline__ void mi_bar_init(uint64_t* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(mi_smem(b)), "r"(count) : "memory");
}

// one bounded wait for a phase; false if it ran out or another role has aborted
template <bool CLUSTER>
__device__ __forceinline__ bool mi_wait_scope(uint32_t bar, uint32_t parity, volatile int* abort, volatile uint64_t* err,
                                              uint32_t limit = MI_WAIT_LIMIT) {
    for (uint32_t it = 0; it < limit; it++) {
        uint32_t ok;
        if (CLUSTER)
            asm volatile(
                "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}\n"
                : "=r"(ok)
                : "r"(bar), "r"(parity)
                : "memory");
        else
            asm volatile(
                "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
                : "=r"(ok)
                : "r"(bar), "r"(parity)
                : "memory");
        if (ok) return true;
        if (abort && *abort) return false;
    }
    if (abort) {
        *abort = 1;
        *err = 1;
        __threadfence_system();
    }
    return false;
}
__device__ __forceinline__ bool mi_wait(uint32_t bar, uint32_t parity, volatile int* abort, volatile uint64_t* err) {
    return mi_wait_scope<false>(bar, parity, abort, err);
}
__device__ __forceinline__ bool mi_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort, volatile uint64_t* err) {
    return __all_sync(0xffffffffu, mi_wait(bar, parity, abort, err));
}
// the same for copies and MMAs in flight while aborting: no flag is looked at
__device__ __forceinline__ void mi_drain(uint32_t bar, uint32_t parity) { mi_wait_scope<false>(bar, parity, nullptr, nullptr); }

__device__ __forceinline__ void mi_arrive(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
// arrives when the MMAs issued so far are complete; PAIR: at the barrier of that offset in both blocks
template <bool PAIR>
__device__ __forceinline__ void mi_commit(uint32_t bar) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
// arrivals at the barrier of that offset in block `rank` of the cluster
__device__ __forceinline__ void mi_arrive_at(uint32_t bar, uint32_t rank, uint32_t count) {
    uint32_t there;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(bar), "r"(rank));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0], %1;\n" ::"r"(there), "r"(count) : "memory");
}
// a, b: the low words of the operands' descriptors
template <bool PAIR>
__device__ __forceinline__ void mi_mma(uint32_t tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\t"
            "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], da, db, %3, p;\n\t}\n" ::"r"(tmem),
            "r"(a), "r"(b), "r"(idesc), "r"(MI_DESC_HI), "r"(add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\t"
            "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], da, db, %3, p;\n\t}\n" ::"r"(tmem),
            "r"(a), "r"(b), "r"(idesc), "r"(MI_DESC_HI), "r"(add)
            : "memory");
}
// PAIR: bar may be the other block's (an address in the cluster's window)
template <bool PAIR>
__device__ __forceinline__ void mi_tma(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3}], [%4];\n" ::"r"(dst),
            "l"(tm), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n" ::"r"(dst),
        "l"(tm), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mi_ld16(uint32_t a, int32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(a));
}
__device__ __forceinline__ void mi_ld8(uint32_t a, int32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(a));
}
__device__ __forceinline__ void mi_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }

// the tokens of token tile u: expert e's rows [first[e], first[e + 1]) in equal shares of a multiple of 16
struct MiTokens {
    int e, n0, cols;
};
__device__ __forceinline__ MiTokens mi_tokens(const int32_t* first, const int32_t* tiles, int E, int u) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {  // the last expert whose first tile is at or before u: the one that has tile u
        const int mid = (lo + hi + 1) >> 1;
        if (tiles[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int n = first[lo + 1] - first[lo], nt = tiles[lo + 1] - tiles[lo];
    const int width = ((n + nt - 1) / nt + 15) & ~15, at = (u - tiles[lo]) * width;
    return MiTokens{lo, first[lo] + at, min(width, n - at)};
}

// the columns of a tile's MMAs: kind::i8 takes multiples of 16 with 128 rows, of 32 with a pair's 256
template <bool PAIR>
__device__ __forceinline__ int mi_columns(int cols) {
    return PAIR ? (cols + 31) & ~31 : (cols + 15) & ~15;
}

// y of C columns (tokens n .. n + cols - 1) for 32 channels from m0 on, one a lane; xs: the tokens' scales.
// The values cross the warp's C x 32 buffer in shared memory, so that a lane stores 16 bytes of a token
// (a 2-byte store a lane and token took 24 instructions a token, most of them addresses and predicates).
template <typename YT, int C>
__device__ __forceinline__ void mi_store(const MiArgs& a, const int32_t (&v)[C], const float* xs, int64_t n, int cols,
                                         int64_t m0, float ws, YT* buf, int lane) {
    __syncwarp();  // the buffer's last values have been read
#pragma unroll
    for (int i = 0; i < C; i++) buf[32 * i + lane] = fp_from_f<YT>((float)v[i] * xs[i] * ws);
    __syncwarp();
    constexpr int E16 = 16 / sizeof(YT), P = 32 / E16;  // values and pieces of 16 bytes
    YT* y = reinterpret_cast<YT*>(a.y) + n * a.ldy + m0;
    if (a.yvec) {
        const int pc = lane % P;
#pragma unroll
        for (int i = 0; i < C * P / 32; i++) {
            const int col = lane / P + i * (32 / P);
            if (col < cols && m0 + pc * E16 < a.M)
                *reinterpret_cast<uint4*>(y + col * a.ldy + pc * E16) = *reinterpret_cast<const uint4*>(buf + 32 * col + pc * E16);
        }
    } else if (m0 + lane < a.M) {
#pragma unroll 4
        for (int i = 0; i < cols; i++) y[i * a.ldy + lane] = buf[32 * i + lane];
    }
}
template <int C>
__device__ __forceinline__ void mi_put(const MiArgs& a, const int32_t (&v)[C], const float* xs, int64_t n, int cols,
                                       int64_t m0, float ws, void* buf, int lane) {
    if (a.y_type == FP_F32)
        mi_store<float>(a, v, xs, n, cols, m0, ws, (float*)buf, lane);
    else if (a.y_type == FP_F16)
        mi_store<__half>(a, v, xs, n, cols, m0, ws, (__half*)buf, lane);
    else
        mi_store<__nv_bfloat16>(a, v, xs, n, cols, m0, ws, (__nv_bfloat16*)buf, lane);
}

// the same for channels that lie apart: single values, m the lane's channel
template <typename YT>
__device__ __forceinline__ void mi_store_apart(const MiArgs& a, const int32_t (&v)[16], const float* xs, int64_t n, int cols,
                                               int64_t m, float ws, bool live) {
    if (!live || m >= a.M) return;
    YT* y = reinterpret_cast<YT*>(a.y) + n * a.ldy + m;
#pragma unroll
    for (int i = 0; i < 16; i++)
        if (i < cols) y[i * a.ldy] = fp_from_f<YT>((float)v[i] * xs[i] * ws);
}
__device__ __forceinline__ void mi_put_apart(const MiArgs& a, const int32_t (&v)[16], const float* xs, int64_t n, int cols,
                                             int64_t m, float ws, bool live) {
    if (a.y_type == FP_F32)
        mi_store_apart<float>(a, v, xs, n, cols, m, ws, live);
    else if (a.y_type == FP_F16)
        mi_store_apart<__half>(a, v, xs, n, cols, m, ws, live);
    else
        mi_store_apart<__nv_bfloat16>(a, v, xs, n, cols, m, ws, live);
}

// (CLASSES) the place in class c of the first of its rows from row g on
__device__ __forceinline__ int mi_class_row(int g, int c, int classes) { return (g - c + classes - 1) / classes; }

template <int BN, bool SPLIT, bool PAIR, bool CLASSES>
__global__ void __launch_bounds__(MI_THREADS, 1)
    matmul_i8_kernel(const __grid_constant__ std::conditional_t<CLASSES, MiClassArgs, MiArgs> a) {
    static_assert(!(PAIR && SPLIT) && !(CLASSES && (PAIR || SPLIT)), "a pair and a class have a tile's whole K");
    constexpr int XB = mi_box_rows(BN), XROWS = PAIR ? BN / 2 : BN;  // token rows of a box, of this block's stage
    constexpr int STAGE = MI_W_BYTES + XROWS * MI_BK;
    constexpr int TM = PAIR ? 2 * MI_BM : MI_BM;  // channels of a tile
    constexpr int SLOTS = SPLIT ? 1 : 2;
    constexpr int TCOLS = SLOTS * BN;
    extern __shared__ uint8_t mi_raw[];
    uint8_t* smem = mi_raw + ((1024 - (mi_smem(mi_raw) & 1023)) & 1023);
    uint8_t* ring = smem;
    int32_t* red = reinterpret_cast<int32_t*>(ring + a.stages * STAGE);  // (SPLIT) partial sums of the other blocks
    __shared__ __align__(8) uint64_t full[MI_MAX_STAGES], empty[MI_MAX_STAGES], accfull[2], accempty[2], fin, redfull;
    __shared__ uint32_t tmem_base;
    __shared__ volatile int s_abort;
    __shared__ int32_t s_part[32];
    __shared__ __align__(16) float s_scale[MI_EPI_WARPS][128];
    __shared__ __align__(16) uint8_t s_out[MI_EPI_WARPS][16 * 32 * 4];
    static_assert(!SPLIT || BN <= 128, "a warp keeps the scales of 128 tokens");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nthr = blockDim.x;
    const int S = a.stages;
    uint32_t crank = 0, csize = 1;
    if (SPLIT || PAIR) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
    }
    int32_t* first = reinterpret_cast<int32_t*>(ring + a.stages * STAGE +
                                                (SPLIT ? (size_t)csize * a.per * MI_BM * sizeof(int32_t) : 0));
    int32_t* tiles = first + a.E + 1;

    if (tid == 0) {
        for (int s = 0; s < S; s++) {
            mi_bar_init(&full[s], 1);
            mi_bar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; s++) {
            mi_bar_init(&accfull[s], 1);
            mi_bar_init(&accempty[s], (PAIR ? 2 : 1) * MI_EPI_WARPS);  // a warp of the epilogue each
        }
        mi_bar_init(&fin, 1);
        mi_bar_init(&redfull, SPLIT ? max(1, MI_EPI_WARPS * ((int)csize - 1)) : 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(mi_smem(&tmem_base)),
                         "n"(TCOLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(mi_smem(&tmem_base)),
                         "n"(TCOLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        }
    }
    // the other blocks' barriers are there before anything arrives at them (SPLIT: awaited by those who send)
    if (SPLIT) asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");
    // what is above overlaps the end of the kernel before this one on the stream; from here on its results are
    // read (with plain loads: an invariant one could be moved up across the wait). The next kernel may be brought
    // onto the SMs that this one leaves.
    if (warp == 0 && lane == 0) {
        if (!CLASSES) asm volatile("prefetch.tensormap [%0];\n" ::"l"(&a.tw) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(&a.tx) : "memory");
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    // the experts' first rows (each offset counted as the largest up to it, inside [0, N]) and the prefix
    // sums of their token tiles
    if (!a.offsets) {
        if (tid == 0) {
            first[0] = 0;
            first[1] = a.N;
        }
        __syncthreads();
    } else {
        const int per = (a.E + nthr) / nthr, x0 = min(a.E + 1, tid * per), x1 = min(a.E + 1, x0 + per);
        int32_t m = 0;
        for (int x = x0; x < x1; x++) m = max(m, a.offsets[x]);
        int32_t inc = m;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc = max(inc, v);
        }
        if (lane == 31) s_part[warp] = inc;
        __syncthreads();
        int32_t run = __shfl_up_sync(0xffffffffu, inc, 1);
        if (lane == 0) run = 0;
        for (int w = 0; w < warp; w++) run = max(run, s_part[w]);
        for (int x = x0; x < x1; x++) {
            run = max(run, a.offsets[x]);
            first[x] = min(run, a.N);
        }
        __syncthreads();
    }
    {
        const int per = (a.E + nthr - 1) / nthr, x0 = min(a.E, tid * per), x1 = min(a.E, x0 + per);
        int32_t sum = 0;
        for (int x = x0; x < x1; x++) sum += (first[x + 1] - first[x] + BN - 1) / BN;
        int32_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += v;
        }
        if (lane == 31) s_part[warp] = inc;
        __syncthreads();
        int32_t run = inc - sum;
        for (int w = 0; w < warp; w++) run += s_part[w];
        for (int x = x0; x < x1; x++) {
            tiles[x] = run;
            run += (first[x + 1] - first[x] + BN - 1) / BN;
        }
        if (x0 < x1 && x1 == a.E) tiles[a.E] = run;
    }
    asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
    if (PAIR) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;\n" ::: "memory");
    const uint32_t tmem = tmem_base;
    const int total_u = tiles[a.E];  // token tiles; tile (u, m) of channel tile m
    // this block's (SPLIT, PAIR: this cluster's) first tile and its step; SPLIT has one tile per cluster
    const int start = (int)(blockIdx.x / csize), walkers = (int)(gridDim.x / csize);
    const int u0 = start / a.mt, mm0 = start % a.mt;
    const int du = SPLIT ? 0x3fffffff : walkers / a.mt, dm = SPLIT ? 0 : walkers % a.mt;
    const int kt0 = SPLIT ? (int)((int64_t)a.nk * crank / csize) : 0;
    const int kt1 = SPLIT ? (int)((int64_t)a.nk * (crank + 1) / csize) : a.nk;
    const int wlead = PAIR ? (int)crank * MI_BM : 0;  // this block's channels of a tile
    volatile uint64_t* err = a.err;

    if (warp == 0) {
        // ---- TMA: the whole warp walks and waits, one lane issues ----
        const bool lead = mi_elect();
        const uint32_t full0 = mi_smem(full), empty0 = mi_smem(empty), ring0 = mi_smem(ring);
        uint32_t fulls = full0;  // where the copies are counted: PAIR, the first block's barriers
        if (PAIR) asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(fulls) : "r"(full0));
        uint32_t s = 0, ph = 1;  // a fresh barrier's "previous phase" counts as complete
        uint32_t issued = 0;
        bool ok = true;
        for (int u = u0, m = mm0; u < total_u && ok;) {
            const MiTokens tk = mi_tokens(first, tiles, a.E, u);
            // PAIR: half of the MMA's columns each, and both blocks' bytes awaited by the issuing block
            const int half = PAIR ? mi_columns<PAIR>(tk.cols) >> 1 : 0;
            const int boxes = ((PAIR ? half : tk.cols) + XB - 1) / XB;
            int xrow = tk.n0 + (PAIR ? (int)crank * half : 0);
            uint32_t bytes = MI_W_BYTES + boxes * XB * MI_BK;
            int wrow = tk.e * a.M + m * TM + wlead;
            const CUtensorMap* tw = &a.tw;
            if constexpr (CLASSES) {
                const int cls = m / a.per_class;
                wrow = mi_class_row(tk.e * a.M, cls, a.classes) + (m - cls * a.per_class) * a.box;
                xrow += cls * a.N;
                tw = &a.wc[cls];
                bytes = (uint32_t)a.box * MI_BK + boxes * XB * MI_BK;
            }
            for (int kt = kt0; kt < kt1; kt++) {
                if (!mi_wait_warp(empty0 + 8 * s, ph, &s_abort, err)) {
                    ok = false;
                    break;
                }
                if (lead) {
                    const uint32_t fb = fulls + 8 * s, dst = ring0 + s * STAGE;
                    if (!PAIR || crank == 0)
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(full0 + 8 * s),
                                     "r"(PAIR ? 2 * bytes : bytes)
                                     : "memory");
                    mi_tma<PAIR>(dst, tw, kt * MI_BK, wrow, fb);
#pragma unroll
                    for (int b = 0; b < XROWS / XB; b++)
                        if (b < boxes)
                            mi_tma<PAIR>(dst + MI_W_BYTES + b * XB * MI_BK, &a.tx, kt * MI_BK, xrow + b * XB, fb);
                }
                issued++;
                if (++s == (uint32_t)S) s = 0, ph ^= 1;
            }
            u += du, m += dm;
            if (m >= a.mt) m -= a.mt, u++;
        }
        if (!ok && lead) {
            if (!PAIR) {
                // every copy that was issued lands before the block ends
                for (uint32_t i = issued > (uint32_t)S ? issued - S : 0; i < issued; i++)
                    mi_drain(full0 + 8 * (i % S), (i / S) & 1u);
            } else {
                // (the other block's part may be missing, so that the phases never complete: 64 ms have to do, of which
                // the copies, on their way when the wait ran out, need a few microseconds)
                for (int i = 0; i < 64; i++) __nanosleep(1000000);
            }
        }
        __syncwarp();
    } else if (warp == 1 && (!PAIR || crank == 0)) {
        // ---- MMA issue: the same way; PAIR: for both blocks ----
        const bool lead = mi_elect();
        const uint32_t full0 = mi_smem(full), empty0 = mi_smem(empty), desc0 = mi_desc_lo(mi_smem(ring));
        uint32_t s = 0, ph = 0, tc = 0;
        bool ok = true;
        for (int u = u0, m = mm0; u < total_u && ok; tc++) {
            const MiTokens tk = mi_tokens(first, tiles, a.E, u);
            const uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(mi_columns<PAIR>(tk.cols) >> 3) << 17) |
                                   ((uint32_t)(TM >> 4) << 24);  // s32 += s8 x s8, both K-major
            const uint32_t slot = tc % SLOTS;
            if (tc >= SLOTS && !__all_sync(0xffffffffu, mi_wait_scope<PAIR>(mi_smem(&accempty[slot]), (tc / SLOTS - 1) & 1u,
                                                                        &s_abort, err)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
            const uint32_t dst = tmem + slot * BN;
            for (int kt = kt0; kt < kt1; kt++) {
                if (!mi_wait_warp(full0 + 8 * s, ph, &s_abort, err)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
                if (lead) {
                    const uint32_t wd = desc0 + s * (STAGE >> 4), xd = wd + (MI_W_BYTES >> 4);
#pragma unroll
                    for (int kc = 0; kc < MI_BK / 32; kc++)
                        mi_mma<PAIR>(dst, wd + 2 * kc, xd + 2 * kc, idesc, (kt > kt0 || kc > 0) ? 1u : 0u);
                    mi_commit<PAIR>(empty0 + 8 * s);
                    if (kt == kt1 - 1) mi_commit<PAIR>(mi_smem(&accfull[slot]));
                }
                if (++s == (uint32_t)S) s = 0, ph ^= 1;
            }
            u += du, m += dm;
            if (m >= a.mt) m -= a.mt, u++;
        }
        // every MMA issued is complete before the tensor memory is freed
        if (lead) {
            mi_commit<PAIR>(mi_smem(&fin));
            mi_drain(mi_smem(&fin), 0);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- (PAIR) the second block stays until the last of the first one's arrivals at its barriers ----
        if (lane == 0) mi_drain(mi_smem(&fin), 0);
        __syncwarp();
    } else {
        // ---- epilogue: warp w reads lanes 32 (w % 4) .. + 31; the two warps of the same lanes take every
        // other chunk of 16 columns of a tile, or, of tiles with few columns, whose time is mostly the way to
        // the scales and back, every other tile. A chunk's load is in flight while the one before is stored
        // (53 experts, 1649 tokens, 2992 x 96: 20.7 us, tiles shared 23.5).
        const int qd = warp & 3, group = (warp - 2) >> 2;
        const bool several = (int64_t)total_u * a.mt > walkers;  // some block has more than one tile
        if (SPLIT) asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
        uint32_t tc = 0;
        for (int u = u0, m = mm0; u < total_u; tc++) {
            const MiTokens tk = mi_tokens(first, tiles, a.E, u);
            const uint32_t slot = tc % SLOTS;
            const bool alone = !SPLIT && several && tk.cols <= 64;  // a group's own tile
            // Every warp arrives once for every tile, the four that pass a tile over when they have seen its
            // accumulator's phase: the slot's next phase then cannot end before all eight have seen this one, and no
            // warp loses count of the phases.
            const auto leave_slot = [&] {
                if (lane != 0) return;
                if (PAIR)
                    mi_arrive_at(mi_smem(&accempty[slot]), 0, 1);
                else
                    mi_arrive(mi_smem(&accempty[slot]), 1);
            };
            if (alone && (int)(tc & 1) != group) {
                if (!mi_wait_warp(mi_smem(&accfull[slot]), (tc / SLOTS) & 1u, &s_abort, err)) break;
                leave_slot();
                u += du, m += dm;
                if (m >= a.mt) m -= a.mt, u++;
                continue;
            }
            const int part = alone ? 0 : group, step = alone ? 16 : 32;
            int64_t m0 = (int64_t)m * TM + wlead + 32 * qd;  // the warp's first channel
            int stride = 1, rows = 32;                       // the channels' distance, how many are the tile's
            if constexpr (CLASSES) {
                const int cls = m / a.per_class, at = (m - cls * a.per_class) * a.box;
                stride = a.classes;
                m0 = cls + (int64_t)stride * (mi_class_row(tk.e * a.M, cls, stride) + at + 32 * qd) - (int64_t)tk.e * a.M;
                rows = a.box - 32 * qd;
            }
            const int64_t mine = m0 + (int64_t)stride * lane;
            const float ws = lane < rows && mine < a.M ? a.w_scale[(int64_t)tk.e * a.M + mine] : 0.0f;
            // the scales of this warp's tokens, before their sums are there: chunk i of 16 columns at 16 i (SPLIT:
            // all columns, for the share may lie anywhere)
            float* xs = s_scale[warp - 2];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int j = lane + 32 * i, col = SPLIT || alone ? j : (j >> 4) * 32 + 16 * part + (j & 15);
                if (col < tk.cols) xs[j] = a.x_scale[tk.n0 + col];
            }
            __syncwarp();
            if (!mi_wait_warp(mi_smem(&accfull[slot]), (tc / SLOTS) & 1u, &s_abort, err)) break;
            asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
            const uint32_t base = tmem + ((uint32_t)(32 * qd) << 16) + slot * BN;
            if (!SPLIT) {
                int32_t v[16], nx[16];
                int c0 = 16 * part;
                if (c0 < tk.cols) {
                    mi_ld16(base + (uint32_t)c0, v);
                    mi_ld_wait();
                }
#pragma unroll 1
                for (; c0 < tk.cols; c0 += step) {
                    if (c0 + step < tk.cols) mi_ld16(base + (uint32_t)(c0 + step), nx);
                    const float* sc = xs + (alone ? c0 : (c0 >> 5) * 16);
                    const int cols = min(16, tk.cols - c0);
                    if constexpr (CLASSES)
                        mi_put_apart(a, v, sc, (int64_t)tk.n0 + c0, cols, mine, ws, lane < rows);
                    else
                        mi_put<16>(a, v, sc, (int64_t)tk.n0 + c0, cols, m0, ws, s_out[warp - 2], lane);
                    mi_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i++) v[i] = nx[i];
                }
            } else {
                // send: columns [d per, (d + 1) per) to block d, at [this block][column][lane]; the two warps of
                // the same lanes take every other block
                const int per = a.per, mrow = 32 * qd + lane;
                for (uint32_t d = (uint32_t)group; d < csize; d += 2) {
                    if (d == crank) continue;
                    const int lo = (int)d * per, hi = min(tk.cols, lo + per);
                    uint32_t at;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at)
                        : "r"(mi_smem(red + (size_t)crank * per * MI_BM + mrow)), "r"(d));
                    for (int c = lo; c < hi; c += 8) {
                        int32_t v[8];
                        mi_ld8(base + (uint32_t)c, v);
                        mi_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(at + (uint32_t)((c - lo + i) * MI_BM * 4)),
                                         "r"(v[i])
                                         : "memory");
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    for (uint32_t d = 0; d < csize; d++)
                        if (d != crank) mi_arrive_at(mi_smem(&redfull), d, 1);
                }
                __syncwarp();
                const bool got =
                    csize == 1 || __all_sync(0xffffffffu, mi_wait_scope<true>(mi_smem(&redfull), 0, &s_abort, err));
                if (!got) break;
                const int lo = (int)crank * per, hi = min(tk.cols, lo + per);
                for (int c0 = lo + 8 * group; c0 < hi; c0 += 16) {
                    int32_t v[8];
                    mi_ld8(base + (uint32_t)c0, v);
                    mi_ld_wait();
                    const int cols = min(8, hi - c0);
                    for (uint32_t b = 0; b < csize; b++) {
                        if (b == crank) continue;
                        const int32_t* src = red + ((size_t)b * per + (c0 - lo)) * MI_BM + mrow;
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            if (i < cols) v[i] += src[i * MI_BM];
                    }
                    mi_put<8>(a, v, xs + c0, (int64_t)tk.n0 + c0, cols, m0, ws, s_out[warp - 2], lane);
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
            __syncwarp();
            leave_slot();
            u += du, m += dm;
            if (m >= a.mt) m -= a.mt, u++;
        }
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
    // no block leaves while another may still write to it or read its operands. SPLIT: a block has had all that the
    // others write to it before it finishes its share, unless a wait ran out.
    if (SPLIT && warp < 2) asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
    if (PAIR || (SPLIT && s_abort))
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;\n" ::: "memory");
    if (warp == 1) {
        if (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "n"(TCOLS));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "n"(TCOLS));
    }
}

// ---- operands that TMA cannot read ----------------------------------------------------------
//
// TMA wants an address and a pitch that are multiples of 16. Rows that are not so are first copied to rows
// that are, in stream-ordered memory from the context's pool (inside a graph its own allocation nodes), by
// one launch for both operands: a thread loads the two aligned 16 bytes that its own lie in and shifts. An expert
// without tokens is passed over. Weights that few tokens meet are not copied but read by classes of rows
// (MiClassArgs): then only the tokens are copied, shifted for every class.
// (Realigning inside the product, with warps that load words into the swizzled stages, took 1224 us on 2352 x 9600 x
// 7454 where this takes 188: every tile of channels did the tokens' rows again.)

struct MiOperand {
    const int8_t* p;
    int64_t ld, rows;
};

// rows of K bytes at src (pitch ld), `copies` times, copy c shifted right by (c step) mod 16 bytes, to rows of
// 16 chunks bytes; zeros around them. M: rows of an expert, with offsets.
struct MiRealign {
    const int8_t* src;
    int8_t* dst;
    int64_t ld;
    const int32_t* offsets;
    uint32_t rows, blocks;         // rows of a copy; blocks of the job
    uint32_t chunks, per, across;  // 16-byte pieces of a row, rows of a block, blocks across a row
    int32_t copies, step, M;
};
constexpr int MI_RE = 4;  // 16-byte pieces of a thread, a block's width apart

__global__ void __launch_bounds__(256) realign_rows_kernel(MiRealign j0, MiRealign j1, int K) {
    // the product's set-up overlaps the last blocks of this (it waits for their end before it reads)
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // (the kernel before this one)
    const bool second = blockIdx.x >= j0.blocks;
    const MiRealign j = second ? j1 : j0;
    const uint32_t b = blockIdx.x - (second ? j0.blocks : 0), down = b / j.across, c0 = (b - down * j.across) * (256 * MI_RE);
    const FpSpan span = fp_span(j.src, j.rows, j.ld, K);
#pragma unroll
    for (int u = 0; u < MI_RE; u++) {
        // a block has several short rows, or a part of a long one
        const uint32_t i = c0 + threadIdx.x + 256 * u, r = j.across == 1 ? i / j.chunks : 0, c = i - r * j.chunks;
        const uint32_t out = down * j.per + r;
        if (r >= j.per || c >= j.chunks || out >= j.rows * j.copies) break;
        uint32_t row = out;
        int first = 16 * (int)c;  // the K index of the piece's first byte
        if (j.copies > 1) {
            const uint32_t copy = out / j.rows;
            row = out - copy * j.rows;
            first -= (int)(copy * j.step) & 15;
        }
        if (j.offsets) {
            const uint32_t e = row / (uint32_t)j.M;
            if (j.offsets[e + 1] <= max(0, j.offsets[e])) continue;
        }
        const int8_t* p = j.src + (int64_t)row * j.ld + first;
        const int lo = max(0, -first), hi = K - first;  // the bytes of the piece inside the row
        FpWords<16> w;
        uint32_t o[4];
        if (hi <= lo) {
#pragma unroll
            for (int q = 0; q < 4; q++) w.w[q] = 0;
        } else if (fp_load16_any(p, span, o)) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int a = lo - 4 * q, b = hi - 4 * q;
                w.w[q] = o[q] & (b >= 4 ? 0xFFFFFFFFu : b <= 0 ? 0u : (1u << (8 * b)) - 1) &
                         (a <= 0 ? 0xFFFFFFFFu : a >= 4 ? 0u : ~((1u << (8 * a)) - 1));
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                w.w[q] = 0;
#pragma unroll
                for (int b = 0; b < 4; b++)
                    if (4 * q + b >= lo && 4 * q + b < hi) w.w[q] |= (uint32_t)(uint8_t)p[4 * q + b] << (8 * b);
            }
        }
        w.store(j.dst + ((int64_t)out * j.chunks + c) * 16);
    }
}

// Scratch rows of a call, given back to the pool in the order of the stream when the call has queued its work
struct MiScratch {
    cudaStream_t st;
    int8_t* p = nullptr;
    explicit MiScratch(cudaStream_t s) : st(s) {}
    ~MiScratch() {
        if (p) cudaFreeAsync(p, st);
    }
    MiScratch(const MiScratch&) = delete;
    MiScratch& operator=(const MiScratch&) = delete;
};

bool mi_readable(const MiOperand& o) { return ((uintptr_t)o.p | (uint64_t)o.ld) % 16 == 0; }

// makes both operands readable for TMA; classes > 0: only the tokens are copied, for so many classes of weight rows
int mi_realign(fp_ctx* c, MiOperand& w, MiOperand& x, int K, const int32_t* offsets, int M, int classes, MiScratch& scratch) {
    MiOperand* op[2] = {!classes && !mi_readable(w) ? &w : nullptr, classes || !mi_readable(x) ? &x : nullptr};
    if (!op[0] && !op[1]) return FP_OK;
    MiRealign job[2] = {};
    size_t bytes = 0, at[2] = {0, 0};
    int64_t blocks = 0;
    for (int i = 0; i < 2; i++) {
        if (!op[i]) continue;
        MiRealign& j = job[i];
        j.src = op[i]->p, j.ld = op[i]->ld, j.rows = (uint32_t)op[i]->rows, j.M = M;
        j.copies = i == 1 && classes ? classes : 1;
        j.step = i == 1 && classes ? (int)(w.ld & 15) : 0;
        j.chunks = (uint32_t)(K + (j.copies > 1 ? 15 : 0) + 15) / 16;
        j.offsets = i == 0 ? offsets : nullptr;
        j.per = std::max(1u, 256 * MI_RE / j.chunks);
        j.across = (j.chunks + 256 * MI_RE - 1) / (256 * MI_RE);
        const int64_t n = ((int64_t)j.rows * j.copies + j.per - 1) / j.per * j.across;
        j.blocks = (uint32_t)n;
        at[i] = bytes;
        bytes += (size_t)16 * j.chunks * j.rows * j.copies;
        blocks += n;
    }
    if (blocks > 0x7fffffffll) return fp_fail(c, FP_ERR_SHAPE, "fp_matmul_i8: operands of over 2^45 bytes with odd pitches");
    if (!c->pool) return fp_fail(c, FP_ERR_OOM, "fp_matmul_i8: no memory pool for realigned rows on this device");
    const cudaError_t e = cudaMallocFromPoolAsync((void**)&scratch.p, bytes, c->pool, scratch.st);
    if (e != cudaSuccess) {
        scratch.p = nullptr;
        cudaGetLastError();
        return fp_fail(c, FP_ERR_OOM,
                       std::string("fp_matmul_i8: ") + std::to_string(bytes) + " bytes for realigned rows: " + cudaGetErrorString(e));
    }
    for (int i = 0; i < 2; i++) {
        if (!op[i]) continue;
        job[i].dst = scratch.p + at[i];
        op[i]->p = job[i].dst, op[i]->ld = 16 * (int64_t)job[i].chunks, op[i]->rows *= job[i].copies;
    }
    int slot;
    fp_op_tic(c, scratch.st, K_REALIGN, 2.0 * (double)bytes, &slot);
    const cudaError_t rc = fp_launch(realign_rows_kernel, dim3((unsigned)blocks), 256, 0, scratch.st, job[0], job[1], K);
    fp_toc(c, scratch.st, slot);
    FP_CUDA(c, rc);
    return FP_OK;
}

// Classes of weight rows to read apart (0: none). Where a group has up to 128 rows and the shifted copies of the
// tokens are at most a quarter of the weights that need no copy: 64 experts of 4512 x 13885 over 1087 tokens take
// 873 us and took 2426 with copied weights, 8192 x 5121 for 64 tokens 27 and 38. The copied rows win where many
// tokens meet each weight: 4096 x 4097 for 128 tokens 34 and 27.
int mi_classes(const MiOperand& w, int64_t E, int64_t M, int64_t N, int64_t rows) {
    if (mi_readable(w) || (uintptr_t)w.p % 16 != 0 || rows > 128) return 0;
    int classes = 16;
    while (classes > 2 && (uint64_t)w.ld * (classes / 2) % 16 == 0) classes /= 2;
    return M >= 4 * classes && classes * N <= std::min(E, N) * M / 4 ? classes : 0;
}

// (fp_ops_selftest) a wait for a barrier that nothing arrives at: a second one has the abort flag to end it
__global__ void __launch_bounds__(64) wait_selftest_kernel(volatile uint64_t* err, uint32_t limit) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ volatile int s_abort;
    if (threadIdx.x == 0) {
        mi_bar_init(&bar, 1);
        s_abort = 0;
    }
    __syncthreads();
    mi_wait_scope<false>(mi_smem(&bar), 0, &s_abort, err, limit);
}

template <int BN, bool SPLIT, bool PAIR, bool CLASSES>
constexpr int mi_kernel_bit() {
    return CLASSES ? 13 : 1 + (BN == 32 ? 0 : BN == 128 ? 4 : 8) + 2 * SPLIT + PAIR;
}

template <int BN, bool SPLIT, bool PAIR, bool CLASSES = false>
int launch_mi(fp_ctx* c, std::conditional_t<CLASSES, MiClassArgs, MiArgs>& a, const MiOperand& w, const MiOperand& x,
              int64_t token_tiles, int split, cudaStream_t st) {
    constexpr int STAGE = MI_W_BYTES + (PAIR ? BN / 2 : BN) * MI_BK;
    constexpr int TM = PAIR ? 2 * MI_BM : MI_BM;
    const int cluster = PAIR ? 2 : split;
    if constexpr (CLASSES) {
        a.box = (int32_t)std::min<int64_t>(MI_BM, ((a.M + a.classes - 1) / a.classes + 7) / 8 * 8);
        a.per_class = (int32_t)(((a.M + a.classes - 1) / a.classes + a.box - 1) / a.box);
        a.mt = a.classes * a.per_class;
        for (int i = 0; i < a.classes; i++) {
            const int64_t at = i * w.ld;  // (the first row of the class, and the bytes before it that align it)
            const int s = (int)(at & 15);
            if (i < w.rows &&
                !fp_tmap_u8_2d(&a.wc[i], w.p + at - s, (uint64_t)(s + a.K), (uint64_t)((w.rows - i + a.classes - 1) / a.classes),
                               (uint64_t)(a.classes * w.ld), MI_BK, (uint32_t)a.box, true))
                return fp_fail(c, FP_ERR_CUDA, "fp_matmul_i8: tensor map encoding failed");
        }
    } else {
        if (!fp_tmap_u8_2d(&a.tw, w.p, (uint64_t)a.K, (uint64_t)w.rows, (uint64_t)w.ld, MI_BK, MI_BM, true))
            return fp_fail(c, FP_ERR_CUDA, "fp_matmul_i8: tensor map encoding failed");
        a.mt = (a.M + TM - 1) / TM;
    }
    const uint64_t xk = (uint64_t)(CLASSES ? x.ld : a.K);  // (classes: the whole of a shifted row)
    if (!fp_tmap_u8_2d(&a.tx, x.p, xk, (uint64_t)x.rows, (uint64_t)x.ld, MI_BK, mi_box_rows(BN), true))
        return fp_fail(c, FP_ERR_CUDA, "fp_matmul_i8: tensor map encoding failed");
    a.per = SPLIT ? (((BN + split - 1) / split) + 7) & ~7 : 0;
    const size_t extra = (SPLIT ? (size_t)split * a.per * MI_BM * 4 : 0) + 8 * ((size_t)a.E + 1) + 1024;
    a.stages = (int)std::min<size_t>(MI_MAX_STAGES, (MI_SMEM - extra) / STAGE);
    if (extra + 2 * STAGE > (size_t)MI_SMEM)  // (three stages at 4096 experts)
        return fp_fail(c, FP_ERR_SHAPE, "fp_matmul_i8: too many experts for the shared memory");
    auto kern = matmul_i8_kernel<BN, SPLIT, PAIR, CLASSES>;
    FP_CUDA(c, fp_op_smem(c, mi_kernel_bit<BN, SPLIT, PAIR, CLASSES>(), kern, MI_SMEM));
    const int64_t tiles = token_tiles * a.mt;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cluster * (SPLIT ? tiles : std::min<int64_t>(tiles, c->num_sms / cluster))));
    cfg.blockDim = dim3(MI_THREADS);
    cfg.dynamicSmemBytes = a.stages * STAGE + extra;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    FP_CUDA(c, cudaLaunchKernelEx(&cfg, kern, a));
    return FP_OK;
}

// clusters of `split` blocks of the splitting kernel that the GPU holds at once (asked once a context)
template <int BN>
int64_t mi_clusters(fp_ctx* c, int split) {
    int16_t& n = c->op_clusters[BN == 32 ? 0 : 1][split];
    if (n == 0) {
        auto kern = matmul_i8_kernel<BN, true, false, false>;
        if (fp_op_smem(c, mi_kernel_bit<BN, true, false, false>(), kern, MI_SMEM) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)split);
        cfg.blockDim = dim3(MI_THREADS);
        cfg.dynamicSmemBytes = MI_SMEM;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)split;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int most = 0;
        if (cudaOccupancyMaxActiveClusters(&most, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            most = 0;
        }
        n = (int16_t)(most + 1);
    }
    return n - 1;
}

// token tiles at most: every group that can have rows has one, and the rows fill the others
int64_t mi_token_tiles(const MiArgs& a, int bn) {
    const int64_t groups = std::min(a.E, a.N);
    return groups == 1 ? (a.N + bn - 1) / bn : groups + a.N / bn;
}

// The sums over K are split when the tiles of a whole K leave SMs idle: as far as all clusters are on the GPU at
// once (a second wave costs what the split gains: 64 tiles of 8192 x 5120, 16 tokens, took 13.8 us in two parts
// and 20.9 in three), from twelve k-tiles on, up to six parts of at least four (700 x 1024 x 1024, eight k-tiles:
// 7.3 us whole, 8.6 in two; 1 x 5120 x 16384, 40 tiles: 37.5, 23.5 and 20.1 us whole and in two and three parts;
// 1 x 1024 x 8192, 8 tiles: 20.7 us whole, 14.1, 10.4 and 9.8 in two, four and six).
template <int BN>
int mi_split(fp_ctx* c, int64_t tiles, int64_t nk) {
    for (int s = nk < 12 ? 1 : (int)std::min<int64_t>(6, nk / 4); s > 1; s--)
        if (tiles <= c->num_sms / s && tiles <= mi_clusters<BN>(c, s)) return s;
    return 1;
}

// Tiles of 32 tokens where a group has no more (deeper stages), and where all of them are on the GPU at once: then more
// SMs share the epilogue, for reading the weights several times (102 x 2895 x 368: 5.1 us, tiles of 128 7.1; 128 x 1024 x
// 1024: 5.9 and 7.5; 128 x 4096 x 2048: 8.1 and 9.2). With a longer K only if a block has no more bytes to load, a
// k-tile's 20 KB against 32, with K split or not (100 x 512 x 4096: 7.9 and 9.8; 64 x 2048 x 8192: 10.3 and 10.8; but 96 x
// 6000 x 4096: 12.9 and 11.9, 128 x 4096 x 8192: 20.8 and 14.5). Tiles of 128 where all such tiles are on the GPU at
// once, K split or whole (512 x 4096 x 4096: 16.2 us, pairs 17.7; 256 x 2048 x 8192: 14.2 and 26.1), and where a tile is
// soon done, so that the epilogue counts and a pair's 256 columns stay empty (96 experts, 3722 tokens, 608 x 240: 11.8
// us, pairs 15.4; 64, 4000, 4096 x 1024: 55 and 60; 64, 6000, 1024 x 1024: 22.9 and 26.2; 802 x 12944 x 128: 15.7 and
// 16.3); else pairs (1024 x 4096 x 4096: 18.2 us, tiles of 128 25.1; 64, 4000, 4096 x 2048: 96.2 and 97.5; 256 x 16384 x
// 1024: 11.4 and 11.8)
int launch_product(fp_ctx* c, MiArgs& a, const MiOperand& w, const MiOperand& x, int64_t rows, cudaStream_t st) {
    const int64_t mt = (a.M + MI_BM - 1) / MI_BM, nk = (a.K + MI_BK - 1) / MI_BK;
    a.nk = (int32_t)nk;
    const int64_t tt = mi_token_tiles(a, 128), narrow = mi_token_tiles(a, 32);
    const int split = mi_split<128>(c, tt * mt, nk), nsplit = mi_split<32>(c, narrow * mt, nk);
    const bool fits = narrow * mt <= c->num_sms;
    if (rows <= 32 || (fits && (nk <= 16 || 20 * ((nk + nsplit - 1) / nsplit) <= 32 * ((nk + split - 1) / split))))
        return nsplit > 1 ? launch_mi<32, true, false>(c, a, w, x, narrow, nsplit, st)
                          : launch_mi<32, false, false>(c, a, w, x, narrow, 1, st);
    if (tt * mt <= c->num_sms || nk <= 4 || (nk < 12 && rows < 256)) {
        return split > 1 ? launch_mi<128, true, false>(c, a, w, x, tt, split, st)
                         : launch_mi<128, false, false>(c, a, w, x, tt, 1, st);
    }
    return launch_mi<256, false, true>(c, a, w, x, mi_token_tiles(a, 256), 1, st);
}

}  // namespace

int fp_matmul_i8(fp_ctx* c, const int8_t* w, int64_t ldw, const float* w_scale, int E, int64_t M, int64_t K,
                 const int8_t* x, int64_t ldx, const float* x_scale, int64_t N, const int32_t* offsets, void* y,
                 int y_type, int64_t ldy, void* stream) {
    const int ys = fp_type_size(y_type);
    if (!ys) return fp_fail(c, FP_ERR_ARG, "fp_matmul_i8: y_type must be FP_F32, FP_F16 or FP_BF16");
    if (M < 1 || M > (1ll << 24) || N < 0 || N > (1ll << 24) || K < 1 || K > 131071 || E < 1 || E > 4096 ||
        E * M > 0x7fffff00ll)
        return fp_fail(c, FP_ERR_SHAPE,
                       "fp_matmul_i8: M outside [1, 2^24], N outside [0, 2^24], K outside [1, 2^17) or E outside [1, 4096]");
    if (E > 1 && !offsets) return fp_fail(c, FP_ERR_ARG, "fp_matmul_i8: several experts need offsets");
    if ((E * M > 1 && ldw < K) || (N > 1 && (ldx < K || ldy < M)))
        return fp_fail(c, FP_ERR_SHAPE, "fp_matmul_i8: a row pitch below the row");
    const bool empty = N == 0;
    if (!empty && (!w || !w_scale || !x || !x_scale || !y)) return fp_fail(c, FP_ERR_ARG, "fp_matmul_i8: null argument");
    if (((uintptr_t)w_scale | (uintptr_t)x_scale | (uintptr_t)offsets) % 4 || (uintptr_t)y % ys)
        return fp_fail(c, FP_ERR_ARG, "fp_matmul_i8: an address is not a multiple of its element size");
    if (!c) return FP_ERR_ARG;
    if (int rc = fp_op_pending(c, "fp_matmul_i8")) return rc;
    if (empty) return FP_OK;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_matmul_i8");
    cudaStream_t st = (cudaStream_t)stream;
    if (N == 1) ldx = (K + 15) & ~15ll, ldy = M;  // a single row has no pitch: one that keeps its alignment
    if (E * M == 1) ldw = (K + 15) & ~15ll;
    // rows of a group: N of a dense product, twice the mean of those that can have rows by expert
    const int64_t rows = E == 1 ? N : 2 * ((N + std::min<int64_t>(E, N) - 1) / std::min<int64_t>(E, N));
    MiOperand ow{w, ldw, E * M}, ox{x, ldx, N};
    const int classes = mi_classes(ow, E, M, N, rows);
    MiScratch scratch(st);
    int rc = mi_realign(c, ow, ox, (int)K, E > 1 ? offsets : nullptr, (int)M, classes, scratch);
    if (rc) return rc;
    MiClassArgs a = {};
    a.w_scale = w_scale, a.x_scale = x_scale, a.offsets = offsets, a.y = y, a.ldy = ldy;
    a.M = (int32_t)M, a.K = (int32_t)K, a.N = (int32_t)N, a.E = E, a.y_type = y_type;
    a.yvec = (M * ys) % 16 == 0 && fp_common_align({(uint64_t)(uintptr_t)y, (uint64_t)ldy * ys}) == 16;
    a.err = &c->mb_dev->op_err;
    a.classes = classes;
    int slot;
    fp_op_tic(c, st, K_MATMUL_I8, (double)std::min<int64_t>(E, N) * M * K + (double)N * (K + ys * (double)M), &slot);
    if (classes) {
        a.nk = (int32_t)((K + 15 + MI_BK - 1) / MI_BK);
        rc = launch_mi<128, false, false, true>(c, a, ow, ox, mi_token_tiles(a, 128), 1, st);
    } else {
        rc = launch_product(c, a, ow, ox, rows, st);
    }
    fp_toc(c, st, slot);
    return rc;
}

int fp_ops_status(fp_ctx* c) { return c ? fp_op_pending(c, "fp_ops_status") : FP_ERR_ARG; }

int fp_ops_trim(fp_ctx* c) {
    if (!c) return FP_ERR_ARG;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_ops_trim");
    if (c->pool) FP_CUDA(c, cudaMemPoolTrimTo(c->pool, 0));
    return FP_OK;
}

int fp_ops_selftest(fp_ctx* c, void* stream) {
    if (!c) return FP_ERR_ARG;
    if (int rc = fp_op_pending(c, "fp_ops_selftest")) return rc;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_ops_selftest");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(64);
    cfg.stream = (cudaStream_t)stream;
    FP_CUDA(c, cudaLaunchKernelEx(&cfg, wait_selftest_kernel, (volatile uint64_t*)&c->mb_dev->op_err, 1u << 10));
    return FP_OK;
}
