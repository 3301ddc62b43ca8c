// Tokens to their experts and back: fp_moe_sort, fp_moe_dispatch, fp_moe_combine, fp_moe_combine_grad.
//
// A layer of E experts takes every token's k choices e[t][j]. Choice i = t k + j has the row
//   pos_i = #{i' : e_i' < e_i} + #{i' < i : e_i' = e_i}
// among the experts' inputs: the experts one after the other, each one's rows in the order of the
// choices (with k = 1 the order of the dispatch statement). The rows go out with
//   rows[pos[t][j]] = x[t]                                  (dispatch)
// and come back with
//   out[t] = base[t] + sum_j weights[t][j] rows[pos[t][j]]  (combine).
// The gradients are the same movements: a dispatched row's back to its token is a combine without
// weights, a combine's are d rows[pos[t][j]] = weights[t][j] dout[t] and
// d weights[t][j] = <dout[t], rows[pos[t][j]]>. Every one of them goes by tokens: a token's k rows are
// read or written by the threads that own the token, so sums have one order and nothing is atomic.
#include <cooperative_groups.h>

#include <algorithm>

#include "fp_ops.cuh"

namespace cg = cooperative_groups;

namespace {

// ---- sort -----------------------------------------------------------------------------------
//
// One thread-block cluster ranks all choices. Warp w of the cluster takes a run of consecutive
// choices and ranks them by expert against a histogram of its own in shared memory: the lanes that hold the
// same expert are found by match.any and take the ranks after the histogram's count in the order of the
// lanes, so the sort is stable. The histograms' prefix sums (over a block's warps, then over the cluster's
// blocks through distributed shared memory, then over the experts) give every warp its first row of each
// expert, which a second pass over the run adds to the ranks. Bound by latency: 8 choices take 2.9 us, 16382
// of 128 experts 7.6, 65536 15 (0.5 MB, 0.1 us of memory traffic; a launch alone is about 2 us). No block waits
// for another but at the cluster's barriers, and nothing is kept in memory between calls.
constexpr int MS_HIST_BYTES = 176 * 1024;
constexpr int MS_MAX_CLUSTER = 8;

constexpr int MS_KEEP = 8;  // choices of a lane that stay in registers between the passes (of longer runs, ranks in pos)

__global__ void __launch_bounds__(1024)
    moe_sort_kernel(const int32_t* __restrict__ e, int64_t n, int E, int warps, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ pos) {
    cg::cluster_group cl = cg::this_cluster();
    unsigned block = cl.block_rank();
    fp_begin(block);
    const int C = (int)cl.num_blocks(), rank = (int)block;
    extern __shared__ int32_t ms_smem[];
    int32_t* hist = ms_smem;             // warps x E
    int32_t* tot = hist + warps * E;     // this block's choices of every expert (read by the cluster)
    int32_t* first = tot + E;            // first row of every expert for this block
    __shared__ int32_t wsum[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nthr = blockDim.x;

    // this warp's run of choices, a multiple of 32
    const int64_t run = ((n + (int64_t)C * warps - 1) / ((int64_t)C * warps) + 31) / 32 * 32;
    const int64_t lo = warp < warps ? min(n, ((int64_t)rank * warps + warp) * run) : n, hi = min(n, lo + run);
    const bool kept = run <= 32 * MS_KEEP;
    int32_t keep[MS_KEEP], rank_in[MS_KEEP];  // the experts (-1: none) and the ranks among the run's of an expert
    auto fetch = [&](int64_t i) {
#pragma unroll
        for (int v = 0; v < MS_KEEP; v++) {
            const int64_t at = i + 32 * v + lane;
            keep[v] = at < hi ? __ldg(e + at) : -1;
            if (keep[v] >= E) keep[v] = -1;
        }
    };
    if (kept) fetch(lo);
    for (int i = tid; i < warps * E; i += nthr) hist[i] = 0;
    __syncthreads();
    int32_t* mine = hist + warp * E;
    for (int64_t i = lo; i < hi; i += 32 * MS_KEEP) {
        if (!kept) fetch(i);
#pragma unroll
        for (int v = 0; v < MS_KEEP; v++) {
            if (i + 32 * v >= hi) break;
            // the choice's rank among the run's of its expert
            const int32_t x = keep[v];
            const uint32_t same = __match_any_sync(0xffffffffu, x);
            int32_t r = 0;
            if (x >= 0) r = mine[x] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (x >= 0 && lane == __ffs(same) - 1) mine[x] = r + __popc(same);
            __syncwarp();
            if (kept)
                rank_in[v] = r;
            else if (i + 32 * v + lane < hi)
                pos[i + 32 * v + lane] = r;
        }
    }
    __syncthreads();
    for (int x = tid; x < E; x += nthr) {
        int32_t s = 0;
#pragma unroll 8
        for (int w = 0; w < warps; w++) {
            const int32_t h = hist[w * E + x];
            hist[w * E + x] = s;
            s += h;
        }
        tot[x] = s;
    }
    if (C > 1)
        cl.sync();
    else
        __syncthreads();
    // experts in runs of `per` for every thread: the cluster's total of each, and its share below this block
    const int per = (E + nthr - 1) / nthr, x0 = min(E, tid * per), x1 = min(E, x0 + per);
    int32_t sum = 0;
    for (int x = x0; x < x1; x++) {
        int32_t below = 0, all = 0, v[MS_MAX_CLUSTER];
#pragma unroll
        for (int b = 0; b < MS_MAX_CLUSTER; b++) v[b] = b < C ? cl.map_shared_rank(tot, b)[x] : 0;
#pragma unroll
        for (int b = 0; b < MS_MAX_CLUSTER; b++) {
            all += v[b];
            below += b < rank ? v[b] : 0;
        }
        first[x] = sum + below;
        sum += all;
        if (rank == 0) offsets[x + 1] = sum;  // within the thread's run; the runs before it are added below
    }
    int32_t inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int32_t before = inc - sum;
    for (int w = 0; w < warp; w++) before += wsum[w];
    for (int x = x0; x < x1; x++) {
        first[x] += before;
        if (rank == 0) offsets[x + 1] += before;
    }
    if (rank == 0 && tid == 0) offsets[0] = 0;
    // every block has read the others' counts; `first` is complete
    if (C > 1)
        cl.sync();
    else
        __syncthreads();
    for (int64_t i = lo; i < hi; i += 32 * MS_KEEP) {
        if (!kept) fetch(i);
#pragma unroll
        for (int v = 0; v < MS_KEEP; v++) {
            if (i + 32 * v >= hi) break;
            const int64_t at = i + 32 * v + lane;
            const int32_t x = keep[v];
            if (at < hi) pos[at] = x < 0 ? -1 : first[x] + mine[x] + (kept ? rank_in[v] : pos[at]);
        }
    }
}

// ---- dispatch -------------------------------------------------------------------------------

constexpr int MO_CHOICES = 4;  // positions (and weights) of a token kept in registers at a time

// Bound by HBM: 8192 x 5120 bf16 to two rows each, 252 MB, takes 41.7 us, 6.0 TB/s (a plain copy here: 6.4).
// A token's row is read once and written k times, so nothing but the positions is read twice.
//
// rows[pos[t][j]] = x[t] in units of A bytes; one token per tpr threads, blockIdx.y a share of the columns. U
// loads of a thread are in flight before its stores.
template <int A, int U>
__global__ void __launch_bounds__(FP_ROW_THREADS)
    moe_dispatch_kernel(const char* __restrict__ x, int64_t T, int nvec, int64_t ldx, const int32_t* __restrict__ pos,
                        int k, int64_t R, char* __restrict__ rows, int64_t ldr, int tpr) {
    unsigned block = blockIdx.x;
    fp_begin(block);
    const int64_t t = (int64_t)block * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (t >= T) return;
    const char* src = x + t * ldx;
    const int step = tpr * gridDim.y;
    for (int c = threadIdx.x % tpr + tpr * blockIdx.y; c < nvec; c += U * step) {
        FpWords<A> v[U];
#pragma unroll
        for (int u = 0; u < U; u++)
            if (c + u * step < nvec) v[u].load(src + (int64_t)(c + u * step) * A);
        for (int j0 = 0; j0 < k; j0 += MO_CHOICES) {
            char* dst[MO_CHOICES];
#pragma unroll
            for (int j = 0; j < MO_CHOICES; j++) {
                const int64_t p = j0 + j < k ? __ldg(pos + t * k + j0 + j) : -1;
                dst[j] = p >= 0 && p < R ? rows + p * ldr : nullptr;
            }
#pragma unroll
            for (int j = 0; j < MO_CHOICES; j++) {
                if (!dst[j]) continue;
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (c + u * step < nvec) v[u].store(dst[j] + (int64_t)(c + u * step) * A);
            }
        }
    }
}

// The same for rows of any bytes and pitch: 16 bytes at a time from the first multiple of 16 in each destination's
// row, x shifted to it (and read for every choice, from L1 after the first), the bytes before and behind one by one.
// blockIdx.z: a share of the choices. 8192 rows of 5121 bf16 to two rows each, 252 MB, take 48 us, 5.2 TB/s.
__global__ void __launch_bounds__(FP_ROW_THREADS)
    moe_dispatch_any_kernel(const uint8_t* __restrict__ x, int64_t T, int64_t bytes, int64_t ldx,
                            const int32_t* __restrict__ pos, int k, int64_t R, uint8_t* __restrict__ rows, int64_t ldr, int tpr) {
    unsigned block = blockIdx.x;
    fp_begin(block);
    const int64_t t = (int64_t)block * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (t >= T) return;
    const uint8_t* src = x + t * ldx;
    const FpSpan span = fp_span(x, T, ldx, bytes);
    const int step = tpr * gridDim.y, at = threadIdx.x % tpr;
    for (int j = blockIdx.z; j < k; j += gridDim.z) {
        const int64_t p = __ldg(pos + t * k + j);
        if (p < 0 || p >= R) continue;
        uint8_t* dst = rows + p * ldr;
        const int head = (int)min((int64_t)(-reinterpret_cast<uintptr_t>(dst) & 15), bytes);
        const int nvec = (int)((bytes - head) / 16);
        if (blockIdx.y == 0) {
            const int tail = (int)(bytes - head) & 15;
            if (at < head) dst[at] = src[at];
            if (at < tail) dst[bytes - tail + at] = src[bytes - tail + at];
        }
        const FpRow<uint8_t, 16, true> from(src + head, span);
        constexpr int U = 1;  // (2: 53 us)
        for (int c = at + tpr * blockIdx.y; c < nvec; c += U * step) {
            FpVec<uint8_t, 16> v[U];
            bool ok = true;
#pragma unroll
            for (int u = 0; u < U; u++)
                if (c + u * step < nvec) ok &= from.load(v[u], c + u * step);
            if (!ok) {
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (c + u * step < nvec) from.slow(v[u], c + u * step);
            }
#pragma unroll
            for (int u = 0; u < U; u++)
                if (c + u * step < nvec) v[u].store(dst + head + (int64_t)(c + u * step) * 16);
        }
    }
}

template <int A>
cudaError_t launch_dispatch(const fp_ctx* c, const void* x, int64_t T, int64_t bytes, int64_t ldx, const int32_t* pos, int k,
                     int64_t R, void* rows, int64_t ldr, cudaStream_t st) {
    const int nvec = (int)(bytes / A);
    constexpr int U = A == 16 ? 2 : 4;
    const FpRowGrid g = fp_row_grid(c, T, nvec, U, true);
    return fp_launch(moe_dispatch_kernel<A, U>, dim3(g.gx, g.gy), g.threads(), 0, st, (const char*)x, T, nvec, ldx, pos, k, R,
                     (char*)rows, ldr, g.tpr);
}

// ---- combine --------------------------------------------------------------------------------

// Bound by HBM: 8192 x 5120 bf16, k = 2, 252 MB, takes 43.3 us, 5.8 TB/s (k = 1: 35 us, 4.8: a block waits for its
// position before its one load a thread); fp32 rows of the odd width 4099, k = 2, 403 MB, 74 us, 5.4 TB/s.
//
// out[t] = base[t] + sum_j w[t][j] rows[pos[t][j]] in fp32, rounded once; V elements per load, U vectors
// of a thread at a time
template <typename RT, typename OT, int V, int U>
__global__ void __launch_bounds__(FP_ROW_THREADS)
    moe_combine_kernel(const RT* __restrict__ rows, int64_t R, int64_t ldr, const int32_t* __restrict__ pos,
                       const float* __restrict__ w, const OT* base, int64_t ldb, int64_t T, int k, int nvec, OT* out,
                       int64_t ldo, int tpr) {
    unsigned block = blockIdx.x;
    fp_begin(block);
    const int64_t t = (int64_t)block * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (t >= T) return;
    const int step = tpr * gridDim.y;
    for (int c = threadIdx.x % tpr + tpr * blockIdx.y; c < nvec; c += U * step) {
        float acc[U][V];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const bool in = base && c + u * step < nvec;
            FpVec<OT, V> b;
            if (in) b.load(base + t * ldb + (int64_t)(c + u * step) * V);
#pragma unroll
            for (int i = 0; i < V; i++) acc[u][i] = in ? b.get(i) : 0.0f;
        }
        // the loads of two choices at a time, then their sums in the order of the choices
        for (int j0 = 0; j0 < k; j0 += 2) {
            const RT* src[2];
            float s[2];
            FpVec<RT, V> v[2][U];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int64_t p = j0 + j < k ? __ldg(pos + t * k + j0 + j) : -1;
                src[j] = p >= 0 && p < R ? rows + p * ldr : nullptr;
                s[j] = w && j0 + j < k ? __ldg(w + t * k + j0 + j) : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (src[j] && c + u * step < nvec) v[j][u].load(src[j] + (int64_t)(c + u * step) * V);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                if (!src[j]) continue;
#pragma unroll
                for (int u = 0; u < U; u++)
#pragma unroll
                    for (int i = 0; i < V; i++) acc[u][i] = fmaf(s[j], v[j][u].get(i), acc[u][i]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (c + u * step >= nvec) break;
            FpVec<OT, V> o;
            o.set(acc[u]);
            o.store(out + t * ldo + (int64_t)(c + u * step) * V);
        }
    }
}

// The same for rows of 16 bits and any width, address and pitch: V elements at a time from the first multiple of 16 bytes
// in each output row, the rows and base shifted to it; the elements before and behind them one by one.
template <typename RT, typename OT, int V>
__global__ void __launch_bounds__(FP_ROW_THREADS)
    moe_combine_odd_kernel(const RT* __restrict__ rows, int64_t R, int64_t ldr, const int32_t* __restrict__ pos,
                           const float* __restrict__ w, const OT* base, int64_t ldb, int64_t T, int k, int M, OT* out,
                           int64_t ldo, int tpr) {
    unsigned block = blockIdx.x;
    fp_begin(block);
    const int64_t t = (int64_t)block * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (t >= T) return;
    const int step = tpr * gridDim.y, at = threadIdx.x % tpr;
    OT* o = out + t * ldo;
    const int head = min((int)((-reinterpret_cast<uintptr_t>(o) & 15) / sizeof(OT)), M), nvec = (M - head) / V;
    const FpSpan span = fp_span(rows, R, ldr, M);
    const int rest = M - nvec * V;  // head and tail
    if (blockIdx.y == 0 && at < rest) {
        const int c = at < head ? at : M - rest + at;
        float acc = base ? fp_to_f(base[t * ldb + c]) : 0.0f;
        for (int j = 0; j < k; j++) {
            const int64_t p = __ldg(pos + t * k + j);
            if (p >= 0 && p < R) acc = fmaf(w ? __ldg(w + t * k + j) : 1.0f, fp_to_f(rows[p * ldr + c]), acc);
        }
        o[c] = fp_from_f<OT>(acc);
    }
    for (int c = at + tpr * blockIdx.y; c < nvec; c += step) {
        float acc[V];
        FpVec<OT, V> b;
        if (base) b = FpRow<OT, V, true>(base + t * ldb + head, fp_span(base, T, ldb, M)).get(c);
#pragma unroll
        for (int i = 0; i < V; i++) acc[i] = base ? b.get(i) : 0.0f;
        // the loads of two choices at a time, then their sums in the order of the choices
        for (int j0 = 0; j0 < k; j0 += 2) {
            bool has[2], ok = true;
            FpRow<RT, V, true> src[2];
            FpVec<RT, V> v[2];
            float s[2];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int64_t p = j0 + j < k ? __ldg(pos + t * k + j0 + j) : -1;
                has[j] = p >= 0 && p < R;
                src[j] = FpRow<RT, V, true>(rows + (has[j] ? p : 0) * ldr + head, span);
                s[j] = w && j0 + j < k ? __ldg(w + t * k + j0 + j) : 1.0f;
                if (has[j]) ok &= src[j].load(v[j], c);
            }
            if (!ok) {
#pragma unroll
                for (int j = 0; j < 2; j++)
                    if (has[j]) src[j].slow(v[j], c);
            }
#pragma unroll
            for (int j = 0; j < 2; j++) {
                if (!has[j]) continue;
#pragma unroll
                for (int i = 0; i < V; i++) acc[i] = fmaf(s[j], v[j].get(i), acc[i]);
            }
        }
        FpVec<OT, V> r;
        r.set(acc);
        r.store(o + head + (int64_t)c * V);
    }
}

// ---- gradients of combine -------------------------------------------------------------------

constexpr int MO_GRAD_THREADS = 512;

// Bound by HBM: 8192 x 5120 bf16, k = 2, 420 MB, takes 68 us, 6.2 TB/s.
//
// One token per tpr threads: its k rows' gradients and the k inner products (fp32, a fixed order: a
// thread's columns, its warp's tree, then the warps). Two choices at a time read dout once; blockIdx.y a
// share of the choices.
template <typename RT, typename OT, int V, int U, bool ANY>
__global__ void __launch_bounds__(MO_GRAD_THREADS)
    moe_grad_kernel(const OT* __restrict__ dout, int64_t ldd, const RT* __restrict__ rows, int64_t R, int64_t ldr,
                    const int32_t* __restrict__ pos, const float* __restrict__ w, int64_t T, int k, int nvec,
                    RT* __restrict__ drows, int64_t lddr, float* __restrict__ dw, int tpr, bool dvec) {
    unsigned block = blockIdx.x;
    fp_begin(block);
    __shared__ float red[2][32];
    const int sub = threadIdx.x / tpr, tt = threadIdx.x % tpr, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)block * (blockDim.x / tpr) + sub;
    const bool live = t < T;
    const FpRow<OT, V, ANY> g(dout + (live ? t : 0) * ldd, fp_span(dout, T, ldd, (int64_t)nvec * V));
    const FpSpan rspan = fp_span(rows, R, ldr, (int64_t)nvec * V);
    for (int j0 = 2 * blockIdx.y; j0 < k; j0 += 2 * gridDim.y) {
        int64_t p[2];
        float s[2], dot[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 2; j++) {
            p[j] = live && j0 + j < k ? __ldg(pos + t * k + j0 + j) : -1;
            if (p[j] >= R) p[j] = -1;
            s[j] = w && live && j0 + j < k ? __ldg(w + t * k + j0 + j) : 1.0f;
        }
        for (int c = tt; c < nvec && (p[0] >= 0 || p[1] >= 0); c += U * tpr) {
            FpVec<OT, V> gv[U];
            FpVec<RT, V> v[2][U];
#pragma unroll
            for (int u = 0; u < U; u++)
                if (c + u * tpr < nvec) gv[u] = g.get(c + u * tpr);
            if (dw) {
#pragma unroll
                for (int j = 0; j < 2; j++)
#pragma unroll
                    for (int u = 0; u < U; u++)
                        if (p[j] >= 0 && c + u * tpr < nvec)
                            v[j][u] = FpRow<RT, V, ANY>(rows + p[j] * ldr, rspan).get(c + u * tpr);
            }
#pragma unroll
            for (int j = 0; j < 2; j++) {
                if (p[j] < 0) continue;
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if (c + u * tpr >= nvec) break;
                    if (dw) {
#pragma unroll
                        for (int i = 0; i < V; i++) dot[j] = fmaf(gv[u].get(i), v[j][u].get(i), dot[j]);
                    }
                    if (drows) {
                        float f[V];
#pragma unroll
                        for (int i = 0; i < V; i++) f[i] = s[j] * gv[u].get(i);
                        FpVec<RT, V> o;
                        o.set(f);
                        RT* d = drows + p[j] * lddr + (int64_t)(c + u * tpr) * V;
                        if (!ANY || dvec) {
                            o.store(d);
                        } else {
#pragma unroll
                            for (int i = 0; i < V; i++) d[i] = fp_from_f<RT>(f[i]);
                        }
                    }
                }
            }
        }
        if (dw) {
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], m);
            float sum = lane ? dot[1] : dot[0];
            if (tpr > 32) {
                if (j0 > 2 * (int)blockIdx.y) __syncthreads();  // red may still be read for the choices before
                if (lane < 2) red[lane][warp] = sum;
                __syncthreads();
                if (tt < 2) {
                    sum = 0.0f;
                    for (int i = 0; i < tpr >> 5; i++) sum += red[tt][sub * (tpr >> 5) + i];
                }
            }
            // 0 where there is no row: nothing was added
            if (live && tt < 2 && j0 + tt < k) dw[t * k + j0 + tt] = sum;
        }
    }
}

// The same for any width, address and pitch, a choice at a time: the inner product in the order of the kernel above, both
// rows shifted to their first values, then the gradient's row from dout once more (from L1), V elements at a time from the
// row's first multiple of 16 bytes.
template <typename RT, typename OT, int V>
__global__ void __launch_bounds__(MO_GRAD_THREADS)
    moe_grad_odd_kernel(const OT* __restrict__ dout, int64_t ldd, const RT* __restrict__ rows, int64_t R, int64_t ldr,
                        const int32_t* __restrict__ pos, const float* __restrict__ w, int64_t T, int k, int M,
                        RT* __restrict__ drows, int64_t lddr, float* __restrict__ dw, int tpr) {
    unsigned block = blockIdx.x;
    fp_begin(block);
    __shared__ float red[32];
    const int sub = threadIdx.x / tpr, tt = threadIdx.x % tpr, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)block * (blockDim.x / tpr) + sub;
    const bool live = t < T;
    const OT* g = dout + (live ? t : 0) * ldd;
    const FpSpan gspan = fp_span(dout, T, ldd, M), rspan = fp_span(rows, R, ldr, M);
    for (int j = blockIdx.y; j < k; j += gridDim.y) {
        const int64_t p = live ? __ldg(pos + t * k + j) : -1;
        const bool has = p >= 0 && p < R;
        if (dw) {
            float dot = 0.0f;
            if (has) {
                const RT* r = rows + p * ldr;
                const FpRow<OT, V, true> gv(g, gspan);
                const FpRow<RT, V, true> rv(r, rspan);
                const int nvec = M / V, rest = M % V;
                for (int c = tt; c < nvec; c += tpr) {
                    FpVec<OT, V> x;
                    FpVec<RT, V> y;
                    const bool gok = gv.load(x, c), rok = rv.load(y, c);
                    if (!gok) gv.slow(x, c);
                    if (!rok) rv.slow(y, c);
#pragma unroll
                    for (int i = 0; i < V; i++) dot = fmaf(x.get(i), y.get(i), dot);
                }
                if (tt < rest) dot = fmaf(fp_to_f(g[nvec * V + tt]), fp_to_f(r[nvec * V + tt]), dot);
            }
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
            if (tpr > 32) {
                if (j > (int)blockIdx.y) __syncthreads();  // red may still be read for the choice before
                if (lane == 0) red[warp] = dot;
                __syncthreads();
                if (tt == 0) {
                    dot = 0.0f;
                    for (int i = 0; i < tpr >> 5; i++) dot += red[sub * (tpr >> 5) + i];
                }
            }
            if (live && tt == 0) dw[t * k + j] = dot;
        }
        if (drows && has) {
            const float s = w ? __ldg(w + t * k + j) : 1.0f;
            RT* d = drows + p * lddr;
            const int head = min((int)((-reinterpret_cast<uintptr_t>(d) & 15) / sizeof(RT)), M), nvec = (M - head) / V;
            const int rest = M - nvec * V;  // head and tail
            if (tt < rest) {
                const int c = tt < head ? tt : M - rest + tt;
                d[c] = fp_from_f<RT>(s * fp_to_f(g[c]));
            }
            const FpRow<OT, V, true> gv(g + head, gspan);
            for (int c = tt; c < nvec; c += tpr) {
                const FpVec<OT, V> x = gv.get(c);
                float f[V];
#pragma unroll
                for (int i = 0; i < V; i++) f[i] = s * x.get(i);
                FpVec<RT, V> o;
                o.set(f);
                o.store(d + head + (int64_t)c * V);
            }
        }
    }
}

template <typename F>
void by_type(int type, F&& f) {
    if (type == FP_F32)
        f((float*)nullptr);
    else if (type == FP_F16)
        f((__half*)nullptr);
    else
        f((__nv_bfloat16*)nullptr);
}

// positions: T x k of them, rows 0 .. R - 1. The kernels step over a token's choices, several at a time, in 32 bits: up to
// 2^30 of them, so that no step passes 2^31.
int check_positions(fp_ctx* c, const char* what, int64_t T, int k, int64_t R) {
    if (T < 0 || T > (1ll << 24) || R < 0 || R > 0x7fffffffll)
        return fp_fail(c, FP_ERR_SHAPE, std::string(what) + ": T outside [0, 2^24] or R outside [0, 2^31)");
    if (k < 1 || k > (1 << 30) || T * k > 0x7fffffffll)
        return fp_fail(c, FP_ERR_SHAPE, std::string(what) + ": k outside [1, 2^30] or T k above 2^31 - 1");
    return FP_OK;
}

}  // namespace

int fp_moe_sort(fp_ctx* c, const int32_t* e, int64_t n, int E, int32_t* offsets, int32_t* pos, void* stream) {
    if (n < 0 || n > 0x7fffffffll || E < 1 || E > 4096)
        return fp_fail(c, FP_ERR_SHAPE, "fp_moe_sort: n outside [0, 2^31) or E outside [1, 4096]");
    if (!offsets || (n && (!e || !pos))) return fp_fail(c, FP_ERR_ARG, "fp_moe_sort: null argument");
    if (((uintptr_t)e | (uintptr_t)offsets | (uintptr_t)pos) % 4)
        return fp_fail(c, FP_ERR_ARG, "fp_moe_sort: an address is not a multiple of its element size");
    if (!c) return FP_ERR_ARG;
    if (int rc = fp_op_pending(c, "fp_moe_sort")) return rc;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_moe_sort");
    cudaStream_t st = (cudaStream_t)stream;
    // One block below 1024 choices, a cluster of eight from there (1024 choices of 128 experts: 4.9 and 4.4 us;
    // 256: 3.7 and 4.1). A block's warps cost time in the sums over them, their rounds of 32 choices in the
    // ranking: about sqrt(2 rounds) warps (8192 choices: 4, 8, 16, 32 warps take 6.9, 5.6, 5.7, 6.7 us), more
    // where that keeps the choices in registers.
    const int64_t rounds = std::max<int64_t>(1, (n + 31) / 32);
    const int most = (int)std::min<int64_t>(32, MS_HIST_BYTES / (4 * (int64_t)E));
    const int blocks = rounds >= 32 ? MS_MAX_CLUSTER : 1;
    const int64_t per = (rounds + blocks - 1) / blocks;
    int warps = 1;
    while (warps < most && ((int64_t)warps * warps < 2 * per || (int64_t)warps * MS_KEEP < per)) warps++;
    const int threads = std::max(32 * warps, 128);
    const size_t smem = sizeof(int32_t) * ((size_t)warps * E + 2 * (size_t)E);
    FP_CUDA(c, fp_op_smem(c, 0, moe_sort_kernel, MS_HIST_BYTES + 8 * 4096));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];  // (as fp_launch, in a cluster)
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    int slot;
    fp_op_tic(c, st, K_MOE_SORT, 8.0 * (double)n + 4.0 * E, &slot);
    const cudaError_t rc = cudaLaunchKernelEx(&cfg, moe_sort_kernel, e, n, E, warps, offsets, pos);
    fp_toc(c, st, slot);
    FP_CUDA(c, rc);
    return FP_OK;
}

int fp_moe_dispatch(fp_ctx* c, const void* x, int64_t T, int64_t row_bytes, int64_t ldx, const int32_t* pos, int k,
                    int64_t R, void* rows, int64_t ldr, void* stream) {
    int rc = check_positions(c, "fp_moe_dispatch", T, k, R);
    if (rc) return rc;
    if (row_bytes < 1 || row_bytes > (1ll << 24)) return fp_fail(c, FP_ERR_SHAPE, "fp_moe_dispatch: row_bytes outside [1, 2^24]");
    if ((T > 1 && ldx < row_bytes) || (R > 1 && ldr < row_bytes))
        return fp_fail(c, FP_ERR_SHAPE, "fp_moe_dispatch: a row pitch below row_bytes");
    const bool empty = T == 0 || R == 0;
    if (!empty && (!x || !pos || !rows)) return fp_fail(c, FP_ERR_ARG, "fp_moe_dispatch: null argument");
    if ((uintptr_t)pos % 4) return fp_fail(c, FP_ERR_ARG, "fp_moe_dispatch: an address is not a multiple of its element size");
    if (!c) return FP_ERR_ARG;
    if ((rc = fp_op_pending(c, "fp_moe_dispatch"))) return rc;
    if (empty) return FP_OK;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_moe_dispatch");
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 1) ldx = 0;
    if (R == 1) ldr = 0;
    const int al = fp_common_align({(uint64_t)(uintptr_t)x, (uint64_t)(uintptr_t)rows, (uint64_t)ldx, (uint64_t)ldr,
                                    (uint64_t)row_bytes});
    int slot;
    cudaError_t launched;
    fp_op_tic(c, st, K_MOE_DISPATCH, (double)row_bytes * (T + T * (double)k) + 4.0 * T * k, &slot);
    // Units of 1, 2 or 4 bytes against 16 shifted ones, us: 8192 rows of 5121 bytes 65.5 and 20.0, 20000 x 2 of 1030 24.6
    // and 22.5; 8192 x 2 of 10242 66.3 and 48.4, 4787 x 3 of 1344 10.0 and 10.6; 8192 x 2 of 16396 89.7 and 80.6, 20000 x
    // 2 of 1028 16.9 and 22.2; few rows: 8 of 10242 2.2 and 2.5. (Units of 8: 865 x 5 of 20664 24.4 and 30.9.)
    if (al <= 4 && row_bytes >= 1024 * al && T * k * row_bytes >= (1 << 21)) {
        const FpRowGrid g = fp_row_grid(c, T, row_bytes / 16, 1, true);
        const int64_t gz = std::max<int64_t>(1, std::min<int64_t>(k, 4 * (int64_t)c->num_sms / ((int64_t)g.gx * g.gy)));
        launched = fp_launch(moe_dispatch_any_kernel, dim3(g.gx, g.gy, (unsigned)gz), g.threads(), 0, st,
                             (const uint8_t*)x, T, row_bytes, ldx, pos, k, R, (uint8_t*)rows, ldr, g.tpr);
    } else if (al >= 16)
        launched = launch_dispatch<16>(c, x, T, row_bytes, ldx, pos, k, R, rows, ldr, st);
    else if (al >= 8)
        launched = launch_dispatch<8>(c, x, T, row_bytes, ldx, pos, k, R, rows, ldr, st);
    else if (al >= 4)
        launched = launch_dispatch<4>(c, x, T, row_bytes, ldx, pos, k, R, rows, ldr, st);
    else if (al >= 2)
        launched = launch_dispatch<2>(c, x, T, row_bytes, ldx, pos, k, R, rows, ldr, st);
    else
        launched = launch_dispatch<1>(c, x, T, row_bytes, ldx, pos, k, R, rows, ldr, st);
    fp_toc(c, st, slot);
    FP_CUDA(c, launched);
    return FP_OK;
}

int fp_moe_combine(fp_ctx* c, const void* rows, int rows_type, int64_t R, int64_t ldr, const int32_t* pos,
                   const float* weights, const void* base, int64_t ldb, int64_t T, int k, int64_t M, void* out,
                   int out_type, int64_t ldo, void* stream) {
    const int rs = fp_type_size(rows_type), os = fp_type_size(out_type);
    if (!rs || !os) return fp_fail(c, FP_ERR_ARG, "fp_moe_combine: a type is not FP_F32, FP_F16 or FP_BF16");
    int rc = check_positions(c, "fp_moe_combine", T, k, R);
    if (rc) return rc;
    if (M < 1 || M > (1ll << 24)) return fp_fail(c, FP_ERR_SHAPE, "fp_moe_combine: M outside [1, 2^24]");
    if ((R > 1 && ldr < M) || (T > 1 && (ldo < M || (base && ldb < M))))
        return fp_fail(c, FP_ERR_SHAPE, "fp_moe_combine: a row pitch below M");
    const bool empty = T == 0;
    if (!empty && ((!rows && R) || !pos || !out)) return fp_fail(c, FP_ERR_ARG, "fp_moe_combine: null argument");
    if ((uintptr_t)rows % rs || ((uintptr_t)base | (uintptr_t)out) % os || ((uintptr_t)pos | (uintptr_t)weights) % 4)
        return fp_fail(c, FP_ERR_ARG, "fp_moe_combine: an address is not a multiple of its element size");
    if (!c) return FP_ERR_ARG;
    if ((rc = fp_op_pending(c, "fp_moe_combine"))) return rc;
    if (empty) return FP_OK;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_moe_combine");
    cudaStream_t st = (cudaStream_t)stream;
    if (R <= 1) ldr = 0;
    if (T == 1) ldo = ldb = 0;
    if (!base) ldb = 0;
    int slot;
    cudaError_t launched = cudaSuccess;
    fp_op_tic(c, st, K_MOE_COMBINE, (double)M * (rs * (double)T * k + os * (double)T * (base ? 2 : 1)) + 8.0 * T * k, &slot);
    by_type(rows_type, [&](auto* rp) {
        using RT = std::remove_pointer_t<decltype(rp)>;
        by_type(out_type, [&](auto* op) {
            using OT = std::remove_pointer_t<decltype(op)>;
            constexpr int V = 16 / sizeof(RT), OA = V * sizeof(OT) < 16 ? V * sizeof(OT) : 16;
            const bool vec = M % V == 0 && fp_common_align({(uint64_t)(uintptr_t)rows, (uint64_t)ldr * rs}) == 16 &&
                             fp_common_align({(uint64_t)(uintptr_t)base, (uint64_t)ldb * os, (uint64_t)(uintptr_t)out,
                                              (uint64_t)ldo * os}) >= OA;
            // single values against shifted vectors, us, k = 2: 8192 x 4099 bf16 72.1 and 60.5, 20000 x 1201 62.0 and 61.0, 300
            // x 1201 3.5 and 3.9 (fp32: 73.8 and 83.3 at 8192 x 4099)
            const bool odd = !vec && rs == 2 && M >= 2048 && T * M >= 1 << 20;
            const int nvec = (int)(vec || odd ? M / V : M);
            auto run = [&](auto kern, int loads, int width) {
                const FpRowGrid g = fp_row_grid(c, T, nvec, loads, true);
                launched = fp_launch(kern, dim3(g.gx, g.gy), g.threads(), 0, st, (const RT*)rows, R, ldr, pos, weights,
                                     (const OT*)base, ldb, T, k, width, (OT*)out, ldo, g.tpr);
            };
            if constexpr (sizeof(RT) == 2) {
                if (odd) return run(moe_combine_odd_kernel<RT, OT, V>, 1, (int)M);
            }
            if (!vec)
                run(moe_combine_kernel<RT, OT, 1, 4>, 4, nvec);
            else if (k <= 2)  // (8192 x 5120, k = 2: 43.2 and 43.9 us with one vector and two; 1024, k = 8: 22.9 and 19.5)
                run(moe_combine_kernel<RT, OT, V, 1>, 1, nvec);
            else
                run(moe_combine_kernel<RT, OT, V, 2>, 2, nvec);
        });
    });
    fp_toc(c, st, slot);
    FP_CUDA(c, launched);
    return FP_OK;
}

int fp_moe_combine_grad(fp_ctx* c, const void* dout, int out_type, int64_t ldd, const void* rows, int rows_type,
                        int64_t R, int64_t ldr, const int32_t* pos, const float* weights, int64_t T, int k, int64_t M,
                        void* drows, int64_t lddr, float* dweights, void* stream) {
    const int rs = fp_type_size(rows_type), os = fp_type_size(out_type);
    if (!rs || !os) return fp_fail(c, FP_ERR_ARG, "fp_moe_combine_grad: a type is not FP_F32, FP_F16 or FP_BF16");
    int rc = check_positions(c, "fp_moe_combine_grad", T, k, R);
    if (rc) return rc;
    if (M < 1 || M > (1ll << 24)) return fp_fail(c, FP_ERR_SHAPE, "fp_moe_combine_grad: M outside [1, 2^24]");
    if ((R > 1 && ((dweights && ldr < M) || (drows && lddr < M))) || (T > 1 && ldd < M))
        return fp_fail(c, FP_ERR_SHAPE, "fp_moe_combine_grad: a row pitch below M");
    if (!drows && !dweights) return fp_fail(c, FP_ERR_ARG, "fp_moe_combine_grad: no gradient is asked for");
    const bool empty = T == 0;
    if (!empty && (!dout || !pos || (dweights && !rows && R))) return fp_fail(c, FP_ERR_ARG, "fp_moe_combine_grad: null argument");
    if (((uintptr_t)rows | (uintptr_t)drows) % rs || (uintptr_t)dout % os ||
        ((uintptr_t)pos | (uintptr_t)weights | (uintptr_t)dweights) % 4)
        return fp_fail(c, FP_ERR_ARG, "fp_moe_combine_grad: an address is not a multiple of its element size");
    if (!c) return FP_ERR_ARG;
    if ((rc = fp_op_pending(c, "fp_moe_combine_grad"))) return rc;
    if (empty) return FP_OK;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_moe_combine_grad");
    cudaStream_t st = (cudaStream_t)stream;
    if (R <= 1 || !dweights) ldr = 0;
    if (R <= 1 || !drows) lddr = 0;
    if (T == 1) ldd = 0;
    const void* rd = dweights ? rows : nullptr;
    int slot;
    cudaError_t launched = cudaSuccess;
    fp_op_tic(c, st, K_MOE_GRAD,
              (double)M * (os * (double)T + rs * (double)T * k * ((drows ? 1 : 0) + (dweights ? 1 : 0))) + 12.0 * T * k, &slot);
    by_type(rows_type, [&](auto* rp) {
        using RT = std::remove_pointer_t<decltype(rp)>;
        by_type(out_type, [&](auto* op) {
            using OT = std::remove_pointer_t<decltype(op)>;
            constexpr int V = 16 / sizeof(RT), OA = V * sizeof(OT) < 16 ? V * sizeof(OT) : 16;
            // (dweights' order of summation hangs on the sizes: not on what else is asked for, nor on addresses)
            const bool whole = M % V == 0, dvec = fp_common_align({(uint64_t)(uintptr_t)drows, (uint64_t)lddr * rs}) == 16;
            const bool aligned = dvec && fp_common_align({(uint64_t)(uintptr_t)rd, (uint64_t)ldr * rs}) == 16 &&
                                 fp_common_align({(uint64_t)(uintptr_t)dout, (uint64_t)ldd * os}) >= OA;
            // single values against shifted vectors, us, k = 2: 8192 x 4099 bf16 117 and 87, 20000 x 601 72 and 59, 20000 x 301
            // 40.8 and 40.8, 20000 x 100 13 and 20
            const bool odd = !whole && rs == 2 && M >= 300;
            const int nvec = (int)(whole || odd ? M / V : M);
            auto grid = [&](int loads, int choices) {  // choices: of a block at a time
                FpRowGrid g = fp_row_grid(c, T, nvec, loads, false);
                // few tokens: wider blocks, the choices over blocks (211 x 9648 fp32, k = 2: 18.7 us without, 10.4)
                if (g.gx < 4u * c->num_sms) {
                    while (g.tpr < MO_GRAD_THREADS && g.tpr * loads < nvec) g.tpr = std::min(MO_GRAD_THREADS, 2 * g.tpr);
                    g.rpb = std::max(1, FP_ROW_THREADS / g.tpr);
                    g.gx = (unsigned)((T + g.rpb - 1) / g.rpb);
                    g.gy = (unsigned)std::min((k + choices - 1) / choices, 32);
                }
                return g;
            };
            auto run = [&](auto kern, int loads) {
                const FpRowGrid g = grid(loads, 2);
                launched = fp_launch(kern, dim3(g.gx, g.gy), g.threads(), 0, st, (const OT*)dout, ldd, (const RT*)rd, R, ldr, pos,
                                     weights, T, k, nvec, (RT*)drows, lddr, dweights, g.tpr, dvec);
            };
            if constexpr (sizeof(RT) == 2) {
                if (odd) {
                    const FpRowGrid g = grid(1, 1);
                    launched = fp_launch(moe_grad_odd_kernel<RT, OT, V>, dim3(g.gx, g.gy), g.threads(), 0, st,
                                         (const OT*)dout, ldd, (const RT*)rd, R, ldr, pos, weights, T, k, (int)M, (RT*)drows, lddr,
                                         dweights, g.tpr);
                    return;
                }
            }
            if (!whole)
                run(moe_grad_kernel<RT, OT, 1, 4, false>, 4);
            else
                aligned ? run(moe_grad_kernel<RT, OT, V, 1, false>, 1) : run(moe_grad_kernel<RT, OT, V, 1, true>, 1);
        });
    });
    fp_toc(c, st, slot);
    FP_CUDA(c, launched);
    return FP_OK;
}
