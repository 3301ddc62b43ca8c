// fp_quantize_rows: activations to int8 with one scale a token.
//
// a_t = max_j |x_tj|, scale_t = a_t / 127 (fp32), q_tj = the integer nearest to 127 x_tj / a_t, ties to
// the even one, exactly. The kernel multiplies by 127 / a_t, rounded up, in fp32: off by less than 127 * 2^-22.
// A 16-bit value that is not at a half itself is further from one than that: 254 x - (2 n + 1) a_t is a multiple of
// x's last place, so 127 x / a_t differs from n + 1/2 by 2^-12 / 127 of itself at least. At a half, 254 x = (2 n + 1)
// a_t, the prime 127 divides 2 n + 1, so that n = 63 and the quotient rounded up goes to 64 as it has to, or it
// divides a_t: with 8 bits the quotient is then exact, with f16's 11 such rows are done value by value. fp32 values
// within 2^-15 of a half are done one by one too. One by one: 254 |x| against (2 n + 1) a_t, exact in double.
//
// A row with a NaN or an infinity has no scale: its scale is NaN and its integers are 0, so every
// product with it is NaN. A row of zeros has scale 0.
// One read of the row: it stays in registers between the maximum and the integers. 8192 x 5120 bf16 into
// experts' rows, 126 MB, takes 26 us, 4.8 TB/s: ten rows of 10 KB are in flight on an SM (64 registers a thread),
// each for about 4.5 us, and that wait bounds it (fewer registers spill: 31 us at 48).
#include <algorithm>

#include "fp_ops.cuh"

namespace {

constexpr int QR_LOADS = 8;              // vectors of a row that a thread keeps in registers
constexpr float QR_MAGIC = 12582912.0f;  // 1.5 * 2^23: t + it has the nearest integer to t in its low bits
constexpr float QR_NEAR = 0.5f - 3.0517578e-5f;

// what a row's values are divided by: 127 / a, and the row scaled by 2^64 where 127 / a may not be finite
struct QuantRow {
    float inv;            // of the fast quotient; 0 in a row of zeros or with a NaN or an infinity
    float up, a, inv_up;  // 1 or 2^64; a up; 127 / (a up)
    bool bad;             // integers 0
    bool exact;           // every value by quant_exact
};

// x's integer as a float: the nearest to t = 127 x / a unless t lies next to a half, then by 254 |x| - (2 n + 1) a
__device__ __forceinline__ float quant_exact(float x, const QuantRow& row) {
    const float ax = fabsf(x) * row.up, t = ax * row.inv_up, r = (t + QR_MAGIC) - QR_MAGIC;
    float n = r;
    if (fabsf(t - r) > QR_NEAR) {
        n = t > r ? r : r - 1.0f;
        const double d = 254.0 * (double)ax - (double)(2.0f * n + 1.0f) * (double)row.a;
        if (d > 0.0 || (d == 0.0 && ((int)n & 1))) n += 1.0f;
    }
    return copysignf(n, x);
}

// integers as floats to V bytes
template <int V>
__device__ __forceinline__ FpWords<V> quant_pack(float (&n)[V], const QuantRow& row) {
    FpWords<V> o;  // (with QR_MAGIC added, the low byte is the integer)
    if constexpr (V == 1) o.w[0] = row.bad ? 0 : __float_as_uint(n[0]);
#pragma unroll
    for (int i = 0; i < V / 4; i++)
        o.w[i] = row.bad ? 0
                         : __byte_perm(__byte_perm(__float_as_uint(n[4 * i]), __float_as_uint(n[4 * i + 1]), 0x0040),
                                       __byte_perm(__float_as_uint(n[4 * i + 2]), __float_as_uint(n[4 * i + 3]), 0x0040),
                                       0x5410);
    return o;
}

// V values to int8, each by quant_exact
template <typename T, int V>
__device__ __forceinline__ FpWords<V> quant_one_by_one(const FpVec<T, V>& w, const QuantRow& row) {
    float n[V];
#pragma unroll
    for (int e = 0; e < V; e++) n[e] = quant_exact(w.get(e), row) + QR_MAGIC;
    return quant_pack<V>(n, row);
}

// V values to int8 by the fast quotient; near: some lie too close to a half for it
template <typename T, int V>
__device__ __forceinline__ FpWords<V> quant_fast(const FpVec<T, V>& w, const QuantRow& row, bool& near) {
    float n[V], off = 0.0f;
#pragma unroll
    for (int e = 0; e < V; e++) {
        const float t = w.get(e) * row.inv;
        n[e] = t + QR_MAGIC;
        if (sizeof(T) == 4) off = fmaxf(off, fabsf(t - (n[e] - QR_MAGIC)));
    }
    near = off > QR_NEAR;
    return quant_pack<V>(n, row);
}

template <typename T, int V>
__device__ __forceinline__ FpWords<V> quant_vec(const FpVec<T, V>& w, const QuantRow& row) {
    bool near;
    const FpWords<V> o = quant_fast<T, V>(w, row, near);
    return near ? quant_one_by_one<T, V>(w, row) : o;
}

// The largest magnitude of values as bits of T (NaN above infinity above every number), two 16-bit values
// to a word
template <typename T, int V>
__device__ __forceinline__ uint32_t quant_largest(const FpVec<T, V>& w, uint32_t m) {
    constexpr int W = FpVec<T, V>::W;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < W; i++) m = max(m, w.w[i] & 0x7fffffffu);
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 2) m = __vimax3_u16x2(m, w.w[i] & 0x7fff7fffu, W > 1 ? w.w[i + (W > 1)] & 0x7fff7fffu : 0u);
    }
    return m;
}

// The row's largest magnitude from every thread's (`tpr` threads a row) and what it means for its values
template <typename T>
__device__ __forceinline__ QuantRow quant_row(uint32_t m, int sub, int tpr, float& amax) {
    __shared__ uint32_t red[32];
    const int lane = threadIdx.x & 31;
    if (sizeof(T) == 2) m = max(m >> 16, m & 0xffffu);
    m = __reduce_max_sync(0xffffffffu, m);
    if (tpr > 32) {
        if (lane == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        const int w0 = sub * (tpr >> 5), nw = tpr >> 5;
        m = __reduce_max_sync(0xffffffffu, red[w0 + (lane < nw ? lane : 0)]);
    }
    FpVec<T, 1> top;
    top.w[0] = m;
    amax = top.get(0);
    QuantRow r;
    r.bad = !(amax < __uint_as_float(0x7f800000u));  // an infinity or NaN
    const bool tiny = amax < 5.421010862427522e-20f && m != 0;  // 2^-64
    r.up = tiny ? 18446744073709551616.0f : 1.0f;
    r.a = amax * r.up;
    r.inv_up = r.bad || m == 0 ? 0.0f : __fdiv_ru(127.0f, r.a);
    r.inv = tiny ? 0.0f : r.inv_up;
    // f16 rows whose maximum is a multiple of 127 have ties at every half
    r.exact = tiny || (std::is_same_v<T, __half> && m != 0 && ((m & 0x3ffu) | (m >= 0x400u ? 0x400u : 0u)) % 127u == 0);
    return r;
}

__device__ __forceinline__ float quant_scale(const QuantRow& r, float amax) {
    return r.bad ? __uint_as_float(0x7fc00000u) : amax / 127.0f;
}

// One row per `tpr` threads (a multiple of 32 that divides the block). V: elements per load; a thread keeps the first
// NV vectors it reads in registers, and reads what is beyond them a second time. x's address and pitch are multiples of V
// elements, K, q's address and its pitch of V.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(256, 4)
    quant_rows_kernel(const T* __restrict__ x, int64_t rows, int K, int64_t ldx, const int32_t* __restrict__ pos, int k,
                      int64_t R, int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale, int tpr) {
    unsigned block = blockIdx.x;
    fp_begin(block);
    const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const int64_t row = (int64_t)block * (blockDim.x / tpr) + sub;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * ldx;
    const int nvec = live ? K / V : 0;
    const int64_t p0 = !live ? -1 : pos ? __ldg(pos + row * k) : row;
    FpVec<T, V> reg[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (t + i * tpr < nvec) {
            reg[i].load(xr + (t + i * tpr) * V);
        } else {
#pragma unroll
            for (int e = 0; e < FpVec<T, V>::W; e++) reg[i].w[e] = 0;
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) m = quant_largest<T, V>(reg[i], m);
    for (int c = t + NV * tpr; c < nvec; c += tpr) {
        FpVec<T, V> w;
        w.load(xr + c * V);
        m = quant_largest<T, V>(w, m);
    }
    float amax;
    const QuantRow r = quant_row<T>(m, sub, tpr, amax);
    if (!live) return;
    const int copies = pos ? k : 1;
    FpWords<V> o[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) o[i] = quant_vec<T, V>(reg[i], r);
    for (int j = 0; j < copies; j++) {
        const int64_t p = j == 0 ? p0 : __ldg(pos + row * k + j);
        if (p < 0 || p >= R) continue;
        if (t == 0) scale[p] = quant_scale(r, amax);
        if (r.exact) continue;
        int8_t* d = q + p * ldq;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (t + i * tpr < nvec) o[i].store(d + (t + i * tpr) * V);
        constexpr int B = V == 4 ? 4 : 1;
        for (int c = t + NV * tpr; c < nvec; c += B * tpr) {
            FpVec<T, V> w[B];
#pragma unroll
            for (int i = 0; i < B; i++)
                if (c + i * tpr < nvec) w[i].load(xr + (c + i * tpr) * V);
#pragma unroll
            for (int i = 0; i < B; i++)
                if (c + i * tpr < nvec) quant_vec<T, V>(w[i], r).store(d + (c + i * tpr) * V);
        }
    }
    if (!r.exact) return;
    // the rows that are done one by one are read again, once for all copies (801 x 1232 f16, 8 copies: 20.7 us with a
    // pass for each copy, 8.2)
#pragma unroll 1
    for (int c = t; c < nvec; c += tpr) {
        FpVec<T, V> w;
        w.load(xr + c * V);
        const FpWords<V> one = quant_one_by_one<T, V>(w, r);
        for (int j = 0; j < copies; j++) {
            const int64_t p = j == 0 ? p0 : __ldg(pos + row * k + j);
            if (p >= 0 && p < R) one.store(q + p * ldq + c * V);
        }
    }
}

// The same for any K, addresses and pitches. The integers of tpr QR_LOADS vectors at a time go through
// shared memory, from where each copy of the row takes 16 bytes at a time for the multiples of 16 of its addresses,
// shifted, and the bytes before and behind them one by one. 8192 x 4099 bf16 into experts' rows, 101 MB, takes 40 us (61
// by single values), 2.5 TB/s: about 150 instructions for 8 values (shifts, quotients, the reduction's share), the
// waits between the passes, and spills bound it (60 bytes of a thread for bf16, 80 fp32, 136 f16, at the 64 registers
// that four blocks of 256 threads leave it).
template <typename T, int V>
__global__ void __launch_bounds__(256, 4)
    quant_odd_rows_kernel(const T* __restrict__ x, int64_t rows, int K, int64_t ldx, const int32_t* __restrict__ pos,
                          int k, int64_t R, int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale, int tpr) {
    unsigned block = blockIdx.x;
    fp_begin(block);
    extern __shared__ uint4 st[];
    const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const int64_t row = (int64_t)block * (blockDim.x / tpr) + sub;
    const bool live = row < rows;
    const FpRow<T, V, true> src(x + (live ? row : 0) * ldx, fp_span(x, rows, ldx, K));
    const int len = live ? K : 0, nvec = len / V, rest = len % V;  // the last values of a row, one for each of its threads
    FpVec<T, 1> last;
    last.w[0] = 0;
    if (t < rest) last.load(src.p + nvec * V + t);
    FpVec<T, V> reg[QR_LOADS];
    auto fill = [&](int c0) {  // a part's vectors
        bool ok = true;
#pragma unroll
        for (int i = 0; i < QR_LOADS; i++) {
#pragma unroll
            for (int e = 0; e < FpVec<T, V>::W; e++) reg[i].w[e] = 0;
            if (c0 + t + i * tpr < nvec) ok &= src.load(reg[i], c0 + t + i * tpr);
        }
        if (!ok) {
#pragma unroll
            for (int i = 0; i < QR_LOADS; i++)
                if (c0 + t + i * tpr < nvec) src.slow(reg[i], c0 + t + i * tpr);
        }
    };
    const int part = tpr * QR_LOADS;
    uint32_t m = quant_largest<T, 1>(last, 0);
    // the last part first, so that the first one stays in registers
    for (int c0 = max(0, (nvec - 1) / part * part); c0 >= 0; c0 -= part) {
        fill(c0);
#pragma unroll
        for (int i = 0; i < QR_LOADS; i++) m = quant_largest<T, V>(reg[i], m);
    }
    float amax;
    const QuantRow r = quant_row<T>(m, sub, tpr, amax);
    const int copies = !live ? 0 : pos ? k : 1;
    const int fit = part * V / 16 + 1;  // the last part has the row's rest too
    const uint4* from = st + sub * fit;
    uint8_t* mine = reinterpret_cast<uint8_t*>(st + sub * fit);
    for (int c0 = 0; c0 == 0 || c0 < K / V; c0 += part) {
        if (c0 > 0) {
            fill(c0);
            __syncthreads();  // the part before has been written
        }
        uint32_t again = r.exact ? (1u << QR_LOADS) - 1 : 0;  // what is done one by one, from another read
#pragma unroll
        for (int i = 0; i < QR_LOADS; i++) {
            bool near;
            if (t + i * tpr < nvec - c0) quant_fast<T, V>(reg[i], r, near).store(mine + (t + i * tpr) * V);
            if (t + i * tpr < nvec - c0 && near) again |= 1u << i;
        }
#pragma unroll 1
        for (int i = 0; again >> i; i++) {
            const int c = c0 + t + i * tpr;
            if ((again >> i & 1) && c < nvec) quant_one_by_one<T, V>(src.get(c), r).store(mine + (c - c0) * V);
        }
        const bool end = nvec <= c0 + part;
        if (end && t < rest)
            mine[(nvec - c0) * V + t] = (uint8_t)(r.bad ? 0 : (int)quant_exact(last.get(0), r));
        __syncthreads();
        const int n = end ? len - c0 * V : part * V;
        for (int j = 0; j < copies; j++) {
            const int64_t p = pos ? __ldg(pos + row * k + j) : row;
            if (p < 0 || p >= R) continue;
            if (t == 0 && c0 == 0) scale[p] = quant_scale(r, amax);
            int8_t* d = q + p * ldq + c0 * V;
            const int head = min((int)(-reinterpret_cast<uintptr_t>(d) & 15), n);
            const int words = (n - head) / 16, tail = (n - head) & 15;
            if (t < head) d[t] = (int8_t)mine[t];
            if (t < tail) d[n - tail + t] = (int8_t)mine[n - tail + t];
            for (int v = t; v < words; v += tpr) {
                FpWords<16> o;
                fp_shift16(from[v], from[v + 1], head, o.w);
                o.store(d + head + 16 * v);
            }
        }
    }
}

template <typename T>
cudaError_t launch_quant(const fp_ctx* c, const void* x, int64_t T_, int64_t K, int64_t ldx, const int32_t* pos, int k,
                  int64_t R, int8_t* q, int64_t ldq, float* scale, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool plain = K % V == 0 && fp_common_align({(uint64_t)(uintptr_t)q, (uint64_t)ldq}) >= V &&
                       fp_common_align({(uint64_t)(uintptr_t)x, (uint64_t)ldx * sizeof(T)}) == 16;
    // short or few odd rows: a value a thread and load (us, with shared memory: 8000 x 77 bf16, k = 2: 8.9 and 11.2; 4000 x
    // 513 8.0 and 5.5; 119 x 513 f16 3.0 and 3.9; 1240 x 1362 bf16 5.3 and 4.9)
    const bool single = !plain && (K <= 512 || (K <= 4096 && T_ * K <= 1 << 18));
    const int64_t nvec = single ? K : K / V;
    // a few warps hold a row in registers, so that many rows are in flight; few rows: a vector a thread
    int tpr = 32;
    const int loads = single ? 2 * QR_LOADS : QR_LOADS;
    while (tpr < 256 && ((int64_t)tpr * loads < nvec || (T_ * tpr < (int64_t)c->num_sms * 256 && tpr < nvec))) tpr += 32;
    const int threads = std::max(128 / tpr, 1) * tpr;
    const unsigned grid = (unsigned)((T_ + threads / tpr - 1) / (threads / tpr));
    auto run = [&](auto kern, int smem) {
        return fp_launch(kern, grid, threads, smem, st, (const T*)x, T_, (int)K, ldx, pos, k, R, q, ldq, scale, tpr);
    };
    if (plain) return run(quant_rows_kernel<T, V, QR_LOADS>, 0);
    if (single) return run(quant_rows_kernel<T, 1, 2 * QR_LOADS>, 0);
    return run(quant_odd_rows_kernel<T, V>, threads / tpr * (tpr * QR_LOADS * V + 16));
}

}  // namespace

int fp_quantize_rows(fp_ctx* c, const void* x, int x_type, int64_t T, int64_t K, int64_t ldx, const int32_t* pos, int k,
                     int64_t R, int8_t* q, int64_t ldq, float* scale, void* stream) {
    if (!fp_type_size(x_type)) return fp_fail(c, FP_ERR_ARG, "fp_quantize_rows: x_type must be FP_F32, FP_F16 or FP_BF16");
    if (T < 0 || T > (1ll << 24) || K < 1 || K > (1ll << 20) || R < 0 || R > 0x7fffffffll)
        return fp_fail(c, FP_ERR_SHAPE, "fp_quantize_rows: T outside [0, 2^24], K outside [1, 2^20] or R outside [0, 2^31)");
    if (pos ? (k < 1 || T * k > 0x7fffffffll) : R < T)
        return fp_fail(c, FP_ERR_SHAPE, pos ? "fp_quantize_rows: k < 1 or T k above 2^31 - 1" : "fp_quantize_rows: R < T");
    if ((T > 1 && ldx < K) || (R > 1 && ldq < K))
        return fp_fail(c, FP_ERR_SHAPE, "fp_quantize_rows: a row pitch below K");
    const bool empty = T == 0 || R == 0;
    if (!empty && (!x || !q || !scale)) return fp_fail(c, FP_ERR_ARG, "fp_quantize_rows: null argument");
    if ((uintptr_t)x % fp_type_size(x_type) || (uintptr_t)scale % 4 || (uintptr_t)pos % 4)
        return fp_fail(c, FP_ERR_ARG, "fp_quantize_rows: an address is not a multiple of its element size");
    if (!c) return FP_ERR_ARG;
    if (int rc = fp_op_pending(c, "fp_quantize_rows")) return rc;
    if (empty) return FP_OK;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_quantize_rows");
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 1) ldx = 16;  // a single row has no pitch: one that keeps its alignment
    if (R == 1) ldq = 16;
    int slot;
    fp_op_tic(c, st, K_QUANT_ROWS, (double)T * K * fp_type_size(x_type) + (double)(pos ? T * k : T) * (K + 4), &slot);
    const auto launch = x_type == FP_F32   ? launch_quant<float>
                        : x_type == FP_F16 ? launch_quant<__half>
                                           : launch_quant<__nv_bfloat16>;
    const cudaError_t rc = launch(c, x, T, K, ldx, pos, k, R, q, ldq, scale, st);
    fp_toc(c, st, slot);
    FP_CUDA(c, rc);
    return FP_OK;
}
