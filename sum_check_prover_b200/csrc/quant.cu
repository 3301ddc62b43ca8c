// fp_quantize_rows: activations to int8 with one scale a token.
//
// a_t = max_j |x_tj|, scale_t = a_t / 127 (fp32), q_tj = the integer nearest to 127 x_tj / a_t, ties to
// the even one. The integer is exact: a product with the fp32 value of 127 / a_t is off by less than
// 127 * 2^-22, so only a value within 2^-15 of a half can round to the wrong side, and those compare
// 254 |x| with (2 n + 1) a_t, whose products are exact in double. Vectors with such a value (one value in
// 16000) are noted by a bit and done again one value at a time after the others.
//
// A row with a NaN or an infinity has no scale: its scale is NaN and its integers are 0, so every
// product with it is NaN. A row of zeros has scale 0.
#include <algorithm>

#include "fp_ops.cuh"

namespace {


constexpr int QR_LOADS = 8;  // vectors of a row that a thread keeps in registers (single values: twice as many)
constexpr float QR_MAGIC = 12582912.0f;  // 1.5 * 2^23: t + it has the nearest integer to t in its low bits
constexpr float QR_NEAR = 0.5f - 3.0517578e-5f;

// V values to int8 by the fp32 quotient (0 in a bad row); `near` is set when one lies next to a half
template <typename T, int V>
__device__ __forceinline__ FpWords<V> quant_vec(const FpVec<T, V>& w, float inv, bool bad, bool& near) {
    uint32_t r[V];
    float off = 0.0f;
#pragma unroll
    for (int e = 0; e < V; e++) {
        const float t = w.get(e) * inv, n = t + QR_MAGIC;
        r[e] = __float_as_uint(n);
        off = fmaxf(off, fabsf(t - (n - QR_MAGIC)));
    }
    near = off > QR_NEAR;
    FpWords<V> o;
    if constexpr (V == 1) {
        o.w[0] = bad ? 0 : r[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; i++)
            o.w[i] = bad ? 0
                         : __byte_perm(__byte_perm(r[4 * i], r[4 * i + 1], 0x0040),
                                       __byte_perm(r[4 * i + 2], r[4 * i + 3], 0x0040), 0x5410);
    }
    return o;
}

// one value exactly
__device__ __forceinline__ int8_t quant_exact(float x, float a) {
    const float t = fabsf(x) * (127.0f / a);
    int r = __float2int_rn(t);
    if (fabsf(t - (float)r) > QR_NEAR) {
        const int n = (int)floorf(t);
        const double d = 254.0 * (double)fabsf(x) - (double)(2 * n + 1) * (double)a;
        r = d > 0 ? n + 1 : d < 0 ? n : n + (n & 1);
    }
    return (int8_t)(x < 0 ? -r : r);
}

// One row per `tpr` threads (a multiple of 32 that divides the block). V: elements per load; a thread
// keeps the first NV vectors it reads in registers, and reads what is beyond them a second time.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512)
    quant_rows_kernel(const T* __restrict__ x, int64_t rows, int K, int64_t ldx, const int32_t* __restrict__ pos, int k,
                      int64_t R, int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale, int tpr, bool qvec) {
    __shared__ uint32_t red[32];
    const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + sub;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * ldx;
    const int nvec = live ? K / V : 0;
    const int64_t p0 = !live ? -1 : pos ? __ldg(pos + row * k) : row;
    FpVec<T, V> reg[NV];
    uint32_t m = 0;  // the largest |x| as bits: NaN above infinity above every number
    auto largest = [&](const FpVec<T, V>& w) {
#pragma unroll
        for (int e = 0; e < V; e++) m = max(m, __float_as_uint(w.get(e)) & 0x7fffffffu);
    };
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (t + i * tpr < nvec) {
            reg[i].load(xr + (t + i * tpr) * V);
        } else {
#pragma unroll
            for (int e = 0; e < FpVec<T, V>::W; e++) reg[i].w[e] = 0;
        }
#pragma unroll
    for (int i = 0; i < NV; i++) largest(reg[i]);
    for (int c = t + NV * tpr; c < nvec; c += tpr) {
        FpVec<T, V> w;
        w.load(xr + c * V);
        largest(w);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (tpr > 32) {
        if (lane == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        const int w0 = sub * (tpr >> 5), nw = tpr >> 5;
        m = __reduce_max_sync(0xffffffffu, red[w0 + (lane < nw ? lane : 0)]);
    }
    if (!live) return;
    const float amax = __uint_as_float(m);
    const bool bad = m >= 0x7f800000u;
    const float inv = bad || m == 0 ? 0.0f : 127.0f / amax;
    // in rows below 2^-64 every value is done exactly, scaled up (127 / a may not be finite)
    const bool tiny = amax < 5.421010862427522e-20f && m != 0;
    const float up = tiny ? 18446744073709551616.0f : 1.0f;
    const int copies = pos ? k : 1;
    FpWords<V> o[NV];
    uint32_t redo = 0;  // the vectors with a value next to a half
#pragma unroll
    for (int i = 0; i < NV; i++) {
        bool near;
        o[i] = quant_vec<T, V>(reg[i], tiny ? 0.0f : inv, bad, near);
        if (near || tiny) redo |= 1u << i;
    }
    for (int j = 0; j < copies; j++) {
        const int64_t p = j == 0 ? p0 : __ldg(pos + row * k + j);
        if (p < 0 || p >= R) continue;
        if (t == 0) scale[p] = bad ? __uint_as_float(0x7fc00000u) : amax / 127.0f;
        int8_t* d = q + p * ldq;
        auto put = [&](int c, const FpWords<V>& w) {
            if (V == 1 || qvec) {
                w.store(d + c * V);
            } else {
#pragma unroll
                for (int e = 0; e < V; e++) d[c * V + e] = (int8_t)(w.w[e >> 2] >> (8 * (e & 3)));
            }
        };
        auto again = [&](int c) {
            for (int e = 0; e < V; e++) d[c * V + e] = quant_exact(fp_to_f(xr[c * V + e]) * up, amax * up);
        };
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (t + i * tpr < nvec) put(t + i * tpr, o[i]);
        for (uint32_t left = redo; left; left &= left - 1) {
            const int c = t + (__ffs(left) - 1) * tpr;
            if (c < nvec) again(c);
        }
        for (int c = t + NV * tpr; c < nvec; c += tpr) {
            FpVec<T, V> w;
            w.load(xr + c * V);
            bool near;
            put(c, quant_vec<T, V>(w, tiny ? 0.0f : inv, bad, near));
            if (near || tiny) again(c);
        }
    }
}

template <typename T>
void launch_quant(const fp_ctx* c, const void* x, int64_t T_, int64_t K, int64_t ldx, const int32_t* pos, int k,
                  int64_t R, int8_t* q, int64_t ldq, float* scale, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = fp_common_align({(uint64_t)(uintptr_t)x, (uint64_t)ldx * sizeof(T), (uint64_t)K * sizeof(T)}) == 16;
    const bool qvec = fp_common_align({(uint64_t)(uintptr_t)q, (uint64_t)ldq}) >= V;
    const int64_t nvec = vec ? K / V : K;
    // a few warps hold a row in registers, so that many rows are in flight; few rows: a vector a thread
    auto run = [&](auto kern, int loads) {
        int tpr = 32;
        while (tpr < 512 && ((int64_t)tpr * loads < nvec || (T_ * tpr < (int64_t)c->num_sms * 256 && tpr < nvec))) tpr += 32;
        const int threads = std::max(128 / tpr, 1) * tpr;
        const unsigned grid = (unsigned)((T_ + threads / tpr - 1) / (threads / tpr));
        kern<<<grid, threads, 0, st>>>((const T*)x, T_, (int)K, ldx, pos, k, R, q, ldq, scale, tpr, qvec || !vec);
    };
    vec ? run(quant_rows_kernel<T, V, QR_LOADS>, QR_LOADS) : run(quant_rows_kernel<T, 1, 2 * QR_LOADS>, 2 * QR_LOADS);
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
    if (empty) return FP_OK;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_quantize_rows");
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 1) ldx = 16;  // a single row has no pitch: one that keeps its alignment
    if (R == 1) ldq = 16;
    int slot;
    fp_op_tic(c, st, K_QUANT_ROWS, (double)T * K * fp_type_size(x_type) + (double)(pos ? T * k : T) * (K + 4), &slot);
    if (x_type == FP_F32)
        launch_quant<float>(c, x, T, K, ldx, pos, k, R, q, ldq, scale, st);
    else if (x_type == FP_F16)
        launch_quant<__half>(c, x, T, K, ldx, pos, k, R, q, ldq, scale, st);
    else
        launch_quant<__nv_bfloat16>(c, x, T, K, ldx, pos, k, R, q, ldq, scale, st);
    fp_toc(c, st, slot);
    FP_CUDA(c, cudaGetLastError());
    return FP_OK;
}
