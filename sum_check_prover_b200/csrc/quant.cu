// fp_quantize_rows: activations to int8 with one scale a token.
//
// a_t = max_j |x_tj|, scale_t = a_t / 127 (fp32), q_tj = the integer nearest to 127 x_tj / a_t, ties to
// the even one. The integer is exact: a product with the fp32 value of 127 / a_t is off by less than
// 127 * 2^-22, so only a value within 2^-14 of a half can round to the wrong side, and those compare
// 254 |x| with (2 n + 1) a_t, whose products are exact in double.
//
// A row with a NaN or an infinity has no scale: its scale is NaN and its integers are 0, so every
// product with it is NaN. A row of zeros has scale 0.
#include <algorithm>

#include "fp_ops.cuh"

namespace {

constexpr int QR_VALUES = 32;  // values of a row that a thread keeps in registers

constexpr float QR_MAGIC = 12582912.0f;  // 1.5 * 2^23: t + it has the nearest integer to t in its low bits

// the integer nearest to 127 x / a for a value that lies next to a half (t: the approximate quotient)
__device__ __noinline__ uint32_t quant_near_half(float x, float a, float t) {
    const int n = (int)floorf(fabsf(t));
    const double d = 254.0 * (double)fabsf(x) - (double)(2 * n + 1) * (double)a;
    const int r = d > 0 ? n + 1 : d < 0 ? n : n + (n & 1);
    return (uint32_t)(x < 0 ? -r : r);
}

// V values to int8
template <typename T, int V>
__device__ __forceinline__ FpVec<int8_t, V> quant_vec(const FpVec<T, V>& w, float up, float a, float inv) {
    FpVec<int8_t, V> o;
    bool near = false;
#pragma unroll
    for (int e = 0; e < V; e++) {
        const float t = fp_to_f(w.v[e]) * up * inv, r = t + QR_MAGIC;
        o.v[e] = (int8_t)__float_as_uint(r);
        near |= fabsf(t - (r - QR_MAGIC)) > 0.5f - 6.1035156e-5f;
    }
    if (near) {
#pragma unroll
        for (int e = 0; e < V; e++) {
            const float x = fp_to_f(w.v[e]) * up, t = x * inv;
            if (fabsf(t - (t + QR_MAGIC - QR_MAGIC)) > 0.5f - 6.1035156e-5f) o.v[e] = (int8_t)quant_near_half(x, a, t);
        }
    }
    return o;
}

// One row per `tpr` threads (a multiple of 32 that divides the block). V: elements per load; a thread
// keeps the first QR_VALUES / V vectors it reads, and reads what is beyond them a second time.
template <typename T, int V>
__global__ void __launch_bounds__(1024)
    quant_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t K, int64_t ldx, const int32_t* __restrict__ pos,
                      int k, int64_t R, int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale, int tpr,
                      bool qvec) {
    constexpr int NV = QR_VALUES / V;
    __shared__ uint32_t red[32];
    const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + sub;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * ldx;
    const int64_t nvec = live ? K / V : 0;
    FpVec<T, V> reg[NV];
    uint32_t m = 0;  // the largest |x| as bits: NaN above infinity above every number
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int64_t c = t + (int64_t)i * tpr;
        if (c < nvec) reg[i] = *reinterpret_cast<const FpVec<T, V>*>(xr + c * V);
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (t + (int64_t)i * tpr < nvec) {
#pragma unroll
            for (int e = 0; e < V; e++) m = max(m, __float_as_uint(fp_to_f(reg[i].v[e])) & 0x7fffffffu);
        }
    }
    for (int64_t c = t + (int64_t)NV * tpr; c < nvec; c += tpr) {
        const FpVec<T, V> w = *reinterpret_cast<const FpVec<T, V>*>(xr + c * V);
#pragma unroll
        for (int e = 0; e < V; e++) m = max(m, __float_as_uint(fp_to_f(w.v[e])) & 0x7fffffffu);
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
    // rows below 2^-64 are scaled up (exactly) so that 127 / a stays finite
    const float up = amax < 5.421010862427522e-20f ? 18446744073709551616.0f : 1.0f;
    const float a = amax * up;
    const float inv = (bad || m == 0) ? 0.0f : 127.0f / a;
    const int copies = pos ? k : 1;
    if (t == 0) {
        const float s = bad ? __uint_as_float(0x7fc00000u) : amax / 127.0f;
        for (int j = 0; j < copies; j++) {
            const int64_t p = pos ? pos[row * k + j] : row;
            if (p >= 0 && p < R) scale[p] = s;
        }
    }
    auto put = [&](int64_t c, const FpVec<T, V>& w) {
        FpVec<int8_t, V> o = {};
        if (inv != 0.0f) o = quant_vec<T, V>(w, up, a, inv);
        for (int j = 0; j < copies; j++) {
            const int64_t p = pos ? pos[row * k + j] : row;
            if (p < 0 || p >= R) continue;
            int8_t* d = q + p * ldq + c * V;
            if (qvec) {
                *reinterpret_cast<FpVec<int8_t, V>*>(d) = o;
            } else {
#pragma unroll
                for (int e = 0; e < V; e++) d[e] = o.v[e];
            }
        }
    };
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int64_t c = t + (int64_t)i * tpr;
        if (c < nvec) put(c, reg[i]);
    }
    for (int64_t c = t + (int64_t)NV * tpr; c < nvec; c += tpr)
        put(c, *reinterpret_cast<const FpVec<T, V>*>(xr + c * V));
}

template <typename T>
void launch_quant(const fp_ctx* c, const void* x, int64_t T_, int64_t K, int64_t ldx, const int32_t* pos, int k,
                  int64_t R, int8_t* q, int64_t ldq, float* scale, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = fp_common_align({(uint64_t)(uintptr_t)x, (uint64_t)ldx * sizeof(T), (uint64_t)K * sizeof(T)}) == 16;
    const bool qvec = fp_common_align({(uint64_t)(uintptr_t)q, (uint64_t)ldq}) >= V;
    const int64_t nvec = vec ? K / V : K;
    const int nv = QR_VALUES / (vec ? V : 1);
    // enough threads to hold the row in registers; more while the rows alone do not fill the GPU
    int tpr = 32;
    while (tpr < 1024 && (int64_t)tpr * nv < nvec) tpr *= 2;
    while (tpr < 1024 && tpr < nvec && T_ * tpr < (int64_t)c->num_sms * 512) tpr *= 2;
    const int threads = std::max(tpr, 128), rpb = threads / tpr;
    const unsigned grid = (unsigned)((T_ + rpb - 1) / rpb);
    if (vec)
        quant_rows_kernel<T, V><<<grid, threads, 0, st>>>((const T*)x, T_, K, ldx, pos, k, R, q, ldq, scale, tpr, qvec);
    else
        quant_rows_kernel<T, 1><<<grid, threads, 0, st>>>((const T*)x, T_, K, ldx, pos, k, R, q, ldq, scale, tpr, true);
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
