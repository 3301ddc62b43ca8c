// fp_matmul_i8: y[n][m] = x_scale[n] w_scale[e][m] sum_k w[e][m][k] x[n][k], e the expert of row n.
//
// The sum is exact in int32 (K <= 2^17 - 1 keeps 2^14 K below 2^31); the three factors are multiplied in
// fp32 in the order sum, token scale, channel scale, and rounded to y's type.
#include <algorithm>

#include "fp_ops.cuh"

namespace {

constexpr int MI_TILE = 64;  // channels and tokens per block
constexpr int MI_BK = 64;    // bytes of K per step

struct MiArgs {
    const int8_t* w;
    const float* w_scale;
    const int8_t* x;
    const float* x_scale;
    const int32_t* offsets;
    void* y;
    int64_t M, K, N, ldw, ldx, ldy;
    int E;
};

// the rows [lo, hi) of expert e, kept inside the N rows and apart from the other experts' whatever the
// offsets say: each offset counts as the largest up to it (all threads of the block)
__device__ __forceinline__ void mi_group(const MiArgs& a, int e, int64_t& lo, int64_t& hi) {
    __shared__ int32_t most;
    lo = 0;
    hi = a.N;
    if (!a.offsets) return;
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    int32_t m = 0;
    for (int i = threadIdx.x; i <= e; i += blockDim.x) m = max(m, a.offsets[i]);
    if (m > 0) atomicMax(&most, m);
    __syncthreads();
    lo = min((int64_t)most, a.N);
    hi = min((int64_t)max(most, a.offsets[e + 1]), a.N);
}

// one block per 64 channels of one expert; it goes over that expert's tokens 64 at a time
template <typename YT>
__global__ void __launch_bounds__(256) matmul_i8_kernel(MiArgs a) {
    __shared__ int32_t sw[MI_TILE][MI_BK / 4 + 1], sx[MI_TILE][MI_BK / 4 + 1];
    const int e = blockIdx.y, tid = threadIdx.x, tm = tid & 15, tn = tid >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * MI_TILE;
    int64_t lo, hi;
    mi_group(a, e, lo, hi);
    for (int64_t n0 = lo; n0 < hi; n0 += MI_TILE) {
        int32_t acc[4][4] = {};
        for (int64_t k0 = 0; k0 < a.K; k0 += MI_BK) {
            __syncthreads();
            for (int i = tid; i < MI_TILE * MI_BK; i += 256) {
                const int r = i / MI_BK, kk = i % MI_BK;
                const bool in = k0 + kk < a.K;
                reinterpret_cast<int8_t*>(&sw[r][0])[kk] = in && m0 + r < a.M ? a.w[((int64_t)e * a.M + m0 + r) * a.ldw + k0 + kk] : 0;
                reinterpret_cast<int8_t*>(&sx[r][0])[kk] = in && n0 + r < hi ? a.x[(n0 + r) * a.ldx + k0 + kk] : 0;
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < MI_BK / 4; q++)
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) acc[i][j] = __dp4a(sw[tm + 16 * i][q], sx[tn + 16 * j][q], acc[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int64_t m = m0 + tm + 16 * i, n = n0 + tn + 16 * j;
                if (m >= a.M || n >= hi) continue;
                const float v = (float)acc[i][j] * a.x_scale[n] * a.w_scale[(int64_t)e * a.M + m];
                reinterpret_cast<YT*>(a.y)[n * a.ldy + m] = fp_from_f<YT>(v);
            }
    }
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
    if (empty) return FP_OK;
    FpDeviceScope dev(c);
    if (dev.err != cudaSuccess) return fp_cuda_check(c, dev.err, "fp_matmul_i8");
    cudaStream_t st = (cudaStream_t)stream;
    MiArgs a{w, w_scale, x, x_scale, offsets, y, M, K, N, ldw, ldx, ldy, E};
    const dim3 grid((unsigned)((M + MI_TILE - 1) / MI_TILE), (unsigned)E);
    int slot;
    fp_op_tic(c, st, K_MATMUL_I8, (double)E * M * K + (double)N * (K + ys * (double)M), &slot);
    if (y_type == FP_F32)
        matmul_i8_kernel<float><<<grid, 256, 0, st>>>(a);
    else if (y_type == FP_F16)
        matmul_i8_kernel<__half><<<grid, 256, 0, st>>>(a);
    else
        matmul_i8_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    fp_toc(c, st, slot);
    FP_CUDA(c, cudaGetLastError());
    return FP_OK;
}
