// What the layer operators (quantise, integer products with scales, MoE sort / dispatch / combine)
// share: element types, vectors of them, and the host side of a call that only queues kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp_internal.h"

// ---- host -----------------------------------------------------------------------------------

// Makes the context's device current for a call and the caller's device current again after it.
struct FpDeviceScope {
    int prev = -1;
    cudaError_t err;
    explicit FpDeviceScope(const fp_ctx* c) {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != c->device)
            err = cudaSetDevice(c->device);
        else
            prev = -1;
    }
    ~FpDeviceScope() {
        if (prev >= 0) cudaSetDevice(prev);
    }
    FpDeviceScope(const FpDeviceScope&) = delete;
    FpDeviceScope& operator=(const FpDeviceScope&) = delete;
};

static inline int fp_type_size(int type) { return type == FP_F32 ? 4 : (type == FP_F16 || type == FP_BF16) ? 2 : 0; }

// fp_tic for an operator: a launch that is being captured into a graph is counted, not timed (its
// events would never hold a time)
static inline void fp_op_tic(fp_ctx* c, cudaStream_t s, int kernel, double bytes, int* slot) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (c->profiling && (cudaStreamIsCapturing(s, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone)) {
        c->launches++;
        *slot = -1;
        return;
    }
    fp_tic(c, s, kernel, bytes, slot);
}

// raises a kernel's limit of dynamic shared memory, once a context (bit: the kernel's number)
template <typename F>
static inline cudaError_t fp_op_smem(fp_ctx* c, int bit, F* kernel, int bytes) {
    if (c->op_smem >> bit & 1) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) c->op_smem |= 1u << bit;
    return e;
}

// the largest power of two, at most 16, that divides every given address or pitch
static inline int fp_common_align(std::initializer_list<uint64_t> v) {
    uint64_t a = 16;
    for (uint64_t x : v) a |= x;
    return (int)(a & (~a + 1));
}

// ---- device ---------------------------------------------------------------------------------

__device__ __forceinline__ float fp_to_f(float x) { return x; }
__device__ __forceinline__ float fp_to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float fp_to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T fp_from_f(float x);
template <>
__device__ __forceinline__ float fp_from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half fp_from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 fp_from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V consecutive elements, loaded and stored in units of up to 16 bytes
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) FpVec {
    T v[V];
};
