// What the layer operators (quantise, integer products with scales, MoE sort / dispatch / combine)
// share: element types, vectors of them, and the host side of a call that only queues kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

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

// What a wait that ran out in an earlier call left: FP_ERR_TIMEOUT, once. Every operator asks before it queues anything.
static inline int fp_op_pending(fp_ctx* c, const char* what) {
    if (!c->mb->op_err) return FP_OK;
    c->mb->op_err = 0;
    return fp_fail(c, FP_ERR_TIMEOUT,
                   std::string(what) + ": a wait of an earlier fp_matmul_i8 ran out on the device; its y is not valid, nor what "
                                       "was made of it since");
}

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

// Launches a kernel that begins with fp_begin: it may come onto the SMs while the kernel before it on the stream runs
// its last blocks, and waits there for that one's end (a programmatic dependent launch).
template <typename... P, typename... A>
static inline cudaError_t fp_launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute pdl;
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// the largest power of two, at most 16, that divides every given address or pitch
static inline int fp_common_align(std::initializer_list<uint64_t> v) {
    uint64_t a = 16;
    for (uint64_t x : v) a |= x;
    return (int)(a & (~a + 1));
}

// How a kernel that goes over rows lays its threads: `tpr` threads (a multiple of 32) take a row of nvec
// vectors, U of them each at a time; `rpb` rows a block; `gy` blocks share a row's columns. Blocks of 128
// threads, which go over a long row in several passes: with blocks that hold a whole row (640 threads) the
// gradients of 8192 x 5120 bf16 rows took 157 us instead of 109, for fewer blocks overlap their reads with
// others' writes. Few rows: a vector a thread, the columns over blocks.
constexpr int FP_ROW_THREADS = 128;
struct FpRowGrid {
    int tpr, rpb;
    unsigned gx, gy;
    int threads() const { return tpr * rpb; }
};
static inline FpRowGrid fp_row_grid(const fp_ctx* c, int64_t rows, int64_t nvec, int U, bool share) {
    FpRowGrid g;
    auto threads = [&](int64_t per) { return (int)std::min<int64_t>(FP_ROW_THREADS, ((nvec + per - 1) / per + 31) / 32 * 32); };
    g.tpr = threads(rows * nvec < (int64_t)c->num_sms * 1024 ? 1 : U);
    g.rpb = FP_ROW_THREADS / g.tpr;
    g.gx = (unsigned)((rows + g.rpb - 1) / g.rpb);
    g.gy = 1;
    if (share)  // columns over blocks while there are SMs for them
        g.gy = (unsigned)std::max<int64_t>(1, std::min((nvec + g.tpr - 1) / g.tpr, 4 * (int64_t)c->num_sms / g.gx));
    return g;
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

// The start of a kernel launched by fp_launch: the next kernel of the stream may be brought onto the SMs that this one
// leaves, and nothing is read or written before the kernel before this one has ended. `index` (the block's number), on
// which every address hangs, comes out of the statements as a new value, so that no load, invariant or not, is moved up
// across the wait. (Renewing the pointers does it too, but keeps them in registers: combine of 8192 x 4099 fp32 took 83
// us for 73.)
__device__ __forceinline__ void fp_begin(unsigned& index) {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;\n" ::: "memory");
    asm volatile("" : "+r"(index)::"memory");
}

// the bytes of a matrix that may be read: from its first value to its last
struct FpSpan {
    const char *lo, *hi;
};
template <typename T>
__device__ __forceinline__ FpSpan fp_span(const T* p, int64_t rows, int64_t ld, int64_t cols) {
    return FpSpan{reinterpret_cast<const char*>(p), reinterpret_cast<const char*>(p + (rows - 1) * ld + cols)};
}

// the 16 bytes from byte `sh` of a and b, one after the other
__device__ __forceinline__ void fp_shift16(const uint4& a, const uint4& b, uint32_t sh, uint32_t* o) {
    uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
    if (sh & 8) w[0] = w[2], w[1] = w[3], w[2] = w[4], w[3] = w[5], w[4] = w[6], w[5] = b.w;
    if (sh & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = w[5];
    const uint32_t bits = 8 * (sh & 3);
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = __funnelshift_r(w[i], w[i + 1], bits);
}

// 16 bytes from any address: the two aligned 16 bytes that they lie in, shifted. False where those are not
// both inside the span (the matrix's ends). Plain loads: invariant ones may be moved up across a griddepcontrol.wait.
__device__ __forceinline__ bool fp_load16_any(const void* p, const FpSpan& span, uint32_t (&o)[4]) {
    const uint32_t sh = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    const char* q = reinterpret_cast<const char*>(p) - sh;
    if (q < span.lo || q + 32 > span.hi) return false;
    fp_shift16(reinterpret_cast<const uint4*>(q)[0], reinterpret_cast<const uint4*>(q)[1], sh, o);
    return true;
}

// BYTES consecutive bytes as words (a lone 1 or 2 bytes in one), loaded and stored in units of up to 16
template <int BYTES>
struct FpWords {
    static constexpr int W = BYTES < 4 ? 1 : BYTES / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const void* p) {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; i++) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        } else if constexpr (BYTES == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (BYTES == 2) {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint8_t*>(p);
        }
    }
    // from a multiple of UNIT, UNIT bytes at a time
    template <int UNIT>
    __device__ __forceinline__ void load_units(const void* p) {
        if constexpr (UNIT == 4) {
#pragma unroll
            for (int i = 0; i < W; i++) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        } else if constexpr (UNIT == 2) {
#pragma unroll
            for (int i = 0; i < W; i++)
                w[i] = (uint32_t) reinterpret_cast<const uint16_t*>(p)[2 * i] | (uint32_t) reinterpret_cast<const uint16_t*>(p)[2 * i + 1] << 16;
        } else {
#pragma unroll
            for (int i = 0; i < W; i++) {
                w[i] = 0;
#pragma unroll
                for (int j = 0; j < 4; j++) w[i] |= (uint32_t) reinterpret_cast<const uint8_t*>(p)[4 * i + j] << (8 * j);
            }
        }
    }
    __device__ __forceinline__ void store(void* p) const {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; i++)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (BYTES == 8) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (BYTES == 4) {
            *reinterpret_cast<uint32_t*>(p) = w[0];
        } else if constexpr (BYTES == 2) {
            *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
        } else {
            *reinterpret_cast<uint8_t*>(p) = (uint8_t)w[0];
        }
    }
};

// V consecutive values
template <typename T, int V>
struct FpVec : FpWords<V * (int)sizeof(T)> {
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(this->w[i]);
        } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            return __uint_as_float((i & 1) ? this->w[i >> 1] & 0xFFFF0000u : this->w[i >> 1] << 16);
        } else {
            return __half2float(__ushort_as_half((unsigned short)((i & 1) ? this->w[i >> 1] >> 16 : this->w[i >> 1] & 0xFFFFu)));
        }
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; i++) this->w[i] = __float_as_uint(f[i]);
        } else if constexpr (V == 1) {
            const T x = fp_from_f<T>(f[0]);
            this->w[0] = *reinterpret_cast<const unsigned short*>(&x);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                    const __nv_bfloat162 x = __floats2bfloat162_rn(f[i], f[i + 1]);
                    this->w[i >> 1] = *reinterpret_cast<const uint32_t*>(&x);
                } else {
                    const __half2 x = __floats2half2_rn(f[i], f[i + 1]);
                    this->w[i >> 1] = *reinterpret_cast<const uint32_t*>(&x);
                }
            }
        }
    }
};

// A row's vectors of V values. ANY: the row begins at any multiple of its element's size, and each 16 bytes are the
// two aligned 16 bytes that they lie in, shifted; `load` is false for a vector whose aligned bytes are not all inside
// the matrix (its first and last ones), which `slow` then reads. `load` has no branches, so that a thread's loads do not
// wait for one another.
template <typename T, int V, bool ANY>
struct FpRow {
    static constexpr int BYTES = V * (int)sizeof(T);
    static constexpr bool SHIFT = ANY && BYTES % 16 == 0;
    const T* p;
    const char* q;
    uint32_t sh;
    int first, end;
    __device__ __forceinline__ FpRow() {}
    __device__ __forceinline__ FpRow(const T* row, const FpSpan& span) : p(row) {
        if constexpr (SHIFT) {
            sh = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15);
            q = reinterpret_cast<const char*>(row) - sh;
            first = q < span.lo;
            end = (int)min((int64_t)0x7fffffff, (int64_t)(span.hi - q - 16) / BYTES);
        }
    }
    __device__ __forceinline__ bool load(FpVec<T, V>& v, int c) const {
        if constexpr (SHIFT) {
            const bool ok = c >= first && c < end;
            const uint4* at = reinterpret_cast<const uint4*>(q + (int64_t)c * BYTES);
            uint4 b[BYTES / 16 + 1];
#pragma unroll
            for (int i = 0; i <= BYTES / 16; i++) b[i] = ok ? __ldg(at + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < BYTES / 16; i++) fp_shift16(b[i], b[i + 1], sh, &v.w[4 * i]);
            return ok;
        } else if constexpr (ANY) {
            slow(v, c);
            return true;
        } else {
            v.load(p + (int64_t)c * V);
            return true;
        }
    }
    __device__ __forceinline__ void slow(FpVec<T, V>& v, int c) const {
        v.template load_units<(int)sizeof(T)>(p + (int64_t)c * V);
    }
    __device__ __forceinline__ FpVec<T, V> get(int c) const {
        FpVec<T, V> v;
        if (!load(v, c)) slow(v, c);
        return v;
    }
};
