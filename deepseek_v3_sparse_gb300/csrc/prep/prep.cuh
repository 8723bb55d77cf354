// prep.cuh -- what the kernels of libdsix_prep share: the element types and
// their vectors, reductions over the threads of a row, argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "../../../include/dsix_prep.h"
#include "../common.cuh"

namespace dsix {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

__device__ __forceinline__ void from_f32(float f, __nv_bfloat16& v) { v = __float2bfloat16_rn(f); }
__device__ __forceinline__ void from_f32(float f, __half& v) { v = __float2half_rn(f); }
__device__ __forceinline__ void from_f32(float f, float& v) { v = f; }

__device__ __forceinline__ float2 to_f32(__nv_bfloat162 v) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&v);
    return make_float2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ float2 to_f32(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ void from_f32(float a, float b, __nv_bfloat162& v) { v = __floats2bfloat162_rn(a, b); }
__device__ __forceinline__ void from_f32(float a, float b, __half2& v) { v = __floats2half2_rn(a, b); }

template <class T>
struct Pair;  // two elements in one register
template <>
struct Pair<__nv_bfloat16> { using type = __nv_bfloat162; };
template <>
struct Pair<__half> { using type = __half2; };

// V elements that are loaded and stored as one access (V * sizeof(T) <= 16
// bytes); two 16-bit elements lie in one register and are converted together.
template <class T, int V>
struct alignas(V * sizeof(T)) Vec {
    static constexpr bool paired = sizeof(T) == 2 && V % 2 == 0;
    T v[V];

    __device__ __forceinline__ void unpack(float (&f)[V]) const {
        if constexpr (paired) {
            using P = typename Pair<T>::type;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 q = to_f32(reinterpret_cast<const P*>(v)[i]);
                f[2 * i] = q.x;
                f[2 * i + 1] = q.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = to_f32(v[i]);
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[V]) {
        if constexpr (paired) {
            using P = typename Pair<T>::type;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) from_f32(f[2 * i], f[2 * i + 1], reinterpret_cast<P*>(v)[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) from_f32(f[i], v[i]);
        }
    }
};

template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
    return *reinterpret_cast<const Vec<T, V>*>(p);
}

template <class T, int V>
__device__ __forceinline__ Vec<T, V> zero_vec() {
    Vec<T, V> z;
    const float f[V] = {};
    z.pack(f);
    return z;
}

template <class T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& v) {
    *reinterpret_cast<Vec<T, V>*>(p) = v;
}

// V floats from p, in 16-byte pieces where V allows (p is then 16-byte aligned)
template <int V>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(p) + i);
            f[4 * i] = q.x;
            f[4 * i + 1] = q.y;
            f[4 * i + 2] = q.z;
            f[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __ldg(p + i);
    }
}

// the first n of B bytes from global to shared memory, asynchronously, zeros behind them
template <int B>
__device__ __forceinline__ void copy_async(void* dst, const void* src, uint32_t n) {
    if constexpr (B == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(B), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Division of n < 2^31 by a number known at launch: with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (high word of n m + n) >> s
// (T. Granlund and P. Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct FastDiv {
    uint32_t d = 1, m = 1, s = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t by) : d(by) {
        while ((1ull << s) < d) ++s;
        m = static_cast<uint32_t>((((1ull << s) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

// Shared memory beyond kPlainSmem has to be asked for, once for each kernel and
// device.
constexpr int kPlainSmem = 46 * 1024;
template <auto kernel>
int allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};  // a bit per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return IX_ERR_CUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return IX_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return IX_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_relaxed);
    return IX_OK;
}

inline bool aligned_to(const void* p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

inline int dtype_bytes(int dtype) { return dtype == IX_FP32 ? 4 : dtype == IX_BF16 || dtype == IX_FP16 ? 2 : 0; }

}  // namespace dsix
