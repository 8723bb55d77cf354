// norm.cuh -- what layer norm's forward and backward kernels share: how a row
// lies over threads, sums over those threads, the weights.
//
// G threads hold a row, U vectors of V elements each: thread t has the vectors
// t, t + G, t + 2G, ...  Up to 32 threads a row lies in (part of) a warp and is
// summed by shuffles; beyond, a CTA holds one row.
#pragma once

#include "prep.cuh"

namespace dsix {

constexpr int kNarrowThreads = 256;  // a CTA of rows that lie within a warp
constexpr int kMaxCols = 32768;

template <int G>
struct RowShape {
    static constexpr bool narrow = G <= 32;
    static constexpr int threads = narrow ? kNarrowThreads : G;
    static constexpr int rows = narrow ? kNarrowThreads / G : 1;  // of a CTA at a time
};

// sum over the G threads of a row; s: 32 floats of shared memory that no
// earlier, still unread sum uses (G > 32 only)
template <int G>
__device__ __forceinline__ float row_sum(float v, float* s) {
    constexpr int W = G < 32 ? G : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (G > 32) {
        if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
        __syncthreads();
        constexpr int N = G / 32;
        v = (threadIdx.x & 31) < N ? s[threadIdx.x & 31] : 0.f;
#pragma unroll
        for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        v = __shfl_sync(0xffffffffu, v, 0);
    }
    return v;
}

// V weights from column c on: f32, or of the activations' type
template <class T, int V>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int c, float (&f)[V]) {
    if (f32) {
        load_f32<V>(static_cast<const float*>(w) + c, f);
    } else {
        const Vec<T, V> v = load_vec<T, V>(static_cast<const T*>(w) + c);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f32(v.v[i]);
    }
}

}  // namespace dsix
