// norm.cuh -- what layer norm's forward and backward kernels share: how a row
// lies over threads, sums over those threads, the weights.
//
// G threads hold a row, U vectors of V elements each: thread t has the vectors
// t, t + G, t + 2G, ...  Up to 32 threads a row lies in (part of) a warp and is
// summed by shuffles; beyond, a CTA holds one row.  The CTAs walk over the rows
// of their own, and a thread loads its part of the next D rows before it sums
// the present one, so that loads are always in flight behind the sums.
#pragma once

#include "prep.cuh"

namespace dsix {

constexpr int kNarrowThreads = 256;  // a CTA of rows that lie within a warp
constexpr int kMaxCols = 32768;
constexpr int kSms = 152;            // the grids' unit: whole multiples fill a GB300

template <int G>
struct RowShape {
    static constexpr bool narrow = G <= 32;
    static constexpr int threads = narrow ? kNarrowThreads : G;
    static constexpr int rows = narrow ? kNarrowThreads / G : 1;  // of a CTA at a time
};

// CTAs of so many threads that an SM holds at about so many registers a thread
constexpr int ctas_per_sm(int threads, int regs) {
    const int n = 65536 / (threads * ((regs + 7) / 8 * 8));
    const int most = 2048 / threads;
    return n < 1 ? 1 : n > most ? most : n;
}

// sums of N numbers over the G threads of a row; s: N * 32 floats of shared
// memory that no earlier, still unread sum uses (G > 32 only)
template <int G, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*s)[32]) {
    constexpr int W = G < 32 ? G : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (G > 32) {
        constexpr int warps = G / 32;
        const int lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) s[k][threadIdx.x >> 5] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = s[k][lane & (warps - 1)];
#pragma unroll
        for (int o = warps / 2; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

// V weights from column c on: f32, or of the activations' type
template <class T, int V>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int c, float (&f)[V]) {
    if (f32)
        load_f32<V>(static_cast<const float*>(w) + c, f);
    else
        load_vec<T, V>(static_cast<const T*>(w) + c).unpack(f);
}

template <int V>
__device__ __forceinline__ void fill(float (&f)[V], float v) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = v;
}

}  // namespace dsix
