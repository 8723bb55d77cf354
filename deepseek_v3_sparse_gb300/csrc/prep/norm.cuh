// norm.cuh -- what layer norm's forward and backward kernels share: how a row
// lies over threads and in shared memory, sums over those threads, the weights.
//
// G threads hold a row, U vectors of V elements each: thread t has the vectors
// t, t + G, t + 2G, ...  (Up to 32 threads a row is summed by shuffles, beyond
// through shared memory, under a barrier of its own.)  What bounds these kernels beside DRAM is the issue of
// instructions, and every thread of a row pays the row's sums, its root and its
// addresses; so a thread has many elements, and the arithmetic is in pairs (two
// f32 operations an instruction).  It holds the weights of its columns in
// registers from row to row.
//
// The CTAs walk over rows of their own.  A thread copies its vectors of coming
// rows into shared memory that it alone reads (16-byte asynchronous copies: no
// barrier, no registers), so loads are in flight all the time.
//
// Rows of an odd width (kShift): where the tensors start on 16 bytes but their
// rows do not, row r begins `shift` = r * stride mod V elements behind a 16-byte
// boundary.  A grid whose step is a multiple of V rows gives every thread rows of
// one and the same shift, so it still has columns of its own: its vectors start
// at the boundary, its column c is that of the vector less the shift, and only
// the first and the last vector of a row are cut.
#pragma once

#include <initializer_list>

#include "prep.cuh"

namespace dsix {

constexpr int kMaxCols = 32768;
constexpr int kRowSmem = 200 * 1024;  // of the rows in flight, at most
constexpr int kSms = 152;  // the grids' unit: whole multiples fill a GB300

// a CTA of at least `least` threads: one row, or several at a time
template <int G, int least>
struct RowShape {
    static constexpr int threads = G > least ? G : least;
    static constexpr int rows = threads / G;
    static_assert(G <= 32 || rows <= 15, "a barrier for each row");
};

// CTAs of so many threads, registers a thread and bytes of shared memory that an SM holds
constexpr int ctas_per_sm(int threads, int regs, int smem) {
    const int by_regs = 65536 / (threads * ((regs + 7) / 8 * 8));
    const int by_smem = smem ? 220 * 1024 / (smem + 2048) : 32;
    const int by_threads = 2048 / threads;
    const int n = by_regs < by_smem ? by_regs : by_smem;
    return n < 1 ? 1 : n > by_threads ? by_threads : n;
}

// sums of N numbers over the G threads of a row; s: N * 32 floats of shared
// memory of the CTA that no earlier, still unread sum uses, and `group` the row's
// place among the CTA's rows (G > 32 only)
template <int G, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*s)[32], int group) {
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
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(G) : "memory");
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = s[k][group * warps + (lane & (warps - 1))];
#pragma unroll
        for (int o = warps / 2; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

// Sums in pairs, of products too.  Vector u's elements go to partial sums in
// turn, so that several independent additions are in flight; where a vector is a
// single element, two vectors make a pair.
template <int E>
struct Pairs {
    static constexpr int N = E >= 8 ? 4 : E >= 4 ? 2 : 1;
    float2 p[N];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = make_float2(0.f, 0.f);
    }
    template <int V>
    __device__ __forceinline__ void add(int u, const float (&f)[V]) {
        if constexpr (V % 2 == 0) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                float2& q = p[(u * (V / 2) + i) % N];
                q = __fadd2_rn(q, make_float2(f[2 * i], f[2 * i + 1]));
            }
        } else {
            float2& q = p[(u / 2) % N];
            (u % 2 ? q.y : q.x) += f[0];
        }
    }
    template <int V>
    __device__ __forceinline__ void add_products(int u, const float (&f)[V], const float (&h)[V]) {
        if constexpr (V % 2 == 0) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                float2& q = p[(u * (V / 2) + i) % N];
                q = __ffma2_rn(make_float2(f[2 * i], f[2 * i + 1]), make_float2(h[2 * i], h[2 * i + 1]), q);
            }
        } else {
            float2& q = p[(u / 2) % N];
            float& one = u % 2 ? q.y : q.x;
            one = fmaf(f[0], h[0], one);
        }
    }
    __device__ __forceinline__ float total() const {
        float2 s = p[0];
#pragma unroll
        for (int i = 1; i < N; ++i) s = __fadd2_rn(s, p[i]);
        return s.x + s.y;
    }
};

template <int V>
__device__ __forceinline__ void fill(float (&f)[V], float v) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = v;
}

// V weights from column c on, which are f32 or of the activations' type; `none`
// where there is no weight.  Under kShift c may be negative and need not be a
// multiple of V.
template <class T, int V, bool kShift>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int c, int cols, float none, float (&f)[V]) {
    fill<V>(f, none);
    if (!w || c >= cols) return;
    if constexpr (kShift) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i >= 0 && c + i < cols)
                f[i] = f32 ? __ldg(static_cast<const float*>(w) + c + i) : to_f32(static_cast<const T*>(w)[c + i]);
    } else if (f32) {
        load_f32<V>(static_cast<const float*>(w) + c, f);
    } else {
        load_vec<T, V>(static_cast<const T*>(w) + c).unpack(f);
    }
}

// y to out[c .. c + V), without the columns that the row does not have
template <class T, int V, bool kShift>
__device__ __forceinline__ void store_row(T* out, int c, int cols, const Vec<T, V>& y) {
    if (!kShift || (c >= 0 && c + V <= cols)) {
        store_vec<T, V>(out + c, y);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i >= 0 && c + i < cols) out[c + i] = y.v[i];
    }
}

// How a call's tensors lie: rows of whole 16-byte vectors, rows that start at
// the same place behind a 16-byte boundary in every tensor, or neither.
enum { kAligned, kShifted, kScattered };
template <int W>
int lie(int cols, std::initializer_list<const void*> bases, std::initializer_list<int64_t> strides) {
    for (const void* p : bases)
        if (!aligned16(p)) return kScattered;
    bool whole = cols % W == 0;
    for (int64_t s : strides) {
        if (s % W != *strides.begin() % W) return kScattered;
        whole = whole && s % W == 0;
    }
    return whole ? kAligned : kShifted;
}

}  // namespace dsix
