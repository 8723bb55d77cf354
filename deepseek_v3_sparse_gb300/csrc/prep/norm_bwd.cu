// norm_bwd.cu -- ix_layer_norm_bwd.
//
// One pass over dy and x gives dx and the column sums: a thread holds the same
// columns of every row it takes, so it adds up their dy * xhat and dy in
// registers.  The CTAs that walk the rows write their sums once, and a second
// kernel adds those in the order of the CTAs (the bits do not depend on which CTA
// ends first).  Rows too wide for a thread's registers to hold the sums beside
// the row take their column sums in a pass of their own.
#include "norm.cuh"

namespace dsix {
namespace {

struct BwdArgs {
    const void *dy, *x, *gamma;
    const float *mean, *rstd;
    void* dx;
    float* part;  // [parts][2][cols], or NULL: no column sums
    int64_t dy_stride, x_stride, dx_stride, rows;
    int cols, weight_f32;
    float inv_cols;
};

// CTAs that write column sums, at most: what their sums cost is bounded, also
// where the columns are many
constexpr int max_parts(int cols) { return kSms * (cols <= 2048 ? 4 : cols <= 4096 ? 3 : 2); }

template <class T, int V, int G, int U, bool kSums>
struct Bwd : RowShape<G> {
    static constexpr int E = U * V, words = U * ((V * sizeof(T) + 3) / 4);
    static constexpr bool hold = E <= 16 && V > 1 && G < 1024;
    static constexpr int ahead = RowShape<G>::narrow && words <= 4 ? 2 : E <= 16 ? 1 : 0;
    // the same shape with and without the column sums
    static constexpr int ctas =
        ctas_per_sm(RowShape<G>::threads, 2 * E + (hold ? E : 0) + (ahead + 1) * 2 * words + 32);
};

template <class T, int V, int G, int U, bool kSums>
__global__ void __launch_bounds__(Bwd<T, V, G, U, kSums>::threads, Bwd<T, V, G, U, kSums>::ctas)
    norm_bwd_kernel(const BwdArgs a) {
    using F = Bwd<T, V, G, U, kSums>;
    __shared__ float s_sum[2][2][32];
    const int t = threadIdx.x % G, sub = threadIdx.x / G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * F::rows;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * F::rows;
    struct Row {
        Vec<T, V> x[U], dy[U];
        float mean, rstd;
    };
    // a row past the end has dy = x = 0 and mean = rstd = 0: it adds nothing
    auto load = [&](Row& r, int64_t row) {
        const bool live = row < a.rows;
        const T* px = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* pd = static_cast<const T*>(a.dy) + row * a.dy_stride;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * G + t) * V;
            r.x[u] = live && c < a.cols ? load_vec<T, V>(px + c) : zero_vec<T, V>();
            r.dy[u] = live && c < a.cols ? load_vec<T, V>(pd + c) : zero_vec<T, V>();
        }
        r.mean = live ? __ldg(a.mean + row) : 0.f;
        r.rstd = live ? __ldg(a.rstd + row) : 0.f;
    };
    auto weight = [&](float(&w)[V], int c) {
        fill<V>(w, 1.f);
        if (a.gamma && c < a.cols) load_weight<T, V>(a.gamma, a.weight_f32, c, w);
    };
    Row ring[F::ahead + 1];
#pragma unroll
    for (int k = 0; k <= F::ahead; ++k) load(ring[k], row0 + k * step + sub);
    float ag[kSums ? F::E : 1], ab[kSums ? F::E : 1], g[F::hold ? U : 1][V];
    if constexpr (kSums) {
        fill<F::E>(ag, 0.f);
        fill<F::E>(ab, 0.f);
    }
    if constexpr (F::hold) {
#pragma unroll
        for (int u = 0; u < U; ++u) weight(g[u], (u * G + t) * V);
    }
    int flip = 0;  // the sums of consecutive rows use other places: one barrier a row is enough
    for (int64_t r0 = row0; r0 < a.rows; r0 += step) {
        const Row& r = ring[0];
        const int64_t row = r0 + sub;
        float sums[2] = {0.f, 0.f};  // of h and h * xhat
        // roundings spelled out: with and without the column sums, dx has the same bits
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * G + t) * V;
            if constexpr (!F::hold) weight(g[0], c);
            if (c < a.cols) {
                float x[V], d[V];
                r.x[u].unpack(x);
                r.dy[u].unpack(d);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = __fmul_rn(__fsub_rn(x[i], r.mean), r.rstd);
                    const float h = __fmul_rn(d[i], g[F::hold ? u : 0][i]);
                    sums[0] = __fadd_rn(sums[0], h);
                    sums[1] = fmaf(h, xh, sums[1]);
                    if constexpr (kSums) {
                        ag[u * V + i] = fmaf(d[i], xh, ag[u * V + i]);
                        ab[u * V + i] += d[i];
                    }
                }
            }
        }
        row_sums<G>(sums, s_sum[flip]);
        flip ^= 1;
        if (row < a.rows) {
            const float mh = __fmul_rn(sums[0], a.inv_cols), mhx = __fmul_rn(sums[1], a.inv_cols);
            T* out = static_cast<T*>(a.dx) + row * a.dx_stride;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * G + t) * V;
                if constexpr (!F::hold) weight(g[0], c);
                if (c < a.cols) {
                    float x[V], d[V];
                    r.x[u].unpack(x);
                    r.dy[u].unpack(d);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float xh = __fmul_rn(__fsub_rn(x[i], r.mean), r.rstd);
                        const float h = __fmul_rn(d[i], g[F::hold ? u : 0][i]);
                        d[i] = __fmul_rn(r.rstd, fmaf(-xh, mhx, __fsub_rn(h, mh)));
                    }
                    Vec<T, V> y;
                    y.pack(d);
                    store_vec<T, V>(out + c, y);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < F::ahead; ++k) ring[k] = ring[k + 1];
        load(ring[F::ahead], row + (F::ahead + 1) * step);
    }
    if constexpr (kSums) {
        float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
        if constexpr (!F::narrow) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = (u * G + t) * V + i;
                    if (c < a.cols) {
                        part[c] = ag[u * V + i];
                        part[a.cols + c] = ab[u * V + i];
                    }
                }
        } else {
            // the CTA's row groups: those of a warp by shuffles, the warps in shared memory
            constexpr int kWarps = F::threads / 32, kCols = G * U * V;
            __shared__ float s_part[kWarps][kCols];
            const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                __syncthreads();
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float v = w ? ab[u * V + i] : ag[u * V + i];
#pragma unroll
                        for (int o = G; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                        if (lane < G) s_part[warp][(u * G + t) * V + i] = v;
                    }
                __syncthreads();
                for (int c = threadIdx.x; c < a.cols; c += F::threads) {
                    float v = 0.f;
#pragma unroll
                    for (int k = 0; k < kWarps; ++k) v += s_part[k][c];
                    part[w * a.cols + c] = v;
                }
            }
        }
    }
}

// column sums alone: a thread has a column of a run of rows
constexpr int kColThreads = 256;
template <class T>
__global__ void __launch_bounds__(kColThreads) norm_cols_kernel(const BwdArgs a) {
    const int c = blockIdx.x * kColThreads + threadIdx.x;
    if (c >= a.cols) return;
    const T* x = static_cast<const T*>(a.x) + c;
    const T* dy = static_cast<const T*>(a.dy) + c;
    float g = 0.f, b = 0.f;
#pragma unroll 4
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float d = to_f32(dy[r * a.dy_stride]);
        g = fmaf(d, (to_f32(x[r * a.x_stride]) - __ldg(a.mean + r)) * __ldg(a.rstd + r), g);
        b += d;
    }
    float* part = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
    part[c] = g;
    part[a.cols + c] = b;
}

// the parts' sums, in their order: 32 columns a CTA, 32 threads a column
__global__ void __launch_bounds__(1024) norm_parts_kernel(const float* part, int parts, int cols, float* dgamma,
                                                          float* dbeta) {
    __shared__ float s[32][33];
    const int i = blockIdx.x * 32 + threadIdx.x;  // column of [dgamma | dbeta]
    float v = 0.f;
    if (i < 2 * cols) {
#pragma unroll 4
        for (int p = threadIdx.y; p < parts; p += 32) v += part[static_cast<int64_t>(p) * 2 * cols + i];
    }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = s[threadIdx.x][threadIdx.y];  // thread (x, y): part x of column y
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int j = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && j < 2 * cols) {
        if (j < cols)
            dgamma[j] = v;
        else
            dbeta[j - cols] = v;
    }
}

template <class T, int V, int G, int U, bool kSums>
int launch(const BwdArgs& a, int* parts, cudaStream_t s) {
    using F = Bwd<T, V, G, U, kSums>;
    const int64_t want = (a.rows + F::rows - 1) / F::rows;
    const int cap = max_parts(a.cols), most = kSms * F::ctas < cap ? kSms * F::ctas : cap;
    const int grid = static_cast<int>(want < most ? want : most);
    if (kSums) *parts = grid;
    norm_bwd_kernel<T, V, G, U, kSums><<<grid, F::threads, 0, s>>>(a);
    return launch_status();
}

template <class T, bool kSums>
int fused(const BwdArgs& a, bool wide, int* parts, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    if (wide) {
        const int n = a.cols / W;
        if (n <= 16) return launch<T, W, 16, 1, kSums>(a, parts, s);
        if (n <= 32) return launch<T, W, 32, 1, kSums>(a, parts, s);
        if (n <= 64) return launch<T, W, 32, 2, kSums>(a, parts, s);
        if (n <= 256) return launch<T, W, 256, 1, kSums>(a, parts, s);
        if (n <= 512) return launch<T, W, 256, 2, kSums>(a, parts, s);
        if (n <= 1024) return launch<T, W, 512, 2, kSums>(a, parts, s);
        if (n <= 2048) return launch<T, W, 512, 4, kSums>(a, parts, s);
        if constexpr (!kSums) {
            if (n <= 4096) return launch<T, W, 1024, 4, false>(a, parts, s);
            if constexpr (W == 4) return launch<T, W, 1024, 8, false>(a, parts, s);
        }
        return IX_ERR_UNSUPPORTED;
    }
    const int n = a.cols;
    if (n <= 32) return launch<T, 1, 32, 1, kSums>(a, parts, s);
    if (n <= 128) return launch<T, 1, 32, 4, kSums>(a, parts, s);
    if (n <= 512) return launch<T, 1, 128, 4, kSums>(a, parts, s);
    if (n <= 2048) return launch<T, 1, 256, 8, kSums>(a, parts, s);
    if (n <= 8192) return launch<T, 1, 512, 16, kSums>(a, parts, s);
    if constexpr (!kSums) return launch<T, 1, 1024, 32, false>(a, parts, s);
    return IX_ERR_UNSUPPORTED;
}

template <class T>
int dispatch(const BwdArgs& a, float* dgamma, float* dbeta, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    int parts = 0, rc = IX_OK;
    if (a.rows > 0) {
        const bool wide = a.cols % W == 0 && a.x_stride % W == 0 && a.dy_stride % W == 0 && a.dx_stride % W == 0 &&
                          aligned16(a.x) && aligned16(a.dy) && aligned16(a.dx);
        if (!dgamma) return fused<T, false>(a, wide, nullptr, s);
        if (a.cols <= (wide ? 2048 * W : 8192)) {
            rc = fused<T, true>(a, wide, &parts, s);
        } else {
            // before dx is written: dx may be dy in place
            parts = static_cast<int>(a.rows < max_parts(a.cols) ? a.rows : max_parts(a.cols));
            norm_cols_kernel<T><<<dim3((a.cols + kColThreads - 1) / kColThreads, parts), kColThreads, 0, s>>>(a);
            rc = launch_status();
            if (rc == IX_OK) rc = fused<T, false>(a, wide, nullptr, s);
        }
        if (rc != IX_OK) return rc;
    }
    if (!dgamma) return IX_OK;
    norm_parts_kernel<<<(2 * a.cols + 31) / 32, dim3(32, 32), 0, s>>>(a.part, parts, a.cols, dgamma, dbeta);
    return launch_status();
}

}  // namespace
}  // namespace dsix

using namespace dsix;

extern "C" size_t ix_layer_norm_bwd_workspace_size(int64_t rows, int cols) {
    if (rows <= 0 || cols <= 0) return 0;
    const int most = max_parts(cols);
    return static_cast<size_t>(rows < most ? rows : most) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

extern "C" int ix_layer_norm_bwd(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                 const void* gamma, int weight_dtype, const float* mean, const float* rstd,
                                 int64_t rows, int cols, void* dx, int64_t dx_stride, float* dgamma, float* dbeta,
                                 int dtype, void* workspace, size_t workspace_bytes, ix_stream_t stream) {
    if (rows < 0 || dy_stride < 0 || x_stride < 0 || cols < 1 || (rows > 1 && dx_stride < cols)) return IX_ERR_SHAPE;
    const int es = dtype_bytes(dtype);
    if (!es || cols > kMaxCols || (weight_dtype != IX_FP32 && weight_dtype != dtype)) return IX_ERR_UNSUPPORTED;
    if (!dgamma != !dbeta) return IX_ERR_NULL;
    if (rows == 0 && !dgamma) return IX_OK;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return IX_ERR_NULL;
    if (rows > 1 && ((dx == dy && dx_stride != dy_stride) || (dx == x && dx_stride != x_stride))) return IX_ERR_SHAPE;
    if (!aligned_to(dy, es) || !aligned_to(x, es) || !aligned_to(dx, es) || !aligned16(gamma) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dgamma, 4) || !aligned_to(dbeta, 4))
        return IX_ERR_ALIGN;
    if (dgamma && rows > 0) {
        if (!workspace || workspace_bytes < ix_layer_norm_bwd_workspace_size(rows, cols)) return IX_ERR_WORKSPACE;
        if (!aligned16(workspace)) return IX_ERR_ALIGN;
    }
    const BwdArgs a{dy, x, gamma, mean, rstd, dx, static_cast<float*>(workspace), dy_stride, x_stride, dx_stride,
                    rows, cols, weight_dtype == IX_FP32, 1.f / static_cast<float>(cols)};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == IX_BF16) return dispatch<__nv_bfloat16>(a, dgamma, dbeta, s);
    if (dtype == IX_FP16) return dispatch<__half>(a, dgamma, dbeta, s);
    return dispatch<float>(a, dgamma, dbeta, s);
}
