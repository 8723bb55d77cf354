// norm_fwd.cu -- ix_layer_norm.
//
// The row is read once and stays in registers, as it came, for the three passes
// over it: the sum, the sum of the centred squares (no cancellation, whatever
// the mean), the output.
#include "norm.cuh"

namespace dsix {
namespace {

struct NormArgs {
    const void* x;
    const void *gamma, *beta;
    void* out;
    float *mean, *rstd;
    int64_t x_stride, out_stride, rows;
    int cols, weight_f32;
    float eps, inv_cols;
};

template <class T, int V, int G, int U>
__global__ void __launch_bounds__(RowShape<G>::threads) norm_fwd_kernel(const NormArgs a) {
    __shared__ float s_sum[2][32];
    const int t = threadIdx.x % G;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * RowShape<G>::rows + threadIdx.x / G;
    const bool live = row < a.rows;
    Vec<T, V> x[U];
    const T* in = static_cast<const T*>(a.x) + row * a.x_stride;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (u * G + t) * V;
        if (live && c < a.cols) {
            x[u] = load_vec<T, V>(in + c);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[u].v[i] = from_f32<T>(0.f);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) sum += to_f32(x[u].v[i]);
    const float mean = row_sum<G>(sum, s_sum[0]) * a.inv_cols;
    float sq = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if ((u * G + t) * V < a.cols) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = to_f32(x[u].v[i]) - mean;
                sq = fmaf(d, d, sq);
            }
        }
    }
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(fmaf(row_sum<G>(sq, s_sum[1]), a.inv_cols, a.eps)));
    if (!live) return;
    if (t == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (u * G + t) * V;
        if (c < a.cols) {
            float g[V], b[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                g[i] = 1.f;
                b[i] = 0.f;
            }
            if (a.gamma) load_weight<T, V>(a.gamma, a.weight_f32, c, g);
            if (a.beta) load_weight<T, V>(a.beta, a.weight_f32, c, b);
            Vec<T, V> y;
#pragma unroll
            for (int i = 0; i < V; ++i) y.v[i] = from_f32<T>(fmaf((to_f32(x[u].v[i]) - mean) * rstd, g[i], b[i]));
            store_vec<T, V>(out + c, y);
        }
    }
}

template <class T, int V, int G, int U>
int launch(const NormArgs& a, cudaStream_t s) {
    const int64_t blocks = (a.rows + RowShape<G>::rows - 1) / RowShape<G>::rows;
    if (blocks > INT32_MAX) return IX_ERR_UNSUPPORTED;
    norm_fwd_kernel<T, V, G, U><<<static_cast<unsigned>(blocks), RowShape<G>::threads, 0, s>>>(a);
    return launch_status();
}

template <class T>
int dispatch(const NormArgs& a, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    const bool wide = a.cols % W == 0 && a.x_stride % W == 0 && a.out_stride % W == 0 && aligned16(a.x) &&
                      aligned16(a.out);
    if (wide) {
        const int n = a.cols / W;
        if (n <= 16) return launch<T, W, 16, 1>(a, s);
        if (n <= 32) return launch<T, W, 32, 1>(a, s);
        if (n <= 64) return launch<T, W, 32, 2>(a, s);
        if (n <= 128) return launch<T, W, 32, 4>(a, s);
        if (n <= 256) return launch<T, W, 128, 2>(a, s);
        if (n <= 512) return launch<T, W, 256, 2>(a, s);
        if (n <= 1024) return launch<T, W, 256, 4>(a, s);
        if (n <= 2048) return launch<T, W, 512, 4>(a, s);
        if (n <= 4096) return launch<T, W, 1024, 4>(a, s);
        if constexpr (W == 4) return launch<T, W, 1024, 8>(a, s);
        return IX_ERR_UNSUPPORTED;
    }
    const int n = a.cols;
    if (n <= 32) return launch<T, 1, 32, 1>(a, s);
    if (n <= 128) return launch<T, 1, 32, 4>(a, s);
    if (n <= 512) return launch<T, 1, 32, 16>(a, s);
    if (n <= 2048) return launch<T, 1, 128, 16>(a, s);
    if (n <= 8192) return launch<T, 1, 512, 16>(a, s);
    return launch<T, 1, 1024, 32>(a, s);
}

}  // namespace
}  // namespace dsix

using namespace dsix;

extern "C" int ix_layer_norm(const void* x, int64_t x_stride, const void* gamma, const void* beta, int weight_dtype,
                             float eps, int64_t rows, int cols, void* out, int64_t out_stride, float* mean,
                             float* rstd, int dtype, ix_stream_t stream) {
    if (rows < 0 || x_stride < 0 || cols < 1 || (rows > 1 && out_stride < cols)) return IX_ERR_SHAPE;
    const int es = dtype_bytes(dtype);
    if (!es || cols > kMaxCols || !(eps >= 0.f) || !isfinite(eps) ||
        (weight_dtype != IX_FP32 && weight_dtype != dtype))
        return IX_ERR_UNSUPPORTED;
    if (rows == 0) return IX_OK;
    if (!x || !out || !mean != !rstd) return IX_ERR_NULL;
    if (x == out && rows > 1 && x_stride != out_stride) return IX_ERR_SHAPE;
    if (!aligned_to(x, es) || !aligned_to(out, es) || !aligned16(gamma) || !aligned16(beta) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return IX_ERR_ALIGN;
    const NormArgs a{x, gamma, beta, out, mean, rstd, x_stride, out_stride, rows, cols, weight_dtype == IX_FP32,
                     eps, 1.f / static_cast<float>(cols)};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == IX_BF16) return dispatch<__nv_bfloat16>(a, s);
    if (dtype == IX_FP16) return dispatch<__half>(a, s);
    return dispatch<float>(a, s);
}
