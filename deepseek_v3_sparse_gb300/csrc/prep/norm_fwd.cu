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
struct Fwd : RowShape<G> {
    static constexpr int E = U * V, words = U * ((V * sizeof(T) + 3) / 4);
    // the weights stay in registers where a thread has few columns
    static constexpr bool hold = E <= 16 && V > 1 && G < 1024;
    static constexpr int ahead = RowShape<G>::narrow && words <= 4 ? 3 : E <= 16 ? 1 : 0;
    static constexpr int ctas = ctas_per_sm(RowShape<G>::threads, (hold ? 2 * E : 0) + (ahead + 1) * words + 36);
};

template <class T, int V, int G, int U>
__global__ void __launch_bounds__(Fwd<T, V, G, U>::threads, Fwd<T, V, G, U>::ctas) norm_fwd_kernel(const NormArgs a) {
    using F = Fwd<T, V, G, U>;
    __shared__ float s_sum[4][1][32];
    const int t = threadIdx.x % G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * F::rows;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * F::rows;
    const int sub = threadIdx.x / G;
    auto load = [&](Vec<T, V>(&x)[U], int64_t row) {
        const T* in = static_cast<const T*>(a.x) + row * a.x_stride;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * G + t) * V;
            x[u] = row < a.rows && c < a.cols ? load_vec<T, V>(in + c) : zero_vec<T, V>();
        }
    };
    Vec<T, V> ring[F::ahead + 1][U];  // the present row and the next ones
#pragma unroll
    for (int k = 0; k <= F::ahead; ++k) load(ring[k], row0 + k * step + sub);
    float g[F::hold ? U : 1][V], b[F::hold ? U : 1][V];
    auto weights = [&](float(&gv)[V], float(&bv)[V], int c) {
        fill<V>(gv, 1.f);
        fill<V>(bv, 0.f);
        if (c < a.cols) {
            if (a.gamma) load_weight<T, V>(a.gamma, a.weight_f32, c, gv);
            if (a.beta) load_weight<T, V>(a.beta, a.weight_f32, c, bv);
        }
    };
    if constexpr (F::hold) {
#pragma unroll
        for (int u = 0; u < U; ++u) weights(g[u], b[u], (u * G + t) * V);
    }
    int flip = 0;  // the sums of consecutive rows use other places: one barrier a sum is enough
    for (int64_t r0 = row0; r0 < a.rows; r0 += step) {
        Vec<T, V>(&x)[U] = ring[0];
        const int64_t row = r0 + sub;
        float sum[1] = {0.f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[V];
            x[u].unpack(f);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[0] += f[i];
        }
        row_sums<G>(sum, s_sum[2 * flip]);
        const float mean = sum[0] * a.inv_cols;
        float sq[1] = {0.f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if ((u * G + t) * V < a.cols) {
                float f[V];
                x[u].unpack(f);
#pragma unroll
                for (int i = 0; i < V; ++i) sq[0] = fmaf(f[i] - mean, f[i] - mean, sq[0]);
            }
        }
        row_sums<G>(sq, s_sum[2 * flip + 1]);
        flip ^= 1;
        const float rstd = __fdiv_rn(1.f, __fsqrt_rn(fmaf(sq[0], a.inv_cols, a.eps)));
        if (row < a.rows) {
            if (t == 0 && a.mean) {
                a.mean[row] = mean;
                a.rstd[row] = rstd;
            }
            T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * G + t) * V;
                if constexpr (!F::hold) weights(g[0], b[0], c);
                if (c < a.cols) {
                    float f[V];
                    x[u].unpack(f);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        f[i] = fmaf((f[i] - mean) * rstd, g[F::hold ? u : 0][i], b[F::hold ? u : 0][i]);
                    Vec<T, V> y;
                    y.pack(f);
                    store_vec<T, V>(out + c, y);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < F::ahead; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) ring[k][u] = ring[k + 1][u];
        load(ring[F::ahead], row + (F::ahead + 1) * step);
    }
}

template <class T, int V, int G, int U>
int launch(const NormArgs& a, cudaStream_t s) {
    using F = Fwd<T, V, G, U>;
    const int64_t want = (a.rows + F::rows - 1) / F::rows, most = kSms * F::ctas;
    norm_fwd_kernel<T, V, G, U><<<static_cast<int>(want < most ? want : most), F::threads, 0, s>>>(a);
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
        if (n <= 128) return launch<T, W, 64, 2>(a, s);
        if (n <= 256) return launch<T, W, 128, 2>(a, s);
        if (n <= 512) return launch<T, W, 256, 2>(a, s);
        if (n <= 1024) return launch<T, W, 512, 2>(a, s);
        if (n <= 2048) return launch<T, W, 1024, 2>(a, s);
        if (n <= 4096) return launch<T, W, 1024, 4>(a, s);
        if constexpr (W == 4) return launch<T, W, 1024, 8>(a, s);
        return IX_ERR_UNSUPPORTED;
    }
    const int n = a.cols;
    if (n <= 32) return launch<T, 1, 32, 1>(a, s);
    if (n <= 128) return launch<T, 1, 32, 4>(a, s);
    if (n <= 512) return launch<T, 1, 64, 8>(a, s);
    if (n <= 2048) return launch<T, 1, 256, 8>(a, s);
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
