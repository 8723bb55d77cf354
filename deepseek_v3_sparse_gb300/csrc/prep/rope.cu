// rope.cu -- rotary positions: the frequencies (host), the table, and the
// rotation of a part of every head.
#include "prep.cuh"

namespace dsix {
namespace {

constexpr int kMaxPairs = 128;
constexpr int kThreads = 256;
constexpr int kMaxHeads = 65536, kMaxDim = 65536;

// ---------------------------------------------------------------------------
// ix_rope_table.  The angle p * f of pair f at position p is held in turns, as
// a 64-bit fixed-point fraction: with F = round(f / (2 pi) * 2^64) mod 2^64, the
// wrapping product p * F is the angle modulo one turn, exact but for F's one
// rounding (p * 2^-65 turns).  The nearest quarter turn is split off in
// integers; what is left, at most an eighth of a turn, goes through sincospif in
// f32 with its relative accuracy intact, also next to the zeros.
// ---------------------------------------------------------------------------
struct TurnTable {
    uint64_t step[kMaxPairs];
};

__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ TurnTable f, int pairs,
                                                              int64_t first, int64_t n, float amplitude,
                                                              float* __restrict__ out) {
    const int64_t total = n * pairs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / pairs;
        const int p = static_cast<int>(i - r * pairs);
        const uint64_t turn = static_cast<uint64_t>(first + r) * f.step[p];
        const uint64_t quarter = (turn + (1ull << 61)) >> 62;
        const int64_t rest = static_cast<int64_t>(turn - (quarter << 62));
        float s, c;
        sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
        const bool swap = quarter & 1;
        float cs = swap ? s : c, sn = swap ? c : s;
        if (quarter == 1 || quarter == 2) cs = -cs;
        if (quarter == 2 || quarter == 3) sn = -sn;
        out[r * 2 * pairs + p] = cs * amplitude;
        out[r * 2 * pairs + pairs + p] = sn * amplitude;
    }
}

// ---------------------------------------------------------------------------
// ix_rope.  A head is cut into items of two vectors of V elements: a pair item
// holds V whole pairs (half layout: a vector of each half; interleaved: two
// adjacent vectors), a copy item two vectors of the rest.  A thread has one item
// of kHeads heads of a token, so the cosines and sines it read serve all of
// them.
// ---------------------------------------------------------------------------
struct RopeSide {
    const void* x;
    void* out;
    int heads, groups;  // groups = ceil(heads / kHeads): head u of group g is g + u * groups
    int64_t xt, xh, ot, oh;
};

struct RopeArgs {
    RopeSide side[2];
    int64_t blocks0;  // CTAs of side 0
    int64_t tokens;
    int pair_items, items;  // per head
    int dim, offset, rot, copy_vecs;
    int interleaved;
    float sign;
    const int64_t* positions;
    const float* cos_sin;
    int64_t max_pos;
    int* status;
};

template <class T, int V, int kHeads>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
    const int which = blockIdx.x >= a.blocks0;
    const RopeSide& d = a.side[which];
    const int64_t idx = (static_cast<int64_t>(blockIdx.x) - (which ? a.blocks0 : 0)) * kThreads + threadIdx.x;
    const int64_t per_token = static_cast<int64_t>(d.groups) * a.items;
    const int64_t t = idx / per_token;
    if (t >= a.tokens) return;
    const int rest = static_cast<int>(idx - t * per_token);
    const int g = rest / a.items, item = rest - g * a.items;
    const int64_t p = __ldg(a.positions + t);
    const T* x = static_cast<const T*>(d.x) + t * d.xt;
    T* out = static_cast<T*>(d.out) + t * d.ot;
    const bool pair = item < a.pair_items;
    int e0, e1;  // first elements of the item's two vectors
    bool has1 = true;
    if (pair) {
        e0 = a.offset + (a.interleaved ? 2 : 1) * item * V;
        e1 = a.interleaved ? e0 + V : e0 + a.rot / 2;
    } else {
        const int v = 2 * (item - a.pair_items);
        e0 = v * V < a.offset ? v * V : v * V + a.rot;
        e1 = (v + 1) * V < a.offset ? (v + 1) * V : (v + 1) * V + a.rot;
        has1 = v + 1 < a.copy_vecs;
    }
    Vec<T, V> v0[kHeads], v1[kHeads];
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
        const int h = g + u * d.groups;
        if (h < d.heads) {
            v0[u] = load_vec<T, V>(x + h * d.xh + e0);
            if (has1) v1[u] = load_vec<T, V>(x + h * d.xh + e1);
        }
    }
    if (p < 0 || p >= a.max_pos) {
        if (rest == 0) flag(a.status, IX_DEV_BAD_POSITION);
        return;
    }
    if (pair) {
        float c[V], s[V];
        const float* row = a.cos_sin + p * a.rot + item * V;
        load_f32<V>(row, c);
        load_f32<V>(row + a.rot / 2, s);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] *= a.sign;
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            if (g + u * d.groups >= d.heads) break;
            float e[2 * V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                e[i] = to_f32(v0[u].v[i]);
                e[V + i] = to_f32(v1[u].v[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int ia = a.interleaved ? 2 * i : i, ib = a.interleaved ? 2 * i + 1 : V + i;
                const float y = e[ia], z = e[ib];
                // the roundings are spelled out: every variant gives the same bits
                e[ia] = fmaf(-z, s[i], __fmul_rn(y, c[i]));
                e[ib] = fmaf(y, s[i], __fmul_rn(z, c[i]));
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v0[u].v[i] = from_f32<T>(e[i]);
                v1[u].v[i] = from_f32<T>(e[V + i]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
        const int h = g + u * d.groups;
        if (h < d.heads) {
            store_vec<T, V>(out + h * d.oh + e0, v0[u]);
            if (has1) store_vec<T, V>(out + h * d.oh + e1, v1[u]);
        }
    }
}

template <class T, int V, int kHeads>
int launch(RopeArgs& a, bool copies, cudaStream_t s) {
    a.pair_items = a.rot / (2 * V);
    a.copy_vecs = copies ? (a.dim - a.rot) / V : 0;
    a.items = a.pair_items + (a.copy_vecs + 1) / 2;
    int64_t blocks[2] = {0, 0};
    for (int w = 0; w < 2; ++w) {
        RopeSide& d = a.side[w];
        if (!d.x) continue;
        d.groups = (d.heads + kHeads - 1) / kHeads;
        blocks[w] = (a.tokens * d.groups * a.items + kThreads - 1) / kThreads;
    }
    a.blocks0 = blocks[0];
    if (blocks[0] + blocks[1] > INT32_MAX) return IX_ERR_UNSUPPORTED;
    rope_kernel<T, V, kHeads><<<static_cast<unsigned>(blocks[0] + blocks[1]), kThreads, 0, s>>>(a);
    return launch_status();
}

template <class T>
int dispatch(RopeArgs& a, bool copies, int sms, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    // 16-byte vectors where every pointer, stride and part of the head allows them
    bool wide = a.offset % W == 0 && (a.rot / 2) % W == 0 && aligned16(a.cos_sin) &&
                (!copies || (a.dim - a.offset - a.rot) % W == 0);
    for (const RopeSide& d : a.side)
        if (d.x)
            wide = wide && aligned16(d.x) && aligned16(d.out) && d.xt % W == 0 && d.ot % W == 0 &&
                   (d.heads == 1 || (d.xh % W == 0 && d.oh % W == 0));
    const int64_t values = a.tokens * a.side[0].heads * a.dim;
    // four heads a thread once that leaves every SM its share of threads
    const bool many = values * static_cast<int64_t>(sizeof(T)) >= static_cast<int64_t>(sms) * 2048 * 128;
    if (wide) return many ? launch<T, W, 4>(a, copies, s) : launch<T, W, 1>(a, copies, s);
    return many ? launch<T, 1, 4>(a, copies, s) : launch<T, 1, 1>(a, copies, s);
}

// an output whose elements are all distinct: heads within tokens, or tokens within heads
bool distinct(int64_t tokens, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
    if ((tokens <= 1 || ts >= (heads - 1) * hs + dim) && (heads <= 1 || hs >= dim)) return true;
    return (heads <= 1 || hs >= (tokens - 1) * ts + dim) && (tokens <= 1 || ts >= dim);
}

}  // namespace
}  // namespace dsix

using namespace dsix;

extern "C" int ix_rope_frequencies(int scaling, int rot, double base, double factor, double original,
                                   double beta_fast, double beta_slow, double* inv_freq) {
    if (rot < 2 || rot > 2 * kMaxPairs || rot % 2 || !(base > 1.0) || !isfinite(base)) return IX_ERR_UNSUPPORTED;
    if (scaling < IX_ROPE_PLAIN || scaling > IX_ROPE_YARN) return IX_ERR_UNSUPPORTED;
    if (scaling != IX_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return IX_ERR_UNSUPPORTED;
    if (!inv_freq) return IX_ERR_NULL;
    if (scaling == IX_ROPE_NTK && rot > 2) base *= pow(factor, static_cast<double>(rot) / (rot - 2));
    double low = 0, high = 0;
    if (scaling == IX_ROPE_YARN) {
        if (!(original > 0) || !isfinite(original) || !(beta_slow > 0) || !(beta_fast >= beta_slow) ||
            !isfinite(beta_fast))
            return IX_ERR_UNSUPPORTED;
        const double two_pi = 6.283185307179586476925;
        auto pair = [&](double turns) { return rot * log(original / (two_pi * turns)) / (2 * log(base)); };
        low = fmax(floor(pair(beta_fast)), 0.0);
        high = fmin(ceil(pair(beta_slow)), rot - 1.0);
    }
    for (int i = 0; i < rot / 2; ++i) {
        double w = pow(base, -2.0 * i / rot);
        if (scaling == IX_ROPE_LINEAR) w /= factor;
        if (scaling == IX_ROPE_YARN) {
            const double g = fmin(fmax((i - low) / fmax(high - low, 0.001), 0.0), 1.0);
            w = w * (1 - g) + w / factor * g;
        }
        inv_freq[i] = w;
    }
    return IX_OK;
}

extern "C" int ix_rope_table(const double* inv_freq, int rot, int64_t first, int64_t n, double amplitude,
                             float* cos_sin, ix_stream_t stream) {
    if (first < 0 || n < 0) return IX_ERR_SHAPE;
    if (rot < 2 || rot > 2 * kMaxPairs || rot % 2 || first > (1ll << 40) || n > (1ll << 40) ||
        first + n > (1ll << 40) || !isfinite(amplitude))
        return IX_ERR_UNSUPPORTED;
    if (!inv_freq) return IX_ERR_NULL;
    TurnTable f{};
    for (int i = 0; i < rot / 2; ++i) {
        if (!isfinite(inv_freq[i])) return IX_ERR_UNSUPPORTED;
        long double turns = static_cast<long double>(inv_freq[i]) / 6.283185307179586476925286766559L;
        turns -= floorl(turns);  // [0, 1]: whole turns per position change nothing
        const long double scaled = roundl(turns * 0x1p64L);
        f.step[i] = scaled >= 0x1p64L ? 0 : static_cast<uint64_t>(scaled);
    }
    if (n == 0) return IX_OK;
    if (!cos_sin) return IX_ERR_NULL;
    if (!aligned16(cos_sin)) return IX_ERR_ALIGN;
    const int sms = num_sms();
    if (sms <= 0) return IX_ERR_CUDA;
    const int64_t want = (n * (rot / 2) + kThreads - 1) / kThreads, cap = static_cast<int64_t>(sms) * 8;
    rope_table_kernel<<<static_cast<int>(want < cap ? want : cap), kThreads, 0,
                        reinterpret_cast<cudaStream_t>(stream)>>>(f, rot / 2, first, n,
                                                                  static_cast<float>(amplitude), cos_sin);
    return launch_status();
}

extern "C" int ix_rope(const ix_rope_tensor* x, const ix_rope_tensor* x2, int dtype, int64_t tokens, int head_dim,
                       int offset, const int64_t* positions, const float* cos_sin, int64_t max_pos, int rot,
                       int flags, ix_stream_t stream) {
    if (!x) return IX_ERR_NULL;
    const ix_rope_tensor* both[2] = {x, x2};
    if (tokens < 0 || max_pos < 0 || head_dim < 1 || offset < 0) return IX_ERR_SHAPE;
    if (head_dim > kMaxDim) return IX_ERR_UNSUPPORTED;
    for (const ix_rope_tensor* d : both)
        if (d && (d->heads < 1 || d->heads > kMaxHeads || d->x_token_stride < 0 || d->x_head_stride < 0 ||
                  !distinct(tokens, d->heads, head_dim, d->out_token_stride, d->out_head_stride)))
            return IX_ERR_SHAPE;
    const int es = dtype_bytes(dtype);
    if (!es || rot < 2 || rot > 2 * kMaxPairs || rot % 2 || offset + static_cast<int64_t>(rot) > head_dim ||
        (flags & ~(IX_ROPE_INTERLEAVED | IX_ROPE_INVERSE)))
        return IX_ERR_UNSUPPORTED;
    if (tokens == 0) return IX_OK;
    if (!positions || (max_pos > 0 && !cos_sin)) return IX_ERR_NULL;
    if (!aligned_to(positions, 8) || !aligned_to(cos_sin, 4)) return IX_ERR_ALIGN;
    RopeArgs a{};
    bool copies = false;
    for (int w = 0; w < 2; ++w) {
        const ix_rope_tensor* d = both[w];
        if (!d) continue;
        if (!d->x || !d->out) return IX_ERR_NULL;
        if (!aligned_to(d->x, es) || !aligned_to(d->out, es)) return IX_ERR_ALIGN;
        if (d->x == d->out) {
            if (d->x_token_stride != d->out_token_stride ||
                (d->heads > 1 && d->x_head_stride != d->out_head_stride))
                return IX_ERR_SHAPE;
        } else {
            copies = copies || head_dim > rot;
        }
        a.side[w] = {d->x, d->out, d->heads, 0, d->x_token_stride, d->x_head_stride, d->out_token_stride,
                     d->out_head_stride};
    }
    a.tokens = tokens;
    a.dim = head_dim;
    a.offset = offset;
    a.rot = rot;
    a.interleaved = (flags & IX_ROPE_INTERLEAVED) ? 1 : 0;
    a.sign = (flags & IX_ROPE_INVERSE) ? -1.f : 1.f;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.max_pos = max_pos;
    a.status = status_ptr();
    const int sms = num_sms();
    if (!a.status || sms <= 0) return IX_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == IX_BF16) return dispatch<__nv_bfloat16>(a, copies, sms, s);
    if (dtype == IX_FP16) return dispatch<__half>(a, copies, sms, s);
    return dispatch<float>(a, copies, sms, s);
}
