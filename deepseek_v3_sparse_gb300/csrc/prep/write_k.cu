// write_k.cu -- ix_norm_rope_write_k: layer norm, rotary positions, fp8 coding
// and the paged write of the indexer key, one pass over the token.
//
// Eight lanes hold a token, 16 consecutive values each, so the three reductions
// of a token (mean, centred squares, amax) are three shuffles each, and a
// rotated pair lies in one lane (interleaved; rot = 16) or in two lanes
// rot / 32 apart, each of which forms its own half of the pair.
#include <float.h>

#include "prep.cuh"

namespace dsix {
namespace {

constexpr int kDim = 128;
constexpr int kBlock = 64;
constexpr int kBlockBytes = kBlock * (kDim + 4);
constexpr int kLanes = 8;             // per token
constexpr int kPer = kDim / kLanes;   // values per lane
constexpr int kThreads = 256;

struct WriteArgs {
    const void* k;
    int64_t k_stride, n;
    const float *gamma, *beta;
    float eps;
    const int64_t* positions;
    const float* cos_sin;
    int64_t max_pos;
    int rot, offset, interleaved;
    const int64_t* slots;
    uint8_t* cache;
    int64_t num_blocks;
    int* status;
};

__device__ __forceinline__ float sum8(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <class T>
__global__ void __launch_bounds__(kThreads) norm_rope_write_kernel(const WriteArgs a) {
    constexpr int V = 16 / sizeof(T), NV = kPer / V;
    const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1);
    const T* kin = static_cast<const T*>(a.k);
    float g[kPer], bt[kPer];
    load_f32<kPer>(a.gamma + sub * kPer, g);
    load_f32<kPer>(a.beta + sub * kPer, bt);
    // where this lane's values lie in the rotated part
    const int e0 = sub * kPer - a.offset;  // a multiple of 16
    const bool rotated = e0 >= 0 && e0 < a.rot;
    const int half = a.rot >> 1;
    const bool second = e0 >= half;
    const int apart = a.rot >= 32 ? a.rot / 32 : 0;
    const int other = (lane & ~(kLanes - 1)) | ((sub + (second ? -apart : apart)) & (kLanes - 1));
    const int64_t tokens = (static_cast<int64_t>(gridDim.x) * kThreads) / kLanes;
    // the loop runs for the warp's first token, so that all lanes meet in the shuffles
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes; t0 - (lane / kLanes) < a.n;
         t0 += tokens) {
        const bool live = t0 < a.n;
        float x[kPer];
        int64_t slot = -1, pos = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = 0.f;
        if (live) {
            slot = __ldg(a.slots + t0);
            pos = __ldg(a.positions + t0);
            const T* row = kin + t0 * a.k_stride + sub * kPer;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const Vec<T, V> v = load_vec<T, V>(row + j * V);
#pragma unroll
                for (int i = 0; i < V; ++i) x[j * V + i] = to_f32(v.v[i]);
            }
        }
        const int64_t blk = slot / kBlock;
        bool write = slot >= 0;
        if (write && (blk >= a.num_blocks || pos < 0 || pos >= a.max_pos)) {
            if (sub == 0) flag(a.status, blk >= a.num_blocks ? IX_DEV_BAD_SLOT : IX_DEV_BAD_POSITION);
            write = false;
        }
        float c[kPer], s[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) c[i] = s[i] = 0.f;
        if (write && rotated) {
            const float* row = a.cos_sin + pos * a.rot;
            if (a.interleaved || a.rot == 16) {  // eight pairs in this lane
                const int p0 = a.interleaved ? e0 >> 1 : 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 cq = __ldg(reinterpret_cast<const float4*>(row + p0) + i);
                    const float4 sq = __ldg(reinterpret_cast<const float4*>(row + half + p0) + i);
                    c[4 * i] = cq.x; c[4 * i + 1] = cq.y; c[4 * i + 2] = cq.z; c[4 * i + 3] = cq.w;
                    s[4 * i] = sq.x; s[4 * i + 1] = sq.y; s[4 * i + 2] = sq.z; s[4 * i + 3] = sq.w;
                }
            } else {
                const int p0 = second ? e0 - half : e0;
                load_f32<kPer>(row + p0, c);
                load_f32<kPer>(row + half + p0, s);
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum += x[i];
        const float mean = sum8(sum) * (1.f / kDim);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            x[i] -= mean;
            sq = fmaf(x[i], x[i], sq);
        }
        const float rstd = __fdiv_rn(1.f, __fsqrt_rn(fmaf(sum8(sq), 1.f / kDim, a.eps)));
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = fmaf(x[i] * rstd, g[i], bt[i]);
        if (a.interleaved) {
            if (rotated) {
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) {
                    const float p = x[2 * i], q = x[2 * i + 1];
                    x[2 * i] = p * c[i] - q * s[i];
                    x[2 * i + 1] = p * s[i] + q * c[i];
                }
            }
        } else if (a.rot == 16) {
            if (rotated) {
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) {
                    const float p = x[i], q = x[i + kPer / 2];
                    x[i] = p * c[i] - q * s[i];
                    x[i + kPer / 2] = p * s[i] + q * c[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float y = __shfl_sync(0xffffffffu, x[i], other);
                // the first of a pair: a c - b s; the second: a s + b c
                if (rotated) x[i] = second ? fmaf(y, s[i], x[i] * c[i]) : fmaf(-y, s[i], x[i] * c[i]);
            }
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float scale = fmaxf(__fdiv_rn(amax, 448.f), FLT_MIN);
        if (write) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = cvt_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)) |
                       (cvt_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)) << 16);
            const int at = static_cast<int>(slot % kBlock);
            uint8_t* base = a.cache + blk * kBlockBytes;
            *reinterpret_cast<uint4*>(base + at * kDim + sub * kPer) = make_uint4(w[0], w[1], w[2], w[3]);
            if (sub == 0) *reinterpret_cast<float*>(base + kBlock * kDim + 4 * at) = scale;
        }
    }
}

}  // namespace
}  // namespace dsix

using namespace dsix;

extern "C" int ix_norm_rope_write_k(const void* k, int64_t k_stride, int dtype, int64_t n, const float* gamma,
                                    const float* beta, float eps, const int64_t* positions, const float* cos_sin,
                                    int64_t max_pos, int rot, int offset, int interleaved,
                                    const int64_t* slot_mapping, uint8_t* cache, int64_t num_blocks, int block_size,
                                    ix_stream_t stream) {
    if (n < 0 || num_blocks < 0 || k_stride < 0 || max_pos < 0) return IX_ERR_SHAPE;
    const int es = dtype_bytes(dtype);
    if (!es || block_size != kBlock || !(eps >= 0.f) || !isfinite(eps)) return IX_ERR_UNSUPPORTED;
    if (!(rot == 16 || (rot > 0 && rot % 32 == 0)) || offset < 0 || offset % 16 || offset + rot > kDim)
        return IX_ERR_UNSUPPORTED;
    if (n == 0) return IX_OK;
    if (!k || !gamma || !beta || !positions || !slot_mapping) return IX_ERR_NULL;
    if ((max_pos > 0 && !cos_sin) || (num_blocks > 0 && !cache)) return IX_ERR_NULL;
    if (!aligned16(k) || ((k_stride * es) & 15) || !aligned16(gamma) || !aligned16(beta) || !aligned16(cos_sin) ||
        !aligned16(cache) || !aligned_to(positions, 8) || !aligned_to(slot_mapping, 8))
        return IX_ERR_ALIGN;
    int* st = status_ptr();
    const int sms = num_sms();
    if (!st || sms <= 0) return IX_ERR_CUDA;
    const WriteArgs a{k, k_stride, n, gamma, beta, eps, positions, cos_sin, max_pos, rot, offset, interleaved ? 1 : 0,
                      slot_mapping, cache, num_blocks, st};
    const int64_t want = (n + kThreads / kLanes - 1) / (kThreads / kLanes), cap = static_cast<int64_t>(sms) * 8;
    const int grid = static_cast<int>(want < cap ? want : cap);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == IX_BF16)
        norm_rope_write_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    else if (dtype == IX_FP16)
        norm_rope_write_kernel<__half><<<grid, kThreads, 0, s>>>(a);
    else
        norm_rope_write_kernel<float><<<grid, kThreads, 0, s>>>(a);
    return launch_status();
}
