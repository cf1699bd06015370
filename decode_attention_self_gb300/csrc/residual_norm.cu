// Residual, gate and the norms around a block, one pass over the rows:
//   h = residual + scale * gate * post(x),   y = pre(h)
// with post and pre nothing, layer norm ((v - mean) / sqrt(mean((v - mean)^2) + eps)) or RMS norm (v / sqrt(mean(v^2) + eps)),
// times weight, plus bias.
//
// A row lives in the registers of `lanes` threads (8 elements per vector, V vectors per thread), so each input is read once and
// each output written once, and layer norm takes its mean first and the squared differences after, without cancellation.
// Everything between the loads and the stores is fp32; y comes from h before it is rounded for storing.  Row sums go
// over warp shuffles, and over shared memory where a row has several warps, in a fixed order.
#include "dr_layer.h"
#include "dr_device.cuh"

namespace dr {
namespace {

constexpr int kMaxRowThreads = 512;
constexpr int kMaxWarps = kMaxRowThreads / 32;

// Eight elements, as they lie in memory.
template <bool f32>
struct Raw;
template <>
struct Raw<false> {
    uint4 w;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(w, f); }
};
template <>
struct Raw<true> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        a = q[0];
        b = q[1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

__device__ __forceinline__ void store8(void *p, int64_t i, bool f32, const float (&f)[8]) {
    if (f32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = (uint32_t)f32_to_bf16_rn(f[2 * j]) | ((uint32_t)f32_to_bf16_rn(f[2 * j + 1]) << 16);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The sum over a row's threads, the same in each of them.  `lanes`: a power of two; of 64 and more a CTA holds one row.
__device__ __forceinline__ float row_sum(float v, int lanes, float *shared) {
    for (int o = min(lanes, 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lanes > 32) {
        const int warps = lanes / 32;
        if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
        for (int i = 0; i < warps; ++i) v += shared[i];
    }
    return v;
}

// The norm of the row that v holds (elements past the row are 0 and stay out of the sums).
template <int V>
__device__ __forceinline__ void norm(float (&v)[V][8], const NormParams &n, const ResidualNormParams &p, int first, int lanes,
                                     float *shared) {
    const float inv = 1.0f / (float)p.Dm;
    if (n.kind == DR_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        const float mean = row_sum(s, lanes, shared) * inv;
        shared += kMaxWarps;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((first + i * lanes) * 8 < p.Dm)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] -= mean;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[i][j], v[i][j], s);
    const float r = 1.0f / sqrtf(row_sum(s, lanes, shared) * inv + n.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = (first + i * lanes) * 8;
        if (d >= p.Dm) break;
        float w[8], b[8];
        if (n.weight) {
            unpack8(*reinterpret_cast<const uint4 *>(n.weight + d), w);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.f;
        }
        if (n.bias) {
            unpack8(*reinterpret_cast<const uint4 *>(n.bias + d), b);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * r, w[j], b[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * w[j];
        }
    }
}

template <int V, bool kXf32, bool kResF32>
__global__ void __launch_bounds__(kMaxRowThreads) residual_norm_kernel(const ResidualNormParams p, const int lanes) {
    __shared__ float sums[4][kMaxWarps];   // a row of slots per sum, so that none is written again while it is read
    const int per_cta = blockDim.x / lanes;
    const int first = threadIdx.x & (lanes - 1);
    const int64_t row = (int64_t)blockIdx.x * per_cta + threadIdx.x / lanes;
    const bool live = row < p.T;   // the other threads take part in the shuffles
    const int64_t t = live ? row : 0;
    pdl_wait();
    Raw<kXf32> rx[V];
    Raw<kResF32> rr[V];
    uint4 rg[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = (first + i * lanes) * 8;
        if (d < p.Dm) {
            rx[i].load(p.x, t * p.x_stride + d);
            if (p.residual) rr[i].load(p.residual, t * p.res_stride + d);
            if (p.gate) rg[i] = *reinterpret_cast<const uint4 *>(p.gate + t * p.gate_stride + d);
        }
    }
    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if ((first + i * lanes) * 8 < p.Dm) {
            rx[i].get(v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
    }
    pdl_trigger();
    if (p.post.kind != DR_NORM_NONE) norm<V>(v, p.post, p, first, lanes, sums[0]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = (first + i * lanes) * 8;
        if (d >= p.Dm) break;
        if (p.gate) {
            float g[8];
            unpack8(rg[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= g[j];
        }
        if (p.residual) {
            float r[8];
            rr[i].get(r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j], p.scale, r[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= p.scale;
        }
        if (p.h && live) store8(p.h, t * p.h_stride + d, p.res_f32, v[i]);
    }
    if (!p.y) return;
    if (p.pre.kind != DR_NORM_NONE) norm<V>(v, p.pre, p, first, lanes, sums[2]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = (first + i * lanes) * 8;
        if (d < p.Dm && live) store8(p.y, t * p.y_stride + d, p.y_f32, v[i]);
    }
}

template <int V>
cudaError_t launch(const ResidualNormParams &p, int lanes, int threads, cudaStream_t stream) {
    const int per_cta = threads / lanes;
    const dim3 grid((unsigned)((p.T + (int64_t)per_cta - 1) / per_cta));
    auto kern = p.x_f32 ? (p.res_f32 ? residual_norm_kernel<V, true, true> : residual_norm_kernel<V, true, false>)
                        : (p.res_f32 ? residual_norm_kernel<V, false, true> : residual_norm_kernel<V, false, false>);
    return launch_kernel(kern, grid, dim3((unsigned)threads), 0, stream, 1, p, lanes);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormParams &p, cudaStream_t stream) {
    const int vecs = p.Dm / 8;
    int V = 1, lanes = 8;
    while (lanes < 256 && lanes < vecs) lanes *= 2;
    while (V < 4 && V * lanes < vecs) V *= 2;
    while (lanes < kMaxRowThreads && V * lanes < vecs) lanes *= 2;
    const int threads = lanes < 64 ? 128 : lanes;
    switch (V) {
        case 1: return launch<1>(p, lanes, threads, stream);
        case 2: return launch<2>(p, lanes, threads, stream);
        default: return launch<4>(p, lanes, threads, stream);
    }
}

}  // namespace dr
