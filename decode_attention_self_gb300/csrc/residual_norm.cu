// Residual, gate and the norms around a block, one pass over the rows:
//   h = residual + scale * gate * post(x),   y = pre(h)
// with post and pre nothing, layer norm ((v - mean) / sqrt(mean((v - mean)^2) + eps)) or RMS norm (v / sqrt(mean(v^2) + eps)),
// times weight, plus bias.
//
// A row lives in the registers of `lanes` threads (8 elements per vector, V vectors per thread), so each input is read once and
// each output written once, and layer norm takes its mean first and the squared differences after, without cancellation.
// Everything between the loads and the stores is fp32; y comes from h before it is rounded for storing.  Row sums go
// over warp shuffles, and over shared memory where a row has several warps, in a fixed order.  Memory bounds many rows,
// latency few; arithmetic comes close to both (packed fp32 instructions: a row of 1024 took 690 instructions a lane without).
// CTAs that stay and take rows in turn were slower than a grid of short ones (fp32 stream of 65536 x 1024: 145 us, 116 now): the
// SMs run at different rates, and a fixed share of the rows cannot follow that.
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
    using T = uint16_t;
    uint4 w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        f[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
        f[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
        f[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
        f[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
    }
};
template <>
struct Raw<true> {
    using T = float;
    float4 a, b;
    __device__ __forceinline__ void load(const T *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        f[0] = make_float2(a.x, a.y);
        f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y);
        f[3] = make_float2(b.z, b.w);
    }
};
using Bf16 = Raw<false>;

__device__ __forceinline__ uint32_t pack2(float2 v) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
    return r;
}
__device__ __forceinline__ void store8(void *p, int64_t i, bool f32, const float2 (&f)[4]) {
    if (f32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        q[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
    }
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The sum over a row's threads, the same in each of them.  `lanes`: a power of two in a warp, or the warps of a CTA.
__device__ __forceinline__ float row_sum(float v, int lanes, float *shared) {
    if (lanes >= 32) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    } else {
        for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    }
    if (lanes > 32) {
        const int warps = lanes / 32;
        if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
        for (int i = 0; i < warps; ++i) v += shared[i];
    }
    return v;
}

// The norm of the row that v holds (elements past the row are 0 and stay out of the sums).  kFull: the row fills its threads.
template <int V, bool kFull>
__device__ __forceinline__ void norm(float2 (&v)[V][4], const NormParams &n, int Dm, int d0, int dstep, int lanes, float *shared) {
    const float inv = 1.0f / (float)Dm;
    if (n.kind == DR_NORM_LAYER) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s = __fadd2_rn(s, v[i][j]);
        const float2 mean = both(-row_sum(s.x + s.y, lanes, shared) * inv);
        shared += kMaxWarps;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (kFull || d0 + i * dstep < Dm)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = __fadd2_rn(v[i][j], mean);
    }
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s = __ffma2_rn(v[i][j], v[i][j], s);
    const float2 r = both(1.0f / sqrtf(row_sum(s.x + s.y, lanes, shared) * inv + n.eps));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = d0 + i * dstep;
        if (!kFull && d >= Dm) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(v[i][j], r);
    }
    if (n.weight)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int d = d0 + i * dstep;
            if (!kFull && d >= Dm) break;
            Bf16 raw;
            float2 w[4];
            raw.load(n.weight + d);
            raw.get(w);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(v[i][j], w[j]);
        }
    if (n.bias)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int d = d0 + i * dstep;
            if (!kFull && d >= Dm) break;
            Bf16 raw;
            float2 b[4];
            raw.load(n.bias + d);
            raw.get(b);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = __fadd2_rn(v[i][j], b[j]);
        }
}

// A CTA takes `rounds` times as many rows as its threads hold, one after the other; a row's inputs are on their way while the
// row before is stored and normed.
template <int V, bool kXf32, bool kResF32, bool kFull>
__global__ void __launch_bounds__(kMaxRowThreads) residual_norm_kernel(const ResidualNormParams p, const int lanes, const int rounds) {
    // slots per sum and, in turn, per row: none is written again while a slower warp may read it
    __shared__ float sums[2][4][kMaxWarps];
    const int per_cta = blockDim.x / lanes;
    const int d0 = (lanes > 32 ? threadIdx.x : threadIdx.x & (lanes - 1)) * 8, dstep = lanes * 8;
    const int64_t base = (int64_t)blockIdx.x * rounds * per_cta;
    int64_t row = base + threadIdx.x / lanes;
    pdl_wait();
    Raw<kXf32> rx[V];
    Raw<kResF32> rr[V];
    Bf16 rg[V];
    const auto load = [&](int64_t t) {
        const auto *x = static_cast<const typename Raw<kXf32>::T *>(p.x) + t * p.x_stride + d0;
        const auto *r = static_cast<const typename Raw<kResF32>::T *>(p.residual) + t * p.res_stride + d0;
        const uint16_t *g = p.gate + t * p.gate_stride + d0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (kFull || d0 + i * dstep < p.Dm) rx[i].load(x + i * dstep);
        if (p.residual)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (kFull || d0 + i * dstep < p.Dm) rr[i].load(r + i * dstep);
        if (p.gate)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (kFull || d0 + i * dstep < p.Dm) rg[i].load(g + i * dstep);
    };
    if (row < p.T) load(row);
    // all threads of a CTA stay together: those without a row take part in the shuffles and barriers
#pragma unroll 1
    for (int round = 0; round < rounds && base + (int64_t)round * per_cta < p.T; ++round, row += per_cta) {
        const bool live = row < p.T;
        float2 v[V][4];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (live && (kFull || d0 + i * dstep < p.Dm)) {
                rx[i].get(v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = both(0.f);
            }
        }
        if (p.post.kind != DR_NORM_NONE) norm<V, kFull>(v, p.post, p.Dm, d0, dstep, lanes, sums[round & 1][0]);
        if (p.gate)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!kFull && d0 + i * dstep >= p.Dm) break;
                float2 g[4];
                rg[i].get(g);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(v[i][j], g[j]);
            }
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!live || (!kFull && d0 + i * dstep >= p.Dm)) break;
                float2 r[4];
                rr[i].get(r);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = __ffma2_rn(v[i][j], both(p.scale), r[j]);
            }
        } else if (p.scale != 1.0f) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(v[i][j], both(p.scale));
        }
        if (round + 1 < rounds && row + per_cta < p.T) load(row + per_cta);
        if (round == 0) pdl_trigger();
        if (p.h && live)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (kFull || d0 + i * dstep < p.Dm) store8(p.h, row * p.h_stride + d0 + i * dstep, p.res_f32, v[i]);
        if (!p.y) continue;
        if (p.pre.kind != DR_NORM_NONE) norm<V, kFull>(v, p.pre, p.Dm, d0, dstep, lanes, sums[round & 1][2]);
        if (live)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (kFull || d0 + i * dstep < p.Dm) store8(p.y, row * p.y_stride + d0 + i * dstep, p.y_f32, v[i]);
    }
}

template <int V, bool kFull>
auto kernel_of(bool x_f32, bool res_f32) {
    return x_f32 ? (res_f32 ? residual_norm_kernel<V, true, true, kFull> : residual_norm_kernel<V, true, false, kFull>)
                 : (res_f32 ? residual_norm_kernel<V, false, true, kFull> : residual_norm_kernel<V, false, false, kFull>);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormParams &p, cudaStream_t stream) {
    const int sms = current_device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Few rows: 8 elements a thread, for the shortest way through a row.  Many: 16 to 32 a thread (to 24 where a stream is fp32),
    // which leaves less to do per element, two rows in turn, the second's inputs on their way during the first, and of these
    // the most that leaves the fewest threads without work.  us: 65536 x 1024, RMS norm of a sum, 8 elements 97, 16 a thread 84, 32
    // 83, 32 and two rows 80, four rows 81 (80 at the rate of a copy); 32768 x 1536, both norms and a gate, 8 elements 121, 16 108, 24
    // 101, 32 (a quarter of the threads idle) 118, with an fp32 stream 126, 118, 107; 32768 x 768 58, 54, 47, 56 and 61, 70, 54.
    // Border: 400 x 1536 8 elements 3.5, 24 4.1; 1000 x 768 4.2 and 3.9, 1000 x 1536 6.2 and 5.1; 128 x 1024 8 elements 2.1, 16 2.4.
    const int vecs = p.Dm / 8;
    const auto lanes_of = [&](int v) {   // threads of a row: a power of two in a warp, or whole warps
        const int n = (vecs + v - 1) / v;
        return n > 32 ? (n + 31) / 32 * 32 : n > 16 ? 32 : n > 8 ? 16 : 8;
    };
    int V = p.T <= 2 * sms || (int64_t)p.T * vecs <= 600LL * sms ? 1 : p.x_f32 || p.res_f32 ? 3 : 4;
    for (int v = V - 1; v > 0; --v)
        if (v * lanes_of(v) < V * lanes_of(V)) V = v;
    if (lanes_of(V) > kMaxRowThreads) V = lanes_of(2) > kMaxRowThreads ? 4 : 2;
    const int lanes = lanes_of(V);
    const int threads = lanes <= 32 ? 128 : lanes, per_cta = threads / lanes;
    const int rounds = (int64_t)p.T / per_cta >= 32LL * sms ? 2 : 1;
    const bool full = V * lanes == vecs, xf = p.x_f32, rf = p.res_f32;
    const auto kernel = V == 1 ? (full ? kernel_of<1, true>(xf, rf) : kernel_of<1, false>(xf, rf))
                        : V == 2 ? (full ? kernel_of<2, true>(xf, rf) : kernel_of<2, false>(xf, rf))
                        : V == 3 ? (full ? kernel_of<3, true>(xf, rf) : kernel_of<3, false>(xf, rf))
                                 : (full ? kernel_of<4, true>(xf, rf) : kernel_of<4, false>(xf, rf));
    const int64_t rows = (int64_t)per_cta * rounds;
    return launch_kernel(kernel, dim3((unsigned)((p.T + rows - 1) / rows)), dim3((unsigned)threads), 0, stream, 1, p, lanes, rounds);
}

}  // namespace dr
