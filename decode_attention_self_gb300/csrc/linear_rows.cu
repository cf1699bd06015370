// Matrix product with an epilogue for up to 32 tokens: out = residual + act(x W^T + bias), bound by W's way from memory.
//
// A CTA takes 8 or 16 output columns and all tokens; its warps share K in steps of 32.  W goes from memory to the operand
// registers of mma.sync (m16n8k16) without shared memory: 16 tokens are the rows of one operand, 8 weight rows the
// columns of the other, and since a sum over k may take its terms in any order, a lane's 16 bytes of a row (8 values of k)
// serve as the k slots that the instruction gives that lane, four for one product and four for the next, in both operands
// alike.  A warp's load reads 64 contiguous bytes of each of 8 rows; a group of kGroup steps is on its way while the group
// before is multiplied.  Each group's products make sums of their own, added in fp32: tensor-core chains cut off rather
// than round (about 1e-9 of the value per term).  The warps' sums meet in shared memory and are added in warp order.
// There are no waits on anything but the kernel before.
#include "linear_epilogue.cuh"

namespace dr {
namespace {

constexpr int kMaxWarps = 16;
// steps of 32 k in flight per warp, and again as many ahead
template <int kEights> constexpr int kGroup = kEights > 2 ? 2 : 4;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of W, which no other CTA reads
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p)
                 : "memory");
    return r;
}

// kEights: tokens in eights, 1, 2 or 4;  kBlocks: blocks of 8 weight rows (gated: the second half multiplies the first)
template <int kEights, int kBlocks>
__global__ void __launch_bounds__(kMaxWarps * 32) linear_rows_kernel(const __grid_constant__ LinearParams p) {
    constexpr int kTiles = (kEights + 1) / 2, kSteps = kGroup<kEights>, kRows = kEights * 8;
    extern __shared__ float sums_raw[];
    const auto sums = reinterpret_cast<float (*)[kRows][kBlocks * 8]>(sums_raw);   // of each warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int blocks = p.gated ? kBlocks / 2 : kBlocks;   // of output columns
    const int n0 = blockIdx.x * blocks * 8;
    const auto first_row = [&](int i) {   // of the weight rows of block i
        return i < blocks ? n0 + i * 8 : p.N + n0 + (i - blocks) * 8;
    };
    const int all_rows = p.gated ? 2 * p.N : p.N;
    // W's rows on their way into L2 while the kernel before this one ends (a hint: nothing is read)
    if (warp == 0 && lane < kBlocks) {
        const int row = first_row(lane);
        const int64_t have = (int64_t)min(8, all_rows - row) * p.K * 2;
        if (have > 0) prefetch_l2(p.W + (int64_t)row * p.K, (uint32_t)min(have, (int64_t)32768));
    }
    pdl_wait();
    pdl_trigger();

    const uint16_t *w[kBlocks];
    bool in_w[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int row = first_row(i) + g;
        in_w[i] = row < all_rows;
        w[i] = p.W + (int64_t)(in_w[i] ? row : 0) * p.K;
    }
    bool in_x[kEights];
    const uint16_t *x[kEights];
#pragma unroll
    for (int e = 0; e < kEights; ++e) {
        in_x[e] = e * 8 + g < p.T;
        x[e] = p.x + (in_x[e] ? e * 8 + g : 0) * p.x_stride;
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);

    float acc[kTiles][kBlocks][4] = {};
    uint4 wv[kSteps][kBlocks];
    const int steps = (p.K + 31) / 32;
    const auto load_w = [&](int s0) {
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int k = (s0 + u * warps) * 32 + t * 8;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) wv[u][i] = k < p.K && in_w[i] ? load_once(w[i] + k) : zero;
        }
    };
    load_w(warp);
#pragma unroll 1
    for (int s0 = warp; s0 < steps; s0 += kSteps * warps) {
        uint4 xv[kSteps][kEights], now[kSteps][kBlocks];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int k = (s0 + u * warps) * 32 + t * 8;
#pragma unroll
            for (int e = 0; e < kEights; ++e) xv[u][e] = k < p.K && in_x[e] ? *reinterpret_cast<const uint4 *>(x[e] + k) : zero;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) now[u][i] = wv[u][i];
        }
        if (s0 + kSteps * warps < steps) load_w(s0 + kSteps * warps);
        __syncwarp();   // lanes past K or the last row loaded nothing; the products want all of them at once
        float part[kTiles][kBlocks][4] = {};
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
                const uint4 a = xv[u][2 * m], b = kEights > 1 ? xv[u][kEights > 1 ? 2 * m + 1 : 0] : zero;
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) {
                    mma(part[m][i], a.x, b.x, a.y, b.y, now[u][i].x, now[u][i].y);
                    mma(part[m][i], a.z, b.z, a.w, b.w, now[u][i].z, now[u][i].w);
                }
            }
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][i][j] += part[m][i][j];
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            *reinterpret_cast<float2 *>(&sums[warp][16 * m + g][i * 8 + 2 * t]) = make_float2(acc[m][i][0], acc[m][i][1]);
            if (kEights > 1) *reinterpret_cast<float2 *>(&sums[warp][(16 * m + g + 8) % kRows][i * 8 + 2 * t]) = make_float2(acc[m][i][2], acc[m][i][3]);
        }
    __syncthreads();

    // a pair of columns a thread
    const int pairs = blocks * 4;
#pragma unroll 1
    for (int i = threadIdx.x; i < p.T * pairs; i += blockDim.x) {
        const int row = i / pairs, c = (i - row * pairs) * 2, n = n0 + c;
        if (n >= p.N) continue;
        const bool both = n + 1 < p.N;
        float a[2] = {0.f, 0.f}, b[2] = {0.f, 0.f};
        float r[2] = {0.f, 0.f}, bias[4] = {0.f, 0.f, 0.f, 0.f};
        const int64_t res_at = (int64_t)row * p.res_stride + n;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (j == 0 || both) {
                if (p.residual)
                    r[j] = p.out_f32 ? static_cast<const float *>(p.residual)[res_at + j]
                                     : __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.residual)[res_at + j] << 16);
                if (p.bias) {
                    bias[j] = lin::bf16_at(p.bias, n + j);
                    if (p.gated) bias[2 + j] = lin::bf16_at(p.bias, (int64_t)p.N + n + j);
                }
            }
        for (int s = 0; s < warps; ++s) {
            const float2 v = *reinterpret_cast<const float2 *>(&sums[s][row][c]);
            a[0] += v.x;
            a[1] += v.y;
            if (p.gated) {
                const float2 u = *reinterpret_cast<const float2 *>(&sums[s][row][blocks * 8 + c]);
                b[0] += u.x;
                b[1] += u.y;
            }
        }
        a[0] += bias[0];
        a[1] += bias[1];
        lin::activate<2>(a, p.act);
        if (p.gated) {
            a[0] *= b[0] + bias[2];
            a[1] *= b[1] + bias[3];
        }
        const LinearOut o = lin::output_of(p, n);
        const int64_t at = (int64_t)row * o.stride + (n - o.col0);
        if (p.residual) {
            a[0] = r[0] + a[0];
            a[1] = r[1] + a[1];
        }
        if (p.out_f32) {
            float *to = static_cast<float *>(o.ptr) + at;
            if (p.vec_out && both) {
                *reinterpret_cast<float2 *>(to) = make_float2(a[0], a[1]);
            } else {
                to[0] = a[0];
                if (both) to[1] = a[1];
            }
        } else {
            uint16_t *to = static_cast<uint16_t *>(o.ptr) + at;
            if (p.vec_out && both) {
                *reinterpret_cast<uint32_t *>(to) = lin::pack2(a[0], a[1]);
            } else {
                to[0] = f32_to_bf16_rn(a[0]);
                if (both) to[1] = f32_to_bf16_rn(a[1]);
            }
        }
    }
}

using Kernel = void (*)(const LinearParams);
Kernel kernel_of(int eights, int blocks) {
    return eights == 4 ? (blocks == 2 ? linear_rows_kernel<4, 2> : linear_rows_kernel<4, 1>)
           : eights == 2 ? (blocks == 2 ? linear_rows_kernel<2, 2> : linear_rows_kernel<2, 1>)
                         : (blocks == 2 ? linear_rows_kernel<1, 2> : linear_rows_kernel<1, 1>);
}
size_t sums_bytes(int eights, int blocks, int warps) { return (size_t)warps * eights * 8 * blocks * 8 * sizeof(float); }

// CTAs of such a kernel that an SM holds (asked once per device).
int resident(int eights, int blocks, int warps) {
    static std::atomic<int> known[64][3][2][3];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    std::atomic<int> *slot = dev < 64 ? &known[dev][eights / 2][blocks - 1][warps / 8] : nullptr;
    if (slot && (n = slot->load(std::memory_order_relaxed)) > 0) return n;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel_of(eights, blocks), warps * 32, sums_bytes(eights, blocks, warps)) !=
            cudaSuccess ||
        n < 1)
        n = 1;
    if (slot) slot->store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace

// Blocks of 8 weight rows per CTA (1 or 2) and warps: as many warps as leave the grid one wave and each of them a full group
// of loads; of the two block counts the one with more warps; where they tie, one, or two where the tokens' rows (more than 8 of
// them, read by every CTA) are worth sharing.  Measured (one and two blocks, warps, us): one token 1024 -> 4096 3.4 (4) and 3.1 (8),
// 1536 -> 6144 5.3 (4) and 6.1 (4), 4096 -> 1024 4.0 (16) and 5.2 (16); 16 tokens 1536 -> 6144 9.6 (4) and 6.5 (4).
cudaError_t launch_linear_rows(const LinearParams &p, int sms, cudaStream_t stream) {
    const int eights = p.T <= 8 ? 1 : p.T <= 16 ? 2 : 4;
    const int rows = p.gated ? 2 * p.N : p.N, steps = (p.K + 31) / 32;
    int best = 0, warps = 0;
    for (int blocks = p.gated ? 2 : 1; blocks <= 2; ++blocks) {
        const int ctas = (rows + blocks * 8 - 1) / (blocks * 8);
        int w = kMaxWarps;
        while (w > 4 && (ctas > sms * resident(eights, blocks, w) || steps < w * (eights == 4 ? kGroup<4> : kGroup<1>))) w /= 2;
        if (w > warps || (w == warps && eights > 1 && ctas >= sms)) {
            best = blocks;
            warps = w;
        }
    }
    const int cols = (p.gated ? best / 2 : best) * 8;
    return launch_kernel(kernel_of(eights, best), dim3((unsigned)((p.N + cols - 1) / cols)), dim3((unsigned)(warps * 32)),
                         sums_bytes(eights, best, warps), stream, 1, p);
}

}  // namespace dr
