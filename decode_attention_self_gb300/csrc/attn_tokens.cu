// Attention of single query tokens over a cache of grouped heads, with a score cap, a distance bias and a visible
// interval of keys per token; also the last step of shared-prefix attention (the row's own keys, and the merge with
// the softmax states of the prefix).
//
//   s_j = cap(scale q.k_j) - slope |p - j|,  j in [lo, hi);   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m)
//
// The g query heads of one kv head share its keys, so the products are 16-key x g matrix products.  They run on the
// warp-level matrix instructions (m16n8k16), with the keys (and then the dimensions) as the 16 rows and the heads as
// the 8 columns:
//   S^T [16 keys][8 heads]  = K [16][64] Q^T        four instructions per 8 heads
//   O^T [64 dims][8 heads] += V^T [64][16] P^T      four instructions per 8 heads
// The order in which dimensions are summed, and which output row is which dimension, is free, so a lane loads K and V
// straight from global memory in 16-byte pieces as the fragments that it needs (no shared memory, no transposing
// loads): lane (r, c) = (lane / 4, lane % 4) holds dims 32i + 8c .. +7 of keys r and r + 8, and dims 8r .. 8r + 7 of
// keys 2c, 2c + 1, 2c + 8, 2c + 9.  P^T comes from S^T by two 8x8 register transposes.
// Bound by memory: 4 KB of K and V per 16 keys (bf16) against about 70 warp instructions; even one head in eight
// columns leaves the matrix instructions mostly idle.
//
// e4m3 caches: the codes convert exactly to f16, and the products run in f16 with fp32 sums: q is brought to
// [0.5, 1) times a power of two per head, which f16 holds exactly down to 2^-15 of the largest element (below that
// the error is under 2^-25 of it), and the weights keep 11 bits.  bf16 caches: weights are rounded to bf16 (8 bits)
// for the product with V, their sum is taken in fp32.
#include <cooperative_groups.h>

#include "dr_prompt.h"
#include "dr_rows.cuh"
#include "dr_score.cuh"

namespace cg = cooperative_groups;

namespace dr {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kD = kHeadDim;
constexpr int kTile = kBlockKeys;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Two e4m3 codes (low 16 bits of w) -> f16x2, exact.
__device__ __forceinline__ uint32_t codes2_f16(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

// One 16-key tile as a lane holds it, in the cache's format.
struct Bf16Tile {
    uint4 k[4];   // key r: dims 8c.., 32+8c..; key r+8: the same
    uint4 v[4];   // dims 8r.. of keys 2c, 2c+1, 2c+8, 2c+9
    static constexpr size_t kRowBytes = kD * 2;
    static constexpr bool kF16 = false;
    __device__ __forceinline__ void load_k(int i, const uint8_t *row, int c) {
        k[2 * i] = ld_stream16(row + 16 * c);
        k[2 * i + 1] = ld_stream16(row + 64 + 16 * c);
    }
    __device__ __forceinline__ void load_v(int i, const uint8_t *row, int r) { v[i] = ld_stream16(row + 16 * r); }
    __device__ __forceinline__ void zero_k(int i) { k[2 * i] = k[2 * i + 1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void zero_v(int i) { v[i] = make_uint4(0, 0, 0, 0); }
    // word w (0..7): dims pair w of this lane's 16 dims of key r + 8*i
    __device__ __forceinline__ uint32_t k_word(int i, int w) const { return (&k[2 * i + (w >> 2)].x)[w & 3]; }
    __device__ __forceinline__ void v_words(int i, uint32_t (&o)[4]) const {
        o[0] = v[i].x; o[1] = v[i].y; o[2] = v[i].z; o[3] = v[i].w;
    }
};
struct Fp8Tile {
    uint4 k[2];   // keys r, r+8: codes of dims 16c ..
    uint2 v[4];
    static constexpr size_t kRowBytes = kD;
    static constexpr bool kF16 = true;
    __device__ __forceinline__ void load_k(int i, const uint8_t *row, int c) { k[i] = ld_stream16(row + 16 * c); }
    __device__ __forceinline__ void load_v(int i, const uint8_t *row, int r) { v[i] = ld_stream8(row + 8 * r); }
    __device__ __forceinline__ void zero_k(int i) { k[i] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void zero_v(int i) { v[i] = make_uint2(0, 0); }
    __device__ __forceinline__ uint32_t k_word(int i, int w) const {
        const uint32_t x = (&k[i].x)[w >> 1];
        return codes2_f16((w & 1) ? x >> 16 : x);
    }
    __device__ __forceinline__ void v_words(int i, uint32_t (&o)[4]) const {
        o[0] = codes2_f16(v[i].x); o[1] = codes2_f16(v[i].x >> 16);
        o[2] = codes2_f16(v[i].y); o[3] = codes2_f16(v[i].y >> 16);
    }
};

constexpr float kSlack = 8.0f;   // the reference of the weights moves when a score passes it by 2^8

// kN: groups of 8 query heads of one kv head.
template <typename Tile, bool kPaged, int kN>
__global__ void __launch_bounds__(kThreads) attn_tokens_kernel(const PromptParams p, int splits) {
    constexpr int kHeads = 8 * kN;
    __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
    __shared__ float s_acc[kWarps][kHeads][kD];
    __shared__ float s_M[kHeads], s_L[kHeads];

    const int split = (int)blockIdx.x % splits;
    const int item = (int)blockIdx.x / splits;
    const int b = item / p.tokens_per_row, i0 = item - b * p.tokens_per_row;
    const int hgroups = (p.g + kHeads - 1) / kHeads;
    const int hk = (int)blockIdx.y / hgroups, hg = (int)blockIdx.y - hk * hgroups;
    const int h0 = hk * p.g + hg * kHeads;                  // first query head
    const int nheads = min(kHeads, p.g - hg * kHeads);      // query heads of this CTA
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;

    pdl_wait();
    int s0 = b, n = 1;
    if (p.row_start) {
        s0 = __ldg(p.row_start + b);
        int s1 = __ldg(p.row_start + b + 1);
        if ((s0 < 0 || s1 < s0 || s1 > p.T) && split == 0 && blockIdx.y == 0 && i0 == 0 && threadIdx.x == 0)
            flag_error(p.err, DR_ERRF_ROW_START);
        s0 = min(max(s0, 0), p.T);
        n = min(max(s1, s0), p.T) - s0;
    }
    if (n == 0 || n > p.few_max || i0 >= n) {   // nothing here, or the tile kernel's row (the same in the cluster)
        pdl_trigger();
        return;
    }
    int L = p.kv_len ? __ldg(p.kv_len + b) : 0;
    const int min_len = p.row_start ? n : 0;
    if (L < min_len || L > p.cap) {
        if (split == 0 && blockIdx.y == 0 && i0 == 0 && threadIdx.x == 0 && p.kv_len) flag_error(p.err, DR_ERRF_SEQ_LEN);
        L = min(max(L, 0), p.cap);
    }
    const int prefix = p.prefix_len ? __ldg(p.prefix_len + b) : 0;
    const uint8_t *kc = static_cast<const uint8_t *>(p.k), *vc = static_cast<const uint8_t *>(p.v);

    for (int i = i0; i < n; i += p.tokens_per_row) {
        const int t = s0 + i;
        const int pos = L - n + i;
        int lo = p.first_key ? max(0, __ldg(p.first_key + t)) : 0;
        int hi = p.causal && p.row_start ? min(L, max(pos + 1, prefix)) : L;
        if (lo >= hi) lo = hi = 0;
        const int tile0 = lo / kTile, tiles = (hi + kTile - 1) / kTile - tile0;
        const int per = (tiles + splits - 1) / splits;
        const int tb = tile0 + min(split * per, tiles), te = tile0 + min((split + 1) * per, tiles);

        // Q^T fragments (columns = heads): lane's 16 dims of head r of each group
        uint32_t qf[kN][8];
        float qfac[kN][2];   // e4m3: what a raw score of heads 2c, 2c+1 has to be multiplied by
        float slope[kN][2];
#pragma unroll
        for (int a = 0; a < kN; ++a) {
            const int h = a * 8 + r;
            uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
            if (h < nheads) {
                const uint16_t *src = p.q + (size_t)t * p.q_stride + (size_t)(h0 + h) * kD;
                w0 = ld_ro16(src + (Tile::kF16 ? 16 * c : 8 * c));
                w1 = ld_ro16(src + (Tile::kF16 ? 16 * c + 8 : 32 + 8 * c));
            }
            if constexpr (Tile::kF16) {
                float x[8], y[8];
                unpack8(w0, x);
                unpack8(w1, y);
                float big = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) big = fmaxf(big, fmaxf(fabsf(x[j]), fabsf(y[j])));
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                const float up = pow2_normaliser(big);   // a power of two; 1 for zero, infinite or NaN
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    qf[a][j] = pack_f16(x[2 * j] * up, x[2 * j + 1] * up);
                    qf[a][4 + j] = pack_f16(y[2 * j] * up, y[2 * j + 1] * up);
                }
                qfac[a][0] = 1.0f / __shfl_sync(0xFFFFFFFFu, up, 8 * c);
                qfac[a][1] = 1.0f / __shfl_sync(0xFFFFFFFFu, up, 8 * c + 4);
            } else {
                qf[a][0] = w0.x; qf[a][1] = w0.y; qf[a][2] = w0.z; qf[a][3] = w0.w;
                qf[a][4] = w1.x; qf[a][5] = w1.y; qf[a][6] = w1.z; qf[a][7] = w1.w;
                qfac[a][0] = qfac[a][1] = 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                slope[a][j] = p.slopes && a * 8 + 2 * c + j < nheads
                                  ? __ldg(p.slopes + h0 + a * 8 + 2 * c + j) * 1.4426950408889634f : 0.f;
        }

        float m[kN][2], mref[kN][2], l[kN][2], acc[kN][4][4];
#pragma unroll
        for (int a = 0; a < kN; ++a) {
            m[a][0] = m[a][1] = -INFINITY;
            mref[a][0] = mref[a][1] = l[a][0] = l[a][1] = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[a][x][y] = 0.f;
        }

        // Byte offset of key 16 * tile of this kv head; false: a block outside the pool.
        auto tile_base = [&](int tile, size_t &base) -> bool {
            if (kPaged) {
                const int blk = __ldg(p.table + (size_t)b * p.max_blocks + tile);
                base = ((size_t)blk * p.Hkv + hk) * kTile * Tile::kRowBytes;
                return (unsigned)blk < (unsigned)p.num_blocks;
            }
            base = (((size_t)b * p.Hkv + hk) * (size_t)p.cap + (size_t)tile * kTile) * Tile::kRowBytes;
            return true;
        };
        // 0: nothing to attend, 1: loaded whole, 2: loaded with keys outside [lo, hi) as zeros
        auto load = [&](int tile, Tile &x) -> int {
            size_t base;
            if (!tile_base(tile, base)) {
                if (lane == 0) flag_error(p.err, DR_ERRF_BLOCK_ID);
                return 0;
            }
            const int key = tile * kTile;
            if (key >= lo && key + kTile <= hi) {
#pragma unroll
                for (int j = 0; j < 2; ++j) x.load_k(j, kc + base + (size_t)(r + 8 * j) * Tile::kRowBytes, c);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x.load_v(j, vc + base + (size_t)(2 * c + (j & 1) + 8 * (j >> 1)) * Tile::kRowBytes, r);
                return 1;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int kk = r + 8 * j;
                if (key + kk >= lo && key + kk < hi) x.load_k(j, kc + base + (size_t)kk * Tile::kRowBytes, c);
                else x.zero_k(j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kk = 2 * c + (j & 1) + 8 * (j >> 1);
                if (key + kk >= lo && key + kk < hi) x.load_v(j, vc + base + (size_t)kk * Tile::kRowBytes, r);
                else x.zero_v(j);
            }
            return 2;
        };
        auto consume = [&](int tile, const Tile &x, bool whole) {
            float s[kN][4];
#pragma unroll
            for (int a = 0; a < kN; ++a) s[a][0] = s[a][1] = s[a][2] = s[a][3] = 0.f;
#pragma unroll
            for (int st = 0; st < 4; ++st) {
                const uint32_t af[4] = {x.k_word(0, 2 * st), x.k_word(1, 2 * st), x.k_word(0, 2 * st + 1),
                                        x.k_word(1, 2 * st + 1)};
#pragma unroll
                for (int a = 0; a < kN; ++a) {
                    if (Tile::kF16) mma_f16(s[a], af, qf[a][2 * st], qf[a][2 * st + 1]);
                    else mma_bf16(s[a], af, qf[a][2 * st], qf[a][2 * st + 1]);
                }
            }
            // s[a][0..3]: (key r, head 2c), (key r, head 2c+1), (key r+8, head 2c), (key r+8, head 2c+1)
            const int key = tile * kTile + r;
            bool grows = false;
#pragma unroll
            for (int a = 0; a < kN; ++a)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float raw = Tile::kF16 ? s[a][y] * qfac[a][y & 1] : s[a][y];
                    float v = p.cap_c1 != 0.f ? capped_score(raw, p.cap_c1, p.cap_c2) : raw * p.sscale;
                    const int kk = key + 8 * (y >> 1);
                    if (p.slopes) v -= slope[a][y & 1] * fabsf((float)(pos - kk));
                    if (!whole && (kk < lo || kk >= hi)) v = -INFINITY;
                    s[a][y] = v;
                    grows = grows || v > m[a][y & 1] + kSlack;
                }
            if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
                for (int a = 0; a < kN; ++a)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float mx = fmaxf(m[a][j], fmaxf(s[a][j], s[a][j + 2]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
                        const float corr = mx == -INFINITY ? 1.f : fast_exp2(m[a][j] - mx);
                        m[a][j] = mx;
                        mref[a][j] = mx == -INFINITY ? 0.f : mx;
                        l[a][j] *= corr;
#pragma unroll
                        for (int x4 = 0; x4 < 4; ++x4) {
                            acc[a][x4][j] *= corr;
                            acc[a][x4][j + 2] *= corr;
                        }
                    }
            }
            uint32_t pf[kN][2];
#pragma unroll
            for (int a = 0; a < kN; ++a) {
                float w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) w[y] = fast_exp2(s[a][y] - mref[a][y & 1]);
                l[a][0] += w[0] + w[2];
                l[a][1] += w[1] + w[3];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    pf[a][j] = transpose8x8(Tile::kF16 ? pack_f16(w[2 * j], w[2 * j + 1])
                                                       : pack_bf16(w[2 * j], w[2 * j + 1]));
            }
            uint32_t vw[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x.v_words(j, vw[j]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t af[4] = {__byte_perm(vw[0][y], vw[1][y], 0x5410), __byte_perm(vw[0][y], vw[1][y], 0x7632),
                                        __byte_perm(vw[2][y], vw[3][y], 0x5410), __byte_perm(vw[2][y], vw[3][y], 0x7632)};
#pragma unroll
                for (int a = 0; a < kN; ++a) {
                    if (Tile::kF16) mma_f16(acc[a][y], af, pf[a][0], pf[a][1]);
                    else mma_bf16(acc[a][y], af, pf[a][0], pf[a][1]);
                }
            }
        };

        Tile cur;
        int tile = tb + warp;
        int got = tile < te ? load(tile, cur) : 0;
        for (; tile < te; tile += kWarps) {
            Tile nxt;
            const int nt = tile + kWarps;
            const int ngot = nt < te ? load(nt, nxt) : 0;
            if (got) consume(tile, cur, got == 1);
            cur = nxt;
            got = ngot;
        }

        // The warp's states: sums over the lanes' keys, then one state per warp in shared memory
#pragma unroll
        for (int a = 0; a < kN; ++a)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[a][j] += __shfl_xor_sync(0xFFFFFFFFu, l[a][j], off);
                const int h = a * 8 + 2 * c + j;
                if (r == 0) {
                    s_m[warp][h] = m[a][j];
                    s_l[warp][h] = l[a][j];
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    s_acc[warp][h][8 * r + 2 * y] = acc[a][y][j];
                    s_acc[warp][h][8 * r + 2 * y + 1] = acc[a][y][j + 2];
                }
            }
        __syncthreads();
        // The CTA's state, in the place of warp 0's
        for (int e = threadIdx.x; e < nheads * kD; e += kThreads) {
            const int h = e / kD, d = e % kD;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
            float ls = 0.f, o = 0.f;
            if (M != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float wt = exp2f(s_m[w][h] - M);
                    ls += wt * s_l[w][h];
                    o += wt * s_acc[w][h][d];
                }
            }
            s_acc[0][h][d] = o;   // this thread alone reads and writes column (h, d)
            if (d == 0) {
                s_M[h] = M;
                s_L[h] = ls;
            }
        }
        cg::cluster_group cluster = cg::this_cluster();
        if (splits > 1) cluster.sync();
        else __syncthreads();
        // Every CTA of the cluster finishes its share of the outputs, the CTAs' states in rank order, then the states
        // of the key ranges attended before
        for (int e = split * kThreads + threadIdx.x; e < nheads * kD; e += splits * kThreads) {
            const int h = e / kD, d = e % kD;
            float M = -INFINITY;
            for (int x = 0; x < splits; ++x) M = fmaxf(M, splits > 1 ? *cluster.map_shared_rank(&s_M[h], x) : s_M[h]);
            const size_t row = (size_t)t * p.Hq + h0 + h, rows = (size_t)p.T * p.Hq;
            for (int x = 0; x < p.nparts; ++x) M = fmaxf(M, p.part_ml[x * rows + row].x);
            float ls = 0.f, o = 0.f;
            if (M != -INFINITY) {
                for (int x = 0; x < splits; ++x) {
                    const float wt = exp2f((splits > 1 ? *cluster.map_shared_rank(&s_M[h], x) : s_M[h]) - M);
                    ls += wt * (splits > 1 ? *cluster.map_shared_rank(&s_L[h], x) : s_L[h]);
                    o += wt * (splits > 1 ? *cluster.map_shared_rank(&s_acc[0][h][d], x) : s_acc[0][h][d]);
                }
                o *= p.out_scale;
                for (int x = 0; x < p.nparts; ++x) {
                    const float2 ml = p.part_ml[x * rows + row];
                    if (ml.x == -INFINITY) continue;   // an empty share
                    const float wt = exp2f(ml.x - M);
                    ls += wt * ml.y;
                    o += wt * p.part_acc[(x * rows + row) * kD + d];
                }
            }
            // a sum of weights that is not zero; NaN scores leave NaN
            const float res = ls == 0.f ? 0.f : o / ls;
            if (p.out_f32) static_cast<float *>(p.out)[row * kD + d] = res;
            else static_cast<uint16_t *>(p.out)[row * kD + d] = f32_to_bf16_rn(res);
        }
        if (splits > 1) cluster.sync();   // the states stay until every CTA has read them
        else __syncthreads();
    }
    pdl_trigger();
}

}  // namespace

// CTAs (one cluster) that share a token's keys: enough to give every SM a few CTAs, each at least 64 keys.
int plan_token_splits(long long items, int Hkv, int g, int max_len, bool fp8, int sms) {
    const long long rows = items * Hkv * ((g + 15) / 16);
    const long long key_bytes = 2LL * kD * (fp8 ? 1 : 2);
    long long s = ((long long)max_len * key_bytes + 256 * 1024 - 1) / (256 * 1024);
    const long long fill = (4LL * sms + rows - 1) / rows;
    if (fill > s) s = fill;
    const long long by_keys = ((long long)max_len + 63) / 64;
    if (s > by_keys) s = by_keys;
    if (s > 8) s = 8;
    return s < 1 ? 1 : (int)s;
}

cudaError_t launch_attn_tokens(const PromptParams &p, bool paged, bool fp8, int splits, cudaStream_t stream) {
    const int kn = p.g > 8 ? 2 : 1;
    const unsigned hgroups = (unsigned)((p.g + 8 * kn - 1) / (8 * kn));
    const dim3 grid((unsigned)((long long)p.B * p.tokens_per_row * splits), (unsigned)p.Hkv * hgroups);
    void (*kern)(PromptParams, int);
#define DR_PICK(TILE, P) (kn == 2 ? attn_tokens_kernel<TILE, P, 2> : attn_tokens_kernel<TILE, P, 1>)
    if (fp8) kern = paged ? DR_PICK(Fp8Tile, true) : DR_PICK(Fp8Tile, false);
    else kern = paged ? DR_PICK(Bf16Tile, true) : DR_PICK(Bf16Tile, false);
#undef DR_PICK
    return launch_kernel(kern, grid, dim3(kThreads), 0, stream, (unsigned)splits, p, splits);
}

}  // namespace dr
