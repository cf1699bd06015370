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
// loads): lane (r, c) = (lane / 4, lane % 4) holds dims 16c .. 16c + 15 of keys r and r + 8, and dims 8r .. 8r + 7 of
// keys 2c, 2c + 1, 2c + 8, 2c + 9.  P^T comes from S^T by two 8x8 register transposes.
// Bound by memory: 4 KB of K and V per 16 keys (bf16); even one head in eight columns leaves the matrix instructions
// mostly idle.  Measured: 128 rows of 512..4096 keys, 16 heads, 190 us (6.7 TB/s); e4m3 123 us (5.2 TB/s, where the
// conversions count).  A ring of bulk copies in shared memory (4 tiles in flight per warp) was slower at every size:
// what the loads wait for is the row's chain length - block id - keys, and fewer CTAs per SM hide less of it.
//
// e4m3 caches: the codes convert exactly to f16, and the products run in f16 with fp32 sums: q is brought below 2^15 by
// a power of two per head, which f16 holds exactly down to 2^-31 of the largest element (below that the error is under
// 2^-39 of it), and the weights keep 11 bits down to 2^-21 of the row's largest (kLift).  bf16 caches: a weight goes to
// the product with V as its upper 8 bits and the rest rounded to bf16, 16 bits in all; their sum is taken in fp32.  With
// groups of up to 4 heads the rests go through columns that are idle otherwise, at no matrix instruction more (the rows
// above: 189.4 us with 8-bit weights, 189.7 so, 196 as products of their own); larger groups take four more per 16 keys
// and 8 heads (groups of 16, 2 kv heads: 55 -> 57 us).
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

// Loads of data read once per call, past L1 (cached in L2 alone).  Behind the tile kernel this grid reads before it waits,
// and L1 may then still hold lines from before the last writer; the writer's lines themselves are in L2, for it finished
// before the tile kernel let this grid start.  32 bytes: the lanes of a key cover its row in one request.
__device__ __forceinline__ void ld_l2_32(const void *p, uint4 &a, uint4 &b) {
    asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
}
__device__ __forceinline__ uint4 ld_l2_16(const void *p) { return __ldcg(static_cast<const uint4 *>(p)); }
__device__ __forceinline__ uint2 ld_l2_8(const void *p) { return __ldcg(static_cast<const uint2 *>(p)); }

// One 16-key tile as a lane holds it, in the cache's format.
struct Bf16Tile {
    uint4 k[4];   // keys r, r+8: dims 16c ..
    uint4 v[4];   // dims 8r.. of keys 2c, 2c+1, 2c+8, 2c+9
    static constexpr size_t kRowBytes = kD * 2;
    static constexpr bool kF16 = false;
    __device__ __forceinline__ void load_k(int i, const uint8_t *row, int c) {
        ld_l2_32(row + 32 * c, k[2 * i], k[2 * i + 1]);
    }
    __device__ __forceinline__ void load_v(int i, const uint8_t *row, int r) {
        v[i] = ld_l2_16(row + 16 * r);
    }
    __device__ __forceinline__ void zero_k(int i) { k[2 * i] = k[2 * i + 1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void zero_v(int i) { v[i] = make_uint4(0, 0, 0, 0); }
    // words 2 st and 2 st + 1 of this lane's 16 dims (8 pairs) of key r + 8 i
    __device__ __forceinline__ void k_words(int i, int st, uint32_t &a, uint32_t &b) const {
        const uint4 &w = k[2 * i + (st >> 1)];
        a = st & 1 ? w.z : w.x;
        b = st & 1 ? w.w : w.y;
    }
    __device__ __forceinline__ void v_words(int i, uint32_t (&o)[4]) const {
        o[0] = v[i].x; o[1] = v[i].y; o[2] = v[i].z; o[3] = v[i].w;
    }
};
struct Fp8Tile {
    uint4 k[2];   // keys r, r+8: codes of dims 16c ..
    uint2 v[4];
    static constexpr size_t kRowBytes = kD;
    static constexpr bool kF16 = true;
    __device__ __forceinline__ void load_k(int i, const uint8_t *row, int c) {
        k[i] = ld_l2_16(row + 16 * c);
    }
    __device__ __forceinline__ void load_v(int i, const uint8_t *row, int r) {
        v[i] = ld_l2_8(row + 8 * r);
    }
    __device__ __forceinline__ void zero_k(int i) { k[i] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void zero_v(int i) { v[i] = make_uint2(0, 0); }
    __device__ __forceinline__ void k_words(int i, int st, uint32_t &a, uint32_t &b) const {
        codes4_f16(st == 0 ? k[i].x : st == 1 ? k[i].y : st == 2 ? k[i].z : k[i].w, a, b);
    }
    __device__ __forceinline__ void v_words(int i, uint32_t (&o)[4]) const {
        codes4_f16(v[i].x, o[0], o[1]);
        codes4_f16(v[i].y, o[2], o[3]);
    }
};

// 16-key tiles of one pass of a warp, and CTAs per SM.  With groups of up to 8 heads two tiles per pass give the chain
// scores - maximum - weights - sums two independent halves: 128 rows of 512..4096 bf16 keys, 16 heads, 4% less
// against one tile at 5 CTAs per SM (rows of 1..256 keys lose 17%); three CTAs or five (spills) are slower.
// Groups of 16 heads take one tile: two would spill.
template <typename Tile, int kN>
__host__ __device__ constexpr int tiles_per_pass() { return kN == 2 ? 1 : 2; }
template <typename Tile, int kN>
__host__ __device__ constexpr int ctas_per_sm() { return kN == 2 ? 3 : Tile::kF16 ? 5 : 4; }
constexpr int kMaxSplits = 8;   // CTAs per token and kv head: one portable cluster

template <int kN>
struct Shared {
    static constexpr int kHeads = 8 * kN, kBlocks = kHeads * kD / kThreads;
    float m[kWarps][kHeads], l[kWarps][kHeads];   // the warps' states
    float acc[kWarps][kHeads][kD];
    float pm[kHeads], pl[kHeads];                 // states attended before: [pass][team]
    alignas(16) float pacc[kHeads][kD];
    // what the cluster's CTAs send: every head's (m, l), and the sums of the outputs that this CTA finishes
    float M[kMaxSplits][kHeads], L[kMaxSplits][kHeads];
    float sent[kMaxSplits + kBlocks][kThreads];   // [block / splits][rank]
};

// kN: groups of 8 query heads of one kv head; kPlain: no cap, no bias; kTwice (bf16, up to 4 heads): columns 4 .. 7 repeat
// the heads of columns 0 .. 3 and carry the rests of their weights.
template <typename Tile, bool kPaged, int kN, bool kPlain, bool kTwice>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<Tile, kN>())
    attn_tokens_kernel(const PromptParams p, int splits) {
    constexpr int kHeads = 8 * kN;
    constexpr int kT = tiles_per_pass<Tile, kN>();  // 16-key tiles of one pass of a warp
    constexpr int kBlocks = kHeads * kD / kThreads;     // blocks of kThreads outputs; block x is finished by rank x % splits
    __shared__ Shared<kN> sh;
    auto &s_m = sh.m, &s_l = sh.l;
    auto &s_acc = sh.acc;
    auto &s_pm = sh.pm, &s_pl = sh.pl;
    auto &s_pacc = sh.pacc;
    auto &s_M = sh.M, &s_L = sh.L;
    auto &s_sent = sh.sent;

    // splits fastest, then heads, then rows: a block of a paged cache holds all heads of its keys side by side
    const int hgroups = (p.g + kHeads - 1) / kHeads, hys = p.Hkv * hgroups;
    const int split = (int)(blockIdx.x % (unsigned)splits), rest = (int)(blockIdx.x / (unsigned)splits);
    const int b = rest / hys, hy = rest - b * hys;
    const int hk = hy / hgroups, hg = hy - hk * hgroups;
    const int h0 = hk * p.g + hg * kHeads;                  // first query head
    const int nheads = min(kHeads, p.g - hg * kHeads);      // query heads of this CTA
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;

    // Behind the tile kernel of the same call nothing but the states that it leaves has to be waited for: it let this grid
    // start once all of its CTAs had waited for the kernels before it.  (The wait still comes, at the end: who waits for
    // this grid waits for that one.)
    if (!p.after_tiles) pdl_wait();
    int s0 = b, n = 1;
    int L = p.kv_len ? __ldcg(p.kv_len + b) : 0;
    const int prefix = p.prefix_len ? __ldcg(p.prefix_len + b) : 0;
    if (p.row_start) {
        s0 = __ldcg(p.row_start + b);
        int s1 = __ldcg(p.row_start + b + 1);
        if ((s0 < 0 || s1 < s0 || s1 > p.T || (b == 0 && s0 != 0)) && split == 0 && hy == 0 && threadIdx.x == 0)
            flag_error(p.err, DR_ERRF_ROW_START);
        s0 = min(max(s0, 0), p.T);
        n = min(max(s1, s0), p.T) - s0;
    }
    if (n == 0 || n > p.few_max) {   // nothing here, or the tile kernel's row (the same in the cluster)
        if (p.after_tiles) pdl_wait();
        return;
    }
    const int min_len = p.row_start ? n : 0;
    if (L < min_len || L > p.cap) {
        if (split == 0 && hy == 0 && threadIdx.x == 0 && p.kv_len) flag_error(p.err, DR_ERRF_SEQ_LEN);
        L = min(max(L, 0), p.cap);
    }
    // What is sent to another CTA's shared memory needs that CTA to have started: announced here, waited for there.
    cg::cluster_group cluster = cg::this_cluster();
    if (splits > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const auto finish = [&](size_t row, int d, float ls, float o) {
        const float res = ls == 0.f ? 0.f : o / ls;   // no key: zero; NaN scores leave NaN (state_max)
        if (p.out_f32) static_cast<float *>(p.out)[row * kD + d] = res;
        else static_cast<uint16_t *>(p.out)[row * kD + d] = f32_to_bf16_rn(res);
    };
    for (int i = 0; i < n; ++i) {
        const int t = s0 + i;
        const int pos = L - n + i;
        int lo = p.first_key ? max(0, __ldcg(p.first_key + t)) : 0;
        int hi = p.causal && p.row_start ? min(L, max(pos + 1, prefix)) : L;
        if (lo >= hi) lo = hi = 0;
        const int tile0 = lo / kTile, tiles = (hi + kTile - 1) / kTile - tile0;
        const int per = (tiles + splits - 1) / splits;
        const int tb = tile0 + min(split * per, tiles), te = tile0 + min((split + 1) * per, tiles);

        // Block ids of the warp's next 32 / kT passes, one per lane: lane e has tile e % kT of pass e / kT
        int ids = 0;
        const auto fetch_ids = [&](int first) {
            const int x = first + lane / kT * (kWarps * kT) + lane % kT;
            ids = x < te ? __ldcg(p.table + (size_t)b * p.max_blocks + x) : -1;
        };
        // Byte offset of tile y of pass n of the warp (tile `tile` of the row); false: past the end, or no such block
        auto tile_base = [&](int n, int y, int tile, size_t &base) -> bool {
            int blk = 0;
            if (kPaged) blk = __shfl_sync(0xFFFFFFFFu, ids, n % (32 / kT) * kT + y);
            if (tile >= te) return false;
            if (kPaged) {
                base = ((size_t)blk * p.Hkv + hk) * kTile * Tile::kRowBytes;
                if ((unsigned)blk < (unsigned)p.num_blocks) return true;
                if (lane == 0) flag_error(p.err, DR_ERRF_BLOCK_ID);
                return false;
            }
            base = (((size_t)b * p.Hkv + hk) * (size_t)p.cap + (size_t)tile * kTile) * Tile::kRowBytes;
            return true;
        };
        const uint8_t *kc = static_cast<const uint8_t *>(p.k), *vc = static_cast<const uint8_t *>(p.v);
        // kT tiles from `first` on: where they lie, which of them are there, and whether all of their keys are attended
        struct Group {
            size_t base[kT];
            unsigned there;
            bool whole;
        };
        auto locate = [&](int n, int first, Group &g) {
            if (kPaged && n % (32 / kT) == 0) fetch_ids(first);
            g.there = 0;
#pragma unroll
            for (int y = 0; y < kT; ++y) g.there |= tile_base(n, y, first + y, g.base[y]) ? 1u << y : 0u;
            g.whole = g.there == (1u << kT) - 1 && first * kTile >= lo && (first + kT) * kTile <= hi;
        };
        // Keys that are not attended are loaded as zeros
        auto load = [&](int first, const Group &g, Tile (&x)[kT]) {
            if (g.whole) {
#pragma unroll
                for (int y = 0; y < kT; ++y) {
                    const uint8_t *kp = kc + g.base[y] + r * Tile::kRowBytes, *vp = vc + g.base[y] + 2 * c * Tile::kRowBytes;
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[y].load_k(j, kp + 8 * j * Tile::kRowBytes, c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[y].load_v(j, vp + ((j & 1) + 8 * (j >> 1)) * Tile::kRowBytes, r);
                }
                return;
            }
#pragma unroll
            for (int y = 0; y < kT; ++y) {
                const bool there = (g.there >> y) & 1;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int kk = r + 8 * j, key = (first + y) * kTile + kk;
                    if (there && key >= lo && key < hi) x[y].load_k(j, kc + g.base[y] + kk * Tile::kRowBytes, c);
                    else x[y].zero_k(j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int kk = 2 * c + (j & 1) + 8 * (j >> 1), key = (first + y) * kTile + kk;
                    if (there && key >= lo && key < hi) x[y].load_v(j, vc + g.base[y] + kk * Tile::kRowBytes, r);
                    else x[y].zero_v(j);
                }
            }
        };
        // The first keys go out before the query is waited for
        Tile x[kT];
        Group cur, nxt;
        int tile = tb + warp * kT, pass = 0;
        if (tile < te) {
            locate(0, tile, cur);
            load(tile, cur, x);
        }

        // Q^T fragments (columns = heads): lane's 16 dims of head r of each group
        uint32_t qf[kN][8];
        float qfac[kN][2], qmul[kN][2];   // e4m3: what a raw score of heads 2c, 2c+1 has to be multiplied by
        float slope[kN][2];
#pragma unroll
        for (int a = 0; a < kN; ++a) {
            const int h = kTwice ? r & 3 : a * 8 + r;
            uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
            if (h < nheads) {
                const uint16_t *src = p.q + (size_t)t * p.q_stride + (size_t)(h0 + h) * kD;
                w0 = ld_l2_16(src + 16 * c);
                w1 = ld_l2_16(src + 16 * c + 8);
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
            qmul[a][0] = qfac[a][0] * p.sscale;
            qmul[a][1] = qfac[a][1] * p.sscale;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = kTwice ? (2 * c + j) & 3 : a * 8 + 2 * c + j;
                slope[a][j] = p.slopes && h < nheads ? __ldcg(p.slopes + h0 + h) * 1.4426950408889634f : 0.f;
            }
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

        while (tile < te) {
            float s[kT][kN][4];
#pragma unroll
            for (int y = 0; y < kT; ++y)
#pragma unroll
                for (int a = 0; a < kN; ++a) s[y][a][0] = s[y][a][1] = s[y][a][2] = s[y][a][3] = 0.f;
#pragma unroll
            for (int st = 0; st < 4; ++st)
#pragma unroll
                for (int y = 0; y < kT; ++y) {
                    uint32_t af[4];
                    x[y].k_words(0, st, af[0], af[2]);
                    x[y].k_words(1, st, af[1], af[3]);
#pragma unroll
                    for (int a = 0; a < kN; ++a) {
                        if (Tile::kF16) mma_f16(s[y][a], af, qf[a][2 * st], qf[a][2 * st + 1]);
                        else mma_bf16(s[y][a], af, qf[a][2 * st], qf[a][2 * st + 1]);
                    }
                }
            // s[y][a][0..3]: (key r, head 2c), (key r, head 2c+1), (key r+8, head 2c), (key r+8, head 2c+1) of tile y
            const int next = tile + kWarps * kT;
            if (next < te) locate(++pass, next, nxt);
            if (!kPlain && p.cap_c1 != 0.f) {
                float raw[kT * kN * 4];
#pragma unroll
                for (int e = 0; e < kT * kN * 4; ++e) {
                    raw[e] = s[e / (kN * 4)][e / 4 % kN][e % 4];
                    if (Tile::kF16) raw[e] *= qfac[e / 4 % kN][e & 1];
                }
                ScoreCap(p.cap_c1, p.cap_c2, p.sscale)(raw);
#pragma unroll
                for (int e = 0; e < kT * kN * 4; ++e) s[e / (kN * 4)][e / 4 % kN][e % 4] = raw[e];
            }
#pragma unroll
            for (int y = 0; y < kT; ++y)
#pragma unroll
                for (int a = 0; a < kN; ++a)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        float v = s[y][a][z];
                        if (kPlain || p.cap_c1 == 0.f) v *= Tile::kF16 ? qmul[a][z & 1] : p.sscale;
                        if (!kPlain && p.slopes)
                            v -= slope[a][z & 1] * fabsf((float)(pos - (tile + y) * kTile - r - 8 * (z >> 1)));
                        s[y][a][z] = v;
                    }
            if (!cur.whole) {
#pragma unroll
                for (int y = 0; y < kT; ++y)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int key = (tile + y) * kTile + r + 8 * j;
                        if (key < lo || key >= hi || !((cur.there >> y) & 1))
#pragma unroll
                            for (int a = 0; a < kN; ++a) s[y][a][2 * j] = s[y][a][2 * j + 1] = -INFINITY;
                    }
            }
            float mx[kN][2];
            bool grows = false;
#pragma unroll
            for (int a = 0; a < kN; ++a)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[a][j] = fmaxf(s[0][a][j], s[0][a][j + 2]);
#pragma unroll
                    for (int y = 1; y < kT; ++y) mx[a][j] = fmaxf(mx[a][j], fmaxf(s[y][a][j], s[y][a][j + 2]));
                    grows = grows || mx[a][j] > m[a][j] + kSlack;
                }
            if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
                for (int a = 0; a < kN; ++a)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = fmaxf(m[a][j], mx[a][j]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
                        const float corr = top == -INFINITY ? 1.f : fast_exp2(m[a][j] - top);
                        m[a][j] = top;
                        mref[a][j] = top == -INFINITY ? 0.f : top - kLift<Tile::kF16>;
                        l[a][j] *= corr;
#pragma unroll
                        for (int x4 = 0; x4 < 4; ++x4) {
                            acc[a][x4][j] *= corr;
                            acc[a][x4][j + 2] *= corr;
                        }
                    }
            }
            // bf16: a weight is its upper 8 bits and the rest rounded to bf16, 16 bits in all
            uint32_t pf[kT][kN][2], pr[kT][kN][2];
            const float own = kTwice && c >= 2 ? 1.f : 0.f, upper = kTwice && c >= 2 ? -1.f : 1.f;
#pragma unroll
            for (int y = 0; y < kT; ++y)
#pragma unroll
                for (int a = 0; a < kN; ++a) {
                    float w[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) w[z] = fast_exp2(s[y][a][z] - mref[a][z & 1]);
                    l[a][0] += w[0] + w[2];
                    l[a][1] += w[1] + w[3];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if constexpr (Tile::kF16) {
                            pf[y][a][j] = transpose8x8(pack_f16(w[2 * j], w[2 * j + 1]));
                        } else {
                            const float2 v = make_float2(w[2 * j], w[2 * j + 1]);
                            const float2 up = make_float2(__uint_as_float(__float_as_uint(v.x) & 0xFFFF0000u),
                                                          __uint_as_float(__float_as_uint(v.y) & 0xFFFF0000u));
                            if constexpr (kTwice) {   // exact: upper bits, or weight minus upper bits
                                const float2 x = __ffma2_rn(up, make_float2(upper, upper),
                                                            __fmul2_rn(v, make_float2(own, own)));
                                pf[y][a][j] = transpose8x8(pack_bf16(x.x, x.y));
                            } else {
                                pf[y][a][j] = transpose8x8(pack_bf16(up.x, up.y));
                                pr[y][a][j] = transpose8x8(pack_bf16(v.x - up.x, v.y - up.y));
                            }
                        }
                    }
                }
#pragma unroll
            for (int y = 0; y < kT; ++y) {
                uint32_t vw[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[y].v_words(j, vw[j]);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const uint32_t af[4] = {
                        __byte_perm(vw[0][z], vw[1][z], 0x5410), __byte_perm(vw[0][z], vw[1][z], 0x7632),
                        __byte_perm(vw[2][z], vw[3][z], 0x5410), __byte_perm(vw[2][z], vw[3][z], 0x7632)};
#pragma unroll
                    for (int a = 0; a < kN; ++a) {
                        if constexpr (Tile::kF16) {
                            mma_f16(acc[a][z], af, pf[y][a][0], pf[y][a][1]);
                        } else {
                            if constexpr (!kTwice) mma_bf16(acc[a][z], af, pr[y][a][0], pr[y][a][1]);
                            mma_bf16(acc[a][z], af, pf[y][a][0], pf[y][a][1]);
                        }
                    }
                }
            }
            if (next < te) load(next, nxt, x);
            tile = next;
            cur = nxt;
        }

        // The warp's states: sums over the lanes' keys, then one state per warp in shared memory
#pragma unroll
        for (int a = 0; a < kN; ++a)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[a][j] += __shfl_xor_sync(0xFFFFFFFFu, l[a][j], off);
                const int h = a * 8 + 2 * c + j;
                const bool rests = kTwice && h >= 4;   // sums of head h - 4, added where they are read
                if (h - (rests ? 4 : 0) >= nheads) continue;
                if (r == 0 && !rests) {
                    s_m[warp][h] = state_max(m[a][j] - kLift<Tile::kF16>, l[a][j]);
                    s_l[warp][h] = l[a][j];
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    s_acc[warp][h][8 * r + 2 * y] = acc[a][y][j];
                    s_acc[warp][h][8 * r + 2 * y + 1] = acc[a][y][j + 2];
                }
            }
        // The states of key ranges attended before: eight teams of 16 lanes take a head and a share of this CTA's states
        // each (four dimensions per lane), and leave one state per team and pass beside the warps'.
        const int tnh = nheads >= 8 ? 8 : nheads > 4 ? 8 : nheads > 2 ? 4 : nheads;   // heads per pass, a power of two
        if (p.part_ml) {
            if (i == 0) pdl_wait();   // the tile kernel's states, and what the workspace held before
            const int team = threadIdx.x >> 4, d4 = threadIdx.x & 15;
            const size_t rows = (size_t)p.T * p.Hq;
#pragma unroll
            for (int pass = 0; pass < kN; ++pass) {
                const int h = pass * 8 + (team & (tnh - 1));
                float M = -INFINITY, ls = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                if (h < nheads) {
                    const size_t row = (size_t)t * p.Hq + h0 + h;
                    const int step = splits * (8 / tnh);
                    for (int x = split + splits * (team / tnh); x < p.nparts; x += 4 * step) {
                        float2 ml[4];   // four states' loads in flight
                        float4 a[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const size_t at = (size_t)min(x + y * step, p.nparts - 1) * rows + row;
                            ml[y] = p.part_ml[at];
                            a[y] = reinterpret_cast<const float4 *>(p.part_acc + at * kD)[d4];
                            if (x + y * step >= p.nparts) ml[y].x = -INFINITY;
                        }
                        const float m2 = fmaxf(fmaxf(M, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
                        if (m2 == -INFINITY) continue;   // no key so far
                        const float w0 = exp2f(M - m2);
                        M = m2;
                        ls *= w0;
                        o = make_float4(o.x * w0, o.y * w0, o.z * w0, o.w * w0);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float w = exp2f(ml[y].x - m2);
                            ls += ml[y].x == -INFINITY ? 0.f : ml[y].y * w;
                            if (ml[y].x != -INFINITY)   // an empty share, or past the last
                                o = make_float4(o.x + a[y].x * w, o.y + a[y].y * w, o.z + a[y].z * w, o.w + a[y].w * w);
                        }
                    }
                }
                const int slot = pass * 8 + team;
                if (d4 == 0) {
                    s_pm[slot] = M;
                    s_pl[slot] = ls;
                }
                reinterpret_cast<float4 *>(s_pacc[slot])[d4] = o;
            }
        }
        __syncthreads();
        // The CTA's state; of a split row it goes to the CTA that finishes the output (distributed shared memory)
        if (splits > 1) {
            if (i == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every CTA has started
            else cluster.sync();                                                      // the last token's are read
        }
        const size_t row0 = (size_t)t * p.Hq + h0;
#pragma unroll 1
        for (int blk = 0; blk < kBlocks; ++blk) {
            const int e = blk * kThreads + threadIdx.x, h = e / kD, d = e % kD;
            if (h >= nheads) break;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
            const int slot0 = (h & ~7) + (h & (tnh - 1));
            if (p.part_ml)
                for (int y = 0; y < 8; y += tnh) M = fmaxf(M, s_pm[slot0 + y]);
            float ls = 0.f, o = 0.f;
            if (M != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float wt = exp2f(s_m[w][h] - M);
                    ls += wt * s_l[w][h];
                    o += wt * (kTwice ? s_acc[w][h][d] + s_acc[w][h + 4][d] : s_acc[w][h][d]);
                }
                o *= p.out_scale;
                if (p.part_ml)
                    for (int y = 0; y < 8; y += tnh) {
                        const float wt = exp2f(s_pm[slot0 + y] - M);
                        ls += wt * s_pl[slot0 + y];
                        o += wt * s_pacc[slot0 + y][d];
                    }
            }
            if (splits == 1) {
                finish(row0 + h, d, ls, o);
            } else {
                const int owner = blk % splits;
                *cluster.map_shared_rank(&s_sent[blk / splits * splits + split][threadIdx.x], owner) = o;
                if (d == 0)
                    for (int y = 0; y < min(splits, kBlocks); ++y) {
                        *cluster.map_shared_rank(&s_M[split][h], y) = M;
                        *cluster.map_shared_rank(&s_L[split][h], y) = ls;
                    }
            }
        }
        if (splits > 1) {
            cluster.sync();   // nothing reads another CTA's memory after it
            // This CTA's share of the outputs, the CTAs' states in rank order
#pragma unroll 1
            for (int blk = 0; blk < kBlocks; ++blk) {
                const int e = blk * kThreads + threadIdx.x, h = e / kD, d = e % kD;
                if (blk % splits != split || h >= nheads) continue;
                float M = -INFINITY;
                for (int y = 0; y < splits; ++y) M = fmaxf(M, s_M[y][h]);
                float ls = 0.f, o = 0.f;
                if (M != -INFINITY)
                    for (int y = 0; y < splits; ++y) {
                        const float wt = exp2f(s_M[y][h] - M);
                        ls += wt * s_L[y][h];
                        o += wt * s_sent[blk / splits * splits + y][threadIdx.x];
                    }
                finish(row0 + h, d, ls, o);
            }
        }
        __syncthreads();
    }
    if (p.after_tiles && !p.part_ml) pdl_wait();
    pdl_trigger();
}

}  // namespace

// CTAs (one cluster) that share a token's keys: at most 512 KiB of K and V each, and as many as fill the GPU in one wave
// (a few CTAs more than fit cost a whole second wave: 8 rows of 16 heads, 64..512 keys, took two thirds longer with 5
// CTAs per row and head than with 4), with at least 64 keys each.
int plan_token_splits(long long items, int Hkv, int g, int max_len, bool fp8, int sms) {
    const int kn = g > 8 ? 2 : 1;
    const long long rows = items * Hkv * ((g + 8 * kn - 1) / (8 * kn));
    const long long key_bytes = 2LL * kD * (fp8 ? 1 : 2);
    long long s = ((long long)max_len * key_bytes + 512 * 1024 - 1) / (512 * 1024);
    const int slots = kn == 2 ? ctas_per_sm<Bf16Tile, 2>() : fp8 ? ctas_per_sm<Fp8Tile, 1>() : ctas_per_sm<Bf16Tile, 1>();
    const long long fill = (long long)slots * sms / rows;
    if (fill > s) s = fill;
    const long long by_keys = ((long long)max_len + 63) / 64;
    if (s > by_keys) s = by_keys;
    if (s > kMaxSplits) s = kMaxSplits;
    return s < 1 ? 1 : (int)s;
}

namespace {

template <typename Tile, bool kPaged, int kN, bool kPlain, bool kTwice = false>
cudaError_t launch_variant(const PromptParams &p, int splits, cudaStream_t stream) {
    auto kern = attn_tokens_kernel<Tile, kPaged, kN, kPlain, kTwice>;
    // The loads in flight live in L1 (128 KB per SM at four CTAs): ask for no more shared memory than the CTAs need.
    // Left to itself an SM keeps the split of the kernel before, and behind the tile kernel, which takes all of it,
    // 128 rows of 64..2048 own keys took a quarter longer.
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = once_per_device(ready, [&] {
        constexpr size_t all = ctas_per_sm<Tile, kN>() * (sizeof(Shared<kN>) + 1024);
        return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    (int)((all * 100 + 228 * 1024 - 1) / (228 * 1024)));
    });
    if (e != cudaSuccess) return e;
    const unsigned hgroups = (unsigned)((p.g + 8 * kN - 1) / (8 * kN));
    return launch_kernel(kern, dim3((unsigned)((long long)p.B * p.Hkv * hgroups * splits)), dim3(kThreads), 0, stream,
                         (unsigned)splits, p, splits);
}

template <typename Tile, bool kPaged>
cudaError_t launch_layout(const PromptParams &p, int splits, cudaStream_t stream) {
    const bool plain = p.cap_c1 == 0.f && !p.slopes;
    if (p.g > 8)
        return plain ? launch_variant<Tile, kPaged, 2, true>(p, splits, stream)
                     : launch_variant<Tile, kPaged, 2, false>(p, splits, stream);
    if (!Tile::kF16 && p.g <= 4)
        return plain ? launch_variant<Tile, kPaged, 1, true, !Tile::kF16>(p, splits, stream)
                     : launch_variant<Tile, kPaged, 1, false, !Tile::kF16>(p, splits, stream);
    return plain ? launch_variant<Tile, kPaged, 1, true>(p, splits, stream)
                 : launch_variant<Tile, kPaged, 1, false>(p, splits, stream);
}

}  // namespace

cudaError_t launch_attn_tokens(const PromptParams &p, bool paged, bool fp8, int splits, cudaStream_t stream) {
    if (fp8) return paged ? launch_layout<Fp8Tile, true>(p, splits, stream) : launch_layout<Fp8Tile, false>(p, splits, stream);
    return paged ? launch_layout<Bf16Tile, true>(p, splits, stream) : launch_layout<Bf16Tile, false>(p, splits, stream);
}

}  // namespace dr
