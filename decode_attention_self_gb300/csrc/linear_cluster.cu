// Matrix product with an epilogue for some tens to hundreds of tokens: out = residual + act(x W^T + bias).
//
// One CTA multiplies up to 128 tokens by NB rows of W over its share of K on the tensor cores: the tokens are the MMA's
// M = 128 operand, the weight rows its N operand, both K-major bf16 in shared memory with the 128-byte swizzle, the fp32
// sums in tensor memory (a lane per token).  What such a call costs is the way of its operands: W from memory, and both
// from L2 into each SM at some 70 bytes a cycle, so tiles and splits are chosen for few bytes per SM (make_plan).  Where the
// tiles leave SMs idle the S CTAs of a cluster share K: each lays its partial sums down in its shared memory and copies them, in
// bulk, to the CTAs that own the rows (rows / S each), which add the S parts in rank order and finish their rows.  The
// order of sums is fixed: results are the same bits from call to call.
//   warps 0-3: TMA producers of 64-wide K chunks, each of every fourth;  warps 4-7: MMA issuers, likewise, each into sums of its
//   own;  all 8 or 16 warps: sums, epilogue.
// Where the tiles of 64 rows would be more than a wave, but those of 256 tokens by 128 rows are not, two CTAs (a cluster) multiply
// such a tile with two-CTA products (kPair): each loads and keeps 128 of the tokens and 64 of the weight rows, which halves what comes
// from L2 per product; the first CTA issues (two warps: a product is four times as long).  512 tokens 1024 -> 4096 with gelu 9.7 us
// by the pairs that stay, 7.9 here: set-up and epilogue of a single tile are what this kernel is short of.
// (One warp takes some 400 cycles to issue a chunk's four products, wait and commit, and 310 to issue its copies, whatever
// their size: with one of each, 128 tokens of 1024 -> 4096 took 8700 cycles for 16 chunks, with two 5300.)
// The kernel runs once through its code, so there is little of it: 16 columns of a token at a time, from tensor memory to the
// outputs.  (By way of shared memory, with a warp's stores side by side, 256 tokens 1024 -> 4096 took 7.7 us, 6.8 at that step.)  A
// pass costs some 1400 cycles, 2400 with gelu, of which little is arithmetic: two warps per scheduler cannot hide its latencies, so
// tiles of 64 and 128 rows have 16 warps.
// Tensor-core sums are cut off, not rounded: each addition may lose the last bit towards zero, so a chain over K drifts by about
// 1e-9 K (measured: 1.0e-6 at K = 1024, 2.1e-6 at 2048).  fp32 outputs therefore break the chain every 512 of K into
// accumulators of their own (pieces), added in fp32; bf16 outputs, whose rounding is 1000 times that, do not.
// Tensor memory and clusters: a CTA that waits for its cluster must not keep another cluster's CTA waiting for tensor
// memory.  A CTA of a cluster takes at least 80 KB of shared memory and at most 256 columns, so that the two that fit on an SM (or
// one and two of the LM head's, 72 KB and 128 columns at the least and most) never need more than the 512 there are.  A CTA that
// shares its tile with no other waits for nobody and may take all 512.
// Every mbarrier wait is bounded; one that runs out sets DR_ERRF_TIMEOUT, and the rows that lack its sums are not written.
#include "dr_tc.cuh"
#include "linear_epilogue.cuh"

namespace dr {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kRows = 128;        // tokens per tile (MMA M)
constexpr int kChunkK = 64;       // K per stage: one 128-byte swizzled row
constexpr int kMaxStages = 8;
constexpr int kPieceChunks = 8;   // fp32 outputs: K of 512 per accumulator
constexpr int kMaxNb = 128;       // weight rows per tile
constexpr int kWays = 4;          // producers, and issuers
constexpr int kPairNb = 128, kPairIssuers = 2;   // a pair's
constexpr size_t kMinSmem = 80 * 1024;
constexpr size_t kMaxSmem = 225 * 1024;

struct ClusterPlan {
    int pair;          // 1: two CTAs multiply a tile of 256 tokens
    int nb;            // weight rows per tile (MMA N): nb output columns, or nb / 2 when gated
    int split;         // CTAs (one cluster) that share K
    int box_rows;      // tokens per tile that are loaded
    int piece_chunks;  // K chunks of an issuer per accumulator
    int stages;
    int cols;          // tensor-memory columns
    int threads;       // 64 per 8 columns of the tile, at most kMaxThreads
    uint32_t recv_at;  // where the parts of a cluster's other CTAs go, behind the ring and the CTA's own sums
    size_t smem;
};

size_t parts_bytes(int rows, const ClusterPlan &pl) { return (size_t)rows * pl.nb * 4; }

struct ClusterArgs {
    LinearParams p;
    ClusterPlan plan;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(tc::smem_u32(bar))
        : "memory");
}
// A copy from this CTA's shared memory to that of another of the cluster, counted on a barrier there.
__device__ __forceinline__ void copy_to_peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "r"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
// (relaxed: the barriers' set-up has a fence of its own, and what is copied is counted)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <bool kF32, bool kPair>
__global__ void __launch_bounds__(kMaxThreads)
    linear_cluster_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                          const __grid_constant__ ClusterArgs args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done, parts;
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up, issued[kWays];   // a wait ran out; the chunk at which each producer ended
    __shared__ __align__(16) float bias[kMaxNb];   // of the tile's sums

    const LinearParams &p = args.p;
    const ClusterPlan &pl = args.plan;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kIssuers = kPair ? kPairIssuers : kWays;
    const int S = kPair ? 1 : pl.split, rank = kPair ? 0 : blockIdx.x, stages = pl.stages;
    const int half = kPair ? blockIdx.x : 0;   // of a pair's tokens and weight rows; the first CTA issues the products of both
    const int bn = p.gated ? pl.nb / 2 : pl.nb;   // output columns of a tile
    const int n0 = blockIdx.y * bn, t0 = (kPair ? blockIdx.z * 2 + half : blockIdx.z) * kRows;
    const int all_chunks = (p.K + kChunkK - 1) / kChunkK;
    const int c_begin = (int)((int64_t)all_chunks * rank / S), c_end = (int)((int64_t)all_chunks * (rank + 1) / S);
    const int chunks = c_end - c_begin;
    const uint32_t bytes_x = pl.box_rows * 128, bytes_w = (kPair ? pl.nb / 2 : pl.nb) * 128;
    const int w0 = !kPair ? n0 : p.gated ? half * p.N + n0 : n0 + half * (pl.nb / 2);   // first of the CTA's weight rows

    // Ring of tokens, ring of weight rows, partial sums of the cluster.  The MMA reads 128 token rows from each stage, however
    // few there are: rows past the stage's own are whatever follows in shared memory (plan: there is as much), and the sums
    // of their lanes are not looked at.
    const uint32_t ring = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
    const uint32_t sx = ring, sw = ring + stages * bytes_x;
    const int rows = max(0, min(kRows, p.T - t0)), share = (rows + S - 1) / S;   // rows of the tile, and that a CTA owns
    const int mine = min(share, rows - rank * share);
    uint8_t *const staged = smem_raw + (ring - tc::smem_u32(smem_raw));              // own sums, over the ring once it is idle
    uint8_t *const received = staged + pl.recv_at;                                   // the other CTAs', part by part

    // accumulators in use: an issuer has one for each piece_chunks of its chunks, in turn with the others
    const auto ceil_div = [](int a, int b) { return (a + b - 1) / b; };
    int pieces = 0;
    for (int w = 0; w < kIssuers; ++w) pieces += ceil_div(ceil_div(max(chunks - w, 0), kIssuers), pl.piece_chunks);

    if (warp == 1) {   // a lane per barrier of a kind
        if (lane < stages) {
            tc::mbar_init(&full[lane], 1);
            tc::mbar_init(&empty[lane], 1);
        }
        if (lane == 0) {
            tc::mbar_init(&done, kIssuers);
            tc::mbar_init(&parts, 1);
            if (S > 1 && mine > 0) tc::mbar_expect_tx(&parts, (uint32_t)((S - 1) * mine * pl.nb) * 4);
            gave_up = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
    }
    // The first weight boxes, one a warp, on their way into L2 while the kernel before this one ends (a hint: nothing is read).
    if (warp < min(chunks, stages) && tc::elect_one()) {
        if (warp == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
        for (int part = 0; part <= (kPair ? 0 : p.gated); ++part)
            asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(&map_w)),
                         "r"((c_begin + warp) * kChunkK), "r"(part ? p.N + n0 : w0)
                         : "memory");
    }
    __syncwarp();
    if (warp == 2) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(&tmem_base)),
                         "r"(pl.cols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(&tmem_base)),
                         "r"(pl.cols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    tc::fence_before();
    __syncthreads();
    if (kPair) {   // both CTAs' barriers are set up, and both have their tensor memory
        cluster_arrive();
        cluster_wait();
    }
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    if (S > 1) cluster_arrive();   // waited for before the first remote write: every CTA of the cluster runs by then
    pdl_wait();
    // The next kernel may start as far as it fits beside this one: it sets up, and prefetches its weights.
    pdl_trigger();
    if (p.bias && threadIdx.x >= 64)
        for (int j = threadIdx.x - 64; j < pl.nb; j += blockDim.x - 64) {
            const int n = n0 + (j < bn ? j : j - bn);
            bias[j] = n < p.N ? lin::bf16_at(p.bias, j < bn ? n : (int64_t)p.N + n) : 0.f;
        }

    if (warp < kWays) {
        // stage s of round r waits for the products of round r - 1.  (Test hook: the stalled tile's first chunk is left out, so
        // the wait for it runs out.)
        const bool stalled = (int)(blockIdx.z * gridDim.y + blockIdx.y) == p.stall_tile;
        int c = warp;
        for (int s = c % stages, r = c / stages; c < chunks; c += kWays) {
            if (r > 0 && !tc::mbar_wait(&empty[s], (r - 1) & 1, &gave_up)) break;
            if (tc::elect_one() && !(stalled && c == 0)) {
                const int k = (c_begin + c) * kChunkK;
                const uint32_t w_at = sw + s * bytes_w;
                if constexpr (kPair) {
                    const uint32_t bar = tc::mapa(tc::smem_u32(&full[s]), 0);
                    if (half == 0) tc::mbar_expect_tx(&full[s], 2 * (bytes_x + bytes_w));
                    tc::pair_load(w_at, &map_w, k, w0, bar);
                    tc::pair_load(sx + s * bytes_x, &map_x, k, t0, bar);
                } else {
                    tc::mbar_expect_tx(&full[s], bytes_x + bytes_w);
                    tma_load_2d(w_at, &map_w, k, n0, &full[s]);
                    if (p.gated) tma_load_2d(w_at + bytes_w / 2, &map_w, k, p.N + n0, &full[s]);
                    tma_load_2d(sx + s * bytes_x, &map_x, k, t0, &full[s]);
                }
            }
            __syncwarp();
            s += kWays;
            if (s >= stages) {
                s -= stages;
                ++r;
            }
        }
        if (lane == 0) issued[warp] = c;
    } else if (warp < kWays + kIssuers && half == 0) {
        const uint32_t idesc = tc::instr_desc(kPair ? 2 * kRows : kRows, pl.nb, false, false);
        const uint64_t dx = tc::smem_desc(sx), dw = tc::smem_desc(sw);
        const int issuer = warp - kWays;
        bool ok = true;
        int c = issuer, in_piece = 0;
        uint32_t d = tmem + issuer * pl.nb;
        for (int s = c % stages, r = c / stages; c < chunks; c += kIssuers) {
            if (!tc::mbar_wait(&full[s], r & 1, &gave_up)) {
                ok = false;
                break;
            }
            tc::fence_after();
            if (tc::elect_one()) {
#pragma unroll
                for (int k = 0; k < kChunkK / 16; ++k) {
                    const uint64_t a = tc::desc_at(dx, s * bytes_x + k * 32), b = tc::desc_at(dw, s * bytes_w + k * 32);
                    if constexpr (kPair) tc::pair_mma(d, a, b, idesc, (in_piece | k) != 0);
                    else tc::mma_ss(d, a, b, idesc, (in_piece | k) != 0);
                }
                // the stage is free once these products have read it
                if constexpr (kPair) tc::pair_commit(&empty[s]);
                else tc::commit(&empty[s]);
            }
            __syncwarp();
            if (++in_piece == pl.piece_chunks) {
                in_piece = 0;
                d += kIssuers * pl.nb;
            }
            s += kIssuers;
            if (s >= stages) {
                s -= stages;
                ++r;
            }
        }
        if (!ok && lane == 0) flag_error(p.err, DR_ERRF_TIMEOUT);
        // on every path: with `done` the products in flight have ended (a commit follows those before it)
        if (tc::elect_one()) {
            if constexpr (kPair) tc::pair_commit(&done, ok ? 3 : 1);   // (the second CTA's wait runs out too)
            else tc::commit(&done);
        }
        __syncwarp();
    }
    __syncthreads();
    const int row = (warp & 3) * 32 + lane;   // whose sums this thread reads
    const int col0 = (warp >> 2) * 16, cols = blockDim.x / 128 * 16;   // this warp's columns: the first, and to the next
    const bool boxed = p.vec_out && (!p.residual || p.vec_res);   // rows of whole 16-byte pieces
    const bool direct = S == 1 && boxed;                          // from tensor memory to the outputs
    lin::Columns<kF32, 16> res;   // on its way during the last products
    if (direct && row < rows && col0 < bn) lin::load_residual(p, t0 + row, n0 + col0, res);
    bool ok = tc::mbar_wait(&done, 0, &gave_up);
    if (gave_up) {
        // copies in flight end by themselves; wait for them before this CTA's shared memory goes away
        if (warp == 0 && lane == 0) {
            for (int w = 0; half == 0 && w < kWays; ++w)   // both CTAs' copies count on the first one's barriers
                for (int c = issued[w] - kWays; c >= max(p.stall_tile < 0 ? 0 : 1, issued[w] - stages); c -= kWays)
                    tc::mbar_drain(&full[c % stages], (c / stages) & 1);
            flag_error(p.err, DR_ERRF_TIMEOUT);
        }
        ok = false;
    }
    ok = __syncthreads_and(ok);
    tc::fence_after();

    const int nb = pl.nb;
    const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const auto sums = [&](int c, float (&v)[16]) {   // columns c .. c+15 of the row, all pieces of K
        tc::ld16_wait(from + c, v);
#pragma unroll 1
        for (int i = 1; i < pieces; i += 2) {   // two at a time
            float one[16], two[16];
            tc::ld16x2_wait(from + i * nb + c, one, from + min(i + 1, pieces - 1) * nb + c, two);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += one[j];
            if (i + 1 < pieces)
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += two[j];
        }
    };
    if (ok && (warp & 3) * 32 < rows) {
        if (direct) {
#pragma unroll 1
            for (int c = col0; c < bn; c += cols) {
                float a[16], b[16];
                sums(c, a);
                if (p.gated) sums(bn + c, b);
                if (row < rows) {
                    lin::finish(p, bias + c, bias + bn + c, t0 + row, n0 + c, a, b, res);
                    if (c + cols < bn) lin::load_residual(p, t0 + row, n0 + c + cols, res);
                }
                __syncwarp();   // whole again: the next sums' instructions want all lanes at once
            }
        } else {
            // To shared memory, [row][nb] fp32 in 16-byte pieces that the row turns, so that a warp's stores spread over the
            // banks.  The ring is idle: all its copies were multiplied.
            float4 *to = reinterpret_cast<float4 *>(staged) + row * (nb / 4);
#pragma unroll 1
            for (int c = col0; c < nb; c += cols) {
                float v[16];
                sums(c, v);
                if (row < rows)
#pragma unroll
                    for (int j = 0; j < 4; ++j) to[(c / 4 + j) ^ (row & 7)] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                __syncwarp();
            }
        }
    }
    tc::fence_before();
    __syncwarp();
    if (S > 1) {
        tc::fence_proxy_async();
        cluster_wait();   // every CTA of the cluster has set its barrier up
    }
    __syncthreads();
    if (kPair) cluster_arrive();
    if (!kPair && warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(pl.cols));
    if (S > 1) {
        if (ok && warp == 0 && lane < S && lane != rank) {   // a lane per owner
            const int theirs = min(share, rows - lane * share);
            const uint32_t slot = (uint32_t)(rank - (rank > lane)) * (theirs * nb * 4);   // parts in rank order, without the owner's
            if (theirs > 0)
                copy_to_peer(tc::mapa(tc::smem_u32(received) + slot, lane), tc::smem_u32(staged) + lane * share * nb * 4, theirs * nb * 4,
                             tc::mapa(tc::smem_u32(&parts), lane));
        }
        __syncwarp();
        if (mine > 0 && !tc::mbar_wait(&parts, 0, &gave_up)) {
            if (threadIdx.x == 0) flag_error(p.err, DR_ERRF_TIMEOUT);
            ok = false;
        }
        ok = __syncthreads_and(ok);
        cluster_arrive();   // this CTA has its parts; none exits before the copies out of it have landed
    }
    const auto part = [&](int s, int r) {   // the sums of this CTA's row r that CTA s of the cluster made
        return s == rank ? reinterpret_cast<const float *>(staged) + (rank * share + r) * nb
                         : reinterpret_cast<const float *>(received) + ((s - (s > rank)) * mine + r) * nb;
    };
    if (ok && boxed && !direct) {   // four columns a thread (their residual loaded before the wait for the parts: no gain)
        const int shift = 29 - __clz(bn);   // bn is a power of two
#pragma unroll 1
        for (int i = threadIdx.x; i < mine << shift; i += blockDim.x) {
            const int r = i >> shift, g = i - (r << shift), key = (rank * share + r) & 7;
            float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
            lin::Columns<kF32, 4> own;
            lin::load_residual(p, t0 + rank * share + r, n0 + g * 4, own);
#pragma unroll 1
            for (int s = 0; s < S; ++s) {
                const float4 *from = reinterpret_cast<const float4 *>(part(s, r));
                const float4 v = from[g ^ key];
                a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
                if (p.gated) {
                    const float4 u = from[(bn / 4 + g) ^ key];
                    b[0] += u.x; b[1] += u.y; b[2] += u.z; b[3] += u.w;
                }
            }
            lin::finish(p, bias + g * 4, bias + bn + g * 4, t0 + rank * share + r, n0 + g * 4, a, b, own);
        }
    } else if (ok && !boxed) {   // a column of eight rows a thread: a warp's accesses lie side by side
        const int shift = 31 - __clz(bn);
#pragma unroll 1
        for (int i = threadIdx.x; i < (mine + 7) / 8 * bn; i += blockDim.x) {
            const int c = i & (bn - 1), r0 = (i >> shift) * 8, have = min(8, mine - r0);
            float a[8], b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = b[j] = 0.f;
#pragma unroll 1
            for (int s = 0; s < S; ++s) {
                const float *from = part(s, r0);
#pragma unroll
                for (int j = 0; j < 8; ++j, from += nb)
                    if (j < have) {
                        const int key = (rank * share + r0 + j) & 7;
                        a[j] += from[((c >> 2) ^ key) * 4 + (c & 3)];
                        if (p.gated) b[j] += from[(((bn + c) >> 2) ^ key) * 4 + (c & 3)];
                    }
            }
            lin::finish_column8<kF32>(p, bias[c], bias[p.gated ? bn + c : c], t0 + rank * share + r0, have, n0 + c, a, b);
        }
    }
    __syncwarp();   // the lanes of a warp had different numbers of pieces
    if (kPair || S > 1) cluster_wait();
    if (kPair && warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(pl.cols));
}

// Tiles and split of a call.  Measured with one wave of tiles of 32 against 64 rows of W, us (both sides at the step that made the
// choice): 128 tokens 1024 -> 4096 5.8 and 6.9, 4096 -> 1024 (4 CTAs per tile) 6.7 and 8.6; 256 tokens 1024 -> 4096, where tiles of 32 are
// two waves, 7.8 and 6.8.  Tiles of 64 against pairs, where both are a wave: 512 tokens 1024 -> 2048 6.3 and 6.7, 1024 tokens 4096 -> 1024
// 12.5 and 13.4.
// A CTA of a split keeps 4 chunks (or 6, 8, 16, us): 128 tokens 1000 -> 500 5.0 (5.6, 5.6, 7.3), 1024 -> 1024 4.8 (5.0, 5.0, 5.1), 2048 ->
// 1024 5.6 (5.6, 5.5, 6.0); 64 tokens 1536 -> 1024 4.4 (4.4, 5.0, 5.4).  Eight chunks are not split: 64 tokens 512 -> 512 3.7 whole, 3.9
// halved.
ClusterPlan make_plan(const LinearParams &p, int sms) {
    ClusterPlan pl;
    const int chunks = (p.K + kChunkK - 1) / kChunkK;
    const int64_t mtiles = (p.T + kRows - 1) / kRows;
    const auto tiles = [&](int nb) {
        const int bn = p.gated ? nb / 2 : nb;
        return mtiles * ((p.N + bn - 1) / bn);
    };
    pl.pair = tiles(64) > sms;
    pl.nb = pl.pair ? kPairNb : tiles(32) <= sms ? 32 : 64;
    pl.threads = pl.nb == 32 ? 256 : kMaxThreads;
    pl.split = 1;
    while (!pl.pair && chunks > 8 && pl.split < 8 && tiles(pl.nb) * pl.split * 2 <= sms && chunks / (2 * pl.split) >= 4) pl.split *= 2;
    const int rows = p.T < kRows ? p.T : kRows;
    pl.box_rows = (rows + 7) / 8 * 8;
    const int most = (chunks + pl.split - 1) / pl.split;   // chunks of a CTA
    const int issuers = pl.pair ? kPairIssuers : kWays;
    const int own_chunks = (most + issuers - 1) / issuers, max_cols = pl.pair || pl.split > 1 ? 256 : 512;
    const auto pieces = [&] { return issuers * ((own_chunks + pl.piece_chunks - 1) / pl.piece_chunks); };
    pl.piece_chunks = p.out_f32 ? kPieceChunks : own_chunks;
    while (pieces() * pl.nb > max_cols) ++pl.piece_chunks;
    pl.cols = 32;
    while (pl.cols < pl.nb * pieces()) pl.cols *= 2;
    // shared memory: the ring, with what its last stage's products may read past it, or after it the CTA's own sums; the parts
    const size_t stage = (size_t)(pl.box_rows + (pl.pair ? pl.nb / 2 : pl.nb)) * 128, own = parts_bytes(rows, pl);
    const size_t parts = pl.split > 1 ? parts_bytes(rows + pl.split, pl) : 0;
    const auto ring = [&](int n) {
        const size_t over = n * stage > (size_t)(n * pl.box_rows + kRows) * 128 ? n * stage : (size_t)(n * pl.box_rows + kRows) * 128;
        return over > own ? over : own;
    };
    // a multiple of kWays: a stage always belongs to the same producer and issuer, so a warp that waits for one of its rounds has
    // seen the round before (a wait by parity cannot tell a phase from the one two before it)
    pl.stages = most <= kWays ? kWays : kMaxStages;
    while (pl.stages > kWays && 1024 + ring(pl.stages) + parts > kMaxSmem) pl.stages -= kWays;
    pl.recv_at = (uint32_t)ring(pl.stages);
    pl.smem = 1024 + ring(pl.stages) + parts;
    if (pl.smem < kMinSmem) pl.smem = kMinSmem;
    return pl;
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const ClusterArgs);
Kernel kernel_of(bool f32, bool pair) {
    return f32 ? linear_cluster_kernel<true, false> : pair ? linear_cluster_kernel<false, true> : linear_cluster_kernel<false, false>;
}

int64_t plan_tiles(const LinearParams &p, const ClusterPlan &pl) {
    const int bn = p.gated ? pl.nb / 2 : pl.nb, bt = pl.pair ? 2 * kRows : kRows;
    return ((int64_t)p.T + bt - 1) / bt * ((p.N + bn - 1) / bn);
}

}  // namespace

bool linear_cluster_takes(const LinearParams &p, int sms) {
    const ClusterPlan pl = make_plan(p, sms);
    if (pl.pair) return !p.out_f32 && p.T > kRows && plan_tiles(p, pl) <= sms / 2;
    return !p.out_f32 || pl.piece_chunks <= kPieceChunks;
}

int linear_cluster_tiles(const LinearParams &p, int sms) { return (int)plan_tiles(p, make_plan(p, sms)); }

cudaError_t launch_linear_cluster(const LinearParams &p, int sms, cudaStream_t stream) {
    ClusterArgs a;
    a.p = p;
    a.plan = make_plan(p, sms);
    const ClusterPlan &pl = a.plan;
    const int bn = p.gated ? pl.nb / 2 : pl.nb;
    CUtensorMap map_x, map_w;
    if (!encode_matrix(&map_x, p.x, false, p.T, p.K, p.x_stride, pl.box_rows, kChunkK) ||
        !encode_matrix(&map_w, p.W, false, (int64_t)p.N * (p.gated ? 2 : 1), p.K, p.K, pl.pair ? pl.nb / 2 : bn, kChunkK))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = once_per_device(ready, [] {
        for (const Kernel k : {kernel_of(false, false), kernel_of(false, true), kernel_of(true, false)}) {
            const cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
            if (err != cudaSuccess) return err;
        }
        return cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    const int cluster = pl.pair ? 2 : pl.split, bt = pl.pair ? 2 * kRows : kRows;
    const dim3 grid((unsigned)cluster, (unsigned)((p.N + bn - 1) / bn), (unsigned)((p.T + bt - 1) / bt));
    return launch_kernel(kernel_of(p.out_f32, pl.pair), grid, dim3((unsigned)pl.threads), pl.smem, stream, (unsigned)cluster, map_x, map_w, a);
}

}  // namespace dr
