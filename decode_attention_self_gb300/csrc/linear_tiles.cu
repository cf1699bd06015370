// Matrix product with an epilogue for prompts: out = residual + act(x W^T + bias), bound by the tensor cores.
//
// Pairs of CTAs (clusters of two) stay on their SMs and take 256 x 256 tiles of the output in turn: 256 tokens by 256
// weight rows (gated: 128 rows and the 128 that are multiplied in, so that both sums of a column meet in one thread).
// A pair's product is one tcgen05.mma of cta_group::2: each CTA holds 128 tokens and half of the weight rows, and the
// hardware feeds both halves to both SMs, so an SM reads 32 KB of shared memory per 64 of K instead of the 48 KB that a
// 128 x 256 tile of its own would take.
//   warp 0      TMA producer of its CTA's halves: 64-wide K chunks in a ring of kStages, counted on the first CTA's barrier
//   warp 1      MMA issuer (first CTA only)
//   warps 4-11  epilogue: warp w owns 32 tokens (tensor-memory lanes) and half of the tile's columns
// The sums of a tile take 256 of the 512 tensor-memory columns; the next tile is multiplied while the epilogue works on
// the one before.  The epilogue goes through a 4 KB box per warp in shared memory (32 tokens of 128 bytes, 128-byte
// swizzle): the residual's box comes in by TMA before the sums are ready, is added to in place and goes out by TMA, so
// rows may end anywhere.  Outputs or residuals whose rows are not 16-byte aligned go between box and memory element by
// element, a row of the box at a time.
// fp32 outputs: tensor-core chains drift by about 1e-9 K, so each 512 of K is a tile's sums of its own, added up in the
// epilogue warps' registers (128 columns a thread).
// Every mbarrier wait is bounded; after one that runs out the pair's further tiles are not written, and copies and
// products in flight are waited for before it exits.
#include "dr_tc.cuh"
#include "linear_epilogue.cuh"

namespace dr {
namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarp = 4, kEpiWarps = 8;
constexpr int kTileT = 256;       // tokens per pair
constexpr int kTileW = 256;       // weight rows per pair (MMA N)
constexpr int kStages = 5;
constexpr int kHalf = 128 * 128;  // bytes of a CTA's tokens or weight rows in a stage
constexpr int kBox = 32 * 128;    // bytes of an epilogue box
constexpr int kPieceChunks = 8;   // fp32 outputs: K of 512 per chain
constexpr int kGroup = 8;         // token tiles that share their weight tiles' stay in L2
constexpr size_t kSmem = 1024 + (size_t)kStages * 2 * kHalf + kEpiWarps * 2 * kBox;

struct TileArgs {
    LinearParams p;
    int32_t chunks;         // of 64 of K
    int32_t piece_chunks;   // chunks per chain
    int32_t token_tiles, col_tiles;
};

struct Maps {
    CUtensorMap x, w, res, out[DR_LINEAR_MAX_OUTS];
};

struct Control {
    uint64_t full[kStages];    // first CTA's: both CTAs' copies of a stage have landed
    uint64_t empty[kStages];   // the products that read the stage are over
    uint64_t sums_full[2];     // a chain's sums are in tensor memory
    uint64_t sums_free[2];     // first CTA's: both CTAs' epilogue warps have read them
    uint64_t res[kEpiWarps][2];
    uint64_t done;
    uint32_t tmem;
    int gave_up;
};

__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A copy into this CTA's shared memory that counts on a barrier of either CTA of the pair (a cluster address).
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void own_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(tc::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void box_store(const CUtensorMap *map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}
template <int n>
__device__ __forceinline__ void stores_read() {   // all but the last n box stores have read their boxes
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// Arrives on the barrier at this place in both CTAs once the products issued so far are over.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            tc::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Tile i: groups of kGroup token tiles take all column tiles in turn, so that both operands' tiles stay in L2.
__device__ __forceinline__ void tile_at(const TileArgs &a, int64_t i, int &tt, int &ct) {
    const int64_t per_group = (int64_t)kGroup * a.col_tiles;
    const int g = (int)(i / per_group);
    const int r = (int)(i - g * per_group), n = min(kGroup, a.token_tiles - g * kGroup);
    ct = r / n;
    tt = g * kGroup + (r - ct * n);
}

// 32 columns n .. n+31 of bias added to the sums; columns past `have` have none.
__device__ __forceinline__ void add_bias(float *v, const uint16_t *bias, int64_t n, int have) {
    if (have >= 32 && n % 8 == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float f[8];
            unpack8(ld_ro16(bias + n + 8 * c), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * c + j] += f[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < have) v[j] += lin::bf16_at(bias, n + j);
    }
}

// Bias, activation and gating of 32 columns from n on.
__device__ __forceinline__ void finish32(const LinearParams &p, float *a, float *b, int n) {
    if (p.bias) {
        add_bias(a, p.bias, n, p.N - n);
        if (p.gated) add_bias(b, p.bias, (int64_t)p.N + n, p.N - n);
    }
    lin::activate<32>(a, p.act);
    if (p.gated) {
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] *= b[j];
    }
}

// An epilogue warp's box of 32 tokens from t0 on and 128 bytes of columns from n on: residual in, sums added, out.
template <bool kF32>
struct Box {
    static constexpr int kCols = kF32 ? 32 : 64;
    const LinearParams &p;
    const Maps &maps;
    uint32_t at;   // 1024-byte aligned shared memory
    int t0, n, lane;

    __device__ __forceinline__ uint32_t chunk(int row, int c) const { return at + row * 128 + ((c ^ (row & 7)) << 4); }

    // element by element, for a residual without 16-byte rows
    __device__ __forceinline__ void read_residual() const {
        const int rows = min(32, p.T - t0);
        for (int r = 0; r < rows; ++r)
            for (int c = lane; c < kCols && n + c < p.N; c += 32) {
                const int64_t from = (int64_t)(t0 + r) * p.res_stride + n + c;
                if constexpr (kF32) {
                    const float v = static_cast<const float *>(p.residual)[from];
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(chunk(r, c >> 2) + (c & 3) * 4), "f"(v) : "memory");
                } else {
                    const uint16_t v = static_cast<const uint16_t *>(p.residual)[from];
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(chunk(r, c >> 3) + (c & 7) * 2), "h"(v) : "memory");
                }
            }
        __syncwarp();
    }
    // columns c0 .. c0+31 of this thread's token
    __device__ __forceinline__ void put32(float *v, int c0) const {
        if constexpr (kF32) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t to = chunk(lane, c);
                if (p.residual) {
                    const uint4 r = lds16(to);
                    v[4 * c] += __uint_as_float(r.x);
                    v[4 * c + 1] += __uint_as_float(r.y);
                    v[4 * c + 2] += __uint_as_float(r.z);
                    v[4 * c + 3] += __uint_as_float(r.w);
                }
                sts16(to, make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                                     __float_as_uint(v[4 * c + 3])));
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t to = chunk(lane, c0 / 8 + c);
                float *u = v + 8 * c;
                if (p.residual) {
                    float f[8];
                    unpack8(lds16(to), f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[j] += f[j];
                }
                sts16(to, make_uint4(lin::pack2(u[0], u[1]), lin::pack2(u[2], u[3]), lin::pack2(u[4], u[5]),
                                     lin::pack2(u[6], u[7])));
            }
        }
    }
    __device__ __forceinline__ void store() const {
        int s = 0;
        for (int i = 1; i < p.n_outs; ++i)
            if (n >= p.out[i].col0) s = i;
        const LinearOut &o = p.out[s];
        const int col = n - o.col0;
        if (p.vec_out) {
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (t0 < p.T && col < o.cols) box_store(&maps.out[s], col, t0, at);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");   // one group per box, if empty
            }
            return;
        }
        __syncwarp();
        const int rows = min(32, p.T - t0);
        for (int r = 0; r < rows; ++r)
            for (int c = lane; c < kCols && col + c < o.cols; c += 32) {
                const int64_t to = (int64_t)(t0 + r) * o.stride + col + c;
                if constexpr (kF32) {
                    float v;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(chunk(r, c >> 2) + (c & 3) * 4) : "memory");
                    static_cast<float *>(o.ptr)[to] = v;
                } else {
                    uint16_t v;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(chunk(r, c >> 3) + (c & 7) * 2) : "memory");
                    static_cast<uint16_t *>(o.ptr)[to] = v;
                }
            }
        __syncwarp();
    }
};

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tiles_kernel(const __grid_constant__ Maps maps, const __grid_constant__ TileArgs args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Control ctl;

    const LinearParams &p = args.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1;   // the cluster's first CTA issues the products of both
    const int64_t tiles = (int64_t)args.token_tiles * args.col_tiles;
    const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;
    const uint32_t ring = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
    const uint32_t sx = ring, sw = ring + kStages * kHalf, boxes = ring + 2 * kStages * kHalf;
    const int tile_cols = p.gated ? kTileW / 2 : kTileW;
    volatile int *gave_up = &ctl.gave_up;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&ctl.full[s], 1);
            tc::mbar_init(&ctl.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&ctl.sums_full[b], 1);
            tc::mbar_init(&ctl.sums_free[b], 2 * kEpiWarps);
        }
        for (int w = 0; w < kEpiWarps; ++w)
            for (int b = 0; b < 2; ++b) tc::mbar_init(&ctl.res[w][b], 1);
        tc::mbar_init(&ctl.done, 1);
        ctl.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.x)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.w)) : "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(&ctl.tmem)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc::fence_before();
    cluster_sync();   // both CTAs' barriers are set up, and both have their tensor memory
    tc::fence_after();
    const uint32_t tmem = ctl.tmem;
    pdl_wait();

    if (warp == 0) {
        int s = 0, r = 0;
        unsigned armed = 0;   // stages whose copies were issued, and how often (parity of the last)
        unsigned parity = 0;
        bool ok = true;
        for (int64_t i = first; ok && i < tiles; i += step) {
            int tt, ct;
            tile_at(args, i, tt, ct);
            const int t = tt * kTileT + (int)rank * 128;
            // rows of W: the pair's 256 in halves, or 128 and those that multiply them
            const int w = p.gated ? (int)rank * p.N + ct * tile_cols : ct * tile_cols + (int)rank * 128;
            for (int c = 0; c < args.chunks; ++c) {
                if (!(c == 0 && i == p.stall_tile)) {
                    if (r > 0 && !tc::mbar_wait(&ctl.empty[s], (r - 1) & 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    if (tc::elect_one()) {
                        const uint32_t bar = mapa(tc::smem_u32(&ctl.full[s]), 0);
                        if (rank == 0) tc::mbar_expect_tx(&ctl.full[s], 4 * kHalf);
                        pair_load(sx + s * kHalf, &maps.x, c * 64, t, bar);
                        pair_load(sw + s * kHalf, &maps.w, c * 64, w, bar);
                    }
                    __syncwarp();
                    armed |= 1u << s;
                    parity = (parity & ~(1u << s)) | ((unsigned)(r & 1) << s);
                }
                if (++s == kStages) {
                    s = 0;
                    ++r;
                }
            }
        }
        pdl_trigger();
        if (!ok) {
            if (lane == 0) flag_error(p.err, DR_ERRF_TIMEOUT);
            // both CTAs' copies count on the first CTA's barriers; the second waits for it at the end
            if (rank == 0)
                for (int k = 0; k < kStages; ++k)
                    if (armed >> k & 1) tc::mbar_drain(&ctl.full[k], parity >> k & 1);
        }
    } else if (warp == 1 && rank == 0) {
        const uint32_t idesc = tc::instr_desc(kTileT, kTileW, false, false);
        const uint64_t dx = tc::smem_desc(sx), dw = tc::smem_desc(sw);
        int s = 0, r = 0;
        int64_t chain = 0;
        bool ok = true;
        for (int64_t i = first; ok && i < tiles; i += step) {
            for (int c = 0; ok && c < args.chunks; ++chain) {
                const int b = (int)(chain & 1);
                if (chain >= 2 && !tc::mbar_wait(&ctl.sums_free[b], (unsigned)((chain >> 1) - 1) & 1, gave_up)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t d = tmem + b * kTileW;
                const int end = min(args.chunks, c + args.piece_chunks);
                for (int c0 = c; c < end; ++c) {
                    if (!tc::mbar_wait(&ctl.full[s], r & 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    if (tc::elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            pair_mma(d, tc::desc_at(dx, s * kHalf + k * 32), tc::desc_at(dw, s * kHalf + k * 32), idesc,
                                     c > c0 || k > 0);
                        pair_commit(&ctl.empty[s]);
                        if (c + 1 == end) pair_commit(&ctl.sums_full[b]);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        ++r;
                    }
                }
            }
        }
        if (!ok) {
            if (lane == 0) flag_error(p.err, DR_ERRF_TIMEOUT);
            if (tc::elect_one()) pair_commit(&ctl.done);
            __syncwarp();
            tc::mbar_drain(&ctl.done, 0);
        }
    } else if (warp >= kEpiWarp) {
        const int e = warp - kEpiWarp, quad = warp & 3, half = e >> 2;
        constexpr int kCols = Box<kF32>::kCols;
        const int n_boxes = tile_cols / 2 / kCols;   // of this warp
        const bool res_tma = p.residual && p.vec_res;
        const uint32_t my_boxes = boxes + e * 2 * kBox;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        unsigned res_asked = 0, res_odd = 0;   // per buffer: whether a residual box was asked for, and an odd number of times
        bool ok = true;
        int64_t chain = 0;
        for (int64_t i = first; ok && i < tiles; i += step) {
            int tt, ct;
            tile_at(args, i, tt, ct);
            Box<kF32> box{p, maps, my_boxes, tt * kTileT + (int)rank * 128 + quad * 32, 0, lane};
            const int n0 = ct * tile_cols + half * (tile_cols / 2);
            const auto ask_residual = [&](int k) {
                if (lane == 0) {
                    tc::mbar_expect_tx(&ctl.res[e][k & 1], kBox);
                    own_load(my_boxes + (k & 1) * kBox, &maps.res, n0 + k * kCols, box.t0, &ctl.res[e][k & 1]);
                }
                res_asked |= 1u << (k & 1);
                res_odd ^= 1u << (k & 1);
            };
            if (lane == 0) stores_read<0>();
            __syncwarp();
            if (res_tma)
                for (int k = 0; k < 2 && k < n_boxes; ++k) ask_residual(k);
            float acc[kF32 ? 128 : 1];
            uint32_t sums = 0;
            if constexpr (kF32) {
                // thread's columns: 128 of the tile, or 64 and the 64 that multiply them
                const int pieces = (args.chunks + args.piece_chunks - 1) / args.piece_chunks;
                for (int k = 0; k < pieces; ++k, ++chain) {
                    const int b = (int)(chain & 1);
                    ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&ctl.sums_full[b], (unsigned)(chain >> 1) & 1, gave_up));
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t from = tmem + lanes + b * kTileW;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int col = p.gated ? (q >> 1) * 128 + half * 64 + (q & 1) * 32 : half * 128 + q * 32;
                        if (k == 0) {
                            tc::ld32(from + col, acc + 32 * q);
                        } else {
                            float more[32];
                            tc::ld32(from + col, more);
                            tc::wait_ld();
                            tc::pin32(more);
#pragma unroll
                            for (int j = 0; j < 32; ++j) acc[32 * q + j] += more[j];
                        }
                    }
                    tc::wait_ld();
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc::pin32(acc + 32 * q);
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) remote_arrive(mapa(tc::smem_u32(&ctl.sums_free[b]), 0));
                }
                if (!ok) break;
            } else {
                const int b = (int)(chain & 1);
                ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&ctl.sums_full[b], (unsigned)(chain >> 1) & 1, gave_up));
                if (!ok) break;
                tc::fence_after();
                sums = tmem + lanes + b * kTileW;
            }
            const auto begin_box = [&](int k) {
                box.at = my_boxes + (k & 1) * kBox;
                box.n = n0 + k * kCols;
                if (k >= 2 && !res_tma) {   // the box's store two boxes ago has read it
                    if (lane == 0) stores_read<1>();
                    __syncwarp();
                }
                if (res_tma) {
                    ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&ctl.res[e][k & 1], ~(res_odd >> (k & 1)) & 1, gave_up));
                } else if (p.residual) {
                    box.read_residual();
                }
            };
            const auto end_box = [&](int k) {
                box.store();
                if (res_tma && k + 2 < n_boxes) {
                    if (lane == 0) stores_read<0>();
                    __syncwarp();
                    ask_residual(k + 2);
                }
            };
            if constexpr (kF32) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= n_boxes) break;
                    begin_box(k);
                    if (!ok) break;
                    finish32(p, acc + 32 * k, acc + (32 * k + 64) % 128, box.n);
                    box.put32(acc + 32 * k, 0);
                    end_box(k);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < n_boxes; ++k) {
                    begin_box(k);
                    if (!ok) break;
#pragma unroll 1
                    for (int c0 = 0; c0 < 64; c0 += 32) {
                        const int col = half * (tile_cols / 2) + k * kCols + c0;
                        float a[32], g[32];
                        tc::ld32(sums + col, a);
                        if (p.gated) tc::ld32(sums + 128 + col, g);
                        tc::wait_ld();
                        tc::pin32(a);
                        if (p.gated) tc::pin32(g);
                        if (k + 1 == n_boxes && c0 == 32) {   // the last sums are read: the next tile may have their place
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) remote_arrive(mapa(tc::smem_u32(&ctl.sums_free[chain & 1]), 0));
                        }
                        finish32(p, a, g, box.n + c0);
                        box.put32(a, c0);
                    }
                    end_box(k);
                }
                ++chain;
            }
        }
        if (!ok) {
            if (lane == 0) flag_error(p.err, DR_ERRF_TIMEOUT);
            for (int b = 0; b < 2; ++b)   // residual boxes still on their way
                if (res_asked >> b & 1) tc::mbar_drain(&ctl.res[e][b], ~(res_odd >> b) & 1);
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    __syncwarp();
    tc::fence_before();
    cluster_sync();   // neither CTA's shared and tensor memory goes while the other may still use it
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Pairs that the device holds at once (per device; 0: not asked yet).
std::atomic<int> pairs_of_device[64];

template <bool kF32>
cudaError_t most_pairs(int sms, int *pairs) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};
    e = once_per_device(ready, [] {
        return cudaFuncSetAttribute(linear_tiles_kernel<kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    });
    if (e != cudaSuccess) return e;
    int n = dev < 64 ? pairs_of_device[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(sms / 2 * 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, linear_tiles_kernel<kF32>, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        if (dev < 64) pairs_of_device[dev].store(n, std::memory_order_relaxed);
    }
    *pairs = n;
    return cudaSuccess;
}

// Tensor map of an output or residual: boxes of 32 tokens and 128 bytes.
bool encode_box(CUtensorMap *map, const void *ptr, int64_t T, int cols, int64_t stride, bool f32) {
    return encode_matrix(map, ptr, f32, T, cols, stride, 32, f32 ? 32 : 64);
}

template <bool kF32>
cudaError_t launch(const LinearParams &p, int sms, cudaStream_t stream) {
    TileArgs a;
    a.p = p;
    a.chunks = (p.K + 63) / 64;
    a.piece_chunks = kF32 ? kPieceChunks : a.chunks;
    const int cols = p.gated ? kTileW / 2 : kTileW;
    a.token_tiles = (p.T + kTileT - 1) / kTileT;
    a.col_tiles = (p.N + cols - 1) / cols;
    Maps m;
    if (!encode_matrix(&m.x, p.x, false, p.T, p.K, p.x_stride, 128, 64) ||
        !encode_matrix(&m.w, p.W, false, (int64_t)p.N * (p.gated ? 2 : 1), p.K, p.K, 128, 64))
        return cudaErrorInvalidValue;
    m.res = m.x;
    for (int i = 0; i < DR_LINEAR_MAX_OUTS; ++i) m.out[i] = m.x;
    if (p.vec_out)
        for (int i = 0; i < p.n_outs; ++i)
            if (!encode_box(&m.out[i], p.out[i].ptr, p.T, p.out[i].cols, p.out[i].stride, kF32)) return cudaErrorInvalidValue;
    if (p.vec_res && !encode_box(&m.res, p.residual, p.T, p.N, p.res_stride, kF32)) return cudaErrorInvalidValue;
    int pairs = 0;
    const cudaError_t e = most_pairs<kF32>(sms, &pairs);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)a.token_tiles * a.col_tiles;
    if (tiles < pairs) pairs = (int)tiles;
    return launch_kernel(linear_tiles_kernel<kF32>, dim3((unsigned)(2 * pairs)), dim3(kThreads), kSmem, stream, 2, m, a);
}

}  // namespace

int linear_tiles_tiles(const LinearParams &p) {
    const int cols = p.gated ? kTileW / 2 : kTileW;
    const int64_t n = (int64_t)((p.T + kTileT - 1) / kTileT) * ((p.N + cols - 1) / cols);
    return n > 0x7FFFFFFF ? 0x7FFFFFFF : (int)n;
}

cudaError_t launch_linear_tiles(const LinearParams &p, int sms, cudaStream_t stream) {
    return p.out_f32 ? launch<true>(p, sms, stream) : launch<false>(p, sms, stream);
}

}  // namespace dr
