// Matrix product with an epilogue for prompts: out = residual + act(x W^T + bias), bound by the tensor cores.
//
// Pairs of CTAs (clusters of two) stay on their SMs and take 256 x 256 tiles of the output in turn: 256 tokens by 256
// weight rows (gated: 128 rows and the 128 that are multiplied in, so that both sums of a column meet in one thread).
// A pair's product is one tcgen05.mma of cta_group::2: each CTA holds 128 tokens and half of the weight rows, and the
// hardware feeds both halves to both SMs, so an SM reads 32 KB of shared memory per 64 of K instead of the 48 KB that a
// 128 x 256 tile of its own would take.
//   warp 0      TMA producer of its CTA's halves: 64-wide K chunks in a ring of kStages, counted on the first CTA's barrier
//   warp 1      MMA issuer (first CTA only)
//   warps 2, 3  carriers, each for eight epilogue warps: bias and residual in, results out, by TMA
//   warps 4-19  epilogue.  Where a pair has several tiles, two sets of eight warps take them in turn, 128 of a tile's sums per
//               token and warp; where it has one, or outputs are fp32, all sixteen share each tile, 64 sums a warp
// The sums of a tile take 256 of the 512 tensor-memory columns; the next tile is multiplied while the epilogue works on
// the one before.  A tile of K = 1024 is multiplied in 8192 cycles, during which reading its operands and writing them by TMA
// take all of shared memory's 128 bytes a cycle: whatever else goes through there costs the products time, and latencies
// are long (a read of tensor memory 2000 cycles, a load of bias 1000, the fence between writing a box and its store 2000).
// So an epilogue warp's results pass shared memory once, as a 4 KB box (32 tokens of 128 bytes, swizzled) that already
// holds the residual; what takes long is done ahead or afterwards by the carriers; and the two sets are half a period apart.
// Outputs or residuals whose rows are not 16-byte aligned are moved by the epilogue warps, a row of 32 columns at a time.
// fp32 outputs: tensor-core chains drift by about 1e-9 K, so each 512 of K is a tile's sums of its own, added up in the
// epilogue warps' registers.
// An epilogue warp reads 64 of its sums at once and waits for them there and then: nothing it reads is in flight while it works
// (reads that ran ahead of the work were slower, too: 16384 tokens 1024 -> 4096 with gelu, sustained, 101 us, now 95).
// Every mbarrier wait is bounded; after one that runs out the pair's further tiles are not written, and copies and
// products in flight are waited for before it exits.
#include <type_traits>

#include "dr_tc.cuh"
#include "linear_epilogue.cuh"

namespace dr {
namespace {

constexpr int kThreads = 640;
constexpr int kEpiWarp = 4, kEpiWarps = 16;
// Registers: the launch has 640 x 96; four warps give some of theirs to the other sixteen.
constexpr int kLaunchRegs = 96, kOtherRegs = 32, kEpiRegs = 112;
static_assert(kEpiWarp * 32 * kOtherRegs + kEpiWarps * 32 * kEpiRegs <= kThreads * kLaunchRegs, "more than the launch has");
constexpr int kTileT = 256;       // tokens per pair
constexpr int kTileW = 256;       // most weight rows per pair (MMA N), and tensor-memory columns of a tile
constexpr int kStages = 5;
constexpr int kHalf = 128 * 128;  // bytes of a CTA's tokens or weight rows in a stage
constexpr int kBox = 32 * 128;    // bytes of an epilogue box
constexpr int kCarrier = 2, kCarried = 8;   // first carrier warp, epilogue warps of each
constexpr int kPieceChunks = 8;   // fp32 outputs: K of 512 per chain
constexpr int kGroup = 8;         // token tiles that share their weight tiles' stay in L2
constexpr size_t kSmem = (size_t)kStages * 2 * kHalf + kEpiWarps * kBox + 2 * kTileW * sizeof(float) + 512;   // and Control

struct TileArgs {
    LinearParams p;
    int32_t chunks;         // of 64 of K
    int32_t piece_chunks;   // chunks per chain
    int32_t token_tiles, col_tiles;
    int32_t tile_w;         // weight rows per pair: 256, or 128 or 64 where tiles are few
    int32_t shared;         // 1: the epilogue warps share each tile; 0: their two sets take tiles in turn
};

struct Maps {
    CUtensorMap x, w, res, out[DR_LINEAR_MAX_OUTS];
};

struct Control {
    uint64_t full[kStages];    // first CTA's: both CTAs' copies of a stage have landed
    uint64_t empty[kStages];   // the products that read the stage are over
    uint64_t sums_full[2];     // a chain's sums are in tensor memory
    uint64_t sums_free[2];     // first CTA's: both CTAs' epilogue warps have read them
    uint64_t box_ready[kEpiWarps];   // the box may be written, and holds the residual
    uint64_t boxes_full[2];          // a carrier's boxes hold results
    uint64_t bias_ready[2];
    uint64_t done;
    uint32_t tmem;
    int gave_up;   // some wait ran out
};

// All threads of both CTAs have come here.  Relaxed: the barriers' set-up has a fence of its own, and at the end nothing is handed
// over (a release would wait for the last stores, some 1400 cycles).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Tile i: groups of kGroup token tiles take all column tiles in turn, so that both operands' tiles stay in L2.
__device__ __forceinline__ void tile_at(const TileArgs &a, int i, int &tt, int &ct) {
    const int per_group = kGroup * a.col_tiles, g = i / per_group;
    const int r = i - g * per_group, n = min(kGroup, a.token_tiles - g * kGroup);
    ct = r / n;
    tt = g * kGroup + (r - ct * n);
}

// 16 bytes c of row `row` of a box with rows of 128 (64) bytes, as TMA's swizzle of that width lays them.
template <bool kNarrow>
__device__ __forceinline__ uint32_t box_chunk(uint32_t at, int row, int c) {
    return kNarrow ? at + row * 64 + ((c ^ (row >> 1 & 3)) << 4) : at + row * 128 + ((c ^ (row & 7)) << 4);
}

// 32 results of this lane's token into its box, from 16-byte piece c0 on, added to what the box holds.
template <bool kF32, bool kNarrow>
__device__ __forceinline__ void put32(float *v, uint32_t at, int lane, int c0, bool add) {
    if constexpr (kF32) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t to = box_chunk<kNarrow>(at, lane, c);
            float *u = v + 4 * c;
            if (add) {
                const uint4 r = lds16(to);
                u[0] += __uint_as_float(r.x);
                u[1] += __uint_as_float(r.y);
                u[2] += __uint_as_float(r.z);
                u[3] += __uint_as_float(r.w);
            }
            sts16(to, make_uint4(__float_as_uint(u[0]), __float_as_uint(u[1]), __float_as_uint(u[2]), __float_as_uint(u[3])));
        }
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t to = box_chunk<kNarrow>(at, lane, c0 + c);
            float *u = v + 8 * c;
            if (add) {
                float f[8];
                unpack8(lds16(to), f);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] += f[j];
            }
            sts16(to, make_uint4(lin::pack2(u[0], u[1]), lin::pack2(u[2], u[3]), lin::pack2(u[4], u[5]), lin::pack2(u[6], u[7])));
        }
    }
}

// 32 columns n .. n+31 of a warp's 32 tokens between registers (lane = token) and rows that may start anywhere (lane =
// column), through a box of 32 x 32 fp32 values, column c of row r at r * 32 + (c ^ r).
template <bool kF32>
struct LooseRows {
    using T = typename std::conditional<kF32, float, uint16_t>::type;

    static __device__ __forceinline__ void add_residual(const LinearParams &p, float *v, float *box, int t0, int n, int lane) {
        const int rows = min(32, p.T - t0);
        const T *res = static_cast<const T *>(p.residual) + (int64_t)t0 * p.res_stride + n + lane;
        for (int r = 0; r < rows; ++r, res += p.res_stride)
            if (n + lane < p.N) {
                if constexpr (kF32) box[r * 32 + (lane ^ r)] = *res;
                else box[r * 32 + (lane ^ r)] = __uint_as_float((uint32_t)*res << 16);
            }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] += box[lane * 32 + (c ^ lane)];   // rows and columns past the end hold anything
        __syncwarp();
    }
    static __device__ __forceinline__ void store(const LinearParams &p, const float *v, float *box, int t0, int n, int lane) {
#pragma unroll
        for (int c = 0; c < 32; ++c) box[lane * 32 + (c ^ lane)] = v[c];
        __syncwarp();
        const LinearOut o = lin::output_of(p, n);   // the 32 columns lie in one output
        const int rows = min(32, p.T - t0), col = n - o.col0 + lane;
        T *to = static_cast<T *>(o.ptr) + (int64_t)t0 * o.stride + col;
        for (int r = 0; r < rows; ++r, to += o.stride)
            if (col < o.cols) {
                const float x = box[r * 32 + (lane ^ r)];
                if constexpr (kF32) *to = x;
                else *to = f32_to_bf16_rn(x);
            }
        __syncwarp();
    }
};

// Which tiles and columns an epilogue warp takes.
struct Share {
    int first, step;    // tiles
    int col0, span;     // columns
    int blocks;         // of 32 columns
    int box_cols;       // columns of a box: 128 bytes, or 64 where a warp's results come 32 bf16 columns at a time
    bool active;
    __device__ __forceinline__ Share(const TileArgs &a, int e, int first_tile, int tile_step, bool f32) {
        const int cols = a.p.gated ? a.tile_w / 2 : a.tile_w, set = e / kCarried, part = e >> 2;
        first = a.shared ? first_tile : first_tile + set * tile_step;
        step = a.shared ? tile_step : 2 * tile_step;
        span = a.shared ? max(32, cols / 4) : cols / 2;
        col0 = (a.shared ? part : part & 1) * span;
        blocks = span / 32;
        box_cols = f32 || a.p.gated || span == 32 ? 32 : 64;
        active = col0 < cols;
    }
};

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tiles_kernel(const __grid_constant__ Maps maps, const __grid_constant__ TileArgs args) {
    extern __shared__ __align__(1024) uint8_t smem[];   // all there is: nothing in front of it
    static_assert(sizeof(Control) <= 512, "kSmem");
    Control &ctl = *reinterpret_cast<Control *>(smem + kSmem - 512);

    const LinearParams &p = args.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1;   // the cluster's first CTA issues the products of both
    const int tiles = args.token_tiles * args.col_tiles, first = blockIdx.x / 2, step = gridDim.x / 2;
    const uint32_t ring = tc::smem_u32(smem);
    const uint32_t sx = ring, sw = ring + kStages * kHalf, boxes = ring + 2 * kStages * kHalf;
    float *const bias = reinterpret_cast<float *>(smem + 2 * kStages * kHalf + kEpiWarps * kBox);   // two tiles' sums'
    const int tile_cols = p.gated ? args.tile_w / 2 : args.tile_w;
    volatile int *gave_up = &ctl.gave_up;
    // whole 16-byte pieces of rows: boxes carried by TMA
    const bool boxed = p.vec_out && (!p.residual || p.vec_res);

    if (warp == 0) {   // a lane per barrier of a kind: one after the other they take some 400 cycles
        if (lane < kStages) {
            tc::mbar_init(&ctl.full[lane], 1);
            tc::mbar_init(&ctl.empty[lane], 1);
        }
        if (lane < 2) {
            const Share share(args, 0, 0, 0, kF32);
            const int warps = args.shared ? 4 * (tile_cols / share.span) : kCarried;   // that take a tile
            tc::mbar_init(&ctl.sums_full[lane], 1);
            tc::mbar_init(&ctl.sums_free[lane], 2 * warps);
            tc::mbar_init(&ctl.boxes_full[lane], args.shared ? max(1, min(kCarried, warps - lane * kCarried)) : kCarried);
            tc::mbar_init(&ctl.bias_ready[lane], 1);
        }
        if (lane < kEpiWarps) tc::mbar_init(&ctl.box_ready[lane], 1);
        if (lane == 0) {
            tc::mbar_init(&ctl.done, 1);
            ctl.gave_up = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.x)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.w)) : "memory");
        }
        __syncwarp();
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

    if (warp < kEpiWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 0) {
            int s = 0, r = 0;
            unsigned armed = 0;   // stages whose copies were issued, and how often (parity of the last)
            unsigned parity = 0;
            bool ok = true;
            for (int i = first; ok && i < tiles; i += step) {
                int tt, ct;
                tile_at(args, i, tt, ct);
                const int t = tt * kTileT + (int)rank * 128;
                // rows of W: the pair's in halves, or the first half and those that multiply it
                const int w = p.gated ? (int)rank * p.N + ct * tile_cols : ct * tile_cols + (int)rank * (args.tile_w / 2);
                for (int c = 0; c < args.chunks; ++c) {
                    if (!(c == 0 && i == p.stall_tile)) {
                        if (r > 0 && !tc::mbar_wait(&ctl.empty[s], (r - 1) & 1, gave_up)) {
                            ok = false;
                            break;
                        }
                        if (tc::elect_one()) {
                            const uint32_t bar = tc::mapa(tc::smem_u32(&ctl.full[s]), 0);
                            if (rank == 0) tc::mbar_expect_tx(&ctl.full[s], 2 * kHalf + args.tile_w * 128);
                            tc::pair_load(sx + s * kHalf, &maps.x, c * 64, t, bar);
                            tc::pair_load(sw + s * kHalf, &maps.w, c * 64, w, bar);
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
            const uint32_t idesc = tc::instr_desc(kTileT, args.tile_w, false, false);
            const uint64_t dx = tc::smem_desc(sx), dw = tc::smem_desc(sw);
            int s = 0, r = 0;
            unsigned chain = 0;
            bool ok = true;
            for (int i = first; ok && i < tiles; i += step) {
                for (int c = 0; ok && c < args.chunks; ++chain) {
                    const int b = (int)(chain & 1);
                    if (chain >= 2 && !tc::mbar_wait(&ctl.sums_free[b], ((chain >> 1) - 1) & 1, gave_up)) {
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
                                tc::pair_mma(d, tc::desc_at(dx, s * kHalf + k * 32), tc::desc_at(dw, s * kHalf + k * 32), idesc,
                                             c > c0 || k > 0);
                            tc::pair_commit(&ctl.empty[s]);
                            if (c + 1 == end) tc::pair_commit(&ctl.sums_full[b]);
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
                if (tc::elect_one()) tc::pair_commit(&ctl.done);
                __syncwarp();
                tc::mbar_drain(&ctl.done, 0);
            }
        } else if (warp >= kCarrier) {
            const int set = warp - kCarrier, e = set * kCarried + (lane & (kCarried - 1));
            const Share share(args, e, first, step, kF32);
            const bool mine = lane < kCarried && share.active;   // a lane per box
            const bool any = Share(args, set * kCarried, first, step, kF32).active;
            const uint32_t at = boxes + e * kBox;
            const int uses = share.span / share.box_cols;   // boxes per tile and warp
            float *const to = bias + set * kTileW;
            unsigned phase = 0;
            bool ok = true;
            for (int i = share.first; any && ok && i < tiles; i += share.step) {
                int tt, ct;
                tile_at(args, i, tt, ct);
                const int n0 = ct * tile_cols;
                if (p.bias) {   // the tile before is done with it
                    for (int j = lane; j < args.tile_w; j += 32) {
                        const int n = n0 + (j & (tile_cols - 1));
                        to[j] = n < p.N ? lin::bf16_at(p.bias, j < tile_cols ? n : (int64_t)p.N + n) : 0.f;
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&ctl.bias_ready[set]);
                }
                for (int u = 0; u < uses; ++u, phase ^= 1) {
                    const int t0 = tt * kTileT + (int)rank * 128 + (e & 3) * 32, n = n0 + share.col0 + u * share.box_cols;
                    if (mine && boxed) {
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the store before has read the box
                        if (p.residual) {
                            tc::mbar_expect_tx(&ctl.box_ready[e], !kF32 && share.box_cols == 32 ? kBox / 2 : kBox);
                            own_load(at, &maps.res, n, t0, &ctl.box_ready[e]);
                        } else {
                            tc::mbar_arrive(&ctl.box_ready[e]);
                        }
                    }
                    __syncwarp();
                    ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&ctl.boxes_full[set], phase, gave_up));
                    if (!ok) break;
                    tc::fence_proxy_async();   // what the epilogue warps wrote, for the stores below
                    if (mine && boxed) {
                        const int s = lin::out_of(p, n);
                        if (t0 < p.T && n - p.out[s].col0 < p.out[s].cols) box_store(&maps.out[s], n - p.out[s].col0, t0, at);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    __syncwarp();
                }
            }
            if (!ok) {
                if (lane == 0) flag_error(p.err, DR_ERRF_TIMEOUT);
                if (boxed && p.residual && mine) tc::mbar_drain(&ctl.box_ready[e], phase);   // on its way
            }
            if (mine) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        const int e = warp - kEpiWarp, set = e / kCarried, quad = warp & 3;
        const Share share(args, e, first, step, kF32);
        const bool shared = kF32 || args.shared, narrow = !kF32 && share.box_cols == 32;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const int pieces = kF32 ? (args.chunks + args.piece_chunks - 1) / args.piece_chunks : 1;
        const uint32_t box = boxes + e * kBox;
        unsigned chain = shared ? 0 : set, box_phase = 0, bias_phase = 0;   // in turn, a set has the even or the odd chains
        bool ok = true;
        const int apart = p.gated ? args.tile_w / 2 : 32;   // from a block's sums to those that multiply it, or the next block's
        const bool two = p.gated || share.span > 32;        // whether there are such
        const auto release = [&] {   // this warp has its sums: the place may have another tile's
            tc::fence_before();
            __syncwarp();
            if (lane == 0) remote_arrive(tc::mapa(tc::smem_u32(&ctl.sums_free[chain & 1]), 0));
            __syncwarp();
            chain += shared ? 1 : 2;
        };
        for (int i = share.first; share.active && ok && i < tiles; i += share.step) {
            float acc[64];
            uint32_t from = 0;
            for (int k = 0; k < pieces; ++k) {
                ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&ctl.sums_full[chain & 1], (chain >> 1) & 1, gave_up));
                if (!ok) break;
                tc::fence_after();
                from = tmem + lanes + (chain & 1) * kTileW + share.col0;
                if (!kF32 || k == 0) {
                    if (two) tc::ld32x2_wait(from, acc, from + apart, acc + 32);
                    else tc::ld32_wait(from, acc);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (q >= 2 && !two) break;
                        float more[16];
                        tc::ld16_wait(from + (q < 2 ? 0 : apart) + (q & 1) * 16, more);
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[16 * q + j] += more[j];
                    }
                }
                if (shared) release();
            }
            if (!ok) break;
            if (p.bias) {
                ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&ctl.bias_ready[set], bias_phase, gave_up));
                if (!ok) break;
                bias_phase ^= 1;
            }
            const float *b = bias + set * kTileW + share.col0;
            // 32 columns: the sums v (gated: times those in g) to the box or the output
            const auto block = [&](float *v, float *g, int k) {
                if (p.bias) {
                    lin::add_bias<32>(v, b + k * 32);
                    if (p.gated) lin::add_bias<32>(g, b + k * 32 + apart);
                }
                lin::activate<32>(v, p.act);
                if (p.gated) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= g[j];
                }
                const bool opens = kF32 || narrow || k % 2 == 0, closes = kF32 || narrow || k % 2 == 1;   // a box
                if (boxed) {
                    if (opens) {
                        if (!__all_sync(0xFFFFFFFFu, tc::mbar_wait(&ctl.box_ready[e], box_phase, gave_up))) return false;
                        box_phase ^= 1;
                    }
                    if (narrow) put32<kF32, true>(v, box, lane, 0, p.residual);
                    else put32<kF32, false>(v, box, lane, opens ? 0 : 4, p.residual);
                } else {
                    int tt, ct;
                    tile_at(args, i, tt, ct);
                    const int t0 = tt * kTileT + (int)rank * 128 + quad * 32, n = ct * tile_cols + share.col0 + k * 32;
                    float *const loose = reinterpret_cast<float *>(smem + (box - ring));
                    if (n < p.N) {
                        if (p.residual) LooseRows<kF32>::add_residual(p, v, loose, t0, n, lane);
                        LooseRows<kF32>::store(p, v, loose, t0, n, lane);
                    }
                }
                if (closes) {
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&ctl.boxes_full[set]);
                    __syncwarp();   // whole again: tensor-memory instructions want all lanes at once
                }
                return true;
            };
            // Two blocks at a time, one in either half of the registers (gated: one, and what multiplies it).
#pragma unroll 1
            for (int k = 0;;) {
                ok = block(acc, acc + 32, k);
                if (ok && !p.gated && share.blocks > 1) ok = block(acc + 32, acc, k + 1);
                k += p.gated ? 1 : 2;
                if (!ok || shared || k >= share.blocks) break;   // (a shared tile's warps have their two at once)
                from += p.gated ? 32 : 64;   // the rest of the set's share
                tc::ld32x2_wait(from, acc, from + apart, acc + 32);
                release();
            }
        }
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

// Weight rows of a pair's tile: fewer where that puts more pairs to work at once.
int tile_width(const LinearParams &p, int pairs) {
    const int64_t token_tiles = (p.T + kTileT - 1) / kTileT;
    int w = kTileW;
    while (w > 64) {
        const int cols = p.gated ? w / 4 : w / 2;
        if (token_tiles * ((p.N + cols - 1) / cols) > pairs) break;
        w /= 2;
    }
    return w;
}

// Tensor map of an output or residual: boxes of 32 tokens.
bool encode_box(CUtensorMap *map, const void *ptr, const LinearParams &p, int cols, int64_t stride, bool wide) {
    return encode_matrix(map, ptr, p.out_f32, p.T, cols, stride, 32, wide ? 64 : 32);
}

template <bool kF32>
cudaError_t launch(const LinearParams &p, int sms, cudaStream_t stream) {
    TileArgs a;
    a.p = p;
    a.chunks = (p.K + 63) / 64;
    a.piece_chunks = kF32 ? kPieceChunks : a.chunks;
    int pairs = 0;
    const cudaError_t e = most_pairs<kF32>(sms, &pairs);
    if (e != cudaSuccess) return e;
    a.tile_w = tile_width(p, pairs);
    const int cols = p.gated ? a.tile_w / 2 : a.tile_w;
    a.token_tiles = (p.T + kTileT - 1) / kTileT;
    a.col_tiles = (p.N + cols - 1) / cols;
    const int64_t tiles = (int64_t)a.token_tiles * a.col_tiles;
    if (tiles > 0x3FFFFFFF) return cudaErrorInvalidValue;   // tiles are counted in 32 bits: 2^46 outputs
    if (tiles < pairs) pairs = (int)tiles;
    a.shared = kF32 || a.tile_w < kTileW || tiles <= pairs;
    const bool wide = !kF32 && !p.gated && a.tile_w == kTileW;
    Maps m;
    if (!encode_matrix(&m.x, p.x, false, p.T, p.K, p.x_stride, 128, 64) ||
        !encode_matrix(&m.w, p.W, false, (int64_t)p.N * (p.gated ? 2 : 1), p.K, p.K, a.tile_w / 2, 64))
        return cudaErrorInvalidValue;
    // maps that the kernel does not use stay copies
    m.res = m.x;
    for (int i = 0; i < DR_LINEAR_MAX_OUTS; ++i) m.out[i] = m.x;
    if (p.vec_out)
        for (int i = 0; i < p.n_outs; ++i)
            if (!encode_box(&m.out[i], p.out[i].ptr, p, p.out[i].cols, p.out[i].stride, wide)) return cudaErrorInvalidValue;
    if (p.vec_res && !encode_box(&m.res, p.residual, p, p.N, p.res_stride, wide)) return cudaErrorInvalidValue;
    return launch_kernel(linear_tiles_kernel<kF32>, dim3((unsigned)(2 * pairs)), dim3(kThreads), kSmem, stream, 2, m, a);
}

}  // namespace

int linear_tiles_tiles(const LinearParams &p, int sms) {
    const int w = tile_width(p, sms / 2), cols = p.gated ? w / 2 : w;
    const int64_t n = (int64_t)((p.T + kTileT - 1) / kTileT) * ((p.N + cols - 1) / cols);
    return n > 0x7FFFFFFF ? 0x7FFFFFFF : (int)n;
}

cudaError_t launch_linear_tiles(const LinearParams &p, int sms, cudaStream_t stream) {
    return p.out_f32 ? launch<true>(p, sms, stream) : launch<false>(p, sms, stream);
}

}  // namespace dr
