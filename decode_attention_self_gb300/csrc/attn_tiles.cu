// Attention of many query rows over a cache on the 5th-generation tensor cores: prompts, chunks of prompts, and the
// prefix that all rows of a batch share.
//
//   S = Q K^T (128 query rows x 128 keys, D = 64),  P = 2^(S' - m),  O = O 2^(m_old - m) + P V,  l = l 2^(..) + sum P
//
// The g query heads of a kv head and consecutive tokens fill a tile's rows together (row = token * g + head), so one
// pass over the keys serves them all.  A CTA holds one tile of 128 rows and walks its keys 128 at a time; two CTAs share
// an SM and their phases drift apart, so that one's products run under the other's exponentials.  Warps of a CTA:
//   softmax (4)    one thread per query row: S to registers, mask, running maximum, weights, P back to tensor memory
//   producers      TMA loads, K by one and V by another, e4m3 both by one (a paged tile is eight 16-key boxes; blocks
//                  outside the pool and past the last visible key come from an out-of-range coordinate: zeros)
//   MMA            S = Q K^T into tensor memory, one key tile ahead of the softmax; O += P V with P read from tensor
//                  memory and V as the MN-major operand
//   helpers        bf16, one: values that no row of the CTA sees become 0.  e4m3, one for K and one for V: that, and
//                  codes to f16 (exact) on the way from the TMA's buffer to the MMA's
// The softmax holds a row's 128 scores in registers and gives S back before the exponentials, so that the next product runs
// under them.  Biases on keys behind the query, and caps with a bias, would make that code too long for the instruction
// cache: such tiles go through tensor memory a quarter at a time in rolled loops.
// The running maximum moves only when a score passes it by 2^8 (log2 units): O is rescaled rarely.  Sums and states are
// fp32; weights are rounded once, to bf16 (e4m3: f16), for the product with V: the instruction takes both operands in one
// type, and the rests of bf16 weights would need 64 more columns of tensor memory (two CTAs fill it) and P V a second time.
//
// What bounds it.  One token of one head costs 256 flops and one exponential per key it sees.  16384 causal tokens of 16
// heads, bf16: 518 us, 1060 TFLOP/s; the products alone would take 288 us at the library GEMM's rate and the exponentials
// 230 us of the special-function units.  P V runs at 45 cycles per instruction where its shape allows 32 (P comes from
// tensor memory), and the maximum, the packing and the moves to and from tensor memory take issue slots beside the
// exponentials.  Two threads per row (half the registers), skipping hidden columns inside the straight way, and P V one
// tile later were each built and were slower.  e4m3: 600 us; CTAs of two tiles, which convert the keys once for both but
// are alone on their SM, took 6% longer.  24 to 52 bytes per thread are spilled.  Short rows are bound by a CTA's start
// and end: 1304 CTAs without any key take 23 us (9 rows of 364..1812 tokens, 4 kv heads in groups of 4), the same rows
// causal 61, causal with a bias 77, with a cap 106, cut into about three documents each 51, documents with a bias 62.
//
// Every wait is bounded (about 2 s): DR_ERRF_TIMEOUT, the CTA writes no output (a state that others join becomes NaN), waits
// for its own copies and products in flight and frees its tensor memory.
#include <math.h>

#include "dr_prompt.h"
#include "dr_rows.cuh"
#include "dr_score.cuh"
#include "dr_tc.cuh"

namespace dr {
namespace {

using namespace tc;

constexpr int kD = kHeadDim;
constexpr int kRows = 128;   // query rows per tile (MMA M) and keys per tile (MMA N of S, K of O)
constexpr int kKeys = 128;
constexpr int kBitsRing = 8;
constexpr int kMaxStages = 3;
constexpr uint32_t kTileBytes = kKeys * kD * 2;   // a K, V or Q tile of 16-bit elements: 16 KB

template <bool kFp8>
struct Config {
    static constexpr int kProducers = kFp8 ? 1 : 2;              // e4m3: one warp loads K and V
    static constexpr int kMmaWarp = 4 + kProducers, kHelper = kMmaWarp + 1;
    static constexpr int kThreads = 256, kCtasPerSm = 2;
    static constexpr int kTma = kFp8 ? 2 : 3;                    // stages that TMA fills (bf16: the MMA reads them)
    static constexpr int kMma = kFp8 ? 2 : kTma;                 // stages that the MMA reads
    static constexpr uint32_t kTmaBytes = kKeys * kD * (kFp8 ? 1 : 2);
    static constexpr uint32_t kQ = 0, kK = kTileBytes, kV = kK + kMma * kTileBytes, kRawK = kV + kMma * kTileBytes,
                              kRawV = kRawK + (kFp8 ? kTma * kTmaBytes : 0), kEnd = kRawV + (kFp8 ? kTma * kTmaBytes : 0);
};
// Registers: softmax threads hold a row of 128 scores; the rest needs few.  The shares add up to the launch's.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 184, kOtherRegs = 72;
static_assert(kSoftmaxRegs + kOtherRegs <= 2 * kLaunchRegs, "register split");
// tensor memory columns: S (128), O (64), P (64, two weights per column)
constexpr uint32_t kTmemCols = 256;

struct Control {   // at Config::kEnd of the dynamic shared memory
    uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t k_ready[kMaxStages], v_ready[kMaxStages], kc_empty[kMaxStages], vc_empty[kMaxStages];
    uint64_t q_full, s_full, s_free, p_full, o_done;
    uint64_t drained;                    // after a wait that ran out: the products in flight
    uint32_t tmem;
    int gave_up, redo, nonfinite;
    int bits[kBitsRing];                 // per tile: which of its eight 16-key blocks are there
    int b, qt, s0, n, L, prefix;         // the CTA's row and tile
    int lo_min, hi_max;                  // keys that some row sees
    int lo_max, hi_min;                  // keys that every row sees
};

// n / d for n < 2^31 by a product and a shift, the method of Granlund and Montgomery (1994) (a division takes some 30 instructions, and the start of a CTA has five).
struct Divisor {
    uint32_t d, mul, shift;
    void set(uint32_t by) {
        d = by;
        shift = 0;
        while ((1u << shift) < by) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - by)) / by + 1);
    }
    __device__ __forceinline__ unsigned of(unsigned n) const { return (n + __umulhi(n, mul)) >> shift; }
};

struct TileParams {
    PromptParams p;
    Divisor splits, heads, group;   // CTAs per tile, key/value heads, query heads per key/value head
};

// Physical byte of 16-byte chunk c of 128-byte row r under the 128-byte swizzle (tile base 1024-byte aligned).
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ bool nonfinite16(uint32_t w, uint32_t exp_mask) {
    return (w & exp_mask) == exp_mask || ((w >> 16) & exp_mask) == exp_mask;
}

// 32-byte store: a thread's output row is 128 bytes or more, and a request of the warp touches 32 rows.
__device__ __forceinline__ void st_32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Zeroes the NaN codes (0x7F, 0xFF) among four e4m3 codes; whether there was one.
__device__ __forceinline__ bool zero_nan_codes(uint32_t &w) {
    const uint32_t t = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // bit 7 of the bytes that hold one
    if (t == 0) return false;
    w &= ~((t >> 7) * 0xFFu);
    return true;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Weights 2^(s mul - mref) of N scores, packed in pairs; their sum (of the weights before they are rounded).
template <int N, bool kF16>
__device__ __forceinline__ float weights(const float (&s)[N], float mul, float mref, uint32_t (&pk)[N / 2]) {
    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
    const float2 mul2 = make_float2(mul, mul), off2 = make_float2(-mref, -mref);
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), mul2, off2);
        float2 y = __ffma2_rn(make_float2(s[c + 2], s[c + 3]), mul2, off2);
        x.x = fast_exp2(x.x);
        x.y = fast_exp2(x.y);
        y.x = fast_exp2(y.x);
        y.y = fast_exp2(y.y);
        sum0 = __fadd2_rn(sum0, x);
        sum1 = __fadd2_rn(sum1, y);
        pk[c / 2] = kF16 ? pack_f16(x.x, x.y) : pack_bf16(x.x, x.y);
        pk[c / 2 + 1] = kF16 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
    }
    return (sum0.x + sum0.y) + (sum1.x + sum1.y);
}

// Keys [lo, hi) that query i of a row of n queries and L keys sees, and its position.
__device__ __forceinline__ void visible(const PromptParams &p, int t, int i, int n, int L, int prefix, int &lo, int &hi,
                                        int &pos) {
    if (p.row_start) {
        pos = L - n + i;
        lo = p.first_key ? max(0, __ldg(p.first_key + t)) : 0;
        hi = p.causal ? min(L, max(pos + 1, prefix)) : L;
    } else {   // shared prefix: every query stands behind it
        pos = L + (p.own_len ? min(max(0, __ldg(p.own_len + t)), p.own_cap) : 0) - 1;
        lo = 0;
        hi = L;
    }
    if (lo >= hi) lo = hi = 0;
}

// kMode: what is done to scores before the softmax
enum : int { kPlain, kBiased, kCapped };   // capped: biased too, or not

template <bool kFp8, bool kPaged, int kMode>
__global__ void __launch_bounds__(Config<kFp8>::kThreads, Config<kFp8>::kCtasPerSm)
    attn_tiles_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const TileParams tp) {
    using C = Config<kFp8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control &ctl = *reinterpret_cast<Control *>(smem + C::kEnd);
    const PromptParams &p = tp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kProducer = 4, kMmaWarp = C::kMmaWarp, kHelper = C::kHelper;

    // never: the swizzled tiles need 1024-byte alignment.  Such a CTA sees no key and ends as after a wait that ran out.
    const bool misplaced = (smem_u32(smem) & 1023u) != 0;
    if (warp == 1) {   // a lane per barrier
        constexpr int kRing = 8 * kMaxStages;
        static_assert(kRing <= 32 && offsetof(Control, q_full) == kRing * 8 && offsetof(Control, tmem) == (kRing + 6) * 8,
                      "order of the barriers");
        uint64_t *bars = reinterpret_cast<uint64_t *>(&ctl);
        // the four softmax warps arrive at q_full, s_free and p_full, one thread or the tensor pipe at the others
        if (lane < kRing + 6)
            mbar_init(bars + lane, lane == kRing || lane == kRing + 2 || lane == kRing + 3 ? 4 : 1);
        if (lane == 0) {
            ctl.lo_min = 0x7FFFFFFF;
            ctl.hi_max = 0;
            ctl.lo_max = 0;
            ctl.hi_min = 0x7FFFFFFF;
            ctl.gave_up = misplaced;
            ctl.redo = ctl.nonfinite = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    } else if (warp == kProducer && lane < 2) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &map_v : &map_k)) : "memory");
    }
    pdl_wait();
    // Tensor memory is taken after the wait and before the next grid may start: no CTA that waits for another grid holds
    // what that grid still has to take.
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        fence_before();
    }

    // Which tile of which row: tiles of the rows in turn, a row's last (longest, when causal) tile of all heads first
    const unsigned unit = tp.heads.of(blockIdx.x), tile_no = tp.splits.of(unit);
    const int hk = (int)(blockIdx.x - unit * tp.heads.d), split = (int)(unit - tile_no * tp.splits.d);
    if (warp == 0) {
        int want = (int)tile_no;
        int b = -1, s0 = 0, n = 0, L = 0, prefix = 0;
        if (!p.row_start) {
            const int tiles = (int)(((unsigned)p.T * (unsigned)p.g + kRows - 1) / (unsigned)kRows);
            if (want < tiles) b = 0;
            n = p.T;
            L = __ldg(p.kv_len);
        } else {
            const bool checks = blockIdx.x == 0;   // this CTA looks every row over
            for (int base = 0; base < p.B && (b < 0 || checks); base += 32) {
                int a = 0, e = 0, len_l = 0, pre_l = 0;
                if (base + lane < p.B) {
                    len_l = __ldg(p.kv_len + base + lane);
                    pre_l = p.prefix_len ? __ldg(p.prefix_len + base + lane) : 0;
                    a = __ldg(p.row_start + base + lane);
                    e = __ldg(p.row_start + base + lane + 1);
                    if (checks && (a < 0 || e < a || e > p.T || (base + lane == 0 && a != 0)))
                        flag_error(p.err, DR_ERRF_ROW_START);
                    a = min(max(a, 0), p.T);
                    e = min(max(e, a), p.T);
                }
                if (b >= 0) continue;
                const int len = e - a;
                const int tiles =
                    len > p.few_max ? (int)(((unsigned)len * (unsigned)p.g + kRows - 1) / (unsigned)kRows) : 0;
                int sum = tiles;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, sum, off);
                    if (lane >= off) sum += o;
                }
                const unsigned m = __ballot_sync(0xFFFFFFFFu, sum > want);
                if (m) {
                    const int src = __ffs(m) - 1;
                    b = base + src;
                    s0 = __shfl_sync(0xFFFFFFFFu, a, src);
                    n = __shfl_sync(0xFFFFFFFFu, len, src);
                    L = __shfl_sync(0xFFFFFFFFu, len_l, src);
                    prefix = __shfl_sync(0xFFFFFFFFu, pre_l, src);
                    const int before = __shfl_sync(0xFFFFFFFFu, sum - tiles, src);
                    const int mine = __shfl_sync(0xFFFFFFFFu, tiles, src);
                    want = mine - 1 - (want - before);
                } else {
                    want -= __shfl_sync(0xFFFFFFFFu, sum, 31);
                }
            }
        }
        if (lane == 0) {
            if (b >= 0) {
                const int min_len = p.row_start ? n : 0;
                if (L < min_len || L > p.cap) {
                    flag_error(p.err, DR_ERRF_SEQ_LEN);
                    L = min(max(L, 0), p.cap);
                }
            }
            ctl.b = b;
            ctl.qt = want;
            ctl.s0 = s0;
            ctl.n = n;
            ctl.L = misplaced ? 0 : L;
            ctl.prefix = prefix;
        }
    }
    __syncthreads();
    fence_after();
    pdl_trigger();
    const uint32_t tmem = ctl.tmem;
    if (ctl.b < 0) {   // past the last tile
        if (warp == kMmaWarp)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
        return;
    }
    const int b = ctl.b, L = ctl.L, n = ctl.n;

    // The keys that the softmax threads' rows see, and those that some and all rows of the CTA see
    const int row = threadIdx.x;
    int lo = 0, hi = 0, pos = 0, orow = 0;   // orow: token * Hq + head
    bool valid = false;
    uint4 qw[8];   // the query, on its way while the keys that it sees are found out
    const unsigned flat0 = (unsigned)ctl.qt * (unsigned)kRows, flat_end = (unsigned)n * (unsigned)p.g;   // T * Hq < 2^31
    if (warp < kProducer) {
        const unsigned flat = flat0 + row;
        valid = flat < flat_end;
        if (valid) {
            const unsigned i = tp.group.of(flat);
            const int token = ctl.s0 + (int)i, head = hk * p.g + (int)(flat - i * (unsigned)p.g);
            const uint16_t *src = p.q + (size_t)token * p.q_stride + (size_t)head * kD;
#pragma unroll
            for (int c = 0; c < 8; ++c) qw[c] = ld_ro16(src + 8 * c);
            visible(p, token, (int)i, n, L, ctl.prefix, lo, hi, pos);
            orow = token * p.Hq + head;
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) qw[c] = make_uint4(0, 0, 0, 0);
        }
    }
    int ulo, uhi, clo, chi;
    if (p.first_key) {
        if (warp < kProducer) {
            const bool sees = hi > lo;
            const int a0 = __reduce_min_sync(0xFFFFFFFFu, sees ? lo : 0x7FFFFFFF);
            const int a1 = __reduce_max_sync(0xFFFFFFFFu, hi);
            const int b0 = __reduce_max_sync(0xFFFFFFFFu, lo);
            const int b1 = __reduce_min_sync(0xFFFFFFFFu, sees ? hi : 0x7FFFFFFF);
            if (lane == 0) {
                atomicMin(&ctl.lo_min, a0);
                atomicMax(&ctl.hi_max, a1);
                atomicMax(&ctl.lo_max, b0);
                atomicMin(&ctl.hi_min, b1);
            }
        }
        __syncthreads();
        ulo = ctl.lo_min;
        uhi = ctl.hi_max;
        clo = ctl.lo_max;
        chi = ctl.hi_min;
        if (ulo >= uhi) ulo = uhi = 0;
    } else {   // from key 0 to an end that does not fall from one token to the next
        const auto end_of = [&](unsigned flat) -> int {
            int a, e, q;
            visible(p, ctl.s0, (int)tp.group.of(flat), n, L, ctl.prefix, a, e, q);
            return e;
        };
        ulo = clo = 0;
        chi = end_of(flat0);
        uhi = end_of(min(flat0 + kRows, flat_end) - 1);
    }

    // Key tiles: tile i covers keys [kbase + 128 i, + 128); this split's run of them
    const int kbase = ulo & ~(kBlockKeys - 1);
    const int all = (int)((unsigned)(uhi - kbase + kKeys - 1) / kKeys);
    const int per = (int)tp.splits.of((unsigned)all + tp.splits.d - 1);
    const int cb = min(split * per, all), ce = min(cb + per, all);
    volatile int *gave_up = &ctl.gave_up;
    // Twice at most.  A value that is not finite makes a sum of every row of its tile NaN (0 times infinity), of rows that
    // do not see it too.  So where some row ends up with sums that are not finite, the CTA goes over its keys once more,
    // with such values kept out of tiles that not every row sees whole, and every row then adds those that it sees.
    const auto again = [&](int pass) -> bool {   // the same in every thread: all of them get here
        fence_before();
        __syncthreads();
        return pass == 0 && *(volatile int *)&ctl.redo && !*gave_up;
    };

    if (warp >= kProducer) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp < kMmaWarp) {
            // bf16: K by the first producer warp, V by the second.  Block ids of four tiles at a time, one per lane, loaded
            // four tiles ahead (a load per tile, waited for in turn, took longer than the tile's arithmetic): lane 8 y + x
            // has block x of tile y of the group.  z of a block that is not there is out of range.
            const bool does_k = warp == kProducer, does_v = kFp8 || warp != kProducer;
            const uint32_t ring_k = smem_u32(smem + (kFp8 ? C::kRawK : C::kK)),
                           ring_v = smem_u32(smem + (kFp8 ? C::kRawV : C::kV));
            const int kv_row = kPaged ? 0 : b * p.Hkv + hk;
            const bool leader = elect_one();
            const auto group_ids = [&](int j) -> int {   // tiles j .. j + 3
                const int key = kbase + j * kKeys + lane * kBlockKeys;
                return j < ce && key < uhi ? __ldg(p.table + (size_t)b * p.max_blocks + key / kBlockKeys) : -1;
            };
            // (Test hook: the stalled CTA's first keys are never asked for, and the waits for them run out.)
            const int skip = does_k && (int)blockIdx.x == p.stall - 1 ? 1 : 0;
            int s = skip, round = 0, pass = 0, ahead = 0;   // ahead: K of a tile whose V could not be loaded
            do {
                int ids = 0, ids_next = 0;
                if (kPaged) ids_next = group_ids(cb);
                for (int j = cb + skip, i = skip; j < ce; ++j, ++i) {
                    unsigned bits = 0xFFu;
                    int z[8] = {};
                    if (kPaged) {
                        if ((i & 3) == 0) {
                            ids = ids_next;
                            ids_next = group_ids(j + 4);
                            // a block that some row sees and that is not in the pool
                            const int key = kbase + j * kKeys + lane * kBlockKeys;
                            if (does_k && key < uhi && key < kbase + ce * kKeys && (unsigned)ids >= (unsigned)p.num_blocks)
                                flag_error(p.err, DR_ERRF_BLOCK_ID);
                            ids = (unsigned)ids < (unsigned)p.num_blocks ? ids * p.Hkv + hk : -1;
                        }
                        bits = (__ballot_sync(0xFFFFFFFFu, ids >= 0) >> ((i & 3) * 8)) & 0xFFu;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            z[x] = __shfl_sync(0xFFFFFFFFu, ids, (i & 3) * 8 + x);
                            if (z[x] < 0) z[x] = p.num_blocks * p.Hkv;
                        }
                    }
                    // Boxes by one lane of a converged warp: eight lanes with one each take turns, and took over 100 cycles
                    // per box
                    const auto load = [&](const CUtensorMap *map, uint32_t dst, uint64_t *full, uint64_t *empty) -> bool {
                        if (round > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(empty, (round - 1) & 1, gave_up))) return false;
                        if (leader) {
                            if (map == &map_k) ctl.bits[i % kBitsRing] = (int)bits;
                            mbar_expect_tx(full, C::kTmaBytes);
                            if (kPaged) {
#pragma unroll
                                for (int x = 0; x < 8; ++x)
                                    tma_load_3d(dst + x * (C::kTmaBytes / 8), map, 0, 0, z[x], full);
                            } else {
                                tma_load_3d(dst, map, 0, kbase + j * kKeys, kv_row, full);
                            }
                        }
                        __syncwarp();
                        return true;
                    };
                    if (does_k && !load(&map_k, ring_k + s * C::kTmaBytes, &ctl.k_full[s], &ctl.k_empty[s])) break;
                    if (does_v && !load(&map_v, ring_v + s * C::kTmaBytes, &ctl.v_full[s], &ctl.v_empty[s])) {
                        ahead = does_k;
                        break;
                    }
                    if (++s == C::kTma) {
                        s = 0;
                        ++round;
                    }
                }
            } while (again(pass++));
            if (*gave_up) {   // the last load of each stage
                const int nv = round * C::kTma + s, nk = nv + ahead;
                for (int x = 0; x < C::kTma; ++x) {
                    if (does_k && nk > x && x >= skip) mbar_drain(&ctl.k_full[x], ((nk - 1 - x) / C::kTma) & 1);
                    if (does_v && nv > x && x >= skip) mbar_drain(&ctl.v_full[x], ((nv - 1 - x) / C::kTma) & 1);
                }
            }
        } else if (warp < kHelper) {
            // The whole warp waits, one lane issues: descriptors stay warp-uniform (computed by one lane alone, each MMA
            // took over 100 cycles to issue; the tensor pipe takes one in 45 to 65).
            constexpr uint32_t id_s = instr_desc(kRows, kKeys, kFp8, false);
            constexpr uint32_t id_o = instr_desc(kRows, kD, kFp8, true);
            uint64_t *k_in = kFp8 ? ctl.k_ready : ctl.k_full, *k_out = kFp8 ? ctl.kc_empty : ctl.k_empty;
            uint64_t *v_out = kFp8 ? ctl.vc_empty : ctl.v_empty;
            const uint64_t dq = smem_desc(smem_u32(smem + C::kQ)), dk = smem_desc(smem_u32(smem + C::kK)),
                           dv = smem_desc(smem_u32(smem + C::kV));
            const bool leader = elect_one();
            const auto wait = [&](uint64_t *bar, uint32_t parity) {
                return (bool)__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, gave_up));
            };
            const auto wait2 = [&](uint64_t *x, uint32_t px, uint64_t *y, uint32_t py) {
                return (bool)__all_sync(0xFFFFFFFFu, mbar_wait2(x, px, y, py, gave_up));
            };
            int s = 0, round = 0, sp = 0, roundp = 0, made = 0, used = 0, pass = 0;
            bool ok = wait(&ctl.q_full, 0);
            do {
                // Step j: S of tile j, then O of tile j - 1.  What is likely there is waited for before what is not.
                if (ok && cb < ce) ok = wait(&k_in[s], round & 1);
                for (int j = cb; j <= ce && cb < ce && ok; ++j) {
                    const int s1 = s + 1 == C::kMma ? 0 : s + 1, round1 = s + 1 == C::kMma ? round + 1 : round;
                    if (j < ce) {
                        if (made > 0) ok = wait(&ctl.s_free, (made - 1) & 1);
                        if (!ok) break;
                        fence_after();
                        const uint64_t ka = desc_at(dk, s * kTileBytes);
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < kD / 16; ++k)
                                mma_ss(tmem, desc_at(dq, 32 * k), desc_at(ka, 32 * k), id_s, k != 0);
                            commit(&ctl.s_full);
                            commit(&k_out[s]);
                        }
                        __syncwarp();
                        ++made;
                    }
                    if (j > cb && j + 1 < ce) ok = wait2(&ctl.v_ready[sp], roundp & 1, &k_in[s1], round1 & 1);
                    else if (j > cb) ok = wait(&ctl.v_ready[sp], roundp & 1);
                    else if (j + 1 < ce) ok = wait(&k_in[s1], round1 & 1);
                    if (!ok) break;
                    if (j > cb) {
                        ok = wait(&ctl.p_full, used & 1);
                        if (!ok) break;
                        fence_after();
                        const uint64_t va = desc_at(dv, sp * kTileBytes);
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                mma_ts(tmem + 128, tmem + 192 + 8 * k, desc_at(va, 2048 * k), id_o, j - 1 > cb || k != 0);
                            commit(&ctl.o_done);
                            commit(&v_out[sp]);
                        }
                        __syncwarp();
                        ++used;
                        if (j == ce) {   // the last stage's arrivals, so that none is under way when the CTA ends
                            ok = wait(&v_out[sp], roundp & 1);
                        }
                        if (++sp == C::kMma) {
                            sp = 0;
                            ++roundp;
                        }
                    }
                    if (j < ce) {
                        s = s1;
                        round = round1;
                    }
                }
            } while (again(pass++));
            if (*gave_up) {
                if (leader) commit(&ctl.drained);
                __syncwarp();
                mbar_drain(&ctl.drained, 0);
            }
        } else if (kFp8) {
            // Codes to f16, K by the first helper warp, V by the second
            const int kv = warp - kHelper;
            constexpr int kChunks = kKeys * 4 / 32, kBatch = 8;   // a lane's chunks of 16 codes
            uint64_t *full = kv ? ctl.v_full : ctl.k_full, *empty = kv ? ctl.v_empty : ctl.k_empty;
            uint64_t *ready = kv ? ctl.v_ready : ctl.k_ready, *free_ = kv ? ctl.vc_empty : ctl.kc_empty;
            bool ok = true;
            int s = 0, round = 0, sc = 0, roundc = 0, pass = 0;
            do {
                for (int j = cb; j < ce && ok; ++j) {
                    const int key0 = kbase + j * kKeys;
                    ok = roundc > 0 ? mbar_wait2(&full[s], round & 1, &free_[sc], (roundc - 1) & 1, gave_up)
                                    : mbar_wait(&full[s], round & 1, gave_up);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const bool edge = kv && (key0 < ulo || key0 + kKeys > uhi);   // values that no row sees: zeros
                    const bool mixed = kv && pass && (key0 < clo || key0 + kKeys > chi);
                    const uint4 *raw = reinterpret_cast<const uint4 *>(smem + (kv ? C::kRawV : C::kRawK) + s * C::kTmaBytes);
                    uint8_t *dst = smem + (kv ? C::kV : C::kK) + sc * kTileBytes;
                    bool bad = false;
                    const auto convert = [&](const uint4 &now, int e) {
                        const int r = (lane >> 2) + e * 8, c = lane & 3;
                        uint4 a, d;
                        codes4_f16(now.x, a.x, a.y);
                        codes4_f16(now.y, a.z, a.w);
                        codes4_f16(now.z, d.x, d.y);
                        codes4_f16(now.w, d.z, d.w);
                        *reinterpret_cast<uint4 *>(dst + swz(r, 2 * c)) = a;
                        *reinterpret_cast<uint4 *>(dst + swz(r, 2 * c + 1)) = d;
                    };
                    // Eight reads in flight and nothing else in the loop: what bounds a helper is the latency of its own
                    // instructions (8192-token prompt: two reads in flight take 17% longer, four 10%; no conversions 5% less)
                    if (!edge && !mixed) {
#pragma unroll
                        for (int e0 = 0; e0 < kChunks; e0 += kBatch) {
                            uint4 w[kBatch];
#pragma unroll
                            for (int e = 0; e < kBatch; ++e) w[e] = raw[lane + (e0 + e) * 32];
#pragma unroll
                            for (int e = 0; e < kBatch; ++e) convert(w[e], e0 + e);
                        }
                    } else {
#pragma unroll 1
                        for (int e = 0; e < kChunks; ++e) {
                            uint4 now = raw[lane + e * 32];
                            const int key = key0 + (lane >> 2) + e * 8;
                            if (key < ulo || key >= uhi) now = make_uint4(0, 0, 0, 0);
                            if (mixed) {   // NaN codes (0x7F, 0xFF)
                                bad |= zero_nan_codes(now.x);
                                bad |= zero_nan_codes(now.y);
                                bad |= zero_nan_codes(now.z);
                                bad |= zero_nan_codes(now.w);
                            }
                            convert(now, e);
                        }
                    }
                    if (bad) ctl.nonfinite = 1;
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&empty[s]);
                        mbar_arrive(&ready[sc]);
                    }
                    if (++sc == C::kMma) {
                        sc = 0;
                        ++roundc;
                    }
                    if (++s == C::kTma) {
                        s = 0;
                        ++round;
                    }
                }
            } while (again(pass++));
        } else {
            // Values that no row sees become zeros (whatever the cache holds there), in the second pass those that are not
            // finite too
            const int ht = lane;
            constexpr int kHt = 32;
            bool ok = true;
            int s = 0, round = 0, pass = 0;
            do {
                for (int j = cb; j < ce && ok; ++j) {
                    const int key0 = kbase + j * kKeys;
                    const bool edge = key0 < ulo || key0 + kKeys > uhi;
                    const bool mixed = pass && (key0 < clo || key0 + kKeys > chi);
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl.v_full[s], round & 1, gave_up));
                    if (!ok) break;
                    uint8_t *vt = smem + C::kV + s * kTileBytes;
                    bool bad = false;
                    if (edge)
                        for (int x = ht; x < kKeys * 8; x += kHt) {
                            const int key = key0 + (x >> 3);
                            if (key < ulo || key >= uhi) *reinterpret_cast<uint4 *>(vt + x * 16) = make_uint4(0, 0, 0, 0);
                        }
                    if (mixed)
#pragma unroll 1
                        for (int x = ht; x < kKeys * 8; x += kHt) {
                            uint4 w = *reinterpret_cast<const uint4 *>(vt + x * 16);
                            if (nonfinite16(w.x, 0x7F80u) || nonfinite16(w.y, 0x7F80u) || nonfinite16(w.z, 0x7F80u) ||
                                nonfinite16(w.w, 0x7F80u)) {
                                uint32_t *ws = &w.x;
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    if ((ws[y] & 0x7F80u) == 0x7F80u) ws[y] &= 0xFFFF0000u;
                                    if ((ws[y] & 0x7F800000u) == 0x7F800000u) ws[y] &= 0x0000FFFFu;
                                }
                                *reinterpret_cast<uint4 *>(vt + x * 16) = w;
                                bad = true;
                            }
                        }
                    if (bad) ctl.nonfinite = 1;
                    if (edge || mixed) fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.v_ready[s]);
                    if (++s == C::kTma) {
                        s = 0;
                        ++round;
                    }
                }
            } while (again(pass++));
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16), to = ts + 128, tpw = ts + 192;
        // The query row goes to the swizzled tile
        float qfac = 1.0f;
        {
            uint8_t *qs = smem + C::kQ;
            if (kFp8) {
                float big = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float x[8];
                    unpack8(qw[c], x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(x[j]));
                }
                const float up = pow2_normaliser(big);
                qfac = 1.0f / up;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float x[8];
                    unpack8(qw[c], x);
                    qw[c] = make_uint4(pack_f16(x[0] * up, x[1] * up), pack_f16(x[2] * up, x[3] * up),
                                      pack_f16(x[4] * up, x[5] * up), pack_f16(x[6] * up, x[7] * up));
                }
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(qs + swz(row, c)) = qw[c];
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.q_full);
        }
        const float scale = p.sscale * qfac;
        const ScoreCap cap(p.cap_c1, p.cap_c2 * qfac, scale);
        const bool capped = kMode == kCapped, biased = kMode == kBiased || (kMode == kCapped && p.slopes != nullptr);
        const float slope = biased && valid ? __ldg(p.slopes + orow % p.Hq) * 1.4426950408889634f : 0.f;
        const float mul = capped || biased ? 1.0f : scale;
        // A row that sees no key (or is none) goes along with the others of its warp; its state is put right at the end
        const bool sees = hi > lo, any_sees = __any_sync(0xFFFFFFFFu, sees);
        int done = 0, pass = 0;   // tiles so far
        do {
            float m = -INFINITY, mref = 0.f, l = 0.f;
            bool ok = !misplaced, s_there = false;
            for (int j = cb; j < ce; ++j) {
                const int key0 = kbase + j * kKeys;
                const bool inside = __all_sync(0xFFFFFFFFu, !sees || (key0 >= lo && key0 + kKeys <= hi));
                // where every visible key lies before the query the bias is linear in the key's number
                const bool linear = kMode != kBiased || __all_sync(0xFFFFFFFFu, !sees || min(hi, key0 + kKeys) <= pos + 1);
                if (!s_there) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl.s_full, done & 1, gave_up));
                if (!ok) break;
                fence_after();
                const int bits = ctl.bits[(j - cb) % kBitsRing];
                float corr = 1.0f;
                const auto raise = [&](float mx) {   // also for the first visible key (m = -inf)
                    if (mx > m + kSlack) {
                        corr = fast_exp2(m - mx);
                        m = mx;
                        mref = mx - kLift<kFp8>;
                        l *= corr;
                    }
                };
                // P and O are the previous tile's until its product is done
                const auto rescale = [&](bool o_there, bool moved) -> bool {
                    if (j == cb) return true;
                    if (!o_there && !__all_sync(0xFFFFFFFFu, mbar_wait(&ctl.o_done, (done - 1) & 1, gave_up))) return false;
                    fence_after();
                    if (moved) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float o[32];
                            ld32(to + 32 * h, o);
                            wait_ld();
                            pin32(o);
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] *= corr;
                            st32(to + 32 * h, o);
                        }
                    }
                    return true;
                };
                if (!any_sees) {
                    // A warp without such rows passes on: what its rows of P and O hold is not used.  It keeps step by the
                    // previous tile's product, or its arrival at p_full would be counted for that tile.
                    if (lane == 0) mbar_arrive(&ctl.s_free);
                    ok = rescale(false, false);
                    if (!ok) break;
                    s_there = false;
                } else if (kMode == kPlain || (kMode == kBiased && linear) || (kMode == kCapped && !biased)) {
                    // The row in registers at once, S given back before the exponentials.  By the rolled way below, documents
                    // without a bias took a fifth longer, and capped rows 7%.
                    float s[kKeys];
                    float top[8];
                    const float base = slope * (float)(key0 - pos);
                    const auto bias = [&] {
                        if constexpr (kMode == kBiased) {
                            const float2 slope2 = make_float2(slope, slope), base2 = make_float2(base, base);
#pragma unroll
                            for (int c = 0; c < kKeys; c += 2) {
                                const float2 off = __ffma2_rn(make_float2((float)c, (float)(c + 1)), slope2, base2);
                                const float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), make_float2(scale, scale), off);
                                s[c] = x.x;
                                s[c + 1] = x.y;
                            }
                        }
                    };
                    const auto top_first = [&] {
#pragma unroll
                        for (int e = 0; e < 8; ++e) top[e] = fmaxf(s[e], s[56 + e]);
#pragma unroll
                        for (int c = 8; c < 56; c += 16)
#pragma unroll
                            for (int e = 0; e < 8; ++e) top[e] = max3(top[e], s[c + 2 * e], s[c + 2 * e + 1]);
                    };
                    const auto top_second = [&] {
#pragma unroll
                        for (int c = 64; c < kKeys; c += 16)
#pragma unroll
                            for (int e = 0; e < 8; ++e) top[e] = max3(top[e], s[c + 2 * e], s[c + 2 * e + 1]);
                    };
                    const auto give_back = [&] {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl.s_free);
                    };
                    ld32(ts, s);
                    ld32(ts + 32, s + 32);
                    wait_ld();
                    pin32(s);
                    pin32(s + 32);
                    ld32(ts + 64, s + 64);
                    ld32(ts + 96, s + 96);
                    const bool whole = inside && bits == 0xFF;
                    // Long prompts gain 5% by an unmasked way of its own; with a bias the code would grow too long for the
                    // instruction cache (documents with a bias took 5% longer)
                    if (kMode == kPlain && whole) {
                        top_first();
                        wait_ld();
                        pin32(s + 64);
                        pin32(s + 96);
                        give_back();
                        top_second();
                    } else {
                        wait_ld();
                        pin32(s + 64);
                        pin32(s + 96);
                        give_back();
                        bias();
                        if constexpr (kMode == kCapped) cap(s);
                        const auto below = [](int x) { return __funnelshift_lc(0xFFFFFFFFu, 0u, min(max(x, 0), 32)); };
                        if (!whole)   // hidden keys, and those of blocks that are not there
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const unsigned there =
                                    (bits >> (2 * k) & 1 ? 0xFFFFu : 0u) | (bits >> (2 * k) & 2 ? 0xFFFF0000u : 0u);
                                const unsigned seen = below(hi - key0 - 32 * k) & ~below(lo - key0 - 32 * k) & there;
#pragma unroll
                                for (int c = 0; c < 32; ++c)
                                    if (!(seen & (1u << c))) s[32 * k + c] = -INFINITY;
                            }
                        top_first();
                        top_second();
                    }
                    raise(fmaxf(max3(max3(top[0], top[1], top[2]), top[3], top[4]), max3(top[5], top[6], top[7])) * mul);
                    // Asked before the exponentials, needed after them
                    const bool o_there = j > cb && __all_sync(0xFFFFFFFFu, mbar_test(&ctl.o_done, (done - 1) & 1));
                    const bool moved = __any_sync(0xFFFFFFFFu, corr != 1.0f);
                    uint32_t pk[kKeys / 2];
                    l += weights<kKeys, kFp8>(s, mul, mref, pk);
                    ok = rescale(o_there, moved);
                    if (!ok) break;
                    s_there = __all_sync(0xFFFFFFFFu, mbar_test(&ctl.s_full, (done + 1) & 1));
                    st32(tpw, pk);
                    st32(tpw + 32, pk + 32);
                } else {
                    // A quarter at a time in rolled loops: capped, biased and masked scores go back to tensor memory and
                    // are read again for the exponentials.  With straight-line code for every combination a quarter of the
                    // requests to the instruction cache missed, and documents with a bias took 18% longer.
                    unsigned hidden = 0;   // quarters that no row of the warp sees
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const int first = key0 + 32 * k, blocks = (bits >> (2 * k)) & 3;
                        if (__all_sync(0xFFFFFFFFu, hi <= first || lo >= first + 32) || blocks == 0) {
                            hidden |= 1u << k;
                            continue;
                        }
                        float s[32];
                        ld32(ts + 32 * k, s);
                        wait_ld();
                        pin32(s);
                        if (capped) {
                            cap(s);
                        } else if (biased) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) s[c] *= scale;
                        }
                        if (biased) {
                            const float d0 = (float)(pos - first);
#pragma unroll
                            for (int c = 0; c < 32; ++c) s[c] = fmaf(-slope, fabsf(d0 - (float)c), s[c]);
                        }
                        if (blocks != 3 || !__all_sync(0xFFFFFFFFu, !sees || (lo <= first && hi >= first + 32))) {
                            const int a = max(lo - first, blocks & 1 ? 0 : kBlockKeys),
                                      e = min(hi - first, blocks & 2 ? 32 : kBlockKeys);   // a block that is not there
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (c < a || c >= e) s[c] = -INFINITY;
                        }
                        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int c = 4; c < 28; c += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e) top[e] = max3(top[e], s[c + 2 * e], s[c + 2 * e + 1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], s[28 + e]);
                        mx = max3(mx, fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                        st32(ts + 32 * k, s);
                    }
                    wait_st();
                    raise(mx * mul);
                    ok = rescale(false, __any_sync(0xFFFFFFFFu, corr != 1.0f));
                    if (!ok) break;
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pk[16];
                        if ((hidden >> k) & 1) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) pk[c] = 0;
                        } else {
                            float s[32];
                            ld32(ts + 32 * k, s);
                            wait_ld();
                            pin32(s);
                            l += weights<32, kFp8>(s, mul, mref, pk);
                        }
                        st16(tpw + 16 * k, pk);
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.s_free);
                    s_there = false;
                }
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full);
                ++done;
            }

            float o[kD];
            if (ok && ce > cb) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl.o_done, (done - 1) & 1, gave_up));
                fence_after();
                ld32(to, o);
                ld32(to + 32, o + 32);
                wait_ld();
                pin32(o);
                pin32(o + 32);
            } else {
#pragma unroll
                for (int c = 0; c < kD; ++c) o[c] = 0.f;
            }
            if (!sees) {
                m = -INFINITY;
                l = 0.f;
#pragma unroll
                for (int c = 0; c < kD; ++c) o[c] = 0.f;
            }
            if (ok && valid && pass == 0) {
                float2 z[2] = {};
                const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < kD; c += 2) z[c / 2 & 1] = __ffma2_rn(make_float2(o[c], o[c + 1]), zero, z[c / 2 & 1]);
                if ((z[0].x + z[0].y) + (z[1].x + z[1].y) != 0.f) *(volatile int *)&ctl.redo = 1;   // NaN: some sum is not finite
            }
            if (!ok) {   // what is joined must not be an earlier call's: NaN
                m = 0.f;
                l = __int_as_float(0x7FC00000);
            }
            if ((ok || p.part_ml) && valid) {
                if (ok && pass && *(volatile int *)&ctl.nonfinite) {
                    // the values left out that this row sees: a positive weight times such a value is such a value
                    for (int j = cb; j < ce; ++j) {
                        const int key0 = kbase + j * kKeys;
                        for (int key = max(lo, key0); key < min(hi, key0 + kKeys); ++key) {
                            size_t at;
                            if (kPaged) {
                                const int blk = __ldg(p.table + (size_t)b * p.max_blocks + key / kBlockKeys);
                                if ((unsigned)blk >= (unsigned)p.num_blocks) continue;
                                at = (((size_t)blk * p.Hkv + hk) * kBlockKeys + key % kBlockKeys) * kD;
                            } else {
                                at = (((size_t)b * p.Hkv + hk) * (size_t)p.cap + key) * kD;
                            }
                            if constexpr (kFp8) {
                                const uint8_t *v = static_cast<const uint8_t *>(p.v) + at;
#pragma unroll
                                for (int c = 0; c < kD; ++c)
                                    if ((v[c] & 0x7F) == 0x7F) o[c] = __int_as_float(0x7FC00000);
                            } else {
                                const uint16_t *v = static_cast<const uint16_t *>(p.v) + at;
#pragma unroll
                                for (int c = 0; c < kD; ++c)
                                    if ((v[c] & 0x7F80) == 0x7F80) o[c] += __uint_as_float((uint32_t)v[c] << 16);
                            }
                        }
                    }
                }
                if (p.part_ml) {
                    const size_t at = (size_t)split * ((size_t)p.T * p.Hq) + orow;
                    p.part_ml[at] = make_float2(state_max(m - kLift<kFp8>, l), l);
                    float *dst = p.part_acc + at * kD;
#pragma unroll
                    for (int c = 0; c < kD; c += 8) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[c + e] * p.out_scale);
                        st_32(dst + c, w);
                    }
                } else {
                    const float inv = l == 0.f ? 0.f : p.out_scale / l;
                    if (l == 0.f)
#pragma unroll
                        for (int c = 0; c < kD; ++c) o[c] = 0.f;
#pragma unroll
                    for (int c = 0; c < kD; c += 2) {
                        const float2 x = __fmul2_rn(make_float2(o[c], o[c + 1]), make_float2(inv, inv));
                        o[c] = x.x;
                        o[c + 1] = x.y;
                    }
                    if (p.out_f32) {
                        float *dst = static_cast<float *>(p.out) + (size_t)orow * kD;
#pragma unroll
                        for (int c = 0; c < kD; c += 8) st_32(dst + c, reinterpret_cast<const uint32_t *>(o + c));
                    } else {
                        uint16_t *dst = static_cast<uint16_t *>(p.out) + (size_t)orow * kD;
#pragma unroll
                        for (int c = 0; c < kD; c += 16) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = pack_bf16(o[c + 2 * e], o[c + 2 * e + 1]);
                            st_32(dst + c, w);
                        }
                    }
                }
            }
            __syncwarp();
        } while (again(pass++));
    }
    if (*gave_up) {   // the same in every thread: the last wait lies before the last barrier
        if (threadIdx.x == 0) flag_error(p.err, DR_ERRF_TIMEOUT);
        __syncthreads();   // the drained copies and products before the memory is given up
    }
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

// out[t][h] from the states of the splits, in split order.  A warp takes two heads of a token, 16 lanes each, four
// dimensions per lane.
__global__ void __launch_bounds__(256) attn_join_kernel(const PromptParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, pairs = (p.Hq + 1) / 2;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= (long long)p.T * pairs) return;
    const int t = (int)(w / pairs), h = (int)(w - (long long)t * pairs) * 2 + (lane >> 4);
    int s0, s1;
    if (find_row(p.row_start, p.B, p.T, t, lane, s0, s1, nullptr, 0, 1) < 0 || s1 - s0 <= p.few_max || h >= p.Hq) return;
    const size_t rows = (size_t)p.T * p.Hq, row = (size_t)t * p.Hq + h;
    float M = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < p.nparts; ++x) {
        const float2 ml = p.part_ml[x * rows + row];
        const float4 a = reinterpret_cast<const float4 *>(p.part_acc + (x * rows + row) * kD)[lane & 15];
        const float m2 = fmaxf(M, ml.x);
        if (m2 == -INFINITY) continue;   // no key so far
        const float w0 = exp2f(M - m2), w1 = exp2f(ml.x - m2);
        M = m2;
        l = l * w0 + ml.y * w1;
        o = make_float4(o.x * w0 + a.x * w1, o.y * w0 + a.y * w1, o.z * w0 + a.z * w1, o.w * w0 + a.w * w1);
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    o = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (p.out_f32)
        reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * kD)[lane & 15] = o;
    else
        reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row * kD)[lane & 15] =
            make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *ptr = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// Cache as [rows][keys][64] (paged: rows = blocks x heads of 16 keys), box [1][box keys][64].  bf16 tiles land with the
// 128-byte swizzle that the MMA reads; e4m3 codes land plainly (the helper warps swizzle what they convert).
bool encode_cache(CUtensorMap *map, const void *ptr, long long rows, int keys, int box_keys, bool fp8) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t e = fp8 ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)keys, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {kD * e, kD * e * (cuuint64_t)keys};
    const cuuint32_t box[3] = {(cuuint32_t)kD, (cuuint32_t)box_keys, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFp8, bool kPaged, int kMode>
cudaError_t launch_variant(const PromptParams &p, int splits, cudaStream_t stream) {
    using C = Config<kFp8>;
    auto kern = attn_tiles_kernel<kFp8, kPaged, kMode>;
    constexpr size_t smem = C::kEnd + sizeof(Control);
    static_assert(smem <= 113 * 1024, "shared memory of two CTAs per SM");
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = once_per_device(ready, [&]() -> cudaError_t {
        cudaFuncAttributes fa;
        const cudaError_t e1 = cudaFuncGetAttributes(&fa, kern);
        if (e1 != cudaSuccess) return e1;
        // the register split draws on what the launch gives: fewer would leave a warpgroup waiting
        if (fa.numRegs != kLaunchRegs)
            return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap mk, mv;
    const long long rows = (long long)(kPaged ? p.num_blocks : (p.row_start ? p.B : 1)) * p.Hkv;
    const int keys = kPaged ? kBlockKeys : p.cap, box = kPaged ? kBlockKeys : kKeys;
    if (rows >= 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    if (!encode_cache(&mk, p.k, rows, keys, box, kFp8) || !encode_cache(&mv, p.v, rows, keys, box, kFp8))
        return cudaErrorInvalidValue;
    // every row may end in a part of a tile; no row has more tiles than tokens
    const long long per_row = p.row_start ? p.B : 1;
    long long tiles = ((long long)p.T * p.g + per_row * (kRows - 1)) / kRows;
    const long long by_tokens = ((long long)p.T * ((p.g + kRows - 1) / kRows));
    if (tiles > by_tokens) tiles = by_tokens;
    TileParams tp;
    tp.p = p;
    tp.splits.set((uint32_t)splits);
    tp.heads.set((uint32_t)p.Hkv);
    tp.group.set((uint32_t)p.g);
    return launch_kernel(kern, dim3((unsigned)(tiles * splits * p.Hkv)), dim3(C::kThreads), smem, stream, 1u, mk,
                         mv, tp);
}

}  // namespace

cudaError_t launch_attn_tiles(const PromptParams &p, bool paged, bool fp8, int splits, cudaStream_t stream) {
    const int mode = p.cap_c1 != 0.f ? kCapped : p.slopes ? kBiased : kPlain;
#define DR_PICK2(F, P)                                                                  \
    (mode == kPlain    ? launch_variant<F, P, kPlain>(p, splits, stream)                \
     : mode == kBiased ? launch_variant<F, P, kBiased>(p, splits, stream)               \
                       : launch_variant<F, P, kCapped>(p, splits, stream))
    if (fp8) return paged ? DR_PICK2(true, true) : DR_PICK2(true, false);
    return paged ? DR_PICK2(false, true) : DR_PICK2(false, false);
#undef DR_PICK2
}

// CTAs that share a tile's keys.  Fewer leave SMs idle, or waiting for the one with the longest run of keys; more cost
// each its start and end, and the states that they leave and that are read again.  The plan takes the s with the least
//   run x step + 5 us, once per wave of CTAs and half a wave more where there are several (they end unevenly),
//   + s x states, written and read at 4 TB/s, + 2.5 us for the launch that joins them (prompts, s > 1),
// run = key tiles per CTA, step = 0.83 us for a CTA that has an SM to itself, 1.25 for two on an SM (e4m3 0.88, 1.35).
// The rows' own keys, streamed beside a shared prefix (own_us of them), hide about a quarter of their time of it; the
// states are read by the same CTAs and are dearer there, up to three times.  Measured, bf16: 300, 500 and 700 tokens on
// 9000, 14000 and 18000 keys, 16 heads: 162 us unsplit, 136 by 2, 134 by 3 or 4, 151 by 8 (the plan: 135); 200 tokens of 4
// heads in groups of 4 on 30000 keys: 197 us, 49 by 5, 57 by 6, 43 by 10 (the plan's), 59 by 12; a prefix of 500 keys for 8
// rows of 16 heads: 9.8 us, 7.8 by 4 (the plan's); of 4096 keys for 128 rows with 64..2048 own: 107 us, 98 by 2 (the plan's),
// 97 by 3, 103 by 10, 113 by 32.  The plan takes ceil(T g / 128) tiles; rows that end within one make more, and many short
// rows over long pasts are split too far: 32 rows of 4 tokens, 4 heads, 16384 keys 150 us, 88 by 2; 64 rows of 20 tokens, 2
// heads, 8192 keys 77 us, 51 by 2.
int plan_tile_splits(int T, int g, int Hkv, int max_len, bool fp8, int sms, bool joined, double own_us) {
    const double units = (double)(((long long)T * g + kRows - 1) / kRows) * Hkv;
    const int tiles = max_len / kKeys + 1;
    const double state_us = (double)T * Hkv * g * (kD + 2) * 4 * 2 / 4e6 * (own_us < 40 ? 1 + own_us / 20 : 3);
    const double alone = fp8 ? 0.88 : 0.83, two = fp8 ? 1.35 : 1.25;
    int best = 1;
    double best_us = 0;
    for (int s = 1; s <= 64 && s <= tiles; ++s) {
        const double run = (tiles + s - 1) / s, waves = units * s / (2 * sms);
        const double cta = run * (units * s <= sms ? alone : two) + 5;
        const double us = fmax((waves > 1 ? waves + 0.5 : 1) * cta, own_us / 4) +
                          (s > 1 ? s * state_us + (joined ? 2.5 : 0) : 0);
        if (s == 1 || us < best_us) {
            best = s;
            best_us = us;
        }
    }
    return best;
}

cudaError_t launch_attn_join(const PromptParams &p, cudaStream_t stream) {
    const long long warps = (long long)p.T * ((p.Hq + 1) / 2);
    return launch_kernel(attn_join_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, stream, 1u, p);
}

}  // namespace dr
