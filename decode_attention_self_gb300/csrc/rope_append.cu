// Rotate q and k by position and append k, v of ragged new tokens to the cache, in one pass.
//
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin),  cos/sin of pos * base^(-2i/R), i = 0 .. R/2 - 1,
//   pairs (i, i + R/2) or, interleaved, (2i, 2i + 1); dims from R on pass through.  The products and the sum are
//   rounded apart in fp32 (no fused multiply-add), then once to bf16, or once to the e4m3 code of x / scale.
//
// Bound by memory: a token reads (Hq + 2 Hkv) * 128 bytes and its table row and writes as much (e4m3: half for k, v).
// One warp serves one token (several warps when there are few tokens): lane (s, c) = (lane / 4, lane % 4) holds a
// pair of 16-byte chunks of head s, s + 8, ... of q, k and v in turn, chosen so that both elements of every rotated
// pair are in the lane, and reads its 16 table values once for all heads.  The first heads are loaded before the token's
// row and position are known, and 24 warps fit an SM (80 registers) in CTAs of four, which leave a shorter tail than CTAs
// of eight: 65536 tokens, 16 + 2 x 16 heads, 125 us, 6.59 TB/s (CTAs of eight 1% more; the loads behind the row search and 16
// warps per SM a fifth more; a run of tokens per warp, whose loads wait for the stores before, 30%).  22000 ragged tokens
// into an e4m3 cache take 26 us, where scales that are powers of two save the division (10% more with it): each warp's
// chain row - position - table is as long as its transfers.
#include "dr_device.cuh"
#include "dr_prompt.h"
#include "dr_rows.cuh"

namespace dr {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 3;   // heads per lane in flight

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)f32_to_bf16_rn(f[2 * i]) | ((uint32_t)f32_to_bf16_rn(f[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of f / scale, inv as in RopeAppendParams
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float scale, float inv) {
    float2 x[4];
    if (inv != 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale));
    }
    uint32_t pk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pk[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(x[i], __NV_SATFINITE, __NV_E4M3);
    return make_uint2(pk[0] | (pk[1] << 16), pk[2] | (pk[3] << 16));
}

template <bool kPaged, bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 6) rope_append_kernel(const RopeAppendParams p, int warps_per_token) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const long long tl = gw / warps_per_token;
    if (tl >= p.T) return;
    const int t = (int)tl, part = (int)(gw - tl * warps_per_token);
    const int c = lane & 3, hs = lane >> 2;
    const int np = p.rot >> 4;   // lanes whose chunks are rotated
    const bool turned = c < np;
    const int u0 = (!kInterleaved && turned) ? c : 2 * c;
    const int u1 = (!kInterleaved && turned) ? c + np : 2 * c + 1;
    const int nq = p.q ? p.Hq : 0, nh = nq + 2 * p.Hkv, hstep = 8 * warps_per_token;
    const uint16_t *qt = p.q + (size_t)t * p.q_stride, *kt = p.k + (size_t)t * p.k_stride,
                   *vt = p.v + (size_t)t * p.v_stride;
    uint4 w0[kBatch], w1[kBatch];
    const auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = h0 + i * hstep;
            if (h < nh) {
                const uint16_t *src = h < nq ? qt + (size_t)h * kHeadDim
                                     : h < nq + p.Hkv ? kt + (size_t)(h - nq) * kHeadDim
                                                      : vt + (size_t)(h - nq - p.Hkv) * kHeadDim;
                // plain loads: q_out may be q itself (each lane reads its chunks before it writes them)
                w0[i] = *reinterpret_cast<const uint4 *>(src + 8 * u0);
                w1[i] = *reinterpret_cast<const uint4 *>(src + 8 * u1);
            }
        }
    };
    load(part * 8 + hs);   // in flight while the row and the position are found
    int s0, s1;
    const int b = find_row(p.row_start, p.B, p.T, t, lane, s0, s1, p.err, gw, (long long)p.T * warps_per_token);
    if (b < 0) return;   // behind the last row: left as it is

    const long long slot = (long long)__ldg(p.start_pos + b) + (t - s0);
    const long long pos = slot + (p.pos_offset ? __ldg(p.pos_offset + b) : 0);
    if (np > 0 && (pos < 0 || pos >= p.rope_len)) {
        if (part == 0 && lane == 0) flag_error(p.err, DR_ERRF_POS);
        return;
    }
    bool store_kv = slot >= 0 && slot < p.cap;
    size_t dst = 0;        // element offset of (row, head 0, slot)
    size_t dst_head = 0;   // elements from one head to the next
    if (kPaged) {
        const int blk = store_kv ? __ldg(p.block_table + (size_t)b * p.max_blocks + (int)slot / kBlockKeys) : -1;
        store_kv = (unsigned)blk < (unsigned)p.num_blocks;
        dst = ((size_t)(store_kv ? blk : 0) * p.Hkv * kBlockKeys + (size_t)(slot % kBlockKeys)) * kHeadDim;
        dst_head = (size_t)kBlockKeys * kHeadDim;
    } else {
        dst = ((size_t)b * p.Hkv * p.cap + (size_t)(store_kv ? slot : 0)) * kHeadDim;
        dst_head = (size_t)p.cap * kHeadDim;
    }
    if (!store_kv && part == 0 && lane == 0) flag_error(p.err, DR_ERRF_POS);

    float cs[8], sn[8];
    if (turned) {
        const float4 *row = reinterpret_cast<const float4 *>(p.rope + (size_t)pos * p.rot) + 2 * c;
        const float4 a0 = __ldg(row), a1 = __ldg(row + 1);
        const float4 b0 = __ldg(row + p.rot / 8), b1 = __ldg(row + p.rot / 8 + 1);
        cs[0] = a0.x; cs[1] = a0.y; cs[2] = a0.z; cs[3] = a0.w; cs[4] = a1.x; cs[5] = a1.y; cs[6] = a1.z; cs[7] = a1.w;
        sn[0] = b0.x; sn[1] = b0.y; sn[2] = b0.z; sn[3] = b0.w; sn[4] = b1.x; sn[5] = b1.y; sn[6] = b1.z; sn[7] = b1.w;
    }
    uint16_t *qo = p.q_out + (size_t)t * p.q_out_stride;
    for (int h0 = part * 8 + hs; h0 < nh; h0 += kBatch * hstep) {
        if (h0 >= kBatch * hstep) load(h0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = h0 + i * hstep;
            if (h >= nh) break;
            const bool is_v = h >= nq + p.Hkv, is_q = h < nq;
            float x[8], y[8];
            unpack8(w0[i], x);
            unpack8(w1[i], y);
            if (turned && !is_v) {
                if (kInterleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a = x[2 * j], d = x[2 * j + 1], e = y[2 * j], f = y[2 * j + 1];
                        x[2 * j] = __fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(d, sn[j]));
                        x[2 * j + 1] = __fadd_rn(__fmul_rn(d, cs[j]), __fmul_rn(a, sn[j]));
                        y[2 * j] = __fsub_rn(__fmul_rn(e, cs[4 + j]), __fmul_rn(f, sn[4 + j]));
                        y[2 * j + 1] = __fadd_rn(__fmul_rn(f, cs[4 + j]), __fmul_rn(e, sn[4 + j]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float a = x[j], d = y[j];
                        x[j] = __fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(d, sn[j]));
                        y[j] = __fadd_rn(__fmul_rn(d, cs[j]), __fmul_rn(a, sn[j]));
                    }
                }
            }
            if (is_q) {
                uint16_t *o = qo + (size_t)h * kHeadDim;
                *reinterpret_cast<uint4 *>(o + 8 * u0) = pack8(x);
                *reinterpret_cast<uint4 *>(o + 8 * u1) = pack8(y);
            } else if (store_kv) {
                const size_t off = dst + (size_t)(h - nq - (is_v ? p.Hkv : 0)) * dst_head;
                if (kFp8) {
                    uint8_t *o = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + off;
                    const float sc = is_v ? p.v_scale : p.k_scale, inv = is_v ? p.v_inv : p.k_inv;
                    *reinterpret_cast<uint2 *>(o + 8 * u0) = codes8(x, sc, inv);
                    *reinterpret_cast<uint2 *>(o + 8 * u1) = codes8(y, sc, inv);
                } else {
                    uint16_t *o = static_cast<uint16_t *>(is_v ? p.v_cache : p.k_cache) + off;
                    *reinterpret_cast<uint4 *>(o + 8 * u0) = pack8(x);
                    *reinterpret_cast<uint4 *>(o + 8 * u1) = pack8(y);
                }
            }
        }
    }
}

// table[p][i] = cos(p * base^(-2i/rot)), table[p][rot/2 + i] = sin(...): angles and functions in 64 bits (a position
// of 2^20 times a frequency near 1 leaves 4 bits of a 32-bit angle's fraction), rounded once to fp32.
__global__ void __launch_bounds__(256) rope_table_kernel(float *table, int max_pos, int rot, double base) {
    pdl_wait();
    pdl_trigger();
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const int half = rot / 2;
    if (idx >= (long long)max_pos * half) return;
    const int pos = (int)(idx / half), i = (int)(idx - (long long)pos * half);
    double s, c;
    sincos((double)pos * pow(base, -2.0 * i / rot), &s, &c);
    table[(size_t)pos * rot + i] = (float)c;
    table[(size_t)pos * rot + half + i] = (float)s;
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams &p, bool paged, cudaStream_t stream) {
    // One warp per token, more while the tokens alone give fewer than 4 warps per SM.
    const int heads = (p.q ? p.Hq : 0) + 2 * p.Hkv;
    int wpt = 1;
    while (wpt < 8 && (long long)p.T * wpt < 4LL * current_device_sms() && 8 * wpt < heads) wpt *= 2;
    const long long warps = (long long)p.T * wpt;
    const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
    void (*kern)(RopeAppendParams, int);
#define DR_PICK(P, F) (p.interleaved ? rope_append_kernel<P, F, true> : rope_append_kernel<P, F, false>)
    if (paged) kern = p.kv_fp8 ? DR_PICK(true, true) : DR_PICK(true, false);
    else kern = p.kv_fp8 ? DR_PICK(false, true) : DR_PICK(false, false);
#undef DR_PICK
    return launch_kernel(kern, dim3(grid), dim3(kThreads), 0, stream, 1u, p, wpt);
}

cudaError_t launch_rope_table(float *table, int max_pos, int rot, double base, cudaStream_t stream) {
    const long long n = (long long)max_pos * (rot / 2);
    return launch_kernel(rope_table_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, 1u, table, max_pos,
                         rot, base);
}

}  // namespace dr
