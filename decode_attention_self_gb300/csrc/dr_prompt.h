// Internal declarations of the prompt-side operators (rotated append, prompt attention, shared-prefix attention).
// Launch helpers take validated arguments; dr_prompt_api.cu owns all argument checking.
#pragma once

#include <atomic>

#include "dr_internal.h"

namespace dr {

// Runs a kernel's one-time setup once per device (done: one bit per device; a failure is tried again).
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t> &done, F &&setup) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = setup();
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

struct RopeAppendParams {
    void *k_cache, *v_cache;            // bf16 or e4m3 cache
    const int32_t *block_table;         // paged only
    int32_t cap, max_blocks, num_blocks, kv_fp8;
    float k_scale, v_scale;
    float k_inv, v_inv;   // 1 / scale where the scale is a power of two, else 0
    const uint16_t *q, *k, *v;          // [T][heads][64] bf16, tokens *_stride elements apart; q may be null
    uint16_t *q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const int32_t *row_start;           // [B+1]
    const int32_t *start_pos;           // [B]
    const int32_t *pos_offset;          // [B] or null
    const float *rope;                  // [rope_len][rot] cos then sin, or null
    int32_t rope_len, rot, interleaved;
    int32_t T, B, Hq, Hkv;
    int32_t *err;
};

cudaError_t launch_rope_append(const RopeAppendParams &p, bool paged, cudaStream_t stream);
cudaError_t launch_rope_table(float *table, int max_pos, int rot, double base, cudaStream_t stream);

// One attention call over a cache of Hkv heads by queries of Hq = g * Hkv heads.
struct PromptParams {
    const uint16_t *q;                  // [T][Hq][64] bf16, tokens q_stride elements apart
    int64_t q_stride;
    const void *k, *v;                  // cache, as dr_kv_cache
    const int32_t *table;
    int32_t cap, max_blocks, num_blocks;
    float sscale;                       // scores in log2 units: raw * sscale (scale * log2 e * k_scale)
    float out_scale;                    // v_scale of an e4m3 cache, else 1
    float cap_c1, cap_c2;               // score cap in log2 units: c1 tanh(raw c2); c1 = 0: no cap
    const float *slopes;                // [Hq] or null: s -= slope * |pos - key|
    const int32_t *row_start;           // [B+1]; null: one query per row, token b = row b
    const int32_t *kv_len;              // [B]; null: no keys (a row's state is its prefix part alone)
    const int32_t *prefix_len;          // [B] or null: keys every query of a row sees, causal or not
    const int32_t *first_key;           // [T] or null: keys before it are hidden from query t
    int32_t causal;
    int32_t T, B, Hq, Hkv, g;
    void *out;                          // [T][Hq][64]
    int32_t out_f32;
    int32_t *err;
    // the most tokens a row may have to be taken by the token kernel (more: the tile kernel's)
    int32_t few_max;
    // token kernel: launched right behind the tile kernel of the same call
    int32_t after_tiles;
    // tile kernel, test hook: CTA stall - 1 never loads its first keys (0: none)
    int32_t stall;
    // tile kernel: queries of a shared prefix stand own_len[t] keys past its end (null: at their row's last keys)
    const int32_t *own_len;
    int32_t own_cap;                    // own_len is clamped to it
    // softmax states of key ranges attended before: [nparts][rows = T*Hq] (m, l) and [nparts][rows][64]; null: none
    float2 *part_ml;
    float *part_acc;
    int32_t nparts;
};

// Query rows one token at a time (memory bound: single tokens of a batch).
cudaError_t launch_attn_tokens(const PromptParams &p, bool paged, bool fp8, int splits, cudaStream_t stream);
// Query rows 128 at a time on the tensor cores.  splits CTAs share a tile's keys; with part_ml set every CTA leaves its
// softmax state there (nparts = splits), else splits is 1 and the outputs are written.
cudaError_t launch_attn_tiles(const PromptParams &p, bool paged, bool fp8, int splits, cudaStream_t stream);
// Joins the states that the tile kernel's splits left (rows of more than few_max tokens).
cudaError_t launch_attn_join(const PromptParams &p, cudaStream_t stream);
int plan_tile_splits(int T, int g, int Hkv, int max_len, bool fp8, int sms, bool joined, double own_us);
int plan_token_splits(long long items, int Hkv, int g, int max_len, bool fp8, int sms);

}  // namespace dr
