// extern "C" boundary of the prompt-side operators: argument checks, plans and launches.  As in dr_api.cu, nothing
// here allocates device memory or synchronises with the host.
#include <math.h>

#include "dr_prompt.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// the attention kernels read keys and write outputs and states 32 bytes at a time
bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Keys per row: the kernels look a few tiles past a row's end in 32-bit key numbers.
constexpr int kMaxCap = 0x7FFFF000;

// Validates a cache description; on success stores the keys a row can hold in *cap.
dr_status check_cache(const dr_kv_cache *c, int *cap) {
    if (!c || !c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return DR_ERR_INVALID_ARG;
    if (c->kv_dtype != DR_KV_BF16 && c->kv_dtype != DR_KV_FP8_E4M3) return DR_ERR_INVALID_ARG;
    if (c->kv_dtype == DR_KV_FP8_E4M3 &&
        (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || isinf(c->k_scale) || isinf(c->v_scale)))
        return DR_ERR_INVALID_ARG;
    if (c->layout == DR_KV_CONTIGUOUS) {
        if (c->max_len < 1 || c->max_len > kMaxCap) return DR_ERR_INVALID_ARG;
        *cap = c->max_len;
        return DR_OK;
    }
    if (c->layout != DR_KV_PAGED) return DR_ERR_INVALID_ARG;
    if (!c->block_table || c->num_blocks < 1 || c->max_blocks_per_seq < 1) return DR_ERR_INVALID_ARG;
    if (c->block_size != dr::kBlockKeys) return DR_ERR_UNSUPPORTED;
    if ((long long)c->max_blocks_per_seq * c->block_size > kMaxCap) return DR_ERR_INVALID_ARG;
    *cap = c->max_blocks_per_seq * c->block_size;
    return DR_OK;
}

// Ragged tokens T in B rows, Hq query heads on Hkv key/value heads.
dr_status check_sizes(int T, int B, int Hq, int Hkv, int D) {
    if (T < 1 || B < 1 || B > 65535 || Hq < 1 || Hkv < 1 || Hq > 4096 || Hq % Hkv != 0) return DR_ERR_INVALID_ARG;
    if ((long long)T * Hq > 0x7FFFFFFFLL) return DR_ERR_INVALID_ARG;
    if (D != dr::kHeadDim || Hq / Hkv > 128) return DR_ERR_UNSUPPORTED;
    return DR_OK;
}

// A token stride in elements: whole tokens, 16-byte steps.
bool bad_stride(int64_t stride, int heads) { return stride < (int64_t)heads * dr::kHeadDim || stride % 8 != 0; }

// 1 / x where x is a power of two and both are normal numbers, so that y / x and y * (1 / x) are the same for every y;
// else 0.
float exact_inverse(float x) {
    int e;
    return frexpf(x, &e) == 0.5f && e > -125 && e < 126 ? 1.0f / x : 0.f;
}

dr_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DR_OK : DR_ERR_CUDA; }

constexpr float kLog2e = 1.4426950408889634f;

void fill_cache(dr::PromptParams &p, const dr_kv_cache *c, int cap) {
    const bool paged = c->layout == DR_KV_PAGED, fp8 = c->kv_dtype == DR_KV_FP8_E4M3;
    p.k = c->k;
    p.v = c->v;
    p.table = paged ? c->block_table : nullptr;
    p.cap = cap;
    p.max_blocks = paged ? c->max_blocks_per_seq : 0;
    p.num_blocks = paged ? c->num_blocks : 0;
    p.out_scale = fp8 ? c->v_scale : 1.f;
}

// What a raw score q.k (codes, for an e4m3 cache) is multiplied by.
float score_scale(const dr_kv_cache *c, float scale) {
    return (scale > 0.f ? scale : 1.0f / sqrtf((float)dr::kHeadDim)) * (c->kv_dtype == DR_KV_FP8_E4M3 ? c->k_scale : 1.f);
}

void fill_scores(dr::PromptParams &p, const dr_kv_cache *c, float scale, const dr_score_opts *o) {
    const float s = score_scale(c, scale);
    p.sscale = s * kLog2e;
    p.slopes = o ? o->slopes : nullptr;
    p.cap_c1 = o ? o->softcap * kLog2e : 0.f;
    p.cap_c2 = o && o->softcap > 0.f ? s / o->softcap : 0.f;
}

// The kernels compute with scale k_scale log2 e and scale k_scale / softcap: refused where one of them overflows.
dr_status check_scores(const dr_kv_cache *c, float scale, const dr_score_opts *o) {
    if (!(scale == scale) || isinf(scale) || isinf(score_scale(c, scale) * kLog2e)) return DR_ERR_INVALID_ARG;
    if (!o) return DR_OK;
    if (!(o->softcap >= 0.f) || o->softcap > 1e30f || (o->softcap > 0.f && o->softcap < 1e-6f)) return DR_ERR_INVALID_ARG;
    if (o->softcap > 0.f && isinf(score_scale(c, scale) / o->softcap)) return DR_ERR_INVALID_ARG;
    if (o->causal != 0 && o->causal != 1) return DR_ERR_INVALID_ARG;
    return DR_OK;
}

// The CTAs per tile that the plan gives either cache type (a call that finds less workspace than its plan wants splits
// less).
int most_splits(int T, int g, int Hkv, int max_len, int sms, bool joined) {
    const int a = dr::plan_tile_splits(T, g, Hkv, max_len, false, sms, joined, 0),
              b = dr::plan_tile_splits(T, g, Hkv, max_len, true, sms, joined, 0);
    return a > b ? a : b;
}

// Softmax states of `splits` key ranges: (m, l) and 64 sums per (token, head).
size_t states_bytes(int splits, int T, int Hq) {
    return (size_t)splits * T * Hq * (dr::kHeadDim + 2) * sizeof(float);
}
// The sums first: they keep the workspace's alignment.
void set_states(dr::PromptParams &p, void *ws, int splits) {
    p.part_acc = static_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(p.part_acc + (size_t)splits * p.T * p.Hq * dr::kHeadDim);
    p.nparts = splits;
}

// dr_prompt_attn's checks, plan and launches; stall_head >= 0 only from the test hook.
dr_status prompt_call(const void *q, int64_t q_stride, const dr_kv_cache *cache, const int32_t *row_start,
                      const int32_t *kv_len, const dr_score_opts *opts, int T, int B, int Hq, int Hkv, int D,
                      int max_len_hint, float scale, void *out, dr_dtype out_dtype, void *ws, size_t ws_bytes,
                      int32_t *err_flag, int stall_head, void *stream) {
    dr_status st = check_sizes(T, B, Hq, Hkv, D);
    if (st != DR_OK) return st;
    int cap = 0;
    st = check_cache(cache, &cap);
    if (st != DR_OK) return st;
    st = check_scores(cache, scale, opts);
    if (st != DR_OK) return st;
    if (!q || !row_start || !kv_len || !out || !aligned16(q) || !aligned32(out) || bad_stride(q_stride, Hq))
        return DR_ERR_INVALID_ARG;
    if (out_dtype != DR_BF16 && out_dtype != DR_F32) return DR_ERR_INVALID_ARG;
    if (!aligned32(ws) || !aligned32(cache->k) || !aligned32(cache->v)) return DR_ERR_INVALID_ARG;
    if (opts && opts->prefix_len && !opts->causal) return DR_ERR_INVALID_ARG;
    dr::PromptParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.q_stride = q_stride;
    fill_cache(p, cache, cap);
    fill_scores(p, cache, scale, opts);
    p.row_start = row_start;
    p.kv_len = kv_len;
    p.causal = opts ? opts->causal : 1;
    p.prefix_len = opts ? opts->prefix_len : nullptr;
    p.first_key = opts ? opts->first_key : nullptr;
    p.T = T;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.g = Hq / Hkv;
    p.out = out;
    p.out_f32 = out_dtype == DR_F32;
    p.err = err_flag;
    const int sms = dr::current_device_sms();
    if (sms <= 0) return DR_ERR_CUDA;
    const bool paged = cache->layout == DR_KV_PAGED, fp8 = cache->kv_dtype == DR_KV_FP8_E4M3;
    const int len = max_len_hint > 0 && max_len_hint < cap ? max_len_hint : cap;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // Rows of one token go to the token kernel, longer ones to the tile kernel (it reads a row's keys once for all
    // its tokens).  The host knows only T and B: one launch when that settles it, else both.
    p.few_max = 1;
    const bool few = B > 1 || T == 1, many = T > B;
    if (!many) p.few_max = 0x7FFFFFFF;
    const int few_splits = dr::plan_token_splits(B, Hkv, p.g, len, fp8, sms);
    if (!many) return from_cuda(dr::launch_attn_tokens(p, paged, fp8, few_splits, cs));
    if (!few) p.few_max = 0;
    dr::PromptParams tp = p;
    tp.stall = stall_head + 1;
    int splits = dr::plan_tile_splits(T, p.g, Hkv, len, fp8, sms, true, 0);
    while (splits > 1 && (!ws || ws_bytes < states_bytes(splits, T, Hq))) --splits;
    if (splits > 1) set_states(tp, ws, splits);
    cudaError_t e = dr::launch_attn_tiles(tp, paged, fp8, splits, cs);
    if (e == cudaSuccess && few) {
        p.after_tiles = 1;
        e = dr::launch_attn_tokens(p, paged, fp8, few_splits, cs);
    }
    if (e == cudaSuccess && splits > 1) e = dr::launch_attn_join(tp, cs);
    return from_cuda(e);
}

// dr_shared_prefix_attn's checks, plan and launches; stall_head >= 0 only from the test hook.
dr_status shared_call(const void *q, int64_t q_stride, const dr_kv_cache *prefix, const int32_t *prefix_len,
                      const dr_kv_cache *cache, const int32_t *seq_len, const dr_score_opts *opts, int B, int Hq, int Hkv,
                      int D, int max_prefix_hint, int max_seq_len_hint, float scale, void *out, dr_dtype out_dtype,
                      void *ws, size_t ws_bytes, int32_t *err_flag, int stall_head, void *stream) {
    dr_status st = check_sizes(B, B, Hq, Hkv, D);
    if (st != DR_OK) return st;
    int pcap = 0, cap = 0;
    st = check_cache(prefix, &pcap);
    if (st != DR_OK) return st;
    if ((cache == nullptr) != (seq_len == nullptr)) return DR_ERR_INVALID_ARG;
    if (cache) {
        st = check_cache(cache, &cap);
        if (st != DR_OK) return st;
    }
    st = check_scores(prefix, scale, opts);
    if (st == DR_OK && cache) st = check_scores(cache, scale, opts);
    if (st != DR_OK) return st;
    if (opts && (opts->prefix_len || opts->first_key)) return DR_ERR_INVALID_ARG;
    if (!q || !prefix_len || !out || !aligned16(q) || !aligned32(out) || bad_stride(q_stride, Hq))
        return DR_ERR_INVALID_ARG;
    if (out_dtype != DR_BF16 && out_dtype != DR_F32) return DR_ERR_INVALID_ARG;
    const int sms = dr::current_device_sms();
    if (!aligned32(prefix->k) || !aligned32(prefix->v) || (cache && (!aligned32(cache->k) || !aligned32(cache->v))))
        return DR_ERR_INVALID_ARG;
    if (!ws || !aligned32(ws) || ws_bytes < states_bytes(1, B, Hq)) return DR_ERR_INVALID_ARG;
    if (sms <= 0) return DR_ERR_CUDA;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);

    dr::PromptParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.q_stride = q_stride;
    fill_cache(p, prefix, pcap);
    fill_scores(p, prefix, scale, opts);
    p.kv_len = prefix_len;
    p.own_len = seq_len;
    p.own_cap = cap;
    p.stall = stall_head + 1;
    p.T = B;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.g = Hq / Hkv;
    p.out = out;
    p.out_f32 = out_dtype == DR_F32;
    p.err = err_flag;
    const int plen = max_prefix_hint > 0 && max_prefix_hint < pcap ? max_prefix_hint : pcap;
    const dr_kv_cache *own = cache ? cache : prefix;   // no own keys: the token kernel only joins
    const bool own_fp8 = own->kv_dtype == DR_KV_FP8_E4M3;
    const int len = !cache ? 1 : max_seq_len_hint > 0 && max_seq_len_hint < cap ? max_seq_len_hint : cap;
    // rows are half as long as the longest, or so; 6.7 TB/s
    const double own_us = !cache ? 0 : (double)B * Hkv * len / 2 * (own_fp8 ? 128 : 256) / 6.7e6;
    int splits = dr::plan_tile_splits(B, p.g, Hkv, plen, prefix->kv_dtype == DR_KV_FP8_E4M3, sms, false, own_us);
    while (splits > 1 && ws_bytes < states_bytes(splits, B, Hq)) --splits;
    set_states(p, ws, splits);
    const cudaError_t e = dr::launch_attn_tiles(p, prefix->layout == DR_KV_PAGED,
                                                prefix->kv_dtype == DR_KV_FP8_E4M3, splits, cs);
    if (e != cudaSuccess) return DR_ERR_CUDA;

    fill_cache(p, own, cache ? cap : pcap);
    fill_scores(p, own, scale, opts);
    p.kv_len = seq_len;
    p.own_len = nullptr;
    p.few_max = 0x7FFFFFFF;
    p.after_tiles = 1;
    return from_cuda(dr::launch_attn_tokens(p, own->layout == DR_KV_PAGED, own_fp8,
                                            dr::plan_token_splits(B, Hkv, p.g, len, own_fp8, sms), cs));
}

}  // namespace

extern "C" {

dr_status dr_rope_table(float *table, int max_pos, int rot_dim, double base, void *stream) {
    if (!table || !aligned16(table) || max_pos < 1 || !(base > 0.0) || isinf(base)) return DR_ERR_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > dr::kHeadDim || rot_dim % 16 != 0) return DR_ERR_UNSUPPORTED;
    return from_cuda(dr::launch_rope_table(table, max_pos, rot_dim, base, static_cast<cudaStream_t>(stream)));
}

dr_status dr_rope_append(const dr_kv_cache *cache, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, void *q_out, int64_t q_out_stride, const int32_t *row_start,
                         const int32_t *start_pos, const int32_t *pos_offset, const float *rope_table, int rope_len,
                         int rot_dim, int interleaved, int T, int B, int Hq, int Hkv, int D, int32_t *err_flag,
                         void *stream) {
    dr_status st = check_sizes(T, B, Hq, Hkv, D);
    if (st != DR_OK) return st;
    int cap = 0;
    st = check_cache(cache, &cap);
    if (st != DR_OK) return st;
    if (!k || !v || !row_start || !start_pos || !aligned16(k) || !aligned16(v)) return DR_ERR_INVALID_ARG;
    if (bad_stride(k_stride, Hkv) || bad_stride(v_stride, Hkv)) return DR_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr)) return DR_ERR_INVALID_ARG;
    if (q && (!aligned16(q) || !aligned16(q_out) || bad_stride(q_stride, Hq) || bad_stride(q_out_stride, Hq)))
        return DR_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return DR_ERR_INVALID_ARG;
    if (rope_table) {
        if (!aligned16(rope_table) || rope_len < 1) return DR_ERR_INVALID_ARG;
        if (rot_dim < 16 || rot_dim > D || rot_dim % 16 != 0) return DR_ERR_UNSUPPORTED;
    }
    dr::RopeAppendParams p = {};
    p.k_cache = cache->k;
    p.v_cache = cache->v;
    p.block_table = cache->block_table;
    p.cap = cap;
    p.max_blocks = cache->max_blocks_per_seq;
    p.num_blocks = cache->num_blocks;
    p.kv_fp8 = cache->kv_dtype == DR_KV_FP8_E4M3;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.k_inv = exact_inverse(p.k_scale);
    p.v_inv = exact_inverse(p.v_scale);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.row_start = row_start;
    p.start_pos = start_pos;
    p.pos_offset = pos_offset;
    p.rope = rope_table;
    p.rope_len = rope_len;
    p.rot = rope_table ? rot_dim : 0;
    p.interleaved = interleaved;
    p.T = T;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.err = err_flag;
    return from_cuda(
        dr::launch_rope_append(p, cache->layout == DR_KV_PAGED, static_cast<cudaStream_t>(stream)));
}

dr_status dr_prompt_attn(const void *q, int64_t q_stride, const dr_kv_cache *cache, const int32_t *row_start,
                         const int32_t *kv_len, const dr_score_opts *opts, int T, int B, int Hq, int Hkv, int D,
                         int max_len_hint, float scale, void *out, dr_dtype out_dtype, void *ws, size_t ws_bytes,
                         int32_t *err_flag, void *stream) {
    return prompt_call(q, q_stride, cache, row_start, kv_len, opts, T, B, Hq, Hkv, D, max_len_hint, scale, out, out_dtype,
                       ws, ws_bytes, err_flag, -1, stream);
}

dr_status dr_prompt_attn_stall_test(const void *q, int64_t q_stride, const dr_kv_cache *cache, const int32_t *row_start,
                                    const int32_t *kv_len, const dr_score_opts *opts, int T, int B, int Hq, int Hkv, int D,
                                    int max_len_hint, float scale, void *out, dr_dtype out_dtype, void *ws, size_t ws_bytes,
                                    int32_t *err_flag, int stall_head, void *stream) {
    if (stall_head < 0 || stall_head >= Hkv) return DR_ERR_INVALID_ARG;
    if (T <= B) return DR_ERR_UNSUPPORTED;
    return prompt_call(q, q_stride, cache, row_start, kv_len, opts, T, B, Hq, Hkv, D, max_len_hint, scale, out, out_dtype,
                       ws, ws_bytes, err_flag, stall_head, stream);
}

size_t dr_prompt_attn_workspace(int T, int B, int Hq, int Hkv, int max_len, int num_sms) {
    if (T < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_len < 1 || num_sms < 1) return 0;
    if (T <= B) return 0;
    const int splits = most_splits(T, Hq / Hkv, Hkv, max_len, num_sms, true);
    return splits > 1 ? states_bytes(splits, T, Hq) : 0;
}

dr_status dr_shared_prefix_attn(const void *q, int64_t q_stride, const dr_kv_cache *prefix, const int32_t *prefix_len,
                                const dr_kv_cache *cache, const int32_t *seq_len, const dr_score_opts *opts, int B,
                                int Hq, int Hkv, int D, int max_prefix_hint, int max_seq_len_hint, float scale,
                                void *out, dr_dtype out_dtype, void *ws, size_t ws_bytes, int32_t *err_flag,
                                void *stream) {
    return shared_call(q, q_stride, prefix, prefix_len, cache, seq_len, opts, B, Hq, Hkv, D, max_prefix_hint,
                       max_seq_len_hint, scale, out, out_dtype, ws, ws_bytes, err_flag, -1, stream);
}

dr_status dr_shared_prefix_attn_stall_test(const void *q, int64_t q_stride, const dr_kv_cache *prefix, const int32_t *prefix_len,
                                           const dr_kv_cache *cache, const int32_t *seq_len, const dr_score_opts *opts, int B,
                                           int Hq, int Hkv, int D, int max_prefix_hint, int max_seq_len_hint, float scale,
                                           void *out, dr_dtype out_dtype, void *ws, size_t ws_bytes, int32_t *err_flag,
                                           int stall_head, void *stream) {
    if (stall_head < 0 || stall_head >= Hkv) return DR_ERR_INVALID_ARG;
    return shared_call(q, q_stride, prefix, prefix_len, cache, seq_len, opts, B, Hq, Hkv, D, max_prefix_hint,
                       max_seq_len_hint, scale, out, out_dtype, ws, ws_bytes, err_flag, stall_head, stream);
}

size_t dr_shared_prefix_attn_workspace(int B, int Hq, int Hkv, int max_prefix, int num_sms) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_prefix < 1 || num_sms < 1) return 0;
    return states_bytes(most_splits(B, Hq / Hkv, Hkv, max_prefix, num_sms, false), B, Hq);
}

}  // extern "C"
