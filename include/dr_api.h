/*
 * dr_api.h -- C ABI of libdecoderattn.so, the decode step of a MusicGen-style
 * multi-codebook audio-token decoder (the Parler-TTS decoder) on NVIDIA GB300
 * (sm_103a).
 *
 * Four operations make up one decode step:
 *   dr_kv_append            write this step's key/value into the cache;
 *   dr_decode_self_attn     one-query causal self-attention over the valid
 *                           length of a static (contiguous) or paged cache,
 *                           bf16 or FP8 E4M3;
 *   dr_decode_cross_attn    one-query attention over the description
 *                           encoder's keys and values;
 *   dr_sample_topk_delayed  temperature, top-k, softmax and categorical draw
 *                           for every codebook in one kernel, under the
 *                           delay pattern.
 * dr_decode_layer does the first three for one layer in one launch; the
 * decoder's two ends around them are dr_lm_head (the merged codebook heads
 * on the newest position, writing the logits the sampler reads) and
 * dr_embed_tokens (the merged embedding lookup of the drawn tokens).
 * Around the step, on the same caches and with grouped heads:
 *   dr_rope_append          rotate q and k by position and append the keys and
 *                           values of ragged new tokens (prompts, or one per row);
 *   dr_prompt_attn          attention of ragged query tokens over the cache, with
 *                           a score cap, a distance bias and causal, prefix and
 *                           document masks;
 *   dr_shared_prefix_attn   single-query attention of a batch whose rows share a
 *                           long prefix, which is read once for all of them.
 * Between a layer's attention calls, for steps and prompts alike:
 *   dr_linear               matrix product (projections, MLP) with bias, activation,
 *                           gating and residual in its epilogue;
 *   dr_residual_norm        the norms after and before a block with its gate,
 *                           residual scale and residual.
 *
 * Conventions shared by every call
 *   - Every pointer argument except `stream` is a DEVICE pointer owned by the
 *     caller.  The library allocates nothing, keeps no pointer after a call
 *     returns, and never synchronises with the host.
 *   - `stream` is a cudaStream_t passed as an opaque pointer (NULL = the
 *     legacy default stream).  Work is enqueued on it asynchronously; the
 *     calls are free of host-device synchronisation.
 *   - bf16 means IEEE bfloat16 (the upper 16 bits of a binary32), stored as
 *     2-byte values.  Tensors are dense and row-major in the order given.
 *   - Host-checkable mistakes (null pointers, bad sizes, misalignment) return
 *     an error status before anything is enqueued.  A failed launch returns
 *     DR_ERR_CUDA.
 *   - Mistakes only the device can see (a length above the capacity, a block
 *     id outside the pool, an append position past the end) never trap: the
 *     kernel clamps or skips the offending row or block and, when `err_flag`
 *     is non-NULL, ORs a DR_ERRF_* bit into *err_flag (a device int32 the
 *     caller zeroes and reads back when it chooses).
 *   - Head dimension D must be 64 (DR_ERR_UNSUPPORTED otherwise); keys and
 *     values have as many heads H as the query (plain multi-head attention),
 *     except in the calls that take Hq and Hkv: there Hq is a multiple of Hkv
 *     (at most 128 times), and query head h uses key/value head h / (Hq/Hkv);
 *     such a call's cache is described with Hkv in the place of H.
 *   - Calls on the same stream are ordered; the library holds no state
 *     between calls, so calls on different streams may overlap as long as
 *     they do not write the same buffers.
 */
#ifndef DR_API_H
#define DR_API_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dr_status {
    DR_OK = 0,
    DR_ERR_INVALID_ARG = 1, /* null pointer, size out of range, misaligned pointer */
    DR_ERR_UNSUPPORTED = 2, /* a valid but unimplemented shape (D != 64, block_size != 16, C > 16, V > 2048,
                               more than 65535 sampler rows) */
    DR_ERR_CUDA = 3         /* the CUDA runtime refused the launch */
} dr_status;

typedef enum dr_kv_layout {
    DR_KV_CONTIGUOUS = 0, /* static cache: k, v are [B][H][max_len][D] */
    DR_KV_PAGED = 1       /* block pool: k, v are [num_blocks][H][block_size][D] */
} dr_kv_layout;

typedef enum dr_dtype { DR_BF16 = 0, DR_F32 = 1 } dr_dtype;

/* Storage format of a self-attention KV cache. */
typedef enum dr_kv_dtype {
    DR_KV_BF16 = 0,    /* bf16 keys and values */
    DR_KV_FP8_E4M3 = 1 /* OCP FP8 E4M3 codes: key = code * k_scale, value = code * v_scale */
} dr_kv_dtype;

/* Device-side error bits (see err_flag above). */
#define DR_ERRF_SEQ_LEN 1  /* a seq_len / enc_len entry outside [1, capacity]; it was clamped */
#define DR_ERRF_BLOCK_ID 2 /* a needed block-table entry outside [0, num_blocks); its keys were skipped */
#define DR_ERRF_POS 4      /* an append position outside [0, capacity) or on an unmapped block; row skipped */
#define DR_ERRF_TOKEN 8    /* a token outside [0, V) in dr_embed_tokens; that codebook's row was skipped */
#define DR_ERRF_TIMEOUT 16 /* a bounded on-chip wait gave up (never expected); that CTA's results were not written,
                              or are NaN where they are joined with others' */
#define DR_ERRF_ROW_START 32 /* row_start does not rise from 0 to at most T; rows were cut to [0, T) */

/* Sampler flags. */
#define DR_SAMPLE_ADVANCE 1 /* after drawing, step[b] += 1 for every row b */

/*
 * A self-attention KV cache (one decoder layer).
 *
 * Static cache (Optimized Parler TTS, "Analysis and improvements": the static
 * caches for causal and cross attention that CUDA-graph capture needs,
 * preallocated to a maximum length):
 *   layout = DR_KV_CONTIGUOUS; k, v = [B][H][max_len][D]; key j of row
 *   (b, h) at ((b*H + h)*max_len + j)*D.  Capacity = max_len keys per row.
 * Paged cache (same page, "Future work" item 1: a PagedAttention-style cache
 * so that no full static cache has to be kept or moved):
 *   layout = DR_KV_PAGED; k, v = [num_blocks][H][block_size][D];
 *   block_table = [B][max_blocks_per_seq] int32; key j of row b lives in block
 *   block_table[b][j / block_size], slot j % block_size; entries a row does
 *   not use may hold any value (conventionally -1).  block_size must be 16.
 *   Capacity = max_blocks_per_seq * block_size keys per row.
 * Element format (kv_dtype): bf16, or FP8 E4M3 codes (the same page's
 * "Future work" item 1 asks for less KV traffic; 8-bit codes halve it).  An
 * e4m3 cache stores code = e4m3(fl32(x / scale)) (IEEE division, round to
 * nearest even, saturating at +-448) and is read back as code * scale, with
 * k_scale for keys and v_scale for values (both > 0; ignored for bf16).
 * k and v must be 16-byte aligned.  The struct itself is read on the host
 * during the call only.
 */
typedef struct dr_kv_cache {
    int32_t layout;             /* dr_kv_layout */
    int32_t max_len;            /* contiguous: keys per (b, h) row; ignored when paged */
    int32_t block_size;         /* paged: keys per block (16); ignored when contiguous */
    int32_t num_blocks;         /* paged: blocks in the pool */
    int32_t max_blocks_per_seq; /* paged: row stride of block_table */
    int32_t kv_dtype;           /* dr_kv_dtype */
    void *k;                    /* keys (device) */
    void *v;                    /* values (device) */
    const int32_t *block_table; /* paged: [B][max_blocks_per_seq] int32 (device); NULL when contiguous */
    float k_scale;              /* e4m3 only: key = code * k_scale */
    float v_scale;              /* e4m3 only: value = code * v_scale */
} dr_kv_cache;

/*
 * dr_kv_append -- store this step's key and value of every row.
 * Source: Optimized Parler TTS, "Analysis and improvements" (static cache
 * for causal attention; each decode step adds one key/value per row).
 *
 *   k_new, v_new : [B][H][D] bf16 (device, 16-byte aligned); quantised to
 *                  e4m3 codes when the cache is DR_KV_FP8_E4M3
 *   pos          : [B] int32 (device); row b's key/value go to position pos[b]
 *                  (the row's valid length becomes pos[b] + 1 for the
 *                  self-attention that follows)
 *   err_flag     : nullable device int32; DR_ERRF_POS is ORed in when
 *                  pos[b] is outside [0, capacity) or, paged, its block-table
 *                  entry is outside the pool; that row is not written.
 * Writes exactly B*H*D elements into each of cache->k and cache->v.
 */
dr_status dr_kv_append(const dr_kv_cache *cache, const void *k_new, const void *v_new, const int32_t *pos, int B,
                       int H, int D, int32_t *err_flag, void *stream);

/*
 * dr_decode_self_attn -- single-query causal self-attention of one decode
 * step over the valid part of a KV cache.
 * Source: Optimized Parler TTS, "Analysis and improvements": the static-cache
 * attention kernel took ~95 us because it moved the whole preallocated cache,
 * against ~13 us for the eager kernel that reads the valid length only; and
 * "Future work" item 1 (paged cache).
 *
 * For every row b and head h:
 *   s_j = scale * (q[b,h,:] . K[b,h,j,:])  for j in [0, seq_len[b])
 *   out[b,h,:] = sum_j softmax(s)_j V[b,h,j,:]
 * Only the seq_len[b] valid keys of each row are read.  Causality for a
 * single query means it sees every valid key, including the one appended in
 * this step.  Accumulation is fp32; the result is written in out_dtype.
 *
 *   q        : [B][H][D] bf16 (device, 16-byte aligned)
 *   cache    : see dr_kv_cache
 *   seq_len  : [B] int32 (device), keys attended per row, 1 <= seq_len[b] <=
 *              capacity; entries outside are clamped to [0, capacity] and
 *              flagged DR_ERRF_SEQ_LEN (a row of length 0 outputs zeros)
 *   max_seq_len_hint : an upper bound the caller knows for max_b seq_len[b]
 *              (<= 0: the capacity).  It only tunes how each row's keys are
 *              split across CTAs (dr_plan_splits); any value gives a result
 *              within the stated accuracy, and the same hint on the same
 *              device gives the same bits (a different split changes only
 *              the order of the fp32 sums).
 *   scale    : softmax scale; <= 0 selects 1/sqrt(D)
 *   out      : [B][H][D] in out_dtype (DR_BF16: round to nearest even)
 *   err_flag : nullable device int32 (DR_ERRF_SEQ_LEN, DR_ERRF_BLOCK_ID)
 */
dr_status dr_decode_self_attn(const void *q, const dr_kv_cache *cache, const int32_t *seq_len, int B, int H, int D,
                              int max_seq_len_hint, float scale, void *out, dr_dtype out_dtype, int32_t *err_flag,
                              void *stream);

/*
 * dr_decode_cross_attn -- single-query attention over the description
 * encoder's keys and values (recomputed every decode step).
 * Source: Optimized Parler TTS, architecture overview (the description,
 * encoded by Flan-T5, is used through cross-attention in the decoder's
 * attention layers) and "Speeding up Parler TTS decoder" (throughput falls
 * as the description grows, because of this cross-attention).
 *
 *   q        : [B][H][D] bf16 (device, 16-byte aligned)
 *   k_enc, v_enc : [B][H][Lc_max][D] bf16 (device, 16-byte aligned)
 *   enc_len  : [B] int32 (device), description length per row, 1 <=
 *              enc_len[b] <= Lc_max (clamped and flagged otherwise)
 *   scale, out, out_dtype, err_flag : as for dr_decode_self_attn
 */
dr_status dr_decode_cross_attn(const void *q, const void *k_enc, const void *v_enc, const int32_t *enc_len, int B,
                               int H, int D, int Lc_max, float scale, void *out, dr_dtype out_dtype,
                               int32_t *err_flag, void *stream);

/*
 * dr_decode_layer -- one decoder layer's attention work of a decode step in
 * one launch: the KV append, the self-attention and the cross-attention.
 * Source: the same passages as the three calls above; fusing them is the
 * launch-count reduction the page's profile motivates (Optimized Parler TTS,
 * "Analysis and improvements": the decoder is overhead-bound, the GPU waits
 * between small kernels).
 *
 * Equivalent to, in this order,
 *   dr_kv_append(cache, k_new, v_new, pos = seq_len - 1, ...)
 *   dr_decode_self_attn(q, cache, seq_len, ..., out, ...)
 *   dr_decode_cross_attn(q_cross, k_enc, v_enc, enc_len, ..., Lc_max, ..., out_cross, ...)
 * with results within the same tolerances (the key at seq_len[b]-1 is taken
 * from k_new/v_new directly and also stored into the cache; rows whose
 * seq_len is outside [1, capacity] are not appended and flag DR_ERRF_POS and
 * DR_ERRF_SEQ_LEN).  Arguments are as for those calls; out and out_cross are
 * both [B][H][D] in out_dtype.  B <= 32767.
 */
dr_status dr_decode_layer(const void *q, const dr_kv_cache *cache, const void *k_new, const void *v_new,
                          const int32_t *seq_len, const void *q_cross, const void *k_enc, const void *v_enc,
                          const int32_t *enc_len, int Lc_max, int B, int H, int D, int max_seq_len_hint, float scale,
                          void *out, void *out_cross, dr_dtype out_dtype, int32_t *err_flag, void *stream);

/*
 * dr_sample_topk_delayed -- one kernel that turns the logits of every
 * codebook of every row into this step's tokens.
 * Source: Optimized Parler TTS, "Future work" item 2 (temperature scaling,
 * top-k and softmax, run as more than ten kernels, should be one fused
 * kernel), "Analysis and improvements" (sampling without a GPU-CPU
 * synchronisation) and the architecture overview (nine DAC codebooks, one
 * token each per step, in a delayed pattern).
 *
 * For every row b and codebook c (0-based):
 *   if step[b] <= c : tokens[b][c] = pad_id (delay pattern: codebook c starts
 *                     one step after codebook c-1); probs row = 0
 *   else:
 *     x_i  = fl32(logits[b][c][i] / temperature), IEEE round-to-nearest
 *     K    = the top_k indices by x descending, equal x -> lower index first
 *     u_i  = (2*(w >> 9) + 1) * 2^-24, w = word (i mod 4) of
 *            Philox4x32-10(counter = {i/4, c, step[b], b},
 *                          key = {seed[b] bits 0-31, bits 32-63})
 *     tokens[b][c] = argmax over i in K of x_i - log(-log(u_i))  (Gumbel-max:
 *                    a categorical draw from softmax over K); equal scores
 *                    -> lower index
 *     probs[b][c][i] = exp(x_i - max_K x) / sum_K exp(x_j - max_K x) for i in
 *                    K, 0 elsewhere (uniform 1/top_k over K if all of K is -inf)
 * Philox4x32-10: Salmon et al., "Parallel Random Numbers: As Easy as 1, 2, 3",
 * SC'11.
 *
 *   logits   : [B][C][ldv] float32 (device); columns [V, ldv) are never read.
 *              NaN logits give an undefined (but in-range or pad) token.
 *              Where some x_i are +inf (an infinite logit, or a temperature
 *              so small that logit / temperature overflows), the token is the
 *              lowest such index and the probabilities are undefined.
 *   B        : batch rows, 1..65535 (DR_ERR_UNSUPPORTED above)
 *   C        : codebooks, 1..16          V : vocabulary, 1..2048, V <= ldv
 *   temperature : > 0 and finite          top_k : 1..V
 *   seeds    : [B] uint64 (device)
 *   step     : [B] int32 (device); read, and incremented when flags has
 *              DR_SAMPLE_ADVANCE (after every codebook of the row has read it)
 *   tokens   : [B][C] int32 (device, written)
 *   probs    : nullable [B][C][V] float32 (device, written when non-NULL)
 */
dr_status dr_sample_topk_delayed(const float *logits, int B, int C, int V, int ldv, float temperature, int top_k,
                                 const uint64_t *seeds, int32_t *step, int32_t pad_id, int32_t *tokens, float *probs,
                                 int flags, void *stream);

/*
 * dr_embed_tokens -- the next step's decoder input from this step's tokens:
 *   out[b][d] = sum_{c=0..C-1} table[c*V + tokens[b][c]][d]
 * Source: Optimized Parler TTS, "Analysis and improvements", other
 * optimizations item 3: the nine codebook embedding lookups merged into one
 * (one merged table, one gather of C rows per batch row).
 *
 *   C      : codebooks, 1..16 (DR_ERR_UNSUPPORTED above 16, as for the sampler)
 *   tokens : [B][C] int32 (device), e.g. the tokens dr_sample_topk_delayed wrote
 *   table  : [C*V][Dm] bf16 (device, 16-byte aligned); codebook c's rows start at c*V
 *   out    : [B][Dm] in out_dtype (device, 16-byte aligned); fp32 sum in c order
 *   Dm     : a multiple of 8
 *   err_flag : nullable; DR_ERRF_TOKEN when a token is outside [0, V) (that
 *            term is left out of the sum)
 */
dr_status dr_embed_tokens(const int32_t *tokens, const void *table, int B, int C, int V, int Dm, void *out,
                          dr_dtype out_dtype, int32_t *err_flag, void *stream);

/*
 * dr_lm_head -- logits of the newest position from the merged codebook heads:
 *   logits[b][c][v] = sum_k hidden[b][k] * W[c*V + v][k]
 * Source: Optimized Parler TTS, "Analysis and improvements", other
 * optimizations items 1-2: the LM head computed for the last position only,
 * and the nine codebook heads merged into one weight matrix.
 *
 *   hidden : [B][K] bf16 (device, 16-byte aligned), the newest position's hidden state
 *   W      : [C*V][K] bf16 (device, 16-byte aligned)
 *   logits : [B][C][ldv] float32 (device), ldv >= V; columns [V, ldv) untouched.
 *            The layout dr_sample_topk_delayed reads.
 *   K      : 256, 512, 768, 1024, 1536 or 2048 (DR_ERR_UNSUPPORTED otherwise)
 *   err_flag : nullable device int32; DR_ERRF_TIMEOUT if a tensor-core CTA's
 *            bounded pipeline wait gave up (its logits are then not written)
 * fp32 accumulation.  Below 4 batch rows each logit is one CUDA-core dot
 * product in a fixed order; from 4 rows on the head is a dense contraction
 * on the tensor cores (tcgen05.mma, bf16 in, fp32 accumulate in tensor
 * memory, K consumed 16 at a time; when the batch is one tile of up to 32
 * rows and the 128-row weight slabs are fewer than the SMs, the two halves of
 * K are accumulated apart and added, the first half's sum first).
 */
dr_status dr_lm_head(const void *hidden, const void *W, int B, int K, int C, int V, int ldv, float *logits,
                     int32_t *err_flag, void *stream);

/*
 * dr_lm_head_stall_test -- TEST HOOK, never needed in use.  The same call as
 * dr_lm_head, except that the CTAs of 128-row weight slab `stall_slab` (logit
 * rows c*V + v in [128*stall_slab, 128*stall_slab + 128)) never load their
 * first K chunk.  The CTA's bounded pipeline wait for it then runs out (after
 * about 2 s): DR_ERRF_TIMEOUT is ORed into *err_flag, that slab's logits are
 * left unwritten, the CTA frees its tensor memory and exits, and every other
 * logit is written as by dr_lm_head.  Nothing faults or hangs, and later calls
 * on the same context work normally.  The tests use it to check the failure
 * path of the waits; the paper has no counterpart.
 *   B >= 4 (the tensor-core head; DR_ERR_UNSUPPORTED below), 0 <= stall_slab
 *   < ceil(C*V / 128) (DR_ERR_INVALID_ARG otherwise); the rest as dr_lm_head.
 */
dr_status dr_lm_head_stall_test(const void *hidden, const void *W, int B, int K, int C, int V, int ldv, float *logits,
                                int32_t *err_flag, int stall_slab, void *stream);

/*
 * dr_decode_self_attn_stall_test -- TEST HOOK, never needed in use.  The
 * same call as dr_decode_self_attn, except that CTA 1 of row
 * stall_row = b*H + h never sends its softmax state to the row's CTA rank 0.
 * That CTA's bounded wait for the state then runs out (after about 2 s):
 * DR_ERRF_TIMEOUT is ORed into *err_flag, that row's output is left
 * unwritten, and every other row is written as by dr_decode_self_attn.
 * Nothing faults or hangs, and later calls on the same context work
 * normally.  The tests use it to check the failure path of the cluster
 * merge's wait; the paper has no counterpart.
 *   0 <= stall_row < B*H (DR_ERR_INVALID_ARG otherwise).  The call must run
 *   the kernel variant whose split rows merge through that wait: at least 2
 *   CTAs per row (dr_plan_splits) and more than 4 CTAs per SM in all
 *   (DR_ERR_UNSUPPORTED otherwise).  The rest as dr_decode_self_attn.
 */
dr_status dr_decode_self_attn_stall_test(const void *q, const dr_kv_cache *cache, const int32_t *seq_len, int B, int H,
                                        int D, int max_seq_len_hint, float scale, void *out, dr_dtype out_dtype,
                                        int32_t *err_flag, int stall_row, void *stream);

/*
 * dr_rope_table -- cos and sin of every position and frequency, the table
 * that dr_rope_append reads (made once, kept by the caller):
 *   table[p][i]             = cos(p * base^(-2i / rot_dim)),  i in [0, rot_dim/2)
 *   table[p][rot_dim/2 + i] = sin(p * base^(-2i / rot_dim))
 * Angles and functions are computed in 64 bits and rounded once to fp32.
 *   table : [max_pos][rot_dim] float32 (device, 16-byte aligned, written)
 *   rot_dim : 16, 32, 48 or 64 (DR_ERR_UNSUPPORTED otherwise);  base > 0
 */
dr_status dr_rope_table(float *table, int max_pos, int rot_dim, double base, void *stream);

/*
 * dr_rope_append -- rotate the queries and keys of ragged new tokens by their
 * positions and append the keys and values to the cache, in one pass.
 *
 * Row b's tokens are t = row_start[b] .. row_start[b+1]-1; token
 * row_start[b] + i goes to cache slot start_pos[b] + i of row b and is
 * rotated for position start_pos[b] + i (+ pos_offset[b]):
 *   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin)
 * on the pairs (i, i + rot_dim/2), or (2i, 2i+1) when interleaved, i in
 * [0, rot_dim/2) of every head; dimensions from rot_dim on and all of v pass
 * through.  Products and sum are rounded apart in fp32; the result is rounded
 * once: to bf16, or to the e4m3 code of fl32(x / scale) as in dr_kv_append.
 * Tokens from row_start[B] on are left as they are (q_out and cache).
 *
 *   cache    : see dr_kv_cache, with Hkv heads; B rows of at most 2^31 - 4096 keys
 *   q        : nullable [T][Hq][D] bf16 (device, 16-byte aligned), tokens q_stride elements apart (a multiple
 *              of 8, at least Hq*D: a slice of a fused projection's output will do)
 *   k, v     : [T][Hkv][D] bf16 likewise, k_stride and v_stride
 *   q_out    : rotated queries, [T][Hq][D] bf16 likewise; null exactly when q is; may be q itself with the same
 *              stride, else it overlaps no input
 *   row_start: [B+1] int32 (device), rising from 0 to at most T (DR_ERRF_ROW_START otherwise: a token then goes by
 *              one of the rows that hold it, or is left out); rows may be empty
 *   start_pos: [B] int32 (device), cache slot of each row's first new token.  DR_ERRF_POS and no key or value is
 *              written where a slot is outside [0, capacity) or its block outside the pool
 *   pos_offset : nullable [B] int32 (device), added to the slot for the rotation (keys before the row's own
 *              cache, such as a shared prefix)
 *   rope_table : [rope_len][rot_dim] float32 as dr_rope_table makes it (device, 16-byte aligned); null: no
 *              rotation.  A position outside [0, rope_len): DR_ERRF_POS, the token is left out altogether
 *   interleaved: 0 or 1
 * Two rows may not write the same slot of the same block.
 */
dr_status dr_rope_append(const dr_kv_cache *cache, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, void *q_out, int64_t q_out_stride, const int32_t *row_start,
                         const int32_t *start_pos, const int32_t *pos_offset, const float *rope_table, int rope_len,
                         int rot_dim, int interleaved, int T, int B, int Hq, int Hkv, int D, int32_t *err_flag,
                         void *stream);

/* How dr_prompt_attn scores and masks keys (read on the host during the call; the arrays are device pointers). */
typedef struct dr_score_opts {
    int32_t causal;            /* 1: the query at position p sees keys up to p; 0: all keys of its row */
    float softcap;             /* > 0 (1e-6 .. 1e30): s -> softcap * tanh(s / softcap); 0: none */
    const float *slopes;       /* nullable [Hq] float32: s -> s - slopes[h] * |p - j| (after the cap) */
    const int32_t *prefix_len; /* nullable [B], causal only: keys j < prefix_len[b] are seen by all queries of row b */
    const int32_t *first_key;  /* nullable [T]: query t sees no key before first_key[t] (packed documents, windows) */
} dr_score_opts;

/*
 * dr_prompt_attn -- attention of ragged query tokens (prompts, chunks of
 * prompts, or one token per row) over the cache that already holds their keys.
 *
 * Row b's queries are t = row_start[b] .. row_start[b+1]-1, n of them; they
 * are the last n of the row's kv_len[b] keys: query row_start[b] + i stands at
 * position p = kv_len[b] - n + i.  For query head h and its key/value head:
 *   s_j = scale * (q . K_j), capped, biased (dr_score_opts)
 *   out[t][h] = sum_j softmax(s)_j V_j over the keys j in [lo, hi),
 *   lo = max(0, first_key[t]), hi = min(kv_len[b], max(p + 1, prefix_len[b])) when causal, else kv_len[b].
 * A query that sees no key outputs zeros.  Scores, softmax statistics and sums
 * are fp32; the weights are rounded for the product with V: over a bf16 cache to
 * 16 bits in rows of one token (and calls with T <= B) and to bf16 in longer
 * rows, where they are an operand of the matrix unit, which takes bf16 beside
 * bf16 values; over an e4m3 cache to f16 (below 2^-21 of the row's largest weight
 * to steps of 2^-31), which also holds the codes and, scaled by a power of two
 * per head, q.  Keys at or past kv_len and keys that no query
 * of the call may see do not reach the result whatever they hold; a NaN in a
 * query or in a key that it sees makes its outputs NaN.  With T <= B a row's
 * tokens are taken one after another (each reads the row's keys again): prompts
 * in a batch of mostly empty rows are faster in a call over their rows alone.
 *
 *   q        : [T][Hq][D] bf16 (device, 16-byte aligned), tokens q_stride elements apart (multiple of 8, >= Hq*D)
 *   cache    : see dr_kv_cache, with Hkv heads; B rows of at most 2^31 - 4096 keys; k and v 32-byte aligned
 *   row_start: [B+1] int32 (device), rising from 0 to at most T (DR_ERRF_ROW_START otherwise); rows may be empty;
 *              outputs of tokens from row_start[B] on are left as they are
 *   kv_len   : [B] int32 (device), keys per row, its new tokens' included: n <= kv_len[b] <= capacity (clamped to
 *              [0, capacity] and flagged DR_ERRF_SEQ_LEN otherwise)
 *   opts     : nullable (causal, nothing else)
 *   max_len_hint : an upper bound the caller knows for kv_len (<= 0: the capacity); tunes the work split only
 *   scale    : <= 0 selects 1/sqrt(D); scale * log2 e and scale / softcap, times k_scale for an e4m3 cache, have
 *              to be finite (DR_ERR_INVALID_ARG otherwise)
 *   out      : [T][Hq][D] in out_dtype (device, 32-byte aligned)
 *   ws       : nullable workspace (device, 32-byte aligned) of ws_bytes; with at least
 *              dr_prompt_attn_workspace bytes few queries over many keys are spread over the GPU.  Its contents
 *              mean nothing before and after the call; calls that may overlap need one each
 *   err_flag : nullable device int32 (DR_ERRF_ROW_START, DR_ERRF_SEQ_LEN, DR_ERRF_BLOCK_ID, DR_ERRF_TIMEOUT)
 */
dr_status dr_prompt_attn(const void *q, int64_t q_stride, const dr_kv_cache *cache, const int32_t *row_start,
                         const int32_t *kv_len, const dr_score_opts *opts, int T, int B, int Hq, int Hkv, int D,
                         int max_len_hint, float scale, void *out, dr_dtype out_dtype, void *ws, size_t ws_bytes,
                         int32_t *err_flag, void *stream);

/*
 * dr_prompt_attn_stall_test -- TEST HOOK, never needed in use.  The same call
 * as dr_prompt_attn, except that one CTA of the tile kernel never loads its
 * first keys: that of the first tile's first key range, key/value head
 * stall_head (the tile: the last 128 (token, query head) pairs of that head in
 * the first row of several tokens).  The CTA's bounded waits then run out
 * (after about 2 s): DR_ERRF_TIMEOUT is ORed into *err_flag, it waits for its
 * copies in flight, frees its tensor memory and exits.  Its outputs are left
 * unwritten, or NaN where key ranges are joined; every other output is written
 * as by dr_prompt_attn.  Nothing faults or hangs, and later calls on the same
 * context work normally.
 *   T > B (DR_ERR_UNSUPPORTED otherwise: no tile kernel), 0 <= stall_head < Hkv
 *   (DR_ERR_INVALID_ARG otherwise); the rest as dr_prompt_attn.
 */
dr_status dr_prompt_attn_stall_test(const void *q, int64_t q_stride, const dr_kv_cache *cache, const int32_t *row_start,
                                    const int32_t *kv_len, const dr_score_opts *opts, int T, int B, int Hq, int Hkv,
                                    int D, int max_len_hint, float scale, void *out, dr_dtype out_dtype, void *ws,
                                    size_t ws_bytes, int32_t *err_flag, int stall_head, void *stream);

/* Host-only: workspace bytes dr_prompt_attn wants for such a call on a GPU with num_sms SMs (0: none needed). */
size_t dr_prompt_attn_workspace(int T, int B, int Hq, int Hkv, int max_len, int num_sms);

/*
 * dr_shared_prefix_attn -- single-query attention of B rows whose first keys
 * are the same: row b attends the prefix's prefix_len[0] keys, then its own
 * seq_len[b] keys.
 *   s_j = scale * (q[b,h] . K_j), capped and biased as in dr_prompt_attn (row b's query stands at position
 *         prefix_len[0] + seq_len[b] - 1; own key j at prefix_len[0] + j)
 *   out[b][h] = sum_j softmax(s)_j V_j over both
 * The prefix is read once per 128 query rows (all rows' heads on its key/value
 * head together), not once per row; the softmax states of the two parts are
 * merged in fp32.  Rounding as in dr_prompt_attn (own keys as rows of one token,
 * the prefix as longer ones).  A row with no key at all outputs zeros.  For
 * several prefixes, one call per group of rows.  A row's own prompt behind the prefix is a dr_prompt_attn call over a block table that
 * begins with the prefix's blocks (one pool, a prefix of whole blocks), with the
 * prefix counted in kv_len.
 *
 *   q        : [B][Hq][D] bf16 (device, 16-byte aligned), rows q_stride elements apart (multiple of 8, >= Hq*D)
 *   prefix   : cache of one row (row 0) with Hkv heads, k and v 32-byte aligned (cache's too); paged: its blocks may
 *              lie in the same pool as cache's
 *   prefix_len : [1] int32 (device), 0 <= prefix_len[0] <= the prefix's capacity (else clamped, DR_ERRF_SEQ_LEN)
 *   cache, seq_len : the rows' own keys, B rows with Hkv heads, and [B] int32 (device), 0 <= seq_len[b] <= capacity
 *              (else clamped, DR_ERRF_SEQ_LEN); both null: rows have no own keys (a description that a batch shares)
 *   opts     : nullable; softcap and slopes are used, prefix_len and first_key must be null
 *   max_prefix_hint, max_seq_len_hint : upper bounds the caller knows (<= 0: the capacities); tune the split only
 *   out      : [B][Hq][D] in out_dtype (device, 32-byte aligned)
 *   ws       : workspace (device, 32-byte aligned) of ws_bytes, at least dr_shared_prefix_attn_workspace with
 *              max_prefix = 1 (DR_ERR_INVALID_ARG below); as much as it asks for the real bound spreads a prefix over
 *              the GPU.  Its contents mean nothing before and after the call; calls that may overlap need one each
 *   err_flag : nullable device int32 (DR_ERRF_SEQ_LEN, DR_ERRF_BLOCK_ID, DR_ERRF_TIMEOUT)
 */
dr_status dr_shared_prefix_attn(const void *q, int64_t q_stride, const dr_kv_cache *prefix, const int32_t *prefix_len,
                                const dr_kv_cache *cache, const int32_t *seq_len, const dr_score_opts *opts, int B,
                                int Hq, int Hkv, int D, int max_prefix_hint, int max_seq_len_hint, float scale,
                                void *out, dr_dtype out_dtype, void *ws, size_t ws_bytes, int32_t *err_flag,
                                void *stream);

/*
 * dr_shared_prefix_attn_stall_test -- TEST HOOK, as dr_prompt_attn_stall_test:
 * the CTA of the prefix's first key range and the first 128 (row, query head)
 * pairs of key/value head stall_head never loads its first keys.  Those
 * outputs are NaN.
 */
dr_status dr_shared_prefix_attn_stall_test(const void *q, int64_t q_stride, const dr_kv_cache *prefix,
                                           const int32_t *prefix_len, const dr_kv_cache *cache, const int32_t *seq_len,
                                           const dr_score_opts *opts, int B, int Hq, int Hkv, int D,
                                           int max_prefix_hint, int max_seq_len_hint, float scale, void *out,
                                           dr_dtype out_dtype, void *ws, size_t ws_bytes, int32_t *err_flag,
                                           int stall_head, void *stream);

/* Host-only: workspace bytes of dr_shared_prefix_attn for prefixes of up to max_prefix keys on num_sms SMs. */
size_t dr_shared_prefix_attn_workspace(int B, int Hq, int Hkv, int max_prefix, int num_sms);

/* Activations of dr_linear, computed in fp32. */
typedef enum dr_act {
    DR_ACT_NONE = 0,
    DR_ACT_RELU = 1,      /* max(a, 0) */
    DR_ACT_GELU = 2,      /* a * Phi(a), Phi the normal distribution function */
    DR_ACT_GELU_TANH = 3, /* a * (1 + tanh(sqrt(2 / pi) * (a + 0.044715 a^3))) / 2 */
    DR_ACT_SILU = 4       /* a / (1 + exp(-a)) */
} dr_act;

/* What dr_linear does with its sums (read on the host during the call; the arrays are device pointers). */
typedef struct dr_linear_opts {
    int32_t act;             /* dr_act */
    int32_t gated;           /* 1: W has 2N rows; the activated first N columns are multiplied by the last N */
    const void *bias;        /* nullable [N] ([2N] when gated) bf16, 16-byte aligned: added before the activation */
    const void *residual;    /* nullable [T][N] in out_dtype: added last; may be the output itself with its stride */
    int64_t residual_stride; /* elements between its tokens, at least N */
} dr_linear_opts;

/* One output of dr_linear: `cols` columns, after those of the outputs before it. */
typedef struct dr_linear_out {
    void *ptr;      /* [T][cols] in out_dtype (device, aligned to its elements) */
    int64_t stride; /* elements between tokens, at least cols */
    int32_t cols;   /* a multiple of 64 (whole heads) for all but the last */
} dr_linear_out;

#define DR_LINEAR_MAX_OUTS 4

/*
 * dr_linear -- matrix product of tokens with a weight matrix, and what follows
 * it in a decoder layer: bias, activation, gating, residual.
 *
 *   a[t][n]   = sum_k x[t][k] * W[n][k] + bias[n]
 *   v[t][n]   = act(a[t][n]), or act(a[t][n]) * a[t][N + n] when gated
 *   out[t][n] = residual[t][n] + v[t][n]
 * Sums and everything after them are fp32, rounded once to out_dtype.  The
 * columns may go to several outputs in turn (queries, keys and values of a
 * merged projection).  Single steps, batches and prompts take kernels of their
 * own, chosen by T, K, N and gated.  The products run on the tensor cores, whose
 * sums are cut off rather than rounded (about 1e-9 of the value, towards zero,
 * per term of K): with fp32 outputs no such sum is longer than 512 terms, and
 * the sums are added in fp32.  A NaN or infinity in a token, weight row or
 * residual reaches that token's, column's or element's outputs and no others;
 * at a = -inf gelu, gelu_tanh and silu give their limit 0.  With outputs of
 * either type activations use the hardware's exponential and reciprocal (2 and
 * 1 units in the last place), and gelu a fit that is within 1e-6 of the tail
 * that it leaves of a: together within 5e-7 + 2^-21 |v|.
 *
 *   x        : [T][K] bf16 (device, 16-byte aligned), tokens x_stride elements apart (a multiple of 8, >= K)
 *   W        : [N][K] bf16, [2N][K] when gated (device, 16-byte aligned)
 *   opts     : nullable (no bias, activation or residual)
 *   T        : 1 .. 2^31 - 4096;  K : a multiple of 8, at most 2^24;  N : the columns of all outputs together, any number
 *              below 2^30
 *   outs     : n_outs (1 .. DR_LINEAR_MAX_OUTS) outputs, read on the host during the call; a residual takes a single
 *              one.  16-byte aligned pointers and strides make them faster, and so for the residual.  Outputs overlap
 *              neither each other nor x, W and bias (DR_ERR_INVALID_ARG where one starts in the place of another)
 *   err_flag : nullable device int32; DR_ERRF_TIMEOUT if a CTA's bounded pipeline wait gave up (its outputs are then
 *              not written)
 * Same inputs, sizes and device give the same bits from call to call.
 */
dr_status dr_linear(const void *x, int64_t x_stride, const void *W, const dr_linear_opts *opts, int T, int K, int N,
                    const dr_linear_out *outs, int n_outs, dr_dtype out_dtype, int32_t *err_flag, void *stream);

/*
 * dr_linear_stall_test -- TEST HOOK, never needed in use.  The same call as
 * dr_linear, except that the CTAs of output tile `stall_tile` never load their
 * first K chunk.  Their bounded waits then run out (after about 2 s):
 * DR_ERRF_TIMEOUT is ORed into *err_flag, that tile's outputs (and those of
 * tiles that the same CTAs would have taken after it) are left unwritten, and
 * every other output is written as by dr_linear.  Nothing faults or hangs, and
 * later calls on the same context work normally.
 *   DR_ERR_UNSUPPORTED where the call's kernel has no waits; DR_ERR_INVALID_ARG
 *   where there is no such tile; the rest as dr_linear.
 */
dr_status dr_linear_stall_test(const void *x, int64_t x_stride, const void *W, const dr_linear_opts *opts, int T, int K,
                               int N, const dr_linear_out *outs, int n_outs, dr_dtype out_dtype, int32_t *err_flag,
                               int stall_tile, void *stream);

/* Norms of dr_residual_norm. */
typedef enum dr_norm_kind {
    DR_NORM_NONE = 0,
    DR_NORM_LAYER = 1, /* (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * weight + bias */
    DR_NORM_RMS = 2    /* v / sqrt(mean(v^2) + eps) * weight + bias */
} dr_norm_kind;

/* A norm over the Dm elements of a token (read on the host during the call; the arrays are device pointers). */
typedef struct dr_norm {
    int32_t kind;       /* dr_norm_kind */
    float eps;          /* >= 0 and finite */
    const void *weight; /* nullable [Dm] bf16, 16-byte aligned (null: ones) */
    const void *bias;   /* nullable [Dm] bf16, 16-byte aligned (null: zeros) */
} dr_norm;

/*
 * dr_residual_norm -- what stands between one block of a decoder layer and the
 * next, in one pass: the norm after a block, its gate and residual scale, the
 * residual, and the norm before the next block.
 *
 *   h[t] = residual[t] + scale * gate[t] * post(x[t])
 *   y[t] = pre(h[t])
 * Each part may be left out: post or pre (null: nothing is normed), gate,
 * residual (h is then the rest), h or y (not written).  Statistics and all
 * arithmetic are fp32; layer norm takes its mean first and the squared
 * differences after.  A norm multiplies by its root's reciprocal, rounded: one
 * rounding more than a division by the root.  y comes from h before h is
 * rounded to its type.  A NaN or infinity stays in its token.
 *
 *   x        : [T][Dm] in x_dtype, tokens x_stride elements apart
 *   gate     : nullable bf16, [Dm] for all tokens (gate_stride 0) or [T][Dm] (gate_stride >= Dm)
 *   scale    : finite
 *   residual : nullable [T][Dm] in h_dtype;  h : nullable [T][Dm] in h_dtype, may be residual or x itself with the
 *              same stride and type
 *   y        : nullable [T][Dm] in y_dtype; may be x or residual itself with the same stride and type where h is not
 *              it; h and y are not both null
 *   T        : 1 .. 2^31 - 4096;  Dm : a multiple of 8, at most 16384 (DR_ERR_UNSUPPORTED above)
 * Pointers are device pointers, 16-byte aligned; strides are in elements, multiples of 16 bytes, at least Dm.  h and y
 * overlap the inputs and each other only as said.
 */
dr_status dr_residual_norm(const void *x, int64_t x_stride, dr_dtype x_dtype, const dr_norm *post, const void *gate,
                           int64_t gate_stride, float scale, const void *residual, int64_t residual_stride, void *h,
                           int64_t h_stride, dr_dtype h_dtype, const dr_norm *pre, void *y, int64_t y_stride,
                           dr_dtype y_dtype, int T, int Dm, void *stream);

/*
 * dr_plan_splits -- host-only query: how many CTAs (one thread-block
 * cluster) share each (b, h) row of an attention call with this batch,
 * head count, length bound and KV storage type (DR_KV_BF16 or
 * DR_KV_FP8_E4M3; the description-encoder rows of dr_decode_cross_attn are
 * DR_KV_BF16) on a GPU with num_sms SMs.  Each CTA of the cluster takes an
 * equal run of whole 16-key blocks of the row.  The plan: at most 256 KiB
 * of K+V per CTA at the longest row, at least 6 CTAs per SM when the rows
 * alone are fewer, at least 64 keys per CTA, at most 8 CTAs -- or 16 (a
 * non-portable cluster) when 8 would each take at least 256 keys and 16 per
 * row come to at most 2 CTAs per SM (a few long rows: batch 1).  Pure
 * arithmetic; touches no device.  Returns 1 for non-positive sizes or an
 * unknown kv_dtype.
 */
int dr_plan_splits(int B, int H, int max_len, int kv_dtype, int num_sms);

/* Static, NUL-terminated description of a status code. */
const char *dr_status_string(dr_status s);

#ifdef __cplusplus
}
#endif

#endif /* DR_API_H */
