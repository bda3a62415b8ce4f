/*
 * kvattn.h -- C ABI of the kvattn decode-attention library (NVIDIA B200, sm_100a).
 *
 * One decode step of attention for a batch of sequences: every sequence contributes
 * one query token, which attends to all of that sequence's cached keys and values.
 * Two forms share the library:
 *
 *  - kvattn_gqa_decode: multi-head (MHA), grouped-query (GQA) and multi-query (MQA)
 *    attention.  n_kv_heads KV heads are each shared by a group of
 *    g = n_q_heads / n_kv_heads consecutive query heads; query head h reads KV head
 *    h / g.  ("Attention variants: MQA, GQA, and MLA", sections "MQA: one KV head for
 *    everyone" and "GQA: interpolating with groups"; "Grouped-Query Attention: Fewer
 *    KV Heads, Same Quality", section "Writing the formula explicitly", where the
 *    1-based group index ceil(i * n_kv / n_q) is this h / g with 0-based indices.)
 *
 *  - kvattn_mla_decode: absorbed multi-head latent attention.  The key up-projection
 *    is already folded into the query, every head scores the one cached latent per
 *    token plus a decoupled RoPE key, and the output stays in latent space (the
 *    value up-projection is applied by the caller).  ("Attention variants: MQA, GQA,
 *    and MLA", section "MLA: cache a latent, not the keys and values".)
 *
 * For serving there are, besides (documented at their declarations): a cache written with a
 * scale per row, its read back and the decode over it (kvattn_rope_append_rowscale,
 * kvattn_gather_rowscale, kvattn_gqa_decode_rowscale), decode of a batch behind a shared
 * prefix (kvattn_gqa_decode_prefix), and the verification of drafted tokens
 * (kvattn_verify_drafts).
 *
 * For each sequence b and query head h, with T = seq_lens[b] and scaled scores
 * s_t (t < T), the two forms write
 *      out[b, h, :] = sum_t softmax(s)_t * value_t       (fp32)
 *      lse[b, h]    = log(sum_t exp(s_t))                 (fp32, natural log)
 * An empty sequence (T == 0) gives out = 0 and lse = -inf.
 *
 * Conventions for every entry point:
 *  - Pointers marked "device" must point to memory of the device that is current on
 *    the calling host thread; "host" pointers to host memory.  The library never
 *    frees, retains or reallocates caller memory.
 *  - bf16 data is passed as uint16_t bit patterns (IEEE bfloat16).
 *  - All arrays are dense and row-major in the shape given (last index fastest).
 *  - Every device pointer must be 16-byte aligned (else KVATTN_ERR_MISALIGNED).
 *  - out and lse are fully overwritten and must not overlap any input.
 *  - stream is a cudaStream_t (NULL = the legacy default stream).  The call only
 *    enqueues work: KVATTN_OK means the kernels were launched; their completion is
 *    observed through the stream.  Arguments are checked on the host before any work
 *    is enqueued; an argument error launches nothing.
 *  - Functions never throw or abort; they return a kvattn_status.
 *  - Scratch memory: the library keeps one workspace per device, grown with
 *    cudaMalloc when a call needs more than it holds and kept until
 *    kvattn_release_workspace(), and the outgrown ones too: captured graphs may use
 *    them.  A call that grows it is not capturable in a CUDA
 *    graph; issue one call of the largest shape before capturing.  A captured decode
 *    call may be replayed any number of times: its kernels derive the work split from
 *    the device-side seq_lens at every launch, so the lengths (not the shapes or
 *    pointers) may change between replays.  Calls that share a device must be ordered
 *    (same stream, or synchronised): they share the workspace.  That holds for the
 *    row-scaled decode too; the appends, kvattn_gather_rowscale and kvattn_verify_drafts
 *    use no workspace and the prefix decode the caller's, so that they may run beside
 *    other calls.
 *  - Thread safety: entry points may be called from several host threads; the
 *    workspace is guarded by a mutex, but see the ordering rule above.
 */
#ifndef KVATTN_H
#define KVATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KVATTN_VERSION 10000 /* major * 10000 + minor * 100 + patch */

typedef enum {
    KVATTN_OK = 0,
    KVATTN_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, n_q % n_kv != 0, non-finite scale, overlap */
    KVATTN_ERR_UNSUPPORTED = 2, /* valid but not implemented: head_dim, latent/rope width, size limits */
    KVATTN_ERR_MISALIGNED = 3,  /* a pointer is not 16-byte aligned */
    KVATTN_ERR_CUDA = 4,        /* a CUDA runtime call failed (see kvattn_last_error_detail) */
    KVATTN_ERR_NO_MEMORY = 5    /* the workspace could not be allocated */
} kvattn_status;

/*
 * GQA / MQA / MHA decode.
 *   q         device bf16 [batch, n_q_heads, head_dim]   one query token per sequence
 *   k_cache   device bf16 [batch, n_kv_heads, max_seq_len, head_dim]
 *   v_cache   device bf16 [batch, n_kv_heads, max_seq_len, head_dim]
 *             (the pages' cache layout (batch, kv_heads, seq, head_dim), "The KV cache
 *             bill, worked numerically"; positions >= seq_lens[b] are never read)
 *   seq_lens  device int32 [batch]   tokens cached for each sequence, 0..max_seq_len;
 *             values outside that range are clamped on the device (the result for such
 *             a sequence is then unspecified, but no memory outside the caches is read)
 *   max_seq_len  cache capacity per sequence (the T stride of the caches), >= 1
 *   batch, n_q_heads, n_kv_heads   > 0, n_q_heads % n_kv_heads == 0, batch <= 4096
 *   head_dim  64 or 128 (others: KVATTN_ERR_UNSUPPORTED)
 *   scale     finite score scale (the pages use 1/sqrt(head_dim))
 *   out       device fp32 [batch, n_q_heads, head_dim]
 *   lse       device fp32 [batch, n_q_heads]  (required, natural log)
 *   stream    cudaStream_t
 * Limits: batch * n_kv_heads * max_seq_len < 2^31.
 */
int kvattn_gqa_decode(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                      const int32_t *seq_lens, int max_seq_len, int batch, int n_q_heads,
                      int n_kv_heads, int head_dim, float scale, float *out, float *lse,
                      void *stream);

/*
 * Absorbed MLA decode (DeepSeek shape: latent_dim 512, rope_dim 64).
 *   q_latent      device bf16 [batch, n_heads, latent_dim]  queries already multiplied
 *                 by the key up-projection (they score the latents directly)
 *   q_rope        device bf16 [batch, n_heads, rope_dim]    rotated decoupled-RoPE queries
 *   latent_cache  device bf16 [batch, max_seq_len, latent_dim]  one latent per token,
 *                 shared by all heads; it is both key (with the RoPE part) and value
 *   rope_cache    device bf16 [batch, max_seq_len, rope_dim]    rotated RoPE keys
 *   seq_lens      device int32 [batch], as for kvattn_gqa_decode
 *   max_seq_len   cache capacity per sequence, >= 1
 *   batch         > 0, <= 1024;  n_heads 1..128
 *   latent_dim    512;  rope_dim 64 (others: KVATTN_ERR_UNSUPPORTED)
 *   scale         finite score scale (DeepSeek: 1/sqrt(128 + 64))
 *   out           device fp32 [batch, n_heads, latent_dim]  (latent space)
 *   lse           device fp32 [batch, n_heads]
 * Score of head h at token t: scale * (q_latent[h] . latent_t + q_rope[h] . rope_t).
 * Every bf16 value is accepted as is (no narrower intermediate format): the weights
 * enter the value product as a bf16 high part plus a bf16 remainder.
 */
int kvattn_mla_decode(const uint16_t *q_latent, const uint16_t *q_rope,
                      const uint16_t *latent_cache, const uint16_t *rope_cache,
                      const int32_t *seq_lens, int max_seq_len, int batch, int n_heads,
                      int latent_dim, int rope_dim, float scale, float *out, float *lse,
                      void *stream);

/*
 * Several new tokens per sequence in one call (multi-token decode: verifying drafted
 * tokens, or a short prompt continuation), with the causal mask of "Attention variants:
 * MQA, GQA, and MLA", section "Implementation, twice" (a query never sees a later
 * token), and optionally a sliding window (the Mistral-style window named in
 * "Grouped-Query Attention: Fewer KV Heads, Same Quality").
 *   q         device bf16 [batch, q_len, n_q_heads, head_dim]: the q_len newest tokens'
 *             queries, oldest first
 *   k_cache, v_cache, seq_lens, max_seq_len: as for kvattn_gqa_decode; the cache already
 *             holds the q_len new tokens at positions seq_lens[b] - q_len .. seq_lens[b] - 1
 *   window    0: no window; w > 0: query i, at position p = seq_lens[b] - q_len + i,
 *             attends to positions p - w < t <= p only (its last w tokens, itself included);
 *             otherwise to all t <= p.  Tiles wholly before the earliest visible position
 *             are not read.
 *   out       device fp32 [batch, q_len, n_q_heads, head_dim];  lse fp32 [batch, q_len, n_q_heads]
 * A query with no visible position (p < 0) gets out = 0 and lse = -inf.  Cached values of the
 * newest q_len tokens have to be finite for all of them, and with a window so do those from
 * the 128 positions before the earliest visible one on: a weight of zero does not hide NaN.
 * q_len == 1 and window == 0 is exactly kvattn_gqa_decode.  head_dim 64 or 128; a window needs head_dim
 * 128 and n_q_heads / n_kv_heads <= 64; batch * q_len <= 4096 (KVATTN_ERR_UNSUPPORTED
 * otherwise).  With head_dim 128 and (n_q_heads / n_kv_heads) * q_len <= 64 one kernel
 * scores a group's heads at all q_len positions against each cache tile; otherwise the
 * call runs as batch * q_len single-token sequences (query i of sequence b is a sequence
 * of length seq_lens[b] - q_len + 1 + i over b's cache rows), which reads the cache once
 * per new token (the repeats mostly from L2).
 */
int kvattn_gqa_decode_multi(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                            const int32_t *seq_lens, int max_seq_len, int batch, int q_len,
                            int n_q_heads, int n_kv_heads, int head_dim, float scale, int window,
                            float *out, float *lse, void *stream);

/*
 * Decode over a quantised (fp8) KV cache.  The pages list quantised caches among what the
 * libraries build around the attention module ("Attention variants: MQA, GQA, and MLA",
 * section "Against the real libraries"); at one byte per cached value the cache a decode
 * step reads halves.  The format is E4M3 (1 sign, 4 exponent bits with bias 7, 3
 * mantissa bits; largest finite magnitude 448; codes 0x7F / 0xFF are NaN) with one
 * float scale per cache tensor: the cached key is value(code) * k_scale, the value
 * value(code) * v_scale.  The result is attention on those dequantised values, as
 * kvattn_gqa_decode_multi computes it (q_len = 1, window = 0: kvattn_gqa_decode).
 *   q           device bf16 [batch, q_len, n_q_heads, head_dim]
 *   k_cache, v_cache  device E4M3 codes (one byte each)
 *               [batch, n_kv_heads, max_seq_len, head_dim]
 *   k_scale, v_scale  finite, > 0
 *   out, lse    device fp32 [batch, q_len, n_q_heads, head_dim], [batch, q_len, n_q_heads]
 * head_dim must be 128 and n_q_heads / n_kv_heads <= 64 (else KVATTN_ERR_UNSUPPORTED);
 * everything else as for kvattn_gqa_decode_multi.  The query
 * and the softmax weights enter the tensor-core products as two E4M3 parts each (~8
 * significant bits), the codes exactly; accumulation is fp32.  Codes past a sequence's
 * length are never read.
 */
int kvattn_gqa_decode_fp8(const uint16_t *q, const uint8_t *k_cache, const uint8_t *v_cache,
                          const int32_t *seq_lens, int max_seq_len, int batch, int q_len,
                          int n_q_heads, int n_kv_heads, int head_dim, float scale, float k_scale,
                          float v_scale, int window, float *out, float *lse, void *stream);

/*
 * kvattn_gqa_decode_fp8 for one new token per sequence over a paged E4M3 cache:
 * k_pages, v_pages [num_pages, n_kv_heads, page_size, head_dim] codes, block_table and
 * seq_lens as for kvattn_gqa_decode_paged, page_size a multiple of 128; q [batch,
 * n_q_heads, head_dim] bf16, out [batch, n_q_heads, head_dim], lse [batch, n_q_heads].
 */
int kvattn_gqa_decode_fp8_paged(const uint16_t *q, const uint8_t *k_pages, const uint8_t *v_pages,
                                const int32_t *block_table, const int32_t *seq_lens, int num_pages,
                                int page_size, int max_pages_per_seq, int batch, int n_q_heads,
                                int n_kv_heads, int head_dim, float scale, float k_scale, float v_scale,
                                float *out, float *lse, void *stream);

/*
 * kvattn_mla_decode over an E4M3 (fp8) latent cache, the MLA form of
 * kvattn_gqa_decode_fp8 (same format; the pages list quantised caches among what the
 * libraries add, "Attention variants: MQA, GQA, and MLA", section "Against the real
 * libraries").  The cached latent of token t is value(latent_cache[b, t, :]) *
 * latent_scale -- the key's latent part and the value alike -- and its RoPE key
 * value(rope_cache[b, t, :]) * rope_scale; the result is kvattn_mla_decode on those
 * dequantised rows.
 *   q_latent, q_rope  device bf16 [batch, n_heads, 512], [batch, n_heads, 64]
 *   latent_cache, rope_cache  device E4M3 codes [batch, max_seq_len, 512],
 *                     [batch, max_seq_len, 64] (one byte each)
 *   latent_scale, rope_scale  finite, > 0
 *   out, lse    device fp32 [batch, n_heads, 512], [batch, n_heads]
 * Everything else, the results' layout and the errors as for kvattn_mla_decode.  The
 * query (each head's, after scaling by a power of two that puts its largest magnitude in
 * [128, 256)) and the softmax weights enter the tensor-core products as an E4M3 high part
 * plus an E4M3 remainder (~8 significant bits), the codes exactly; accumulation is fp32.
 * Codes past a sequence's length are never read.
 */
int kvattn_mla_decode_fp8(const uint16_t *q_latent, const uint16_t *q_rope, const uint8_t *latent_cache,
                          const uint8_t *rope_cache, const int32_t *seq_lens, int max_seq_len, int batch,
                          int n_heads, int latent_dim, int rope_dim, float scale, float latent_scale,
                          float rope_scale, float *out, float *lse, void *stream);

/*
 * Several new tokens per sequence for absorbed MLA (the causal mask as for
 * kvattn_gqa_decode_multi; no window): query i of sequence b, at position
 * p = seq_lens[b] - q_len + i, attends to the cached tokens t <= p.
 *   q_latent, q_rope  device bf16 [batch, q_len, n_heads, 512], [batch, q_len, n_heads, 64]
 *   latent_cache, rope_cache  device [batch, max_seq_len, 512], [batch, max_seq_len, 64]:
 *             bf16 (e4m3 == 0) or E4M3 codes with latent_scale / rope_scale as for
 *             kvattn_mla_decode_fp8 (e4m3 != 0; the scales are ignored otherwise)
 *   out, lse  device fp32 [batch, q_len, n_heads, 512], [batch, q_len, n_heads]
 * A query with no visible position gets out = 0 and lse = -inf.  batch * q_len <= 1024.
 * The call runs as batch * q_len single-token sequences over b's cache rows (the cache
 * read once per new token, the repeats mostly from L2); q_len == 1 is kvattn_mla_decode
 * (kvattn_mla_decode_fp8).  Everything else as for kvattn_mla_decode.
 */
int kvattn_mla_decode_multi(const uint16_t *q_latent, const uint16_t *q_rope, const void *latent_cache,
                            const void *rope_cache, const int32_t *seq_lens, int max_seq_len, int batch, int q_len,
                            int n_heads, int latent_dim, int rope_dim, float scale, int e4m3, float latent_scale,
                            float rope_scale, float *out, float *lse, void *stream);

/*
 * kvattn_mla_decode_fp8 over a paged cache: latent_pages [num_pages, page_size, 512] and
 * rope_pages [num_pages, page_size, 64] E4M3 codes, block_table and seq_lens as for
 * kvattn_gqa_decode_paged, page_size a multiple of 64.
 */
int kvattn_mla_decode_fp8_paged(const uint16_t *q_latent, const uint16_t *q_rope, const uint8_t *latent_pages,
                                const uint8_t *rope_pages, const int32_t *block_table, const int32_t *seq_lens,
                                int num_pages, int page_size, int max_pages_per_seq, int batch, int n_heads,
                                int latent_dim, int rope_dim, float scale, float latent_scale, float rope_scale,
                                float *out, float *lse, void *stream);

/*
 * kvattn_gqa_decode over a paged KV cache: the cache is a pool of pages and each
 * sequence lists its pages in a block table (the serving-engine layout the pages name,
 * "Attention variants: MQA, GQA, and MLA", section "Against the real libraries": vLLM's
 * PagedAttention).  Token t of sequence b lives in page block_table[b][t / page_size],
 * row t % page_size.
 *   k_pages, v_pages  device bf16 [num_pages, n_kv_heads, page_size, head_dim]
 *   block_table       device int32 [batch, max_pages_per_seq]: physical page of each
 *                     logical page; entries past a sequence's last page are not read.
 *                     Every entry that is read must lie in [0, num_pages).
 *   seq_lens          device int32 [batch], 0 <= len <= max_pages_per_seq * page_size
 *   page_size         a multiple of 64 (the tensor-core kernel for groups of >= 4 heads
 *                     runs when it is a multiple of 128; otherwise the warp-level kernel)
 * Everything else, the results and the errors are those of kvattn_gqa_decode.  Rows
 * of a sequence's last page past its length are never read.
 */
int kvattn_gqa_decode_paged(const uint16_t *q, const uint16_t *k_pages, const uint16_t *v_pages,
                            const int32_t *block_table, const int32_t *seq_lens, int num_pages,
                            int page_size, int max_pages_per_seq, int batch, int n_q_heads,
                            int n_kv_heads, int head_dim, float scale, float *out, float *lse,
                            void *stream);

/*
 * kvattn_mla_decode over a paged latent cache: latent_pages [num_pages, page_size,
 * latent_dim] and rope_pages [num_pages, page_size, rope_dim] bf16, block_table and
 * seq_lens as for kvattn_gqa_decode_paged; page_size a multiple of 64.  Everything else
 * as for kvattn_mla_decode.
 */
int kvattn_mla_decode_paged(const uint16_t *q_latent, const uint16_t *q_rope,
                            const uint16_t *latent_pages, const uint16_t *rope_pages,
                            const int32_t *block_table, const int32_t *seq_lens, int num_pages,
                            int page_size, int max_pages_per_seq, int batch, int n_heads,
                            int latent_dim, int rope_dim, float scale, float *out, float *lse,
                            void *stream);

/*
 * The step either side of the decode: rotary position embedding (RoPE) of the new
 * token's query and key, and the append of its key and value to the cache at its
 * position.  The pages rotate queries and keys before they meet the cache and write the
 * new token to the cache before attending ("Attention variants: MQA, GQA, and MLA",
 * section "MLA: cache a latent, not the keys and values"); the rotation itself is the
 * textbook one: pair i of a head_dim-wide vector at position p turns by the angle
 * p * rope_base^(-2i / head_dim), the pairs being (2i, 2i+1) when interleaved != 0 and
 * (i, i + head_dim/2) otherwise.  The angle is formed in fp64; results are rounded to
 * bf16 once.
 *   q          device bf16 [batch, n_q_heads, head_dim]: rotated in place
 *   k_new      device bf16 [batch, n_kv_heads, head_dim]: the new token's keys (not
 *              rotated); their rotation goes to k_cache[b, j, positions[b], :]
 *   v_new      device bf16 [batch, n_kv_heads, head_dim]: copied to
 *              v_cache[b, j, positions[b], :]
 *   positions  device int32 [batch]: the new token's position (its index in the cache).
 *              A position outside [0, max_seq_len) writes nothing into the caches (q is
 *              still rotated with it).  The caller's seq_lens for the following decode
 *              are positions + 1.
 *   k_cache, v_cache  device bf16 [batch, n_kv_heads, max_seq_len, head_dim]
 *   head_dim   even, <= 1024;  rope_base > 0 and finite (e.g. 10000)
 * Errors as for kvattn_gqa_decode; q and the caches must not overlap each other or the
 * inputs.  Asynchronous on `stream`.
 */
int kvattn_rope_append(uint16_t *q, const uint16_t *k_new, const uint16_t *v_new,
                       const int32_t *positions, uint16_t *k_cache, uint16_t *v_cache,
                       int max_seq_len, int batch, int n_q_heads, int n_kv_heads, int head_dim,
                       float rope_base, int interleaved, void *stream);

/*
 * kvattn_rope_append into an E4M3 (fp8) cache, the producer side of
 * kvattn_gqa_decode_fp8: q is rotated in place (bf16) as above; the new token's rotated
 * key is stored as E4M3 codes of key / k_scale and its value as codes of value /
 * v_scale (the quotient taken in fp32, correctly rounded; the nearest code, ties to
 * even, magnitudes past 448 saturated to +-448, NaN to the NaN code), so that the
 * cached value is code * scale as the decode reads it.
 *   k_cache, v_cache  device E4M3 codes [batch, n_kv_heads, max_seq_len, head_dim]
 *   k_scale, v_scale  finite, > 0 (the scales the cache was quantised with)
 * Everything else, including positions outside the cache, as for kvattn_rope_append.
 */
int kvattn_rope_append_fp8(uint16_t *q, const uint16_t *k_new, const uint16_t *v_new,
                           const int32_t *positions, uint8_t *k_cache, uint8_t *v_cache,
                           int max_seq_len, int batch, int n_q_heads, int n_kv_heads, int head_dim,
                           float rope_base, int interleaved, float k_scale, float v_scale,
                           void *stream);

/*
 * The same for absorbed MLA: q_rope [batch, n_heads, rope_dim] is rotated in place, the
 * new token's decoupled rotary key rope_new [batch, rope_dim] is rotated into
 * rope_cache[b, positions[b], :], and its latent latent_new [batch, latent_dim] is
 * copied (unrotated: the latent carries no position) into latent_cache[b, positions[b], :]
 * ("Attention variants: MQA, GQA, and MLA", section "MLA: cache a latent, not the keys
 * and values").  latent_dim and rope_dim even; the rest as for kvattn_rope_append.
 */
int kvattn_mla_rope_append(uint16_t *q_rope, const uint16_t *latent_new, const uint16_t *rope_new,
                           const int32_t *positions, uint16_t *latent_cache, uint16_t *rope_cache,
                           int max_seq_len, int batch, int n_heads, int latent_dim, int rope_dim,
                           float rope_base, int interleaved, void *stream);

/*
 * kvattn_mla_rope_append into an E4M3 cache, the producer side of kvattn_mla_decode_fp8:
 * q_rope is rotated in place (bf16); the rotated RoPE key is stored as E4M3 codes of
 * key / rope_scale and the latent as codes of latent / latent_scale (the quotient taken
 * in fp32, correctly rounded; nearest code, ties to even, saturated at 448, NaN to the
 * NaN code), as kvattn_rope_append_fp8 encodes.
 *   latent_cache, rope_cache  device E4M3 codes [batch, max_seq_len, latent_dim],
 *                             [batch, max_seq_len, rope_dim]
 *   latent_scale, rope_scale  finite, > 0
 * Everything else as for kvattn_mla_rope_append.
 */
int kvattn_mla_rope_append_fp8(uint16_t *q_rope, const uint16_t *latent_new, const uint16_t *rope_new,
                               const int32_t *positions, uint8_t *latent_cache, uint8_t *rope_cache,
                               int max_seq_len, int batch, int n_heads, int latent_dim, int rope_dim,
                               float rope_base, int interleaved, float latent_scale, float rope_scale,
                               void *stream);

/*
 * A paged E4M3 cache with one scale per cached row.
 *
 * A row is one token's key (or value) of one KV head.  Its scale comes from the row itself,
 *     scale = a / 448,  a = max(max_i |y_i|, 2^-55),   code_i = E4M3(y_i * (448 / a))
 * (nearest, ties to even, saturated; a is at most the largest finite float, NaN elements are
 * passed over in a and become the NaN code), and the cached value is code_i * scale.  So a
 * cache is quantised as it is written, without calibrated tensor scales, and an outlier token
 * costs no other token precision.  ("Attention variants: MQA, GQA, and MLA", section "Against
 * the real libraries", names quantised caches and paged caches; the pages give no format.)
 *   k_pages, v_pages    device E4M3 codes [num_pages, n_kv_heads, page_size, head_dim]
 *   k_scales, v_scales  device fp32 [num_pages, n_kv_heads, page_size]
 *   a slot              page * page_size + row
 *   num_pages * n_kv_heads * page_size < 2^31
 *
 * kvattn_rope_append_rowscale writes n_tokens new tokens of any sequences (one each in a
 * decode step, a whole prompt in a prefill) and rotates their queries and keys:
 *   q          device bf16 [n_tokens, n_q_heads, head_dim], or NULL (then q_out is NULL and
 *              n_q_heads 0); the rotated queries go to q_out (same shape), which may be q itself
 *              with the same stride (in place)
 *   k_new, v_new  device bf16 [n_tokens, n_kv_heads, head_dim]
 *   *_stride   elements from one token to the next (a multiple of 8, at least the token's
 *              own elements): slices of a fused projection are read in place
 *   positions  device int32 [n_tokens]: the angle's position; NULL allowed without rotation
 *   slots      device int64 [n_tokens]: where each token goes; a slot outside the pool (such
 *              as -1) is not written (its query is still rotated).  Slots must be distinct:
 *              a slot given twice holds a mixture of its tokens afterwards.
 *   rope_base  as for kvattn_rope_append; 0: no rotation (q is copied to q_out)
 *   head_dim   a multiple of 16, <= 256
 * The angle is formed in fp64 and the scales and codes from the fp32 rotated values.
 * n_tokens may be 0 (nothing is launched).  q_out, the pools and the scales must not overlap
 * each other or the inputs (but for q in place).  Rows of one stride that lie between each
 * other, as q_out's between the keys and values of a fused projection, do not overlap.
 */
int kvattn_rope_append_rowscale(const uint16_t *q, const uint16_t *k_new, const uint16_t *v_new,
                                const int32_t *positions, const int64_t *slots, uint16_t *q_out, uint8_t *k_pages,
                                uint8_t *v_pages, float *k_scales, float *v_scales, int n_tokens, int n_q_heads,
                                int n_kv_heads, int head_dim, int64_t q_stride, int64_t q_out_stride, int64_t k_stride,
                                int64_t v_stride, int num_pages, int page_size, float rope_base, int interleaved,
                                void *stream);

/*
 * Reads rows of a row-scaled cache back to bf16 (code * scale, rounded once):
 *   slots         device int64 [n_tokens]; a slot outside the pool gives a row of zeros
 *   k_out, v_out  device bf16 [n_kv_heads, n_tokens, head_dim], heads k_head_stride /
 *                 v_head_stride elements apart (a multiple of 8): the layout
 *                 kvattn_gqa_decode_prefix takes its prefix in, and a part of a longer one; they
 *                 must not overlap the inputs or each other (heads that alternate in one
 *                 buffer do not)
 * head_dim a multiple of 16, <= 256.  n_tokens may be 0.
 */
int kvattn_gather_rowscale(const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scales, const float *v_scales,
                           const int64_t *slots, uint16_t *k_out, uint16_t *v_out, int n_tokens, int n_kv_heads,
                           int head_dim, int64_t k_head_stride, int64_t v_head_stride, int num_pages, int page_size,
                           void *stream);

/*
 * Decode over a row-scaled cache, the form of kvattn_gqa_decode_fp8 (several new tokens and a
 * window included) with a scale per row: s_t = scale * k_scale_t (q . kcode_t),
 * out = sum_t softmax(s)_t v_scale_t vcode_t.
 *   q            device bf16 [batch, q_len, n_q_heads, head_dim]
 *   block_table  device int32 [batch, max_pages_per_seq] as for kvattn_gqa_decode_paged, or NULL:
 *                a contiguous cache, one page a sequence (num_pages = batch,
 *                max_pages_per_seq = 1, page_size = the capacity)
 *   out          device bf16 [batch, q_len, n_q_heads, head_dim], rounded once: the type the
 *                output projection reads;  lse fp32 [batch, q_len, n_q_heads]
 * The codes and the query enter the tensor-core products in f16 (the codes exactly, the query
 * times a power of two), the softmax weights times their token's value scale in f16 relative to
 * the unit's largest (11 significant bits); accumulation is fp32.
 * head_dim 128, n_q_heads / n_kv_heads <= 64, page_size a multiple of 128 (paged); batch *
 * q_len <= 4096.  A page outside the pool reads as rows of zeros.  Scales from 2^-40 to 2^40
 * keep full precision.  Codes and scales past a sequence's length are never read into a result,
 * and neither are those of positions that a query must not see (before its window; newer
 * tokens than it): NaN there leaves its result alone.  Everything else as for
 * kvattn_gqa_decode_fp8.
 */
int kvattn_gqa_decode_rowscale(const uint16_t *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scales,
                               const float *v_scales, const int32_t *block_table, const int32_t *seq_lens, int num_pages,
                               int page_size, int max_pages_per_seq, int batch, int q_len, int n_q_heads, int n_kv_heads,
                               int head_dim, float scale, int window, uint16_t *out, float *lse, void *stream);

/*
 * Decode for a batch whose sequences share a prefix: every new token attends to the same
 * prefix tokens and then, causally, to its own sequence's cache.  The prefix is read once for
 * every 256 query rows of a KV head (all sequences' rows make one matrix product with it), not
 * once per sequence.
 *   q          device bf16 [batch, q_len, n_q_heads, head_dim], the newest tokens, oldest first
 *   k_prefix, v_prefix  device bf16 [n_kv_heads, max_prefix_len, head_dim]
 *   prefix_len device int32 [1], 0..max_prefix_len (clamped): tokens of the shared prefix
 *   k_cache, v_cache  device bf16 [batch, n_kv_heads, max_seq_len, head_dim]: each sequence's
 *              own tokens, which follow the prefix
 *   seq_lens   device int32 [batch]: own tokens, the q_len new ones included, 0..max_seq_len
 *              (clamped).  Query i of sequence b attends to the whole prefix and to own
 *              positions t <= seq_lens[b] - q_len + i (none where that is negative).
 *   out        device bf16 [batch, q_len, n_q_heads, head_dim];  lse fp32 [batch, q_len,
 *              n_q_heads] over prefix and own tokens.  A query with nothing to attend to
 *              (prefix_len 0 and no own token) gets out = 0 and lse = -inf.
 *   workspace  device, 16-byte aligned, at least the bytes that
 *              kvattn_gqa_decode_prefix_workspace gives for the same sizes: scratch of this one
 *              call, never kept.  Calls that may run at the same time (other streams, other
 *              captured graphs) need a workspace each; the library allocates nothing.
 *   head_dim 64 or 128; (n_q_heads / n_kv_heads) * q_len <= 128; batch * q_len <= 4096;
 *   batch * n_kv_heads * max_seq_len and n_kv_heads * max_prefix_len < 2^31, and fewer than
 *   about 2^27 tiles of 128 tokens in all, the prefix's counted for every 256 rows.
 * The softmax weights enter the value products as bf16 (8 significant bits; kvattn_gqa_decode
 * keeps about 16 of them in two parts); sums and outputs accumulate in fp32, for cached values
 * of up to 2^80 in size.  Rows at or past prefix_len and seq_lens[b] are never read into a
 * result.  With q_len > 1 a new token's cached value has to be finite also for the older new
 * tokens, which give it weight zero.
 *
 * kvattn_gqa_decode_prefix_paged takes prefix and own tokens from one page pool:
 *   k_pages, v_pages  device bf16 [num_pages, n_kv_heads, page_size, head_dim], page_size a
 *              multiple of 128
 *   prefix_table  device int32 [max_prefix_pages], the prefix's pages;  block_table device
 *              int32 [batch, max_pages_per_seq], each sequence's own pages (after the prefix).
 *              A page outside the pool reads as zeros.
 * Its workspace is that of max_prefix_len = max_prefix_pages * page_size and max_seq_len =
 * max_pages_per_seq * page_size.
 */
int kvattn_gqa_decode_prefix_workspace(int max_prefix_len, int max_seq_len, int batch, int q_len, int n_q_heads,
                                       int n_kv_heads, int head_dim, size_t *bytes);
int kvattn_gqa_decode_prefix(const uint16_t *q, const uint16_t *k_prefix, const uint16_t *v_prefix,
                             const int32_t *prefix_len, int max_prefix_len, const uint16_t *k_cache,
                             const uint16_t *v_cache, const int32_t *seq_lens, int max_seq_len, int batch, int q_len,
                             int n_q_heads, int n_kv_heads, int head_dim, float scale, uint16_t *out, float *lse,
                             void *workspace, size_t workspace_bytes, void *stream);
int kvattn_gqa_decode_prefix_paged(const uint16_t *q, const uint16_t *k_pages, const uint16_t *v_pages,
                                   const int32_t *prefix_table, const int32_t *prefix_len, int max_prefix_pages,
                                   const int32_t *block_table, const int32_t *seq_lens, int num_pages, int page_size,
                                   int max_pages_per_seq, int batch, int q_len, int n_q_heads, int n_kv_heads,
                                   int head_dim, float scale, uint16_t *out, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream);

/*
 * Verification of drafted tokens (speculative sampling): which of a sequence's drafts the
 * target model's probabilities accept, and the token that follows them, from random numbers
 * of the caller.  The step after kvattn_gqa_decode_multi (or a prefix / row-scaled decode)
 * has scored the drafts.
 * Draft i (token x, target probabilities p_i, draft probabilities q_i) is accepted while
 * u_accept[b, i] * q_i(x) < p_i(x).  At the first refusal n the next token is drawn from
 * max(p_n - q_n, 0), normalised (from p_n where that is zero everywhere); with all of the
 * sequence's drafts accepted, from p_n with n = draft_lens[b].  The draw is the first token
 * v with sum_{w <= v} r_w > u_sample[b] * sum_w r_w; products and sums are taken in 64 bits.
 *   target_probs  device [batch, n_drafts + 1, vocab], fp32 (bf16 == 0) or bf16, vocabulary
 *                 contiguous, the other axes target_batch_stride / target_pos_stride elements
 *   draft_probs   device [batch, n_drafts, vocab] of the same type with its strides, or NULL:
 *                 point drafts (probability 1 at the drafted token, as a greedy or a lookup
 *                 draft has)
 *   draft_tokens  device int32 [batch, n_drafts]; one outside [0, vocab) is refused
 *   draft_lens    device int32 [batch], drafts of each sequence (clamped to 0..n_drafts), or
 *                 NULL: n_drafts each
 *   u_accept, u_sample  device fp32 [batch, n_drafts], [batch], uniform in [0, 1)
 *   accepted      device int32 [batch]: n
 *   tokens        device int32 [batch, n_drafts + 1]: the accepted drafts, the drawn token, -1
 * n_drafts may be 0 (then a plain draw from target_probs; draft_tokens and u_accept may be
 * NULL); n_drafts <= 1024, batch <= 4096, vocab <= 2^28.  Probabilities need not sum to one and
 * are not infinite; target entries of zero or less and NaN are never accepted or drawn, draft
 * entries below zero count as zero; a row without a positive entry gives token -1.
 * Rows whose strides and pointers are multiples of 16 bytes are read in vectors, others by
 * element.
 */
int kvattn_verify_drafts(const void *target_probs, const void *draft_probs, const int32_t *draft_tokens,
                         const int32_t *draft_lens, const float *u_accept, const float *u_sample, int32_t *accepted,
                         int32_t *tokens, int batch, int n_drafts, int vocab, int bf16, int64_t target_batch_stride,
                         int64_t target_pos_stride, int64_t draft_batch_stride, int64_t draft_pos_stride, void *stream);

/* Human-readable name of a kvattn_status value (static string, never NULL). */
const char *kvattn_status_string(int status);

/* Detail of the last KVATTN_ERR_CUDA / KVATTN_ERR_NO_MEMORY on this host thread. */
const char *kvattn_last_error_detail(void);

/* KVATTN_VERSION of the loaded library. */
int kvattn_version(void);

/* Frees the workspace of every device (waits for that device to be idle first).  Graphs that
 * captured calls are not to be replayed afterwards. */
void kvattn_release_workspace(void);

/*
 * Device-side error flags of the current device.  Every wait inside the kernels is
 * bounded; a wait that runs out sets a bit here and the kernel returns early (its
 * output is then invalid).  Bit 0: pipeline data wait, bit 1: pipeline slot wait,
 * bit 2: cluster peer wait, bit 3: tensor-core completion wait.  Reading synchronises
 * the device.  Returns a kvattn_status; *flags receives the bits.
 */
int kvattn_read_device_flags(unsigned int *flags);
int kvattn_clear_device_flags(void);

/*
 * Kernels this library has launched (enqueued successfully) from the calling host thread
 * since the library was loaded: a decode call adds one (the decode kernel), or two when a
 * combine kernel merges units cut between workers, plus one when several new tokens run
 * as a virtual batch; an append, a read back and a verification add one; a prefix decode adds
 * two (decode and merge), or three where the batch is above 640 sequences.  Read it before and
 * after a call to count that call's kernels.
 */
unsigned long long kvattn_kernel_launches(void);

/*
 * Test hook for the bounded waits: launches one CTA on `stream` (a cudaStream_t, NULL:
 * the default stream) whose thread waits, with the same bounded wait the kernels use but
 * cut to about limit_us microseconds of SM clock (1 .. 1000000), for a shared-memory
 * barrier that nothing completes.  The wait runs out, sets bit 0 of the device flags and
 * the kernel returns: no fault, no trap, the context stays usable.  Returns
 * KVATTN_ERR_INVALID_ARG for a limit out of range, else the launch status.
 */
int kvattn_debug_wait_probe(int limit_us, void *stream);

/*
 * Test and tuning knob (process-wide): when workers > 0 the next calls use exactly
 * that many workers (CTAs or CTA pairs) and at least min_tiles tiles per worker,
 * which forces the split/combine path on small inputs.  workers == 0 restores the
 * built-in heuristic.
 */
void kvattn_debug_set_workers(int workers, int min_tiles);

/*
 * Test and tuning knob (process-wide): which kernel kvattn_gqa_decode runs.
 *   0  built-in choice (the tensor-memory kernel for head_dim 128 and groups of at
 *      least 4 query heads, the warp-level kernel otherwise)
 *   1  always the warp-level MMA kernel
 *   2  always the tensor-memory (tcgen05) kernel; calls it cannot serve (head_dim 64,
 *      or a batch too large for its shared memory) return KVATTN_ERR_UNSUPPORTED
 * Other values mean 0.  kvattn_gqa_decode_noalloc always runs the warp-level kernel.
 */
void kvattn_debug_set_gqa_kernel(int which);

/*
 * kvattn_gqa_decode without any allocation by the library.  The pages have no
 * counterpart to this call; it exists for callers that must not have a library call
 * cudaMalloc: serving engines that reserve nearly all device memory for their own
 * KV-cache pool (a stray allocation can fail or fragment it), and loops that cannot
 * afford cudaMalloc's implicit synchronisation.
 *   Arguments, layouts, results and errors are those of kvattn_gqa_decode; the call
 *   always runs the warp-level kernel (see kvattn_debug_set_gqa_kernel).
 *   Scratch: a fixed 6 MiB array inside the library, present on every GPU that loads
 *   the library until the process exits.  It holds the built-in plan of any batch on a
 *   device of up to 160 SMs (one worker per SM); a plan that needs more (a larger
 *   device, or kvattn_debug_set_workers forcing many workers) returns
 *   KVATTN_ERR_UNSUPPORTED with the sizes in kvattn_last_error_detail.  It calls no
 *   cudaMalloc, cudaFree or other allocating routine.
 *   The first call on a device looks up the array's device address (once per device,
 *   with that device current); make that first call before any stream capture.
 *   All calls share the one array and it keeps the last call's contents: calls that
 *   overlap on the GPU (different streams without ordering, or several host threads)
 *   race on it and give wrong results.  Order them on one stream.
 */
int kvattn_gqa_decode_noalloc(const uint16_t *q, const uint16_t *k_cache,
                              const uint16_t *v_cache, const int32_t *seq_lens, int max_seq_len,
                              int batch, int n_q_heads, int n_kv_heads, int head_dim, float scale,
                              float *out, float *lse, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KVATTN_H */
