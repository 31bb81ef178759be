/*
 * exact_causal_attention_gb300 -- C ABI of the paged K/V cache's operators beyond the
 * one-token decode and append of attn.h: attention of a chunk of new tokens per
 * request, the score forms (tanh cap, distance bias, window, visible prefix) for it and
 * for the one-token decode, the append of a chunk, the attention weight every
 * cached token received, and eviction by that weight.
 *
 * Everything attn.h says of layout, ownership, streams, launch order, bounded waits,
 * status codes and attn_device_status holds here.  The cache's layout is that of
 * attn_decode_paged: [num_pages, 2, page_size, Hkv, D] 16-bit (index 0 = K, 1 = V),
 * block_table [B, max_pages] int32, lengths [B] int32, page_size 8, 16, 32 or 64, D 64
 * or 128, num_pages * 2 * page_size < 2^31 and max_pages * page_size < 2^31 - 512.
 *
 * A ragged chunk of new tokens: request b owns rows q_offsets[b] .. q_offsets[b + 1] - 1
 * of the packed tensors, n_b of them, and lengths[b] counts its whole context with
 * these tokens (as attn_paged_append counts the token it writes): row i of the request
 * stands at position lengths[b] - n_b + i.  n_b may be 0, and a chunk may be the whole
 * context.  q_offsets [B + 1] int32 starts at 0 and does not decrease; packed rows
 * from q_offsets[B] on belong to no request and are neither read nor written.
 *
 * What the device finds wrong in its own data is skipped, never followed, and reported
 * by attn_device_status as ATTN_ERR_BAD_INDEX: a block-table entry outside
 * [0, num_pages) (its tokens count as not visible), a length outside
 * [0, max_pages * page_size] (taken at the nearest end), offsets that decrease
 * or leave [0, total rows] (the request counts as having no rows), a chunk
 * longer than its context (rows at negative positions).
 *
 * Score forms, for a row at position p and the key at position j of its context:
 *     s = scale * q . k                          softcap = 0
 *     s = softcap * tanh(scale * q . k / softcap)   softcap > 0 (finite)
 *     s = s - alibi_slopes[h] * |p - j|          alibi_slopes: device, [Hq] fp32, or NULL
 * and the key is visible iff it lies below lengths[b] and
 *     j <= p  and  (window = 0 or j > p - window),     window >= 0
 *     or j < prefix_lens[b]                       prefix_lens: device, [B] int32, or NULL
 * so prefix_lens is a prefix that every row sees both ways, and with a window the tokens
 * that stay visible whatever the window (values below 0 count as 0, above the length as
 * the length).  Block-table entries of pages that no row sees (outside the window and
 * the prefix) are not followed and may hold anything.  Positions are places in the
 * cache: after an eviction they are the places of the kept tokens.
 */
#ifndef EXACT_CAUSAL_ATTENTION_GB300_ATTN_CACHE_H_
#define EXACT_CAUSAL_ATTENTION_GB300_ATTN_CACHE_H_

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * attn_prefill_paged -- attention of a ragged chunk of new tokens over the paged cache
 * (which already holds their K and V, see attn_paged_append_chunk), grouped heads as
 * in attn_decode_paged:
 *     O[r, h] = sum_j softmax_j(s) V[j, h / g],    lse[r, h] = ln sum_j e^s.
 *   q           : device, [total_q, Hq, D] fp16, 16-byte aligned, read only.
 *   q_offsets   : device, [B + 1] int32.
 *   out         : device, [total_q, Hq, D] fp16; lse: device, [total_q, Hq] fp32 or
 *                 NULL.  Written for every row of a request; O = 0 and lse = -inf for a row that
 *                 sees no key.
 *   total_q     : >= 0 (0: nothing is launched).   B : 1 .. 4096.
 *   workspace   : device, 256-byte aligned, at least attn_prefill_workspace_bytes of
 *                 the same sizes; its contents on entry do not matter.  Two calls must not share
 *                 one while both may be running (two captured graphs neither).
 * out must not overlap q or the cache.  P is rounded to the 16-bit type for the P V
 * product; scores, the softmax's sums and O accumulate in fp32.  Values of the cache at and past
 * lengths[b] do not matter (they may be NaN); those below it should be finite, as
 * a row's hidden keys share its tiles.
 */
int attn_prefill_paged(const void* q, const void* cache, const int* block_table, const int* lengths,
                       const int* q_offsets, void* out, float* lse, int total_q, int B, int Hq, int Hkv,
                       int D, int page_size, int max_pages, int num_pages, float scale, float softcap,
                       int window, const float* alibi_slopes, const int* prefix_lens, void* workspace,
                       size_t workspace_bytes, attn_stream_t stream);

/* attn_prefill_paged_bf16 -- the same with bf16 q, cache and out. */
int attn_prefill_paged_bf16(const void* q, const void* cache, const int* block_table, const int* lengths,
                            const int* q_offsets, void* out, float* lse, int total_q, int B, int Hq,
                            int Hkv, int D, int page_size, int max_pages, int num_pages, float scale,
                            float softcap, int window, const float* alibi_slopes, const int* prefix_lens,
                            void* workspace, size_t workspace_bytes, attn_stream_t stream);

/* Workspace bytes of attn_prefill_paged; 0 when none is needed or the sizes are
 * invalid.  Needs no GPU. */
size_t attn_prefill_workspace_bytes(int total_q, int B, int Hq, int Hkv, int D, int page_size,
                                    int max_pages);

/*
 * attn_paged_append_chunk -- writes the ragged chunk's K and V into the paged cache:
 * row (r, kind, head) of new_kv [total, 2, Hkv, D] (16-bit, 16-byte aligned) of
 * request b's i-th token goes to position t = lengths[b] - n_b + i,
 * cache[block_table[b, t / page_size]][kind][t % page_size][head].  With one row a
 * request it is attn_paged_append.  The element type does not matter.
 */
int attn_paged_append_chunk(const void* new_kv, void* cache, const int* block_table, const int* lengths,
                            const int* q_offsets, int total, int B, int Hkv, int D, int page_size,
                            int max_pages, int num_pages, attn_stream_t stream);

/*
 * attn_paged_mass -- the attention weight every cached token received from a ragged
 * chunk, summed over the chunk's rows and the g query heads of each key/value head:
 *     mass[b, kvh, j] (+)= sum_{rows r of b} sum_{h / g = kvh} e^(s - lse[r, h])   (visible j)
 *   q, q_offsets : as attn_prefill_paged; q_offsets NULL means one row a request (a
 *                  decode step: total_q = B).
 *   lse          : device, [total_q, Hq] fp32, the log-sum-exp that attn_prefill_paged or
 *                  attn_decode_paged gave for the same rows (rows of -inf add nothing).
 *   mass         : device, [B, Hkv, max_pages * page_size] fp32.  accumulate = 0 writes it
 *                  in full (0 where no row looks); otherwise it is added to, and
 *                  places that no row looks at are left alone.
 * The other arguments as attn_prefill_paged (B up to 4096).  Sums are taken in fp32 in a fixed order:
 * the same call gives the same bits.
 */
int attn_paged_mass(const void* q, const float* lse, const void* cache, const int* block_table,
                    const int* lengths, const int* q_offsets, float* mass, int accumulate, int total_q, int B,
                    int Hq, int Hkv, int D, int page_size, int max_pages, int num_pages, float scale,
                    float softcap, int window, const float* alibi_slopes, const int* prefix_lens,
                    attn_stream_t stream);

/* attn_paged_mass_bf16 -- the same with a bf16 q and cache. */
int attn_paged_mass_bf16(const void* q, const float* lse, const void* cache, const int* block_table,
                         const int* lengths, const int* q_offsets, float* mass, int accumulate, int total_q,
                         int B, int Hq, int Hkv, int D, int page_size, int max_pages, int num_pages, float scale,
                         float softcap, int window, const float* alibi_slopes, const int* prefix_lens,
                         attn_stream_t stream);

/*
 * attn_paged_evict -- shrinks every request that holds more than `budget` tokens to
 * `budget` of them, per key/value head: the last `recent` tokens stay, and of the others
 * those with the largest mass (ties: the lowest position; a NaN ranks below every number).  The kept
 * tokens keep their order and move to positions 0 .. budget - 1 of the same pages, so
 * that pages past budget / page_size are free; rows behind them are left as they were.
 *   mass        : device, [B, Hkv, max_pages * page_size] fp32.
 *   kept        : device, [B, Hkv, budget] int32, written in full: the position every kept
 *                 token had, in order, then -1.
 *   new_lengths : device, [B] int32: min(lengths[b], budget).  May be `lengths`.
 *   mass_out    : device, shaped like mass, written in full: the kept tokens' mass, then 0.
 *                 May be `mass`, or NULL.
 *   budget      : 1 .. max_pages * page_size.   recent : 0 .. budget.
 * Two requests must not share a page that holds tokens of both, as eviction moves rows in place.
 * Distances (alibi_slopes, window) are taken between the new places afterwards.
 */
int attn_paged_evict(void* cache, const int* block_table, const int* lengths, const float* mass, int* kept,
                     int* new_lengths, float* mass_out, int B, int Hkv, int D, int page_size, int max_pages,
                     int num_pages, int budget, int recent, attn_stream_t stream);

/*
 * attn_decode_paged_form -- attn_decode_paged with the score forms above (the row of
 * request b stands at position lengths[b] - 1).  With softcap 0, window 0 and NULL
 * slopes it is attn_decode_paged.  Here the visible tokens of all requests are cut into
 * segments of one size, so that requests of unequal lengths finish together:
 *   kv_splits : the most segments a request may get, 1 .. 64 (see
 *               attn_decode_form_default_splits); the workspace is attn_decode_paged's
 *               for that many.
 */
int attn_decode_paged_form(const void* q, const void* cache, const int* block_table, const int* lengths,
                           void* out, float* lse, int B, int Hq, int Hkv, int D, int page_size, int max_pages,
                           int num_pages, float scale, float softcap, int window, const float* alibi_slopes,
                           const int* prefix_lens, int kv_splits, void* workspace, size_t workspace_bytes,
                           attn_stream_t stream);

/* attn_decode_paged_form_bf16 -- the same with bf16 q, cache and out. */
int attn_decode_paged_form_bf16(const void* q, const void* cache, const int* block_table, const int* lengths,
                                void* out, float* lse, int B, int Hq, int Hkv, int D, int page_size,
                                int max_pages, int num_pages, float scale, float softcap, int window,
                                const float* alibi_slopes, const int* prefix_lens, int kv_splits,
                                void* workspace, size_t workspace_bytes, attn_stream_t stream);

/* A bound on the segments a request gets, for the current device: some times the
 * mean that fills it.  Negative attn_status on bad sizes or a non-sm_103 device. */
int attn_decode_form_default_splits(int B, int Hq, int Hkv, int page_size, int max_pages);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_CAUSAL_ATTENTION_GB300_ATTN_CACHE_H_ */
