/*
 * spec_kv.h -- the paged key/value cache around the verify step, on one GPU (sm_103a).
 *
 * A round of speculative decoding scores L_b draft tokens and the token before them in one
 * target pass (Kangaroo guide, section 3; LayerSkip guide, "Verification Phase"), and rolls the
 * cache back behind the accepted prefix (LayerSkip guide, "Shared KV cache"; Kangaroo guide,
 * "Production advantages": PagedAttention). These entry points are the cache's part of that
 * round, in the order in which it calls them:
 *   spec_block_tables   accepted lengths and new lengths -> pages, slots and positions;
 *   spec_qk_norm_rope   norms of queries and keys per head, and the position rotation;
 *   spec_kv4_append     keys and values of the new tokens into the cache, in 4 bits;
 *   spec_kv4_attention  causal attention of the new tokens over the cache.
 * The hidden states that follow go to spec_verify_hidden (or their logits to spec_verify), whose
 * out_accept_len is the accept_len of the next round's spec_block_tables.
 *
 * Memory: every pointer is DEVICE memory owned by the caller. All calls are asynchronous on
 * `stream` (a cudaStream_t, NULL for the legacy default stream), do not synchronise and may be
 * captured into a graph (spec_kv4_attention after one call on the same stream outside capture).
 * spec_kv4_attention keeps a workspace of fixed size for each device and stream; a captured call
 * keeps that of the stream it was captured on, so its replays must not overlap other calls of
 * that stream, or replays of other graphs captured on it.
 *
 * Errors: arguments are checked on the host before anything is launched, as in spec_verify.h. A
 * copy that spec_kv4_attention waits for in vain raises the stream's error word; what that call and
 * later ones on the stream wrote is not valid until spec_verify_device_error has reported it.
 *
 * The cache. uint8 [num_pages][Hkv][page_size * (D + D/8)], 16-byte aligned: a page holds
 * page_size tokens (16, 32, 64 or 128) of every key/value head, D = 64 or 128 values a head, as
 * page_size / 16 blocks of 16 tokens a head. A value is e2m1 code * e4m3 scale * tensor scale,
 * with one e4m3 scale for 16 neighbouring values of a token. A block is, in this order,
 *   key codes     [16 tokens][D/2]        byte j: value 2j in the low 4 bits, 2j+1 in the high;
 *   key scales    [16 tokens][D/16];
 *   value codes   [8 token pairs][D]      one byte a value: the even token in the low 4 bits, the
 *                                         odd one in the high; the D bytes of pair p are 8
 *                                         chunks, chunk g at place g ^ (2 (p % 4)) when D = 128
 *                                         and g ^ (4 (p / 2 % 2)) when D = 64;
 *   value scales  [8 token pairs][D/16][2 tokens].
 * A token's slot is page * page_size + its place in the page.
 */
#ifndef SPEC_KV_H
#define SPEC_KV_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one page of one head: page_size * (D + D/8); 0 for a page size or D not supported. */
size_t spec_kv4_page_bytes(int page_size, int D);

/*
 * Block tables and slot maps of B sequences (B <= 8192) for the next round, in one launch.
 *   ctx_lens     [B]   tokens of the sequence in the cache before the last round
 *   accept_len   [B]   outcome of the last round (out_accept_len of the verify step), or NULL:
 *                      a >= 0 keeps a + 1 more tokens (the token before the drafts and the a
 *                      accepted ones), a < 0 none
 *   new_lens     [B]   tokens that the sequence brings to this round (the last emitted token and
 *                      its drafts, or a prompt); 0: it waits; < 0: it has ended
 *   block_table  [B][max_blocks]  in and out: page of each block of page_size tokens
 *   held         [B]   pages that the sequence holds
 *   ring         [ring_size]      in and out: free pages, a ring buffer; entry i of the queue is
 *                      ring[i mod ring_size], ring_size >= pages in existence
 *   counters     [2]   int64: queue entries taken so far, entries put back so far; the entries
 *                      from counters[0] to counters[1] - 1 are the free pages
 * With c = ctx_lens + accept_len + 1 (0 when the sequence has ended), n = max(new_lens, 0) and
 * need = ceil((c + n) / page_size), sequences in ascending order take need - held pages from the
 * front of the queue or put held - need pages (those of their last blocks) back at its end; pages put
 * back by this call are taken by a later one. Written:
 *   out_ctx_lens [B]   c;    out_held [B]  pages now held;    out_counters [2]
 *   out_kv_lens  [B]   c plus the tokens scheduled
 *   out_status   [B]   1 scheduled, 0 nothing to schedule, or, with no token scheduled:
 *                      -1 the free pages run out (the sequence keeps what it holds),
 *                      -2 lengths that do not fit (held outside 0..max_blocks; and unless the
 *                         sequence has ended, ctx_lens < 0, c > held * page_size, or
 *                         need > max_blocks): the sequence is left as it was, out_ctx_lens =
 *                         ctx_lens,
 *                      -3 its tokens do not fit in max_tokens (it keeps its pages). A sequence
 *                         fails so when the tokens of it and all before it that have pages pass max_tokens
 *   out_cu_new   [B+1] first token of each sequence in the round's token order, then their number
 *   out_slots    [max_tokens] int64, out_positions [max_tokens], out_seq_ids [max_tokens]: slot,
 *                      position and sequence of each token; -1, 0, -1 past the last one
 * Integers are int32 where nothing else is said. The outputs of lengths, held and counters must
 * be other buffers than the inputs (two sets in turn serve a loop): a call on the same inputs
 * writes the same values again. max_blocks * page_size must stay below 2^31, max_tokens and
 * ring_size below 2^31 - 1.
 */
sv_status spec_block_tables(int B, int page_size, int max_blocks, int max_tokens,
                            const int32_t* ctx_lens, const int32_t* accept_len,
                            const int32_t* new_lens, int32_t* block_table, const int32_t* held,
                            int32_t* ring, int ring_size, const int64_t* counters,
                            int32_t* out_ctx_lens, int32_t* out_held, int64_t* out_counters,
                            int32_t* out_kv_lens, int32_t* out_status, int32_t* out_cu_new,
                            int64_t* out_slots, int32_t* out_positions, int32_t* out_seq_ids,
                            void* stream);

/*
 * Root-mean-square norm of every query and key head and the rotation by position, in one pass:
 * y = x / sqrt(mean(x^2) + eps) * weight, then for j < rot/2 the pair (y[j], y[j + rot/2]), or
 * (y[2j], y[2j+1]) when `interleaved`, is rotated by the angle positions[t] * inv_freq[j].
 *   q  [T][Hq][D], k [T][Hkv][D] of dtype (Hkv may be 0), element (t, h, i) at
 *      t * token_stride + h * D + i, so that both may lie in one projection's output
 *   q_weight, k_weight [D] of dtype, or NULL for ones
 *   positions [T] int32; inv_freq [rot/2] double, finite; 0 <= rot <= D, rot even
 *   out_q, out_k: dtype, with token strides of their own; out_q == q and out_k == k (with the
 *      same strides) work in place, any other overlap does not
 * D is even and at most 512. The norm is held in float32; the angle is reduced as a 64-bit
 * fraction of a turn, exact to 2^-32 turns at any position (|inv_freq| of 2^54 and more counts as 0).
 */
sv_status spec_qk_norm_rope(int T, int Hq, int Hkv, int D, int rot, int interleaved,
                            sv_dtype dtype, const void* q, long long q_token_stride,
                            const void* k, long long k_token_stride, const void* q_weight,
                            const void* k_weight, const int32_t* positions,
                            const double* inv_freq, float eps, void* out_q,
                            long long out_q_token_stride, void* out_k,
                            long long out_k_token_stride, void* stream);

/*
 * Keys and values of T tokens into the cache. For 16 neighbouring values x of a head:
 * scale = e4m3(max|x| * float32(1 / (6 g))), at most 448, and code = e2m1(x / (scale * g)), both to
 * nearest with ties to even, the quotient in float32 and held at +-6; g is k_scale or v_scale
 * (finite, > 0). 16 values that hold a NaN or an infinity get a NaN scale: they read as NaN.
 *   k, v [T][Hkv][D] of dtype, rows as in spec_qk_norm_rope, 16-byte aligned (pointers, strides)
 *   slots [T] int64: slot of each token; a token whose slot is outside 0..num_pages*page_size-1
 *      is not written. The slots of one call are distinct.
 *   out_k, out_v: NULL, or bfloat16 [T][Hkv][D], 16-byte aligned: the values that the cache now
 *      stands for (so that a prompt's own attention sees what later rounds will read); written
 *      for every token
 * The other token of a value pair keeps its code, whether it is written before, after or by the
 * same call.
 */
sv_status spec_kv4_append(int T, int Hkv, int D, int page_size, int num_pages, sv_dtype dtype,
                          const void* k, long long k_token_stride, const void* v,
                          long long v_token_stride, const int64_t* slots, float k_scale,
                          float v_scale, void* cache, void* out_k, void* out_v, void* stream);

/*
 * Causal attention of each sequence's new tokens over the cache. Sequence b has the query rows
 * cu_new[b] .. cu_new[b+1] - 1 of q and kv_lens[b] tokens in the cache, the new ones among them:
 * row i of its n sees tokens 0 .. kv_lens[b] - n + i. out = softmax(scale * q k^T) v over the
 * tokens seen; a row that sees none (kv_lens < n) gives zeros and a log-sum of -inf. Tokens
 * that a row does not see have no part in it, whatever the cache holds there.
 *   q   bfloat16 [T][Hq][D], row as in spec_qk_norm_rope; Hq a multiple of Hkv, query head h
 *       reads key/value head h / (Hq / Hkv)
 *   block_table [B][max_blocks] int32; a page outside 0..num_pages-1 is not read, and the rows
 *       that see one of its tokens are NaN. kv_lens above max_blocks * page_size count as that.
 *   cu_new [B+1] int32, ascending; entries are held to 0..T
 *   scale, k_scale, v_scale: finite; the cache's tensor scales as in spec_kv4_append
 *   max_new: the largest number of new tokens of a sequence, as far as the caller knows. It picks
 *       the kernel's tiles; any value gives the same results to rounding.
 *   out bfloat16 [T][Hq][D] contiguous; out_lse float32 [T][Hq]: natural log of the softmax's
 *       sum, or NULL. Rows of no sequence are not written.
 * Scores, softmax and sums are held in float32; products take float16 operands: keys and values
 * are exact in it, queries too (each row scaled by a power of two; what is below 2^-28 of its
 * largest value, or below 2^-116, is rounded), the softmax's weights are rounded to it (by up to
 * 2^-11 of each, or 2^-32 of the row's largest where that is more).
 * A tile of rows reads all tokens of its sequence, also those that none of its rows sees: of a
 * prompt with nothing before it, half of the work is on those.
 */
sv_status spec_kv4_attention(int B, int T, int Hq, int Hkv, int D, int page_size, int num_pages,
                             int max_blocks, const void* q, long long q_token_stride,
                             const void* cache, const int32_t* block_table,
                             const int32_t* kv_lens, const int32_t* cu_new, float scale,
                             float k_scale, float v_scale, int max_new, void* out,
                             float* out_lse, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_KV_H */
