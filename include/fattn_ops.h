/*
 * fattn_ops.h — C ABI of libfattn, continued: what stands around the attention
 * calls of fattn.h in a model that trains on, or serves, long contexts.
 *
 *   - rotary positions on q and k (fattn_rope), and their serving form, which
 *     also puts the new tokens' k and v into the paged cache
 *     (fattn_rope_append_paged);
 *   - shaped scores: attention whose scores are capped by a tanh, carry a bias
 *     that depends on the distance, and see a window, a document or a prefix
 *     (fattn_fwd_shaped, its gradient fattn_bwd_shaped, query chunks and single
 *     tokens over the paged cache: fattn_fwd_paged_shaped,
 *     fattn_decode_paged_shaped);
 *   - a cache in 8 bits: new tokens rotated, quantized and put into their pages
 *     (fattn_rope_append_paged_fp8), and attention over it (fattn_decode_paged_fp8,
 *     fattn_fwd_paged_fp8);
 *   - a budget for the cache: the attention weight that its tokens receive
 *     (fattn_key_weights_paged), and the eviction of all but the heaviest
 *     (fattn_evict_paged).
 *
 * The conventions of fattn.h hold: DEVICE pointers owned by the caller, host
 * checks before anything is launched, work enqueued on `stream`, no
 * allocation, no synchronisation, problems found on the device recorded in the
 * status word (fattn_debug_read_status). Strides count elements. After a wait that ran
 * out (FATTN_ERR_TIMEOUT) the outputs of the call have no meaning: what was finished before
 * is written, the rest is not. fattn_key_weights_paged with weights_out == weights_in has
 * then changed a part of its input: to repeat it, restore the weights first, or give it
 * another weights_out from the start.
 */
#ifndef FATTN_OPS_H
#define FATTN_OPS_H

#include "fattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fattn_rope — rotary positions.
 *
 * For every token (row) with position p and every head, pair i of the first
 * rotary_dim elements, t = p * inv_freq[i]:
 *   y_a = A (x_a cos t - x_b sin t),  y_b = A (x_b cos t + x_a sin t)
 * with (a, b) = (i, i + rotary_dim / 2), or (2i, 2i + 1) if interleaved != 0.
 * Elements from rotary_dim on are copied. inverse != 0 rotates by -t: with the
 * same amplitude A that is the transposed map, the gradient of the call.
 * The angle is reduced modulo a full turn in 64-bit fixed point (2^-64 turns),
 * so far positions lose nothing; products are fp32, rounded once.
 *
 * q [rows, Hq, d], q_out likewise; k [rows, Hk, d], k_out likewise, both NULL
 * (with Hk = 0) to rotate q alone. dtype FATTN_BF16 or FATTN_FP32. Elements of a
 * head are contiguous; q_row / q_head, qo_*, k_*, ko_* are the strides between rows
 * and heads, >= 0 (inputs) or such that no two outputs overlap. An output may be
 * its input (same pointer and strides); it may not overlap it otherwise.
 * positions: DEVICE int32 [rows], any value, or NULL: row r is position r % period.
 * inv_freq: DEVICE double [rotary_dim / 2], radians per position.
 * Pointers need the alignment of their type; 16-byte aligned pointers and strides
 * (and rotary_dim, d - rotary_dim) take 16-byte accesses.
 * rows == 0 is an empty problem. Errors: INVALID_ARG (NULL or misaligned pointers,
 *   negative sizes or strides, k without k_out, odd rotary_dim or one outside
 *   [0, d], period <= 0 without positions, an amplitude that is not finite, an
 *   unknown dtype); UNSUPPORTED (d > 1024, Hq + Hk > 4096).
 */
fattn_status fattn_rope(const void* q, void* q_out, const void* k, void* k_out, const int32_t* positions, int period,
                        const double* inv_freq, int rows, int Hq, int Hk, int d, int rotary_dim, long long q_row,
                        long long q_head, long long qo_row, long long qo_head, long long k_row, long long k_head,
                        long long ko_row, long long ko_head, int interleaved, int inverse, float amplitude,
                        fattn_dtype dtype, cudaStream_t stream);

/*
 * fattn_rope_append_paged — the serving form: q and k of new tokens rotated, k
 * and v written into their slots of the paged cache, in one launch.
 *
 * The B chunks are packed as fattn_fwd_paged reads them: rows
 * [cu_seqlens_q[b], cu_seqlens_q[b + 1]) are the last tokens of sequence b's
 * seqlens_k[b] context tokens (the new ones included), so row r is token
 * t = seqlens_k[b] - cu_seqlens_q[b + 1] + r, slot t % page_size of page
 * block_table[b * max_pages_per_seq + t / page_size]. q [total_q, Hq, d] (NULL: no
 * q) goes to q_out [total_q, Hq, d] (densely packed, not overlapping q); k and v
 * [total_q, Hkv, d] to kcache and vcache [num_pages, page_size, Hkv, d]; all bf16.
 * positions int32 [total_q], or NULL: the position of row r is its t.
 * Rows at or past cu_seqlens_q[B] are padding: nothing is read or written for them.
 * Two tokens of one call must not share a slot. Any page_size >= 1; d, rotary_dim,
 * inv_freq, interleaved, amplitude and the strides as in fattn_rope.
 * A row whose t is outside [0, max_pages_per_seq * page_size), or whose table entry
 * is outside [0, num_pages), is skipped and recorded as FATTN_ERR_DEVICE_CHECK.
 * Errors: as fattn_rope, with INVALID_ARG for a NULL cache, table, seqlens_k or
 *   cu_seqlens_q or non-positive cache sizes; UNSUPPORTED also for
 *   max_pages_per_seq * page_size >= 2^31.
 */
fattn_status fattn_rope_append_paged(const void* q, void* q_out, const void* k, const void* v, void* kcache,
                                     void* vcache, const int32_t* block_table, const int32_t* seqlens_k,
                                     const int32_t* cu_seqlens_q, const int32_t* positions, const double* inv_freq,
                                     int B, int total_q, int Hq, int Hkv, int d, int rotary_dim, int page_size,
                                     int max_pages_per_seq, int num_pages, long long q_row, long long q_head,
                                     long long k_row, long long k_head, long long v_row, long long v_head,
                                     int interleaved, float amplitude, cudaStream_t stream);

/*
 * Shaped scores. For the query at position i (in key coordinates: the row's
 * index, for chunks plus the context before the chunk) and key j,
 *   s = scale q.k
 *   s = softcap tanh(s / softcap)            if softcap > 0
 *   s = s - slopes[h] |i - j|                if slopes != NULL
 * and key j is visible iff
 *   j <= i                                   if causal != 0,
 *   |i - j| < window                         if window > 0,
 *   key_begin[row] <= j < key_end[row]       where given (either may be NULL).
 * O = softmax(s) V over the visible keys, lse the logsumexp; a row that sees no
 * key gets O = 0, lse = -inf. A capped score keeps the relative precision of a 32-bit
 * score whatever the cap is; from 2^100 on a cap is none.
 *
 * slopes: DEVICE fp32 [Hq], any sign. key_begin, key_end: DEVICE int32, one per
 * query row ([B, N]; [total_q] for chunks), keys of the row's own sequence; they
 * must not decrease from a row to the next of its sequence (a row that sees nothing
 * has begin = end, at least the previous row's end and at most the next row's begin:
 * padding behind a document begins and ends where the document ends). Packed documents
 * (begin = the document's first row, end = one past its last), prefixes (end = max(i + 1,
 * prefix end)) and padding are such ranges; so are their unions with causal and
 * window. Ranges that decrease are recorded as FATTN_ERR_DEVICE_CHECK: by the
 * attention calls where a row's keys are outside its tile's (its output is wrong then, and
 * right otherwise), by the gradient always (the keys' gradients would be wrong).
 * Work goes by 128 x 128 tiles: a tile in which no row sees a key is not computed,
 * and keys before the lowest one that 256 consecutive rows see, rounded down to a
 * multiple of 128, are not read for them. Within the computed tiles hidden keys
 * get weight 0, so every row of the inputs must be finite.
 *
 * fattn_fwd_shaped — dense prefill: bf16, layouts of fattn_fwd (q, o [B, N, Hq,
 *   d]; k, v [B, N, Hkv, d]; lse [B, Hq, N], may be NULL).
 * Errors (all four): those of the plain call; INVALID_ARG also for a softcap that
 *   is negative or not finite (or so small that scale / softcap is not), a negative
 *   window, misaligned slopes or ranges.
 */
fattn_status fattn_fwd_shaped(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                              int N, int d, int causal, float scale, float softcap, const float* slopes, int window,
                              const int32_t* key_begin, const int32_t* key_end, cudaStream_t stream);

/*
 * fattn_fwd_paged_shaped_workspace_size — bytes of scratch that num_splits > 1 needs:
 * the partials lse [total_q, Hq, S] and O [total_q, Hq, S, d], fp32, each region 256-byte
 * aligned. Returns 0 for num_splits <= 1 or non-positive arguments.
 */
size_t fattn_fwd_paged_shaped_workspace_size(int total_q, int Hq, int d, int num_splits);

/*
 * fattn_fwd_paged_shaped — query chunks over the paged cache: fattn_fwd_paged with
 * shaped scores; the position of a chunk's query i is i + seqlens_k[b] - Lq_b.
 * Pages before token 128 floor(t / 128), t the first token that any row of the
 * chunk sees, are not read, nor are their table entries.
 * num_splits = S >= 1: with few query tiles and long contexts the work is split along
 *   the keys: every 128-row query tile's K/V tiles are cut into S runs, worked on
 *   independently and joined with the online-softmax rule by a second launch. workspace: DEVICE
 *   scratch of fattn_fwd_paged_shaped_workspace_size bytes, 256-byte aligned, contents ignored
 *   (S = 1: none, NULL). INVALID_ARG for S < 1, WORKSPACE for a missing, small or misaligned one.
 */
fattn_status fattn_fwd_paged_shaped(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                                    const int32_t* seqlens_k, const int32_t* cu_seqlens_q, void* o, float* lse, int B,
                                    int Hq, int Hkv, int d, int page_size, int max_pages_per_seq, int num_pages,
                                    int total_q, int max_seqlen_q, int causal, float scale, float softcap,
                                    const float* slopes, int window, const int32_t* key_begin, const int32_t* key_end,
                                    int num_splits, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fattn_bwd_shaped_workspace_size — bytes of scratch fattn_bwd_shaped needs: fattn_bwd's
 * two fp32 arrays, then the queries that see each key, int32 pairs [B, Npad], 256-byte
 * aligned, and, with Hq > Hkv and few key tiles, room for the query heads' shares of dV
 * and dK, fp32 [2, B, N, Hq, d]. Returns 0 for non-positive arguments.
 */
size_t fattn_bwd_shaped_workspace_size(int B, int Hq, int Hkv, int N, int d);

/*
 * fattn_bwd_shaped — gradients of fattn_fwd_shaped with respect to q, k and v:
 * fattn_bwd with P rebuilt from the shaped scores and dS multiplied by the cap's
 * derivative 1 - tanh^2. o and lse are fattn_fwd_shaped's for the same arguments;
 * the slopes are constants (no gradient). Rows that see no key and keys that no row
 * sees get gradient 0. workspace: DEVICE, >= fattn_bwd_shaped_workspace_size(B, Hq, Hkv, N, d)
 * bytes, 256-byte aligned, contents ignored.
 */
fattn_status fattn_bwd_shaped(const void* q, const void* k, const void* v, const void* o, const float* lse,
                              const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d,
                              int causal, float scale, float softcap, const float* slopes, int window,
                              const int32_t* key_begin, const int32_t* key_end, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/*
 * fattn_decode_paged_shaped — one query token per sequence, at position
 * seqlens[b] - 1: fattn_decode_paged with a cap, a distance bias and a window. With
 * a window the splits share the pages that it touches: a sequence's visible pages,
 * counted from the page of its first visible token, are cut into S chunks of
 * C = ceil(n / S) pages, n = min(max_pages_per_seq, (window + page_size - 2) /
 * page_size + 1); pages before are not read. Workspace as fattn_decode_paged.
 */
fattn_status fattn_decode_paged_shaped(const void* q, const void* kcache, const void* vcache,
                                       const int32_t* block_table, const int32_t* seqlens, int num_splits, void* o,
                                       float* lse, int B, int Hq, int Hkv, int d, int page_size, int max_pages_per_seq,
                                       int num_pages, float scale, float softcap, const float* slopes, int window,
                                       void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Windows with sinks. The shaped scores with one more rule: beside its window a query always sees the first
 * `sinks` keys of its sequence. Key j is visible iff
 *   (|i - j| < window  or  j < sinks)  and  j <= i if causal != 0;
 * window = 0 hides nothing (sinks then mean nothing). Key ranges are not taken. Tiles and pages between the
 * sinks and the window are neither read nor computed, so memory may have been reclaimed there: their table
 * entries are not read either (chunks: from the first 128-key tile past the sinks to the window of the first
 * of 256 consecutive rows, rounded down to a multiple of 128).
 * Arguments, layouts, workspaces (but the gradient's) and errors are those of the shaped calls, with INVALID_ARG for sinks < 0.
 *
 * fattn_fwd_sinks         — dense prefill (fattn_fwd_shaped).
 * fattn_bwd_sinks         — its gradient (fattn_bwd_shaped). A sink's dK and dV sum over every later row, in a fixed
 *   order. workspace: fattn_bwd_sinks_workspace_size bytes, fattn_bwd_shaped's and room for fp32 shares of the sinks' key
 *   tiles, which are worked on in pieces: at most 128 tiles of 2 * 128 * d for every sequence and head.
 * fattn_fwd_paged_sinks   — query chunks over the paged cache (fattn_fwd_paged_shaped, and its workspace).
 * fattn_decode_paged_sinks — single tokens (fattn_decode_paged_shaped). The splits share the pages of the sinks and of
 *   the window: n = min(max_pages_per_seq, (window + page_size - 2) / page_size + 1 + ceil(sinks / page_size)).
 */
fattn_status fattn_fwd_sinks(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                             int N, int d, int causal, float scale, float softcap, const float* slopes, int window,
                             int sinks, cudaStream_t stream);
size_t fattn_bwd_sinks_workspace_size(int B, int Hq, int Hkv, int N, int d, int causal, int window, int sinks);
fattn_status fattn_bwd_sinks(const void* q, const void* k, const void* v, const void* o, const float* lse,
                             const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d,
                             int causal, float scale, float softcap, const float* slopes, int window, int sinks,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream);
fattn_status fattn_fwd_paged_sinks(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                                   const int32_t* seqlens_k, const int32_t* cu_seqlens_q, void* o, float* lse, int B,
                                   int Hq, int Hkv, int d, int page_size, int max_pages_per_seq, int num_pages,
                                   int total_q, int max_seqlen_q, int causal, float scale, float softcap,
                                   const float* slopes, int window, int sinks, int num_splits, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream);
fattn_status fattn_decode_paged_sinks(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                                      const int32_t* seqlens, int num_splits, void* o, float* lse, int B, int Hq, int Hkv,
                                      int d, int page_size, int max_pages_per_seq, int num_pages, float scale,
                                      float softcap, const float* slopes, int window, int sinks, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream);

/*
 * fattn_bwd_strided — the gradients above for an o that is a view: element (b, i, h, c) is o[b * o_batch + i * o_row +
 * h * o_head + c] (heads first in memory, a slice of a wider tensor, a broadcast), strides >= 0 and multiples of 8 elements.
 * shaped == 0: fattn_bwd (softcap, window and sinks 0, no slopes and key ranges); else fattn_bwd_sinks, with key ranges where
 * sinks == 0. Everything else, bits included, is theirs for the packed o. Errors: theirs, and INVALID_ARG for other strides.
 */
fattn_status fattn_bwd_strided(const void* q, const void* k, const void* v, const void* o, const float* lse,
                               const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d,
                               int causal, float scale, int shaped, float softcap, const float* slopes, int window,
                               int sinks, const int32_t* key_begin, const int32_t* key_end, long long o_batch,
                               long long o_row, long long o_head, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/*
 * The 8-bit cache: kcache, vcache [num_pages, page_size, Hkv, d] E4M3 codes ('fn' variant: no
 * infinities), kscale, vscale fp32 [num_pages, Hkv]; token t of a sequence is slot t % page_size of page
 * block_table[b * max_pages_per_seq + t / page_size], its k in head h is kscale[page, h] * code, its v
 * likewise. Scales of pages in use are finite and at least 2^-100; the append writes powers of two. d in {64, 128},
 * page_size in {16, 32, 64, 128}. Where rows are streamed a key counts, in O and in lse, while its weight times its page's V
 * scale is at least 2^-118 of the largest such product that the row sees: any key whose weight matters if V's scales lie within
 * 2^90 of each other.
 *
 * fattn_rope_append_paged_fp8 — fattn_rope_append_paged into the 8-bit cache: q and k of new tokens
 * rotated, q written to q_out (bf16), k and v as codes, in one launch. Per page, head and cache, with a the
 * largest finite magnitude of the page's new values (k rotated, in fp32):
 *   need = the least power of two with a <= 448 need, at least 2^-100;
 *   a page whose slots before the new tokens hold context has scale max(old, need), and if that is above the
 *   old one the codes of its other slots become RN(code * old / new); any other page has scale need (its old one is not
 *   read) and its other slots mean nothing;
 *   new codes = RN(value / scale); infinities and NaN become NaN codes.
 * A token with NaN codes is not finite for the attention calls: hidden keys have weight 0, as with shaped scores, and 0 times NaN is
 * NaN, so its V may reach rows of its own sequence that do not see it (drafted tokens before it). Rows of other sequences, and
 * what lies in a page past its sequence's end, are not concerned.
 * Which slots hold context follows from seqlens_k alone. A page that is appended to must not be shared with another sequence, and
 * no two tokens of a call share a slot. Everything else (chunks, positions, padding rows, strides, skipped rows) is as in
 * fattn_rope_append_paged. Errors: as there; UNSUPPORTED also for other d or page sizes, or
 * num_pages * page_size >= 2^31; codes must be 16-byte aligned.
 */
fattn_status fattn_rope_append_paged_fp8(const void* q, void* q_out, const void* k, const void* v, void* kcache,
                                         void* vcache, float* kscale, float* vscale, const int32_t* block_table,
                                         const int32_t* seqlens_k, const int32_t* cu_seqlens_q, const int32_t* positions,
                                         const double* inv_freq, int B, int total_q, int Hq, int Hkv, int d,
                                         int rotary_dim, int page_size, int max_pages_per_seq, int num_pages,
                                         long long q_row, long long q_head, long long k_row, long long k_head,
                                         long long v_row, long long v_head, int interleaved, float amplitude,
                                         cudaStream_t stream);

/*
 * fattn_decode_paged_fp8 — one query token per sequence over the 8-bit cache: fattn_decode_paged_sinks with its
 * arguments, outputs and workspace (fattn_decode_workspace_size). num_splits bounds the pieces that one sequence's visible
 * tokens of a KV head are cut into (1: none): up to 16 of equal length where max_pages_per_seq and the window leave little
 * work, else, up to 96, what makes the thread blocks' shares of all sequences' tokens equal. A table much wider than the
 * sequences need costs time for short ones.
 * q bf16. Products of q with codes are exact in fp32 sums, weights are rounded to fp16 (11 bits) for the product with V.
 * Equal calls give equal bits. B == 0 is an empty problem. A table entry outside the pool hides its tokens and records
 * FATTN_ERR_DEVICE_CHECK, as do lengths outside the table.
 */
fattn_status fattn_decode_paged_fp8(const void* q, const void* kcache, const void* vcache, const float* kscale,
                                    const float* vscale, const int32_t* block_table, const int32_t* seqlens,
                                    int num_splits, void* o, float* lse, int B, int Hq, int Hkv, int d, int page_size,
                                    int max_pages_per_seq, int num_pages, float scale, float softcap, const float* slopes,
                                    int window, int sinks, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fattn_fwd_paged_fp8_workspace_size — bytes of scratch fattn_fwd_paged_fp8 needs. Few query rows
 * (max_seqlen_q * Hq / Hkv <= FATTN_FP8_STREAM_ROWS(Hq / Hkv)): the pieces' partials, as for single tokens. More: a bf16
 * copy of the sequences' pages, 4 Hkv d page_size bytes for each of B * max_pages_per_seq, their table, and the partials of
 * fattn_fwd_paged_shaped_workspace_size. Returns 0 for non-positive arguments.
 */
#define FATTN_FP8_STREAM_ROWS(group) (48 * ((group) + 1))
size_t fattn_fwd_paged_fp8_workspace_size(int B, int Hq, int Hkv, int d, int page_size, int max_pages_per_seq, int total_q,
                                          int max_seqlen_q, int num_splits);

/*
 * fattn_fwd_paged_fp8 — query chunks over the 8-bit cache: fattn_fwd_paged_sinks with its arguments and outputs.
 * Few query rows stream the codes as single tokens do; with more, the pages that any of them sees are expanded to
 * bf16 (exact for scales that are powers of two, else one rounding) in the workspace and read by the tensor-core prefill.
 * num_splits >= 1: the pieces at most of a group of up to 32 streamed rows, or the prefill's splits. workspace: 256-byte
 * aligned, contents ignored, always needed.
 * A table entry outside the pool is recorded as FATTN_ERR_DEVICE_CHECK and, as in fattn_fwd_paged, its tokens read as zeros
 * (K and V, so a score of 0 before the distance bias), whichever way the rows take; single tokens do not see them.
 * Errors: those of fattn_fwd_paged_sinks and of the cache; UNSUPPORTED also for total_q * Hq * num_splits >= 2^31, with few
 *   rows for more tokens than an int counts (B * Hkv * ceil(rows / 32) * max_pages_per_seq * page_size / 16 about 2^31), with more
 *   for (B * max_pages_per_seq + 1) * page_size >= 2^31, and for B > 65535 in splits.
 */
fattn_status fattn_fwd_paged_fp8(const void* q, const void* kcache, const void* vcache, const float* kscale,
                                 const float* vscale, const int32_t* block_table, const int32_t* seqlens_k,
                                 const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq, int Hkv, int d,
                                 int page_size, int max_pages_per_seq, int num_pages, int total_q, int max_seqlen_q,
                                 int causal, float scale, float softcap, const float* slopes, int window, int sinks,
                                 int num_splits, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fattn_key_weights_paged — the attention weight that the tokens of a paged cache
 * receive from query chunks:
 *   weights_out[b, hkv, t] = decay weights_in[b, hkv, t]
 *                            + sum over the heads of group hkv and the queries of chunk b of e^{s - lse}
 * for t < seqlens_k[b]; slots from seqlens_k[b] on are set to 0, or in place (weights_out ==
 * weights_in) left as they are. s is the shaped score (softcap, slopes, window as above; causal as in fattn_fwd_paged), lse the
 * logsumexp that the attention call with the same arguments wrote. Sums are fp32, in a fixed order.
 *
 * q, kcache, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q: as fattn_fwd_paged (for single
 *   tokens q is [B, Hq, d] and cu_seqlens_q = 0, 1, ..., B); any page_size >= 1.
 * lse: DEVICE fp32, head h and row r at lse[h * lse_head + r * lse_row]: fattn_fwd_paged's [Hq,
 *   total_q] (total_q, 1) and fattn_decode_paged's [B, Hq] (1, Hq) both serve. A row of -inf gives nothing,
 *   one of NaN makes the weights of the keys that it sees NaN.
 * weights_in (NULL: zeros; then decay is not used), weights_out: DEVICE fp32
 *   [B, Hkv, max_pages_per_seq * page_size]; they may be the same array.
 * max_seqlen_q: host upper bound on the chunks' queries; it chooses between the streaming kernel (few
 *   query rows) and the tensor-core kernel, whose pipeline waits are bounded as the other calls' are.
 * A sequence whose lengths are inconsistent, or with more queries than max_seqlen_q, is skipped (its weights are left as they are), a table entry outside the pool gives its tokens
 *   nothing; both record FATTN_ERR_DEVICE_CHECK.
 * Errors: as fattn_fwd_paged and the shaped calls; INVALID_ARG also for a decay that is not finite,
 *   negative lse strides; UNSUPPORTED for d not in {64, 128}, B or Hkv > 65535.
 */
fattn_status fattn_key_weights_paged(const void* q, const void* kcache, const int32_t* block_table,
                                     const int32_t* seqlens_k, const int32_t* cu_seqlens_q, const float* lse,
                                     long long lse_head, long long lse_row, const float* weights_in, float* weights_out,
                                     int B, int Hq, int Hkv, int d, int page_size, int max_pages_per_seq, int num_pages,
                                     int total_q, int max_seqlen_q, int causal, float scale, float softcap,
                                     const float* slopes, int window, float decay, cudaStream_t stream);

/*
 * fattn_evict_paged — every KV head of every sequence cut down to `keep` tokens.
 *
 * Of a sequence's n = seqlens[b] tokens, every head keeps on its own m = min(n, keep): all of them if
 * n <= keep, else the first `first`, the last `recent` and, of the others, the heaviest by
 * weights_in[b, hkv, t] (of equal weights the lowest index; NaN is below every number). The kept
 * tokens, in their order, become tokens 0 .. m - 1: K and V rows move to those slots (bit for bit),
 * and seqlens_out[b] = m, weights_out[b, hkv, :m] their weights (0 in the rest of the row),
 * kept[b, hkv, :m] their old indices (-1 in the rest). Keys carry their rotary positions with them;
 * distances measured by slot (a window, a distance bias) no longer are those of the text.
 *
 * dst_table: DEVICE int32 [B, dst_max_pages], the pages (of the same pool) the kept tokens go to, not
 *   in use by any sequence of the call; or NULL: in place, in the sequence's own first pages
 *   (dst_max_pages = max_pages_per_seq), which then no other sequence may share.
 * weights_in [B, Hkv, max_pages_per_seq * page_size], weights_out [B, Hkv, dst_max_pages * page_size]
 *   (may be weights_in if the sizes agree), kept [B, Hkv, keep]; seqlens_out [B] is not seqlens.
 * A seqlens entry outside its table counts as an empty sequence; a row whose page is outside the pool
 *   is not moved; both record FATTN_ERR_DEVICE_CHECK. bf16 caches, any page_size >= 1.
 * Errors: INVALID_ARG (NULL or misaligned pointers, non-positive sizes, first + recent > keep, kept tokens
 *   that do not fit dst_max_pages, seqlens_out == seqlens); UNSUPPORTED (d not a multiple of 8 up to
 *   1024, B * Hkv > 65535, tables of 2^31 - 32768 tokens or more).
 */
fattn_status fattn_evict_paged(void* kcache, void* vcache, const int32_t* block_table, const int32_t* seqlens,
                               const float* weights_in, const int32_t* dst_table, int32_t* seqlens_out,
                               float* weights_out, int32_t* kept, int B, int Hkv, int d, int page_size,
                               int max_pages_per_seq, int num_pages, int dst_max_pages, int keep, int recent, int first,
                               cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FATTN_OPS_H */
