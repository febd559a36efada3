/*
 * fattn_ops.h — C ABI of libfattn, continued: what stands around the attention
 * calls of fattn.h in a model that trains on, or serves, long contexts.
 *
 *   - rotary positions on q and k (fattn_rope), and their serving form, which
 *     also puts the new tokens' k and v into the paged cache
 *     (fattn_rope_append_paged).
 *
 * The conventions of fattn.h hold: DEVICE pointers owned by the caller, host
 * checks before anything is launched, work enqueued on `stream`, no
 * allocation, no synchronisation, problems found on the device recorded in the
 * status word (fattn_debug_read_status). Strides count elements.
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

#ifdef __cplusplus
}
#endif

#endif /* FATTN_OPS_H */
