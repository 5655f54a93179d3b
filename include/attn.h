/* libgdn: a paged key-value cache and the attention that reads it (C ABI).
 *
 * The hybrid backbone puts one attention layer beside three GDN layers; at long context that
 * layer reads only the tokens its compressed indexer (qsa.h) lists ("論文解説: Qwen3.8-Next の
 * 設計" (ta-paperlens), sections "GDNの中身" and "部品②: QSA").  These calls are that layer's
 * serving side:
 *
 *   gdn_kv_append        rotate a call's queries and keys and put its keys and values into
 *                        the cache;
 *   gdn_attn_decode      attention of the newest token (or up to 8 drafted ones) of every
 *                        sequence over its whole cache;
 *   gdn_qsa_attn_decode  the same over the token lists of gdn_qsa_index_decode / _multi and
 *                        the newest tokens;
 *   gdn_attn_prefill     attention of prompts (packed, each behind tokens cached earlier).
 *
 * With p the position of a query, h its head and h' = h / (H_q / H_kv) its key head:
 *
 *     x_t = scale * q . k_t                 (k_t, v_t: key and value of token t, head h')
 *     x_t = softcap * tanh(x_t / softcap)   unless softcap is 0 (else 1e-4 .. 1e6)
 *     out = sum_t exp(x_t) v_t / sum_t exp(x_t),   lse = ln sum_t exp(x_t)
 *
 * over the tokens t that the query sees (each call says which).  A query that sees none
 * gets out = 0 and lse = -inf.  Scores, running maxima and sums are fp32; with bf16 inputs
 * the weights exp(x_t - max) are rounded to bf16 for the product with v, and the cap is off by up to
 * 2^-20 of the score.
 *
 * scale is any finite number, without a cap at most 2.3e38 in magnitude (else
 * GDN_ERR_INVALID_ARG).  Every q . k, and without a cap every scale q . k (2.3e38 at most), of a
 * visible token must be finite in fp32: a score that overflows is not a number in out and lse.
 *
 * The cache.  Token t of sequence n is row t % page_size of page
 * page_table[n, t / page_size].  A token is absent (nobody sees it, and appending it writes
 * nothing) when t / page_size >= max_pages or that entry lies outside [0, num_pages), so
 * entries that no live token uses may hold anything.  Rows of the cache that hold no live
 * token may hold anything too (NaN included); queries, and the keys and values of live
 * tokens, must be finite.  Two sequences may share pages that neither appends to.
 *
 * Ownership and errors follow gdn.h: the caller owns every buffer (device memory unless
 * stated); nothing allocates, frees or synchronises; argument checks run on the host and
 * return before anything is enqueued.  Outputs overlap no input, except q_out as stated below.
 */
#ifndef LIBGDN_ATTN_H
#define LIBGDN_ATTN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ATTN_MAX_QUERIES 8     /* largest n_queries of the decode calls               */
#define GDN_ATTN_MAX_LIST 16384    /* largest list_len of gdn_qsa_attn_decode             */
#define GDN_ROPE_MAX_AXES 3        /* largest number of position axes                     */

/* A paged cache (a host struct; the call reads it before it returns). */
typedef struct {
    void *k, *v;                   /* [num_pages, page_size, H_kv, d], 16-byte aligned    */
    const int32_t *page_table;     /* DEVICE [num_seqs, max_pages]                        */
    int32_t num_pages, max_pages;
    int32_t page_size;             /* a power of two, 16 .. 1024                          */
    int32_t H_kv, d;               /* key heads; head dim, 64 or 128                      */
    gdn_dtype dtype;               /* of k, v and of every q, k, v, out below             */
} gdn_paged_kv;

/* rope_sections' frequencies are dealt in turn (t, h, w, t, h, w, ...) instead of in runs. */
#define GDN_ROPE_INTERLEAVED 1u

/* Append.  Token i of sequence n goes to position pos0[n] + i; its key is rotated, its value
 * copied, and, when q is given, its queries are rotated into q_out.
 *   k, v       : [T_total, H_kv, d], tokens k_stride / v_stride elements apart (so a fused
 *                projection's output can be passed as it is); heads and dims contiguous.
 *   q, q_out   : [T_total, H_q, d] or both NULL; q has tokens q_stride elements apart,
 *                q_out is contiguous and may equal a contiguous q.
 *   cu_seqlens : DEVICE int32[num_seqs + 1] token offsets (non-decreasing, from 0), or NULL
 *                for num_seqs sequences of T_total / num_seqs tokens each.  Tokens from
 *                cu_seqlens[num_seqs] on are left alone (q_out too).
 *   pos0       : DEVICE int32[num_seqs] position of each sequence's first token, or NULL
 *                for 0.  A token at a negative position is not put into the cache.
 * The rotation turns the pairs (i, i + rope_dims / 2), i < rope_dims / 2, by the angle
 * position * inv_freq[i]; dims from rope_dims on pass through.
 *   rope_dims  : 0 (no rotation) or a multiple of 16 up to d.
 *   inv_freq   : DEVICE fp32 [rope_dims / 2].  The angle is formed and reduced in 64 bits.
 *   rope_pos   : DEVICE int32 [n_axes, T_total] positions to rotate at, or NULL: the token's
 *                cache position (then n_axes is 1).
 *   rope_sections: HOST int32[n_axes], the number of frequencies of each axis (sum
 *                rope_dims / 2), or NULL with one axis.  Axis 0 takes the first
 *                rope_sections[0] frequencies, axis 1 the next ones, and so on; with
 *                GDN_ROPE_INTERLEAVED frequency i belongs to axis a = i % n_axes as long as
 *                i < n_axes * rope_sections[a], else to axis 0.
 * Pointers 16-byte aligned (the int32 and fp32 tables 4), strides multiples of 16 bytes.
 * If two tokens of a call fall on the same row, what it holds then is not defined (parts of both). */
gdn_status gdn_kv_append(const gdn_paged_kv *kv, const void *k, const void *v, const void *q,
                         void *q_out, int64_t k_stride, int64_t v_stride, int64_t q_stride,
                         const int32_t *cu_seqlens, const int32_t *pos0, int32_t num_seqs,
                         int64_t T_total, int32_t H_q, const float *inv_freq, int32_t rope_dims,
                         const int32_t *rope_pos, const int32_t *rope_sections, int32_t n_axes,
                         uint32_t flags, cudaStream_t stream);

/* Bytes of device workspace the two decode calls need on the current device.  The first 16
 * bytes are the device error word, as in gdn.h: zero-fill them before first use for
 * gdn_get_device_error to be read; the calls write there nothing but an error, and need no other
 * contents, so one workspace can serve decode calls and prompts in turn.  Calls that share one must
 * not overlap on the GPU.  The size does not depend on the lengths, so a captured graph can be
 * replayed as the sequences grow.  0 for sizes the calls refuse. */
size_t gdn_attn_decode_workspace_size(int32_t n_queries, int32_t H_q, int32_t H_kv, int32_t d,
                                      gdn_dtype dtype);

/* Decode.  Query j of sequence n sits at position p = q_pos[n] + j and sees the tokens
 * 0 <= t <= p, with window > 0 only those with t > p - window.
 *   q, out   : [num_seqs, n_queries, H_q, d], 1 <= n_queries <= GDN_ATTN_MAX_QUERIES
 *   q_pos    : DEVICE int32 [num_seqs]; a query at a negative position sees nothing, so an idle
 *              slot has q_pos = -n_queries
 *   lse      : [num_seqs, n_queries, H_q] fp32 or NULL
 * The tokens' keys and values, the queries' own among them, are in the cache already.
 * (Many drafted tokens of wide groups run on gdn_attn_prefill's bf16 kernel, with its bounded
 * waits: a timeout is recorded in the workspace's error word.) */
gdn_status gdn_attn_decode(const void *q, const int32_t *q_pos, const gdn_paged_kv *kv,
                           void *out, float *lse, int32_t num_seqs, int32_t n_queries,
                           int32_t H_q, float scale, float softcap, int32_t window,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Decode over lists.  Query j of sequence n, at p = q_pos[n] + j, sees the newest `recent`
 * tokens p - recent < t <= p (t >= 0) and the listed tokens 0 <= t <= p - recent.  Other
 * entries of a list (the -1 that pads it, tokens of the newest ones, later tokens) are
 * skipped; a token listed twice counts twice.
 *   token_idx : DEVICE int32 [num_seqs, n_queries, list_len], as the indexer writes it
 *               (0 <= list_len <= GDN_ATTN_MAX_LIST; NULL when list_len is 0)
 *   recent    : 0 .. 65536
 * The other arguments are those of gdn_attn_decode. */
gdn_status gdn_qsa_attn_decode(const void *q, const int32_t *q_pos, const gdn_paged_kv *kv,
                               const int32_t *token_idx, int32_t list_len, int32_t recent,
                               void *out, float *lse, int32_t num_seqs, int32_t n_queries,
                               int32_t H_q, float scale, float softcap, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream);

/* Bytes of device workspace that let gdn_attn_prefill use its fastest form for these sizes on the
 * current device, at least 256; 0 for sizes it refuses.  varlen: nonzero when cu_seqlens is given.
 * It depends on what the page table can hold, not on the lengths.  Calls that share a workspace
 * must not overlap on the GPU.
 *
 * Prompts.  Query i of sequence n sits at position p = pos0[n] + i; with e = pos0[n] plus the
 * sequence's tokens in this call, it sees the tokens 0 <= t < e with t <= p, with window > 0
 * only those with t > p - window, and with prefix_len those with t < prefix_len[n] too (a
 * prefix that is seen both ways).
 *   q, out     : [T_total, H_q, d]; rows from cu_seqlens[num_seqs] on are left alone
 *   cu_seqlens : DEVICE int32[num_seqs + 1], or NULL for num_seqs sequences of
 *                T_total / num_seqs tokens each
 *   pos0       : DEVICE int32[num_seqs] tokens cached before this call (>= 0), or NULL for 0
 *   prefix_len : DEVICE int32[num_seqs] or NULL; GDN_ERR_UNSUPPORTED together with a window
 *   lse        : [T_total, H_q] fp32 or NULL
 *   workspace  : device memory whose first 16 bytes hold the device error word (zero-filled
 *                before first use; gdn_get_device_error reads it), or NULL: a device-side
 *                timeout is then not reported.  With gdn_attn_prefill_workspace_size bytes a
 *                call of few query rows behind a long context is split over the context's
 *                length (results differ by rounding); with less it runs in one piece.
 * Keys and values of the call's own tokens are in the cache already. */
size_t gdn_attn_prefill_workspace_size(const gdn_paged_kv *kv, int32_t varlen, int32_t num_seqs,
                                       int64_t T_total, int32_t H_q);
gdn_status gdn_attn_prefill(const void *q, const gdn_paged_kv *kv, const int32_t *cu_seqlens,
                            const int32_t *pos0, const int32_t *prefix_len, void *out,
                            float *lse, int32_t num_seqs, int64_t T_total, int32_t H_q,
                            float scale, float softcap, int32_t window, void *workspace,
                            size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBGDN_ATTN_H */
