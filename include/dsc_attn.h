/*
 * dsc_attn.h -- C ABI of the attention operators of libdsc.so: what follows
 * the short convolution on the Q, K and V projections ("Dynamic Short
 * Convolutions Improve Transformers", technical summary, Methodology,
 * "Placement": the convolution acts on Q, K and V before the rotary position
 * embedding).
 *
 *   rotation   dsc_fwd_rope_varlen, dsc_bwd_rope_varlen
 *   attention  dsc_fwd_attn_varlen, dsc_bwd_attn_varlen  (packed documents)
 *   serving    dsc_kv_append, dsc_decode_attn            (paged key-value cache)
 *
 * The conventions of dsc.h hold here too (caller-owned device pointers,
 * 16-byte aligned; the caller's stream; workspaces passed in; no
 * synchronisation, no allocation; status codes; nothing is launched when
 * validation fails), with these additions.
 *
 *  - Rows and heads.  q holds T rows of Hq heads of d elements, k and v T rows
 *    of Hkv heads; Hq % Hkv == 0, and query head h reads key/value head
 *    h / (Hq / Hkv).  The heads of a row are contiguous; consecutive rows are
 *    q_stride, k_stride and v_stride elements apart, so q, k and v may be views
 *    of one [T, (Hq + 2 Hkv) d] projection.  Strides are at least the row's
 *    width and rows start at multiples of 16 bytes (else DSC_ERR_INVALID_ARG,
 *    DSC_ERR_MISALIGNED).  d is a multiple of 8, 8 <= d <= 128.
 *  - Packed documents are given as in the *_varlen calls of dsc.h: cu_seqlens
 *    int32 [n_docs + 1] on the device, document i being rows cu_seqlens[i] ..
 *    cu_seqlens[i+1]-1; empty documents are allowed.  Offsets are clamped into
 *    [0, T] and a document that would end before it starts is empty, so a
 *    malformed array gives wrong values, never an access out of bounds (the
 *    attention takes documents that overlap so often that they need more tiles
 *    than n_docs documents in T rows can have for no documents at all).  Rows
 *    that no document holds (padding behind the last one) are not read; the
 *    outputs' rows there are set to zero, lse to -infinity.
 *  - dtype DSC_BF16: q, k, v, o, dout, dq, dk, dv and the caches are bf16;
 *    products accumulate in fp32, softmax statistics are fp32, and the
 *    probabilities (and dS in the backward) are rounded to bf16 as operands of
 *    the tensor cores' second product.  DSC_F32: everything fp32.  lse is
 *    always fp32.
 *  - The weighted values are summed up before the division by the weights' sum,
 *    no weight above one: the number of keys times the largest |v| must stay
 *    below fp32's largest number (3.4e38), or the sum becomes infinite.
 *  - Limits: 1 <= T <= 2^30, T * Hq < 2^38, Hq <= 1024, n_docs <= 2^24 and, for
 *    the attention over documents, (T / 32 + n_docs + 2) * Hq < 2^31 - 2^20
 *    (else DSC_ERR_UNSUPPORTED).
 */
#ifndef DSC_ATTN_H
#define DSC_ATTN_H

#include "dsc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of an attention problem.  scale multiplies q.k (usually 1/sqrt(d));
 * it must be positive and finite. */
typedef struct {
    int64_t T, Hq, Hkv, d;
    int64_t q_stride, k_stride, v_stride;
    int32_t dtype; /* dsc_dtype */
    float scale;
} dsc_attn_problem;

/* Shape of a rotation (and append) problem.  rot: the leading elements of each
 * head that are rotated (even, 0 <= rot <= d); the others pass through.
 * interleaved: 0 pairs elements (i, i + rot/2), 1 pairs (2i, 2i+1). */
typedef struct {
    int64_t T, Hq, Hkv, d, rot;
    int64_t q_stride, k_stride, v_stride;
    int32_t dtype; /* dsc_dtype */
    int32_t interleaved;
} dsc_rope_problem;

/* A paged cache: k_cache and v_cache are [n_pages, Hkv, page, d], dense;
 * block_table int32 [sequences, max_pages]: token t of sequence s lies in page
 * block_table[s][t / page], slot t % page.  page >= 1; n_pages, max_pages >= 1
 * and max_pages * page <= 2^30.  A table entry outside [0, n_pages) is a
 * missing page: nothing is written to it, and a token on it counts as masked
 * when it is read. */
typedef struct {
    int64_t n_pages, page, max_pages;
} dsc_paged_cache;

/* ------------------------------------------------------------- attention ---
 * Per document of n rows, head h, kv head h' = h / (Hq/Hkv):
 *   S_ij  = scale * q_i . k_j                    for j <= i (causal)
 *   lse_i = log sum_{j<=i} exp(S_ij),   o_i = sum_{j<=i} exp(S_ij - lse_i) v_j
 * o is [T, Hq, d] dense, lse [Hq, T] dense fp32. */
DSC_API size_t dsc_fwd_attn_varlen_workspace_bytes(const dsc_attn_problem *p, int64_t n_docs);
DSC_API dsc_status dsc_fwd_attn_varlen(const dsc_attn_problem *p, const int32_t *cu_seqlens, int64_t n_docs,
                                       const void *q, const void *k, const void *v, void *o, float *lse,
                                       void *workspace, size_t workspace_bytes, void *stream);

/* Gradients, from the forward's o and lse and the gradient dout [T, Hq, d]
 * (dense) of o:
 *   P_ij = exp(S_ij - lse_i),  D_i = dout_i . o_i = sum_j P_ij dout_i . v_j
 *   dS_ij = P_ij (dout_i . v_j - D_i)
 *   dq_i = scale sum_j dS_ij k_j
 *   dk_j = scale sum_{h in group, i>=j} dS_ij q_i,   dv_j = sum_{h in group, i>=j} P_ij dout_i
 * dq [T, Hq, d], dk and dv [T, Hkv, d] with rows dq_stride, dk_stride and
 * dv_stride elements apart (they may be views of one gradient of a packed
 * projection; the elements between rows are not touched).  With DSC_BF16, D
 * is summed up from P in fp32 and o is not read; a row that is not
 * finite may also show in the rows of its own tile of 128 that it does not reach
 * by the formula (a masked pair's zero is multiplied with it); with DSC_F32 and
 * in the forward it does not.  Deterministic: no sum depends on the order in
 * which blocks run. */
DSC_API size_t dsc_bwd_attn_varlen_workspace_bytes(const dsc_attn_problem *p, int64_t n_docs);
DSC_API dsc_status dsc_bwd_attn_varlen(const dsc_attn_problem *p, const int32_t *cu_seqlens, int64_t n_docs,
                                       const void *q, const void *k, const void *v, const void *o, const float *lse,
                                       const void *dout, void *dq, int64_t dq_stride, void *dk, int64_t dk_stride,
                                       void *dv, int64_t dv_stride, void *workspace, size_t workspace_bytes,
                                       void *stream);

/* Failure-detection self-test of the tensor-core kernels' hand-over of work, as
 * dsc_selftest_timeout: one small kernel whose waits for an item run out (limit
 * about 5 ms).  No item is taken, and the next dsc_check() on the stream
 * returns DSC_ERR_TIMEOUT and clears it (DSC_ERR_CUDA if one was taken). */
DSC_API dsc_status dsc_selftest_attn_timeout(void *stream);

/* -------------------------------------------------------------- rotation ---
 * Row t of a document at place m (0 for its first row): each pair (a, b) of a
 * head becomes (a cos x - b sin x, a sin x + b cos x), x = m * inv_freq[i],
 * i = 0 .. rot/2 - 1 the pair's index, inv_freq fp32 [rot/2] on the device
 * (may be NULL when rot = 0).  The angle is formed and reduced in fp64, so far
 * positions keep their phase.  q_out [T, Hq, d] and k_out [T, Hkv, d] are
 * dense.  v_stride is ignored. */
DSC_API dsc_status dsc_fwd_rope_varlen(const dsc_rope_problem *p, const int32_t *cu_seqlens, int64_t n_docs,
                                       const void *q, const void *k, const float *inv_freq, void *q_out, void *k_out,
                                       void *stream);
/* Gradient: the rotation by the negative angles, of dq and dk. */
DSC_API dsc_status dsc_bwd_rope_varlen(const dsc_rope_problem *p, const int32_t *cu_seqlens, int64_t n_docs,
                                       const void *dq, const void *dk, const float *inv_freq, void *dq_out,
                                       void *dk_out, void *stream);

/* --------------------------------------------------------------- serving ---
 * Append new rows to a paged cache.  Sequence s brings n_s rows: rows
 * cu_seqlens[s] .. cu_seqlens[s+1]-1, or row s alone when cu_seqlens is NULL
 * (then n_seqs = T).  seq_lens int32 [n_seqs] (device) counts the sequence's
 * tokens with the new ones, so the new rows take the positions seq_lens[s] -
 * n_s + i.  Each row's k is rotated by its position and written with v to the
 * row's slot; q is rotated into q_out [T, Hq, d] and, when k_out is not NULL,
 * the rotated k also into k_out [T, Hkv, d] (both dense).  q and q_out may be
 * NULL together (then Hq is ignored but still checked).  Rows at a negative
 * position, beyond max_pages * page or on a missing page write no slot.  Rows
 * that no sequence holds write no slot and zeros to q_out and k_out.  Two rows
 * that fall on the same slot leave some elements of either there. */
DSC_API dsc_status dsc_kv_append(const dsc_rope_problem *p, const dsc_paged_cache *c, const int32_t *cu_seqlens,
                                 int64_t n_seqs, const int32_t *seq_lens, const int32_t *block_table, const void *q,
                                 const void *k, const void *v, const float *inv_freq, void *q_out, void *k_out,
                                 void *k_cache, void *v_cache, void *stream);

/* Attention of one new token per sequence over the first seq_lens[s] slots of
 * its cache (the new token's own key and value among them: append first).
 * p->T sequences; q [T, Hq, d] with rows q_stride apart (k_stride and v_stride
 * are ignored); o [T, Hq, d] dense, lse [T, Hq] fp32 or NULL.  Lengths are
 * clamped into [0, max_pages * page]; a sequence with nothing to read (length
 * 0, or every page missing) gets zeros and lse -infinity.  The cache's length
 * is split over the GPU and the parts are joined in a fixed order. */
DSC_API size_t dsc_decode_attn_workspace_bytes(const dsc_attn_problem *p, const dsc_paged_cache *c);
DSC_API dsc_status dsc_decode_attn(const dsc_attn_problem *p, const dsc_paged_cache *c, const int32_t *seq_lens,
                                   const int32_t *block_table, const void *q, const void *k_cache,
                                   const void *v_cache, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                   void *stream);

#ifdef __cplusplus
}
#endif
#endif /* DSC_ATTN_H */
