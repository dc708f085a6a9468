/*
 * gdn2_attn.h -- C ABI of the attention-layer operators that run beside the
 * GDN-2 forward of gdn2.h, in the same library: a model that mixes GDN-2
 * layers with softmax-attention layers feeds both from one packed batch
 * (cu_seqlens).  A GDN-2 layer carries a state per sequence, an attention
 * layer a paged key/value cache.
 *
 *   gdn2_qk_norm_rope    RMS norm of the queries and keys of each head and
 *                        the rotary position embedding, in one pass
 *   gdn2_kv_append       the new tokens' keys (normed, rotated) and values
 *                        into a paged cache; the queries may ride along
 *   gdn2_paged_attn_fwd  softmax attention of the new tokens (1 .. many per
 *                        sequence) over the paged cache
 *
 * The conventions of gdn2.h hold: device pointers, buffers owned by the
 * caller, no allocation, no synchronisation, argument errors found on the
 * host before anything is enqueued, GDN2_ERR_ARCH on a device other than
 * compute capability 10.3.
 */
#ifndef GDN2_ATTN_H
#define GDN2_ATTN_H

#include "gdn2.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Problem description.  Tensors hold bf16 or fp16 (`dtype`, all alike).
 * Strides are in ELEMENTS; like base pointers they are multiples of 16
 * bytes, and the channel stride is 1.
 *
 *   q, q_out, out    [T_tot, HQ,  D]   strides (token, head)
 *   k, k_out, v      [T_tot, HKV, D]
 *   q_weight, k_weight  [D]            at `dtype`, contiguous
 *   inv_freq         [rot_dim / 2]     double: angle per position (radians)
 *   positions        [T_tot]           int32, or int64 with positions_i64 = 1
 *   k_cache, v_cache [num_pages, page_size, HKV, D], strides (page, token in
 *                    the page, head): token-major and head-major pages are
 *                    both views of this shape
 *   block_table      [N, max_pages]    int32; entry j of row n is the page of
 *                    tokens j * page_size .. of sequence n; table_stride is at
 *                    least max_pages
 *   cu_seqlens       [N + 1]           int32, or int64 with cu_seqlens_i64 = 1:
 *                    the new tokens of sequence n are rows cu[n] .. cu[n + 1)
 *   kv_lens          [N]               int32: tokens of sequence n in the cache
 *                    once the new ones are in, so new token j of sequence n
 *                    has place kv_lens[n] - (cu[n + 1] - cu[n]) + j
 *   lse              [T_tot, HQ]       fp32, contiguous
 *
 * Supported: D in {64, 128}; rot_dim a multiple of 16 in 0 .. D; page_size a
 * multiple of 8; num_pages >= 1; HQ a multiple of HKV with at most 128 query
 * heads per key head (gdn2_qk_norm_rope takes any two head counts); T_tot and
 * max_pages * page_size below 2^31 - 2^16.
 */
typedef struct gdn2_attn_dims {
    int64_t T_tot;
    int64_t num_pages;
    int64_t q_stride[2], k_stride[2], v_stride[2];
    int64_t qo_stride[2];      /* q_out, or out                                    */
    int64_t ko_stride[2];      /* k_out                                            */
    int64_t kc_stride[3], vc_stride[3];
    int64_t table_stride;      /* between rows of block_table                      */
    int32_t N, HQ, HKV, D;
    int32_t page_size, max_pages;
    int32_t dtype;             /* GDN2_DTYPE_BF16 or GDN2_DTYPE_F16                */
    int32_t cu_seqlens_i64, positions_i64;
    int32_t norm;              /* 1: RMS norm of q and k rows before the rotation  */
    int32_t rot_dim;           /* leading channels that are rotated; 0: none       */
    int32_t rope_interleaved;  /* 0: pairs (i, i + rot_dim / 2); 1: (2i, 2i + 1)   */
    int32_t causal;            /* 1: a token attends to keys up to its own place   */
    int32_t window_left;       /* >= 0 (with causal): and not further back than    */
                               /* this many; -1: no window                         */
    float norm_eps;
    float rope_factor;         /* on cos and sin (attention factor of some         */
                               /* long-context scalings); 1 for none               */
} gdn2_attn_dims;

/*
 * Fill `dims` for contiguous tensors (caches [num_pages, page_size, HKV, D]):
 * bf16, int32 cu_seqlens and positions, norm on with eps 1e-6, rot_dim = D in
 * the half layout with factor 1, causal without a window.  Host-only.
 */
GDN2_API gdn2_status gdn2_attn_dims_init(gdn2_attn_dims *dims, int64_t T_tot, int32_t N, int32_t HQ, int32_t HKV,
                                         int32_t D, int64_t num_pages, int32_t page_size, int32_t max_pages);

/*
 * Norm and rotation of queries and keys.  Per row x of D channels, in fp32:
 *
 *     x <- x / sqrt(mean(x^2) + norm_eps) * weight          (norm = 1)
 *     (x_a, x_b) <- rope_factor (x_a cos - x_b sin, x_a sin + x_b cos),
 *                   angle = position * inv_freq[i], for each pair i
 *
 * and one rounding to `dtype` at the end.  The angle is reduced in 64-bit fixed
 * point before the sine and cosine: for frequencies up to 1 it is off by less
 * than |position| 2^-60 radians, nothing at 16 bits for int32 positions and up
 * to some 2^40; int64 positions far past that turn by angles that mean nothing.
 *
 *   q, q_out            both NULL: queries are left out; likewise k, k_out
 *                       (not both pairs)
 *   q_weight, k_weight  may be NULL: weight 1; not used with norm = 0
 *   inv_freq, positions may be NULL when rot_dim = 0
 *   q_out, k_out        may be q, k themselves (same strides): in place; any
 *                       other overlap with an input is GDN2_ERR_ALIAS
 *
 * One launch; no workspace.
 */
GDN2_API gdn2_status gdn2_qk_norm_rope(const void *q, const void *k, const void *q_weight, const void *k_weight,
                                       const double *inv_freq, const void *positions, void *q_out, void *k_out,
                                       const gdn2_attn_dims *dims, void *stream);

/* Workspace bytes of gdn2_kv_append (a 64-byte status area; 0 if the shape is
 * unsupported).  Host-only. */
GDN2_API size_t gdn2_kv_append_workspace_bytes(const gdn2_attn_dims *dims);

/*
 * Append the new tokens to the paged cache: keys normed and rotated as in
 * gdn2_qk_norm_rope, values as they are, each at its place's page and slot.
 * With q, the queries are normed and rotated into q_out in the same launch.
 *
 *   q, q_out       both NULL: keys and values only; q_out may be q
 *   positions      the rotation's positions; NULL: the places
 *   k_cache, v_cache  must not overlap an input; they may interleave in one
 *                  allocation, but not be the same tensor
 *
 * The cache's other slots are not touched.  No two new tokens may share a
 * slot (two sequences with the same page in reach of their new tokens): which
 * one stays would be left open.  A token whose place is negative or past
 * max_pages * page_size, or whose table entry is not in 0 .. num_pages - 1, is
 * left out and the device status (gdn2_device_status on the workspace) says
 * GDN2_ERR_PAGES; a bad cu_seqlens is reported as GDN2_ERR_CU_SEQLENS, and
 * then nothing is written outside the outputs, but what is written is
 * undefined.  One launch.
 */
GDN2_API gdn2_status gdn2_kv_append(const void *q, const void *k, const void *v, const void *q_weight,
                                    const void *k_weight, const double *inv_freq, const void *positions,
                                    const void *cu_seqlens, const int32_t *kv_lens, const int32_t *block_table,
                                    void *q_out, void *k_cache, void *v_cache, const gdn2_attn_dims *dims,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace gdn2_paged_attn_fwd needs for `dims` (0 if the
 * shape is unsupported).  Host-only. */
GDN2_API size_t gdn2_paged_attn_workspace_bytes(const gdn2_attn_dims *dims);

/*
 * Softmax attention of the new tokens over the paged cache, which holds their
 * keys and values already (gdn2_kv_append).  Query head h reads key head
 * h / (HQ / HKV).  For the new token at place p of a sequence with kv_len
 * cached tokens, over the keys c < kv_len with c <= p (causal) and
 * c >= p - window_left (window_left >= 0):
 *
 *     out = sum_c softmax_c(scale q . k_c) v_c,   lse = log sum_c exp(scale q . k_c)
 *
 * A row with no key left (kv_lens[n] smaller than the sequence's new tokens)
 * gives out = 0, lse = -inf.
 *
 *   scale   <= 0 means 1/sqrt(D)
 *   lse     may be NULL
 *   out     must not overlap an input
 *   caches  no zero strides (broadcast pages or heads)
 *
 * Scores, softmax statistics and sums are fp32; the weights are rounded to
 * `dtype` for the product with v.  What the cache holds past kv_len, or before
 * the window of a sequence's first new token, does not matter, NaN and
 * infinities included, and pages wholly before that window may be gone: their
 * table entries are not read.  A NaN or an infinity among the values that one
 * new token attends to may reach other new tokens of its sequence whose mask
 * leaves it out (as 0 x NaN).  A kv_len below 0 or past max_pages * page_size is
 * reported as GDN2_ERR_PAGES and a bad cu_seqlens as
 * GDN2_ERR_CU_SEQLENS (gdn2_device_status on the workspace); the call then
 * writes nothing.  A table entry in reach that is not in 0 .. num_pages - 1 is
 * reported as GDN2_ERR_PAGES; the outputs of its sequence are then undefined.
 */
GDN2_API gdn2_status gdn2_paged_attn_fwd(const void *q, const void *k_cache, const void *v_cache,
                                         const void *cu_seqlens, const int32_t *kv_lens, const int32_t *block_table,
                                         float scale, void *out, float *lse, const gdn2_attn_dims *dims,
                                         void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN2_ATTN_H */
