/*
 * molora_decoder.h — C ABI of the operators that a decoder layer needs around
 * the per-token adapters: routing by scores, causal attention with a window
 * and sink tokens (forward and backward), a paged key-value cache, the
 * attention of one new token over it, and the synthetic decoder's serving form
 * that runs them.
 *
 * The conventions of molora.h hold for every entry point: device pointers
 * belong to the current HIP device, the caller owns every buffer, every call
 * only enqueues on `stream` (capturable, no allocation, no synchronisation),
 * argument errors are found on the host before anything is enqueued, and
 * data-dependent conditions are not errors.  Results are deterministic: no
 * atomics enter any sum.
 */
#ifndef MOLORA_DECODER_H
#define MOLORA_DECODER_H

#include "molora.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOLORA_E4M3 = 2 }; /* 8-bit float, 4 exponent and 3 mantissa bits (OCP e4m3fn), next to MOLORA_BF16 */
enum { MOLORA_SCORE_SOFTMAX = 0, MOLORA_SCORE_SIGMOID = 1 };

/* ------------------------------------------------------------------------
 * Routing by scores: the top-k gate with a balance bias and adapter groups.
 *   logits  device fp32 [N][K]: gate logits
 *   bias    device fp32 [K] or NULL: added to the scores for the selection
 *           only (load balance without a loss term); it gets no gradient
 *   score   MOLORA_SCORE_SOFTMAX: s = softmax(logits) over the K adapters;
 *           MOLORA_SCORE_SIGMOID: s = 1 / (1 + exp(-logits))
 *   n_group, topk_group  adapters [g K / n_group, (g + 1) K / n_group) form
 *           group g; a group's mark is the sum of its two largest s + bias
 *           (of the only one where it has one), and the topk_group groups of
 *           the largest marks are kept
 *   idx     device int32 [N][k] out: the k largest s + bias of the kept
 *           groups, in ascending adapter index
 *   w       device fp32 [N][k] out: factor * s of the chosen adapters,
 *           divided by their sum when renorm != 0
 * Equal values are taken in ascending index.  The selection is the one of s +
 * bias in 64 bits (the kernel decides in 32 bits where the margin is wider
 * than their error and repeats a closer decision in 64); without a bias and
 * with one group it is the order of the logits themselves.  The weights are
 * in 32 bits.
 * An adapter whose logit is NaN or -inf is absent: its score is 0, it takes no
 * part in the softmax and is never chosen; neither is one whose bias is NaN or
 * -inf.  A group with no adapter to choose is kept only after all others.
 * Slots for which nothing is left to choose come last, with idx -1 and weight
 * 0 (unrouted, as molora_dispatch understands it).  +inf logits count as the
 * largest finite number.  A renormalised sum of 0 gives weights 0.
 * Supported: 1 <= K <= 64, 1 <= k <= min(K, 8), n_group divides K,
 * 1 <= topk_group <= n_group, k <= topk_group * K / n_group, N * K < 2^31,
 * N < 2^29, factor finite.
 *
 * molora_route_scores_backward: dL/dlogits with the selection held fixed.
 *   idx     as written by molora_route_scores (entries outside [0, K) receive
 *           nothing); the indices of one token are distinct
 *   dw      device fp32 [N][k]: dL/dw (molora_backward's dw)
 *   dlogits device fp32 [N][K] out: 0 for absent adapters.  Softmax scores:
 *           s_e (g_e - sum_j s_j g_j) over all adapters, with g_j = dL/ds_j;
 *           sigmoid scores: s_e (1 - s_e) g_e.
 * Same score, renorm and factor as the forward; the same limits.
 * Errors (nothing enqueued): shapes -> MOLORA_ENOTSUP; NULL or misaligned
 * pointers, an unknown score -> MOLORA_EINVAL.
 * ------------------------------------------------------------------------ */
int molora_route_scores(const float *logits, const float *bias, int N, int K, int k, int score,
                        int n_group, int topk_group, int renorm, float factor, int32_t *idx,
                        float *w, void *stream);
int molora_route_scores_backward(const float *logits, const int32_t *idx, const float *dw, int N,
                                 int K, int k, int score, int renorm, float factor,
                                 float *dlogits, void *stream);

/* ------------------------------------------------------------------------
 * Causal attention of packed sequences.
 * Sequence b holds the query rows [q_off[b], q_off[b+1]) and the key and value
 * rows [kv_off[b], kv_off[b+1]); its last query stands at its last key, so
 * query i of Lq has position p = i + Lkv - Lq.  It sees key j when j <= p and,
 * with a window, j > p - window or j < sinks (the first tokens that stay
 * visible).  o_i = sum_j softmax_j(scale q_i . k_j) v_j per head; a row that
 * sees nothing gets o = 0 and lse = -inf.
 *   q, o    device bf16 rows [Tq] of n_heads heads of head_dim values
 *   k, v    device bf16 rows [Tkv] of n_kv_heads heads; query head h reads
 *           head h / (n_heads / n_kv_heads)
 *   lse     device fp32 [n_heads][Tq] out or NULL: log sum_j exp(scale q.k_j)
 *   molora_rows describes one of them: element strides between tokens and
 *           between heads, multiples of 8; the values of a head are contiguous
 *           and 16-byte aligned (so q, k and v may lie in one buffer)
 *   q_off, kv_off  device int32 [n_seq + 1], non-decreasing, kv_off NULL: the
 *           same as q_off.  Offsets are limited to [0, Tq] and [0, Tkv].
 *   window  0: none (sinks has no effect); else at least 1
 * o must not overlap q, k or v (parts of one buffer may interleave).
 * Rows of o and entries of lse outside every sequence are left as they were,
 * and rows of q, k and v outside every sequence are not read into any result.
 * Infinities and NaN reach the results of the pairs that see them and no
 * others (rows of sums that share a tile with one are taken again, more slowly).
 * Products are bf16 with fp32 accumulation; the softmax runs in fp32 and its
 * weights enter the second product as bf16; o is rounded once at the store.
 * Where few query rows face many keys the keys are split over workgroups and
 * a second launch joins the parts.
 *   ws      device workspace of the call's *_workspace() bytes (which read the
 *           shape's numbers, not its pointers), 256-byte aligned, no initial
 *           contents (size 0: may be NULL); calls that share it must not
 *           overlap
 *
 * molora_attn_backward: dq, dk, dv (laid out as molora_rows like q, k, v) from
 * do = dL/do and the forward's o and lse.  Gradients of shared key-value heads
 * are summed in fp32 over their query heads.  Rows outside every sequence are
 * left as they were; rows that nothing sees get 0.
 * Supported: head_dim 64 or 128, 1 <= n_kv_heads, n_heads a multiple of it and
 * at most 1024, n_seq, Tq, Tkv >= 0 and below 2^24, (Tq / 128 + n_seq) *
 * n_heads and (Tkv / 128 + n_seq) * n_kv_heads below 2^24, token strides below 2^23,
 * scale positive and finite, sinks <= 2^24.
 * Errors (nothing enqueued): shapes -> MOLORA_ENOTSUP; NULL or misaligned
 * pointers, bad strides, outputs whose rows overlap, a negative window or
 * sinks, a bad scale -> MOLORA_EINVAL; a short workspace -> MOLORA_ENOSPC.
 * ------------------------------------------------------------------------ */
typedef struct {
  void *p;                  /* device bf16 */
  long long token, head;    /* element strides */
} molora_rows;
typedef struct {
  int n_seq, n_heads, n_kv_heads, head_dim;
  int Tq, Tkv;              /* rows of q (and o) and of k and v */
  const int32_t *q_off, *kv_off;
  int window, sinks;
  float scale;
} molora_attn_shape;
int molora_attn_forward_workspace(const molora_attn_shape *shape, size_t *bytes);
int molora_attn_forward(const molora_attn_shape *shape, const molora_rows *q, const molora_rows *k,
                        const molora_rows *v, const molora_rows *o, float *lse, void *ws,
                        size_t ws_bytes, void *stream);
int molora_attn_backward_workspace(const molora_attn_shape *shape, size_t *bytes);
int molora_attn_backward(const molora_attn_shape *shape, const molora_rows *dout, const molora_rows *q,
                         const molora_rows *k, const molora_rows *v, const molora_rows *o,
                         const float *lse, const molora_rows *dq, const molora_rows *dk,
                         const molora_rows *dv, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Paged key-value cache.  A pool of pages, each of page_size tokens of every
 * key-value head; sequence b's token at position j lies in page
 * table[b][j / page_size] at row j % page_size.
 *   k, v    device [n_pages][n_kv_heads][page_size][head_dim], bf16 or e4m3
 *   k_scale, v_scale  e4m3: device uint8 [n_pages][n_kv_heads][page_size],
 *           byte e, 1 <= e <= 254, standing for the factor 2^(e - 127) of its
 *           row; bf16: NULL
 * Supported: head_dim 64 or 128, page_size 16, 32, 64, 128 or 256.
 *
 * molora_kv_append writes the newest rows of every sequence: the rows
 * [q_off[b], q_off[b+1]) of k and v become the last ones of lens[b] tokens,
 * i.e. row i goes to position lens[b] - (q_off[b+1] - q_off[b]) + i - q_off[b].
 *   k, v    molora_rows of T tokens of the cache's heads
 *   q_off   device int32 [n_seq + 1], NULL: one row per sequence
 *   table   device int32 [n_seq][table_width]
 *   lens    device int32 [n_seq], lengths with the new rows
 * Rows whose position is negative or not below table_width * page_size, or
 * whose table entry is outside [0, n_pages), are skipped.  A page must not be
 * written by two sequences in one call.
 * e4m3: a row is stored as rne(x 2^-n) with the smallest n >= -112 that brings
 * its largest finite magnitude within 448, and byte n + 127 (a row of zeros:
 * n = -112).  Infinities become +-448, NaN stays NaN.
 *
 * molora_attn_decode: the attention of one new token per sequence, standing at
 * the last of its lens[b] positions, whose key and value are in the cache.
 *   q, o    molora_rows of n_seq rows of n_heads heads; o may be q
 *   lse     device fp32 [n_seq][n_heads] out or NULL
 *   lens    device int32 [n_seq]; a negative length counts as 0, one above
 *           table_width * page_size as that; length 0 gives o = 0, lse = -inf
 * Visible are the positions molora_attn_forward would see (window, sinks); a
 * position whose table entry is outside [0, n_pages) is not visible, and
 * nothing of a row that is not visible is used, whatever it holds: pages
 * between the sinks and the window may be freed.
 * A sequence's positions are split over workgroups, on the device and by its
 * own length; a second launch joins the parts.
 *   ws      device workspace of molora_attn_decode_workspace() bytes, 256-byte
 *           aligned, no initial contents (size 0: may be NULL); calls that
 *           share it must not overlap
 * Supported: n_heads a multiple of n_kv_heads and at most 1024,
 * n_seq * n_heads < 2^24, table_width * page_size < 2^30.
 * Errors as molora_attn_forward.
 * ------------------------------------------------------------------------ */
typedef struct {
  void *k, *v;
  uint8_t *k_scale, *v_scale;
  int n_pages, n_kv_heads, page_size, head_dim;
  int dtype; /* MOLORA_BF16 or MOLORA_E4M3 */
} molora_kv_cache;
int molora_kv_append(const molora_kv_cache *cache, const molora_rows *k, const molora_rows *v, int T,
                     int n_seq, const int32_t *q_off, const int32_t *table, int table_width,
                     const int32_t *lens, void *stream);
int molora_attn_decode_workspace(const molora_kv_cache *cache, int n_seq, int n_heads,
                                 int table_width, size_t *bytes);
int molora_attn_decode(const molora_kv_cache *cache, const molora_rows *q, const molora_rows *o,
                       float *lse, int n_seq, int n_heads, const int32_t *table, int table_width,
                       const int32_t *lens, int window, int sinks, float scale, void *ws,
                       size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The synthetic decoder of molora_xf_forward in its serving form, over one
 * paged cache per layer (d / 128 heads of 128 values, all of one page_size)
 * that share table and lens.
 * molora_xf_prefill runs the prompts that open n_seq sequences, N packed tokens
 * with the rows [q_off[b], q_off[b+1]) of sequence b: every layer appends its
 * keys and values to its cache and attends as molora_attn_forward does.
 * lens[b] has to be the number of sequence b's rows.
 * molora_xf_decode runs one new token per sequence: every layer appends it
 * at position lens[b] - 1 and attends over the cache (molora_attn_decode).
 * The projections, adapters, norms and rounding points are molora_xf_forward's,
 * and so are d, f, layers, k and the routing (offsets, perm, perm_w, inv of
 * molora_dispatch for the N, or n_seq, tokens).  window, sinks: as
 * molora_attn_forward, the same for every layer.
 *   x_in, x_out  device bf16 [N][d] (n_seq rows for molora_xf_decode; x_out
 *                may equal x_in); rows outside every sequence are undefined
 *   ws           molora_xf_serve_workspace() bytes for N tokens (n_seq for
 *                molora_xf_decode), 256-byte aligned, no initial contents
 * The layers' adapters have one rank (padded to a multiple of 16), else
 * MOLORA_ENOTSUP.
 * Errors as molora_xf_forward and the operators above.
 * ------------------------------------------------------------------------ */
int molora_xf_serve_workspace(int d, int f, int n_layers, const molora_xf_layer *layers,
                              const molora_kv_cache *caches, int n_seq, int N, int table_width, int k,
                              size_t *bytes);
int molora_xf_prefill(int d, int f, int n_layers, const molora_xf_layer *layers,
                      const molora_kv_cache *caches, int n_seq, int N, const int32_t *q_off,
                      const int32_t *table, int table_width, const int32_t *lens, int window, int sinks,
                      const void *x_in, void *x_out, int k, const int32_t *offsets, const int32_t *perm,
                      const float *perm_w, const int32_t *inv, void *ws, size_t ws_bytes, void *stream);
int molora_xf_decode(int d, int f, int n_layers, const molora_xf_layer *layers,
                     const molora_kv_cache *caches, int n_seq, const int32_t *table, int table_width,
                     const int32_t *lens, int window, int sinks, const void *x_in, void *x_out, int k,
                     const int32_t *offsets, const int32_t *perm, const float *perm_w, const int32_t *inv,
                     void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOLORA_DECODER_H */
