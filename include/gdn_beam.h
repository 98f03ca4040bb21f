/*
 * gdn_beam.h -- C ABI of beam search over a hybrid decoder: the selection of the best
 * continuations of every group of beams, and the reordering of their recurrent states, page
 * tables and pages after it.  Part of libgdn.so; statuses, dtypes, streams, scratch and
 * error reporting as in gdn.h: arguments are checked synchronously, work is enqueued on
 * `stream`, errors found by a kernel (an index outside its range) are reported by
 * gdn_sync_check() as GDN_ERR_INVALID_ARG, and leave what they concern unspecified.
 * Pointers are device memory but where said otherwise; int32 and fp32 arrays are aligned to
 * 4 bytes (GDN_ERR_ALIGNMENT).
 *
 * B groups (requests) have W beams each, 1 <= W <= 32 (GDN_ERR_UNSUPPORTED above); beam w of
 * group b is beam b W + w of the call.
 */
#ifndef GDN_BEAM_H
#define GDN_BEAM_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The n best of the W V continuations of every group, best first:
 *     score(w, v) = scores[b][w] + logits[b W + w][v] - log sum_u exp(logits[b W + w][u]).
 *   logits    [B W][V] of dtype dt, rows stride_row elements apart (any number; the base
 *             is aligned to its elements).
 *   scores    fp32 [B][W].
 *   done      uint8 [B][W], or NULL: a beam that is done (not 0) goes on with token `eos`
 *             alone, at the score that it has; its other continuations score -infinity.
 *   out_scores, out_beam, out_token   fp32, int32, int32 [B][n]: the continuation's score,
 *             its beam w and its token v.
 *   n         1 .. 32 (GDN_ERR_UNSUPPORTED above), at most W V.
 *   V         at most 2^22 (GDN_ERR_UNSUPPORTED above).
 * Equal scores go to the lowest (w, v).  Scores are compared as sums of two fp32 numbers (48
 * bits), formed from the logits exactly and from a logarithm that is within some 2^-21 of its
 * own, whatever the logits' magnitude; they are rounded to fp32 in out_scores, and count as
 * -infinity where that overflows.  Within a beam they fall with the logits: what rounding would
 * put above a larger logit's counts as equal to it.
 * A logit of -infinity scores -infinity, and so do all continuations of a beam whose score is
 * -infinity or whose logits all are.  A NaN or +infinity among a beam's logits makes all its
 * continuations NaN, and a NaN ranks before every number, so that it is seen.  The logits of a
 * beam that is done, or whose score is -infinity, do not matter, but are memory that is read
 * all the same.  Scores are numbers or -infinity.  The same inputs give the same bits, and equal
 * rows of a call equal scores.
 */
gdn_status gdn_beam_select(const void *logits, int64_t stride_row, const float *scores,
                           const uint8_t *done, int eos, float *out_scores, int32_t *out_beam,
                           int32_t *out_token, int B, int W, int V, int n, gdn_dtype dt,
                           void *stream);

/* `count` rows of `bytes` bytes each, one after the other from `data` (16-byte aligned;
 * bytes a multiple of 16): the states of a layer by lane, or the pages of a cache. */
typedef struct {
    void *data;
    int64_t bytes;
    int count;
} gdn_beam_pool;

/* Page tables of the beams, and the pages that each lane may write.  All beams of a group
 * have the same number of tokens. */
typedef struct {
    const int32_t *page_table;    /* [B W][max_pages], rows table_stride apart */
    int32_t *table_out;           /* [B W][max_pages], rows out_stride apart */
    const int32_t *own_pages;     /* [lanes][max_pages], rows own_stride apart */
    const int32_t *kv_len;        /* [B W] */
    int max_pages, page_size;     /* page_size: a power of two */
    int64_t table_stride, out_stride, own_stride;
} gdn_beam_tables;

/*
 * Makes beam w of group b go on from beam parent[b][w] of the group, for all w at once.
 *
 * A lane is a place for one beam: a row of every pool of states, and pages own_pages[lane]
 * for every place of a page table.  slots[b][w] is the lane that beam w has; the lanes of
 * a call's beams are distinct.  Of the beams that go on from the same one, the lowest
 * keeps its parent's lane, and nothing of it moves; the others take, in order, the lanes of
 * the group's beams from which none goes on, in order, and what the parent has is copied
 * there: only so much is read and written.  (gdn_decode takes slots_out as its slots.)
 *   parent, slots, slots_out   int32 [B][W]; lanes below `lanes`.
 *   states    HOST array of n_states pools with `lanes` rows (at most 4096 pools with the
 *             caches).
 *   tables    NULL without caches.  A beam that keeps its parent's lane gets its parent's
 *             table row.  One that takes another gets the parent's pages that are full, which
 *             the two share from now on, and from place kv_len / page_size on the pages
 *             own_pages of its lane; where the parent's last page is partly filled, the
 *             whole page is copied to the first of these.  A full page is not written any
 *             more, so sharing it needs no count: own_pages[lane][i] is in use by other
 *             beams at place i alone, and place i is written only while it is a beam's last.
 *   caches    HOST array of n_caches pools of pages (every layer's, in 4 or 8 bits) that go
 *             by this table.
 * slots_out and table_out do not overlap the inputs.  B at most 2^20.
 */
gdn_status gdn_beam_reorder(const int32_t *parent, const int32_t *slots, int32_t *slots_out, int B,
                            int W, int lanes, const gdn_beam_pool *states, int n_states,
                            const gdn_beam_tables *tables, const gdn_beam_pool *caches,
                            int n_caches, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_BEAM_H */
