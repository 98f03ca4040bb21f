/*
 * gdn_attn.h -- C ABI of the softmax-attention layers that stand between gated
 * delta rule layers in a hybrid decoder: rotary positions, a paged key/value
 * cache held in 4 or in 8 bits, and attention over that cache.  Part of libgdn.so;
 * statuses, dtypes, streams, scratch and error reporting as in gdn.h:
 * arguments are checked synchronously, work is enqueued on `stream`, errors
 * found by a kernel (a position outside its table, a page outside the pool, a
 * length outside its bound, offsets that do not pack the tokens) are reported by
 * gdn_sync_check() as GDN_ERR_INVALID_ARG, and leave the rows concerned
 * unspecified.
 *
 * Rows.  q, k, v and o are rows of d contiguous elements, found by strides, so
 * [B][H][T][d], [B][T][H][d], [tokens][H][d] and [H][tokens][d] all pass as
 * they are.  The base pointers of rows, pages, cos and sin and the strides of rows
 * are multiples of 16 bytes, the int32 and fp32 arrays' of 4 (GDN_ERR_ALIGNMENT).
 * Query head i reads key/value head i / (Hq / H): Hq is a multiple of the cache's
 * head count (GDN_ERR_INVALID_ARG).
 *
 * Tokens.  The cache entry points work on the last tokens of N sequences,
 * packed in sequence order: sequence b has the tokens [cu_seqlens[b],
 * cu_seqlens[b+1]), from cu_seqlens[0] = 0 to cu_seqlens[N] = n_tokens, or, where
 * cu_seqlens is NULL, n_tokens / N tokens each.
 * kv_len[b] counts the sequence's tokens INCLUDING these n_b, so the j-th of
 * them lies at place kv_len[b] - n_b + j.  A token whose place is negative (an
 * idle slot of a batch: kv_len[b] = 0) is not written, reads back as zero, and
 * sees nothing; its query is turned like any other, by a position that has to
 * lie in the table.
 *
 * Cache.  `pages` is [n_pages][H][gdn_kv_page_bytes(page_size, d)] bytes.  The
 * block of one (page, head) holds, in this order,
 *     key codes    [page_size][d / 2]      value codes    [page_size][d / 2]
 *     key scales   [page_size][d / 16]     value scales   [page_size][d / 16]
 * A code is an e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; the
 * element of even index in the low half of its byte); 16 neighbours along d
 * share a scale, an e4m3 number; and each head may have a further fp32 scale
 * for its keys and one for its values (`head_scale` [2][H], NULL: 1):
 *     element = e2m1 * e4m3 * head_scale[0 or 1][h].
 * 9/8 d bytes hold a token's key and value of one head (144 at d = 128).
 * Place p of sequence b lies in page page_table[b * table_stride + p / page_size], row
 * p % page_size.  What lies in rows that no sequence counts is never used.
 *
 * Cache in 8 bits (gdn_kv8_*).  `pages` is [n_pages][H][gdn_kv8_page_bytes(page_size,
 * d)] bytes.  The block of one (page, head) holds, in this order,
 *     key codes    [page_size][d]          value codes    [page_size][d]
 *     exponents    [page_size / 128, at least 1][16]
 * A code is an e4m3 number.  16 places of a head share an exponent byte e for their
 * keys and one for their values, 0 <= e <= 22:
 *     element = e4m3 * 2^(e - 15) * head_scale[0 or 1][h],
 * and the bytes of places 128 i + 16 j are bytes j (keys) and 8 + j (values) of the
 * 16 bytes i.  A token's key and value of one head take 2 d + 1/8 bytes (pages of 128).
 * Everything else is as in 4 bits; a gdn_kv describes either.
 *
 * Sizes.  A call has at most 2^31 - 256 tokens, and a page table as many places a
 * sequence (GDN_ERR_UNSUPPORTED).
 */
#ifndef GDN_ATTN_H
#define GDN_ATTN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of d elements: (sequence or batch item b, head h, token t) starts at
 * data + b * stride_seq + h * stride_head + t * stride_tok elements.  Packed
 * tokens ignore stride_seq. */
typedef struct {
    void *data;
    int64_t stride_seq, stride_head, stride_tok;
    int heads;
} gdn_rows;

/*
 * Rotary positions: the first d_rot elements of a row form d_rot / 2 pairs, and
 * pair i is turned by the angle whose cosine and sine are
 * cos[p][i], sin[p][i], p = pos[axes[i]][token].
 *   cos, sin      device fp32 [table_len][d_rot / 2].
 *   pos           device int32; the position on axis a of token t of batch item
 *                 b is pos[a * stride_axis + b * stride_seq + t] (packed
 *                 tokens: b = 0); in [0, table_len).
 *   axes          HOST array of d_rot / 2 axis numbers below n_axes (time,
 *                 height, width of an image or video patch, dealt over the
 *                 pairs in any way), or NULL: every pair goes by axis 0.
 *   n_axes        1 .. 4.
 *   flags         GDN_ROPE_ADJACENT: pair i is elements (2 i, 2 i + 1); else
 *                 (i, i + d_rot / 2).  GDN_ROPE_INVERSE (gdn_rope only): turns
 *                 back, which is also the gradient of the turn.
 * d_rot is a multiple of 16 up to d (in gdn_kv_append, without
 * GDN_ROPE_ADJACENT, a multiple of 32).  Products are formed and summed in fp32,
 * each rounded (no fused multiply-add), and the result is rounded once.
 */
typedef struct {
    const float *cos, *sin;
    const int32_t *pos;
    const uint8_t *axes;
    int64_t stride_axis, stride_seq;
    int table_len, d_rot, n_axes;
    unsigned flags;
} gdn_rotary;
enum { GDN_ROPE_ADJACENT = 1, GDN_ROPE_INVERSE = 2 };

/* The cache and the tokens of a call (above); all pointers device memory.
 * page_size is 16, 32, 64, 128 or 256, d is 64, 128 or 256
 * (GDN_ERR_UNSUPPORTED). */
typedef struct {
    void *pages;
    const float *head_scale;      /* [2][heads] or NULL */
    const int32_t *page_table;    /* [N][max_pages], rows table_stride apart */
    const int32_t *kv_len;        /* [N] */
    const int32_t *cu_seqlens;    /* [N + 1] or NULL */
    int n_pages, page_size, heads, d;
    int N, max_pages, n_tokens;
    int64_t table_stride;
} gdn_kv;

/* Bytes of one (page, head) block, page_size * d * 9 / 8; 0 if unsupported. */
int64_t gdn_kv_page_bytes(int page_size, int d);

/*
 * Turns the rows of q and, where k is not NULL, of k, in one launch.  B items
 * of T tokens; d a multiple of 16 up to 256.  The outputs have their own
 * strides and may be the inputs themselves (not otherwise overlap them).
 */
gdn_status gdn_rope(const gdn_rows *q, const gdn_rows *q_out, const gdn_rows *k,
                    const gdn_rows *k_out, int B, int T, int d, const gdn_rotary *rot,
                    gdn_dtype dt, void *stream);

/*
 * Appends keys and values to the cache, in one launch: turns k by `rot` (NULL:
 * not turned), then holds k and v in 4 bits at their places.  With m the
 * largest magnitude of 16 neighbours over the head's scale, their e4m3 scale is
 * min(m / 6, 448) to nearest, and an element becomes the nearest e2m1 number to
 * its quotient, at most 6 (ties to even; m / 6 and the quotients by an fp32
 * reciprocal).  A NaN makes its 16 neighbours read back as NaN; infinities
 * saturate.  Where q is not NULL its rows are turned as well, into q_out (dtype
 * dt; may be q itself), for the attention that follows.
 */
gdn_status gdn_kv_append(const gdn_kv *kv, const gdn_rows *k, const gdn_rows *v,
                         const gdn_rows *q, const gdn_rows *q_out, const gdn_rotary *rot,
                         gdn_dtype dt, void *stream);

/* Reads the call's tokens back from the cache into k and v, as the values they
 * stand for: e2m1 * e4m3 is exact, its product with the head's scale is rounded
 * to fp32, and that to dt. */
gdn_status gdn_kv_read(const gdn_kv *kv, const gdn_rows *k, const gdn_rows *v, gdn_dtype dt,
                       void *stream);

/*
 * Attention of the call's tokens over their sequences' cached keys and values:
 *     o = sum_t softmax_t(scale * q . k_t) v_t,
 * for the token at place p over the places t with
 *     t <= p (GDN_ATTN_CAUSAL) or t < kv_len[b];  t > p - window (window > 0).
 * A row that sees no place gives o = 0 and lse = -infinity.
 *   q, o      rows of dtype dt, Hq heads each.
 *   lse       device fp32 [n_tokens][Hq], the logarithm of the sum of
 *             exp(scale * q . k_t), or NULL.
 *   max_len, max_new   HOST bounds on kv_len and on the tokens of one sequence,
 *             from which the launch is planned (a larger device value is
 *             reported as GDN_ERR_INVALID_ARG by gdn_sync_check()).  max_new
 *             also chooses the kernel for the whole call (bf16, d <= 128: above
 *             16 rows max_new * Hq / H, in 8 bits 32, the one for many rows), so a bound far
 *             above what the sequences have costs time.
 * The cache's numbers enter the tensor cores exactly (e2m1 * e4m3 fits fp16);
 * with bf16 rows the probabilities are rounded to fp16 (11 bits, down to 2^-22
 * of the row's largest at least; the kernel for many rows leaves out what lies
 * below 2^-33 of it), with fp32 rows queries and probabilities are carried as two
 * fp16 numbers each.  Sums, maxima and outputs are fp32 until o is rounded.
 * Scratch for splitting long sequences comes from the library's pool.  The same
 * inputs give the same bits.
 */
enum { GDN_ATTN_CAUSAL = 1 };
gdn_status gdn_kv_attn(const gdn_kv *kv, const gdn_rows *q, const gdn_rows *o, float *lse,
                       int max_len, int max_new, float scale, int window, unsigned flags,
                       gdn_dtype dt, void *stream);

/* Bytes of one (page, head) block in 8 bits, 2 page_size d and 16 for every 128 places
 * (at least once); 0 if unsupported. */
int64_t gdn_kv8_page_bytes(int page_size, int d);

/*
 * gdn_kv_append on a cache in 8 bits, in one launch.  The exponent of a block of 16
 * places is the least under which the largest magnitude among the call's tokens in it,
 * over the head's scale, is at most 448 (so 22 where there is an infinity); a block that
 * has tokens before them keeps at least the one that it has, and where it grows their
 * codes are divided by the same power of two, to nearest even.  An element becomes the
 * nearest e4m3 number to its quotient, at most 448 (ties to even; quotients by the head's
 * scale are products with its fp32 reciprocal, here and in the largest magnitude).  What is above the
 * range, 57344 times the head's scale, becomes that; a NaN makes the 16 neighbours
 * along d that it is among NaN, and they do not count for the exponent.  A page that a
 * call writes belongs to one sequence of the call.
 */
gdn_status gdn_kv8_append(const gdn_kv *kv, const gdn_rows *k, const gdn_rows *v,
                          const gdn_rows *q, const gdn_rows *q_out, const gdn_rotary *rot,
                          gdn_dtype dt, void *stream);

/* gdn_kv_read from a cache in 8 bits: e4m3 * 2^(e - 15) is exact, its product with the
 * head's scale is rounded to fp32, and that to dt. */
gdn_status gdn_kv8_read(const gdn_kv *kv, const gdn_rows *k, const gdn_rows *v, gdn_dtype dt,
                        void *stream);

/* gdn_kv_attn over a cache in 8 bits: the same arguments, rows seen and roundings (e4m3 *
 * 2^(e - 15) fits fp16 as well).  A NaN among the values reaches the outputs of its own
 * element, or of the 16 neighbours that gdn_kv8_append gives it to, in the rows that see
 * its place. */
gdn_status gdn_kv8_attn(const gdn_kv *kv, const gdn_rows *q, const gdn_rows *o, float *lse,
                        int max_len, int max_new, float scale, int window, unsigned flags,
                        gdn_dtype dt, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTN_H */
