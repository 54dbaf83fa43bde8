/*
 * qdr_cache.h -- C ABI of what a server does around the paged key/value cache
 * of qdr_mixer.h: rotary positions (of tensors, and of the keys on their way
 * into the cache), page tables of requests that go on, fork, end and begin,
 * pages copied and moved together, states of a pool copied, and attention of
 * requests that share their first tokens.
 *
 * The conventions of qdr.h and qdr_mixer.h hold for every entry point here:
 * device pointers (4-byte aligned) of the caller's, asynchronous work on
 * `stream`, host-side argument errors before anything is enqueued, no C++
 * exception across the ABI, token counts `cu`, contexts and page tables as
 * there, a workspace to itself for every call that may run at the same time.
 * Every call that takes a stream can be captured into a HIP graph.
 */
#ifndef QDR_CACHE_H
#define QDR_CACHE_H

#include "qdr_mixer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further bit of a cache's device error word. */
#define QDR_DEVERR_FULL 8u   /* rows that found too few free pages */

/* ---- rotary positions ---- */

typedef struct qdr_rotary qdr_rotary;   /* opaque; owned by the library */

/* Which channels turn together: channel i and i + channels/2, or 2i and 2i+1. */
enum { QDR_ROTARY_HALF = 0, QDR_ROTARY_PAIRS = 1 };

/* How the pairs' frequencies f_i = base^(-2i/channels) (radians a token) are
 * stretched for contexts longer than the `context` they were trained for; with
 * w(f) = context f / (2 pi), a pair's turns in it:
 *   PLAIN   not at all (factor, context, low and high are not looked at)
 *   LINEAR  f / factor
 *   TURNS   k f + (1 - k) f / factor,  k = (w(f) - low) / (high - low), cut to [0, 1]
 *   INDEX   the same with k = 1 - (i - a) / max(b - a, 0.001), cut to [0, 1]:
 *           c(w) = channels ln(context / (2 pi w)) / (2 ln base) is the index of
 *           the pair with w turns, a = max(floor(c(high)), 0),
 *           b = min(ceil(c(low)), channels - 1); amplitude 0.1 ln(factor) + 1
 * amplitude is 1 with the others.  base > 1, factor >= 1, context > 0,
 * 0 < low < high, all finite.  Host computation in doubles: freq gets channels/2 values. */
enum { QDR_ROTARY_PLAIN = 0, QDR_ROTARY_LINEAR = 1, QDR_ROTARY_TURNS = 2, QDR_ROTARY_INDEX = 3 };
qdr_status qdr_rotary_frequencies(int32_t rule, int32_t channels, double base, double factor, double context,
                                  double low, double high, double *freq, double *amplitude);

typedef struct {
  int32_t d;             /* must be 128                                        */
  int32_t channels;      /* a head's first channels turn: a multiple of 16, 16
                            to 128; the others stay as they are                */
  int32_t layout;        /* QDR_ROTARY_HALF or QDR_ROTARY_PAIRS                */
  const double *freq;    /* HOST [channels/2]: radians a token, magnitude <=
                            2^20; copied                                       */
  double amplitude;      /* rotated channels are multiplied by it; a finite fp32 */
} qdr_rotary_desc;

/* Create a rotation on the current HIP device.  Synchronises the device. */
qdr_status qdr_rotary_create(const qdr_rotary_desc *desc, qdr_rotary **out);
/* Free it.  Synchronises its device first.  NULL is accepted. */
qdr_status qdr_rotary_destroy(qdr_rotary *rotary);

/* Rows turned by their positions: the pair (a, b) of row t becomes
 *   amplitude (a cos p f - b sin p f,  a sin p f + b cos p f),  p = positions[t].
 * The angle is right to 2^-31 of a turn at any int32 position where f is at most
 * a turn a token (multiples of a turn are dropped in whole numbers), and to as
 * many times that as f has turns a token above.  Its sine and cosine, times
 * amplitude, are fp32, off by 6 x 2^-24 |amplitude| at most, and so are products
 * and sums.  A negative position turns back: with the positions negated the call
 * is the rotation's gradient (and, divided by amplitude^2, its inverse).
 * x, y: row t at t * stride elements, [heads][128] in a row; x_stride, y_stride
 * from heads*128 to 2^30.  y may be x with the same stride; other overlaps race.
 * fp32, or bfloat16 (y rounded to nearest even, strides even).  heads up to 2^17.
 * A workgroup takes min(32, 128 / heads) tokens, at least one, of up to 128 heads,
 * and a call of 2^24 workgroups or more is refused: 2^29 tokens of one to four
 * heads, 2^26 of 32. */
qdr_status qdr_rotate(qdr_rotary *rotary, const int32_t *positions, int32_t T, int32_t heads, const float *x,
                      int64_t x_stride, float *y, int64_t y_stride, void *stream);
qdr_status qdr_rotate_bf16(qdr_rotary *rotary, const int32_t *positions, int32_t T, int32_t heads,
                           const uint16_t *x, int64_t x_stride, uint16_t *y, int64_t y_stride, void *stream);

/* qdr_kv_write of keys that are turned on the way, and the queries turned
 * beside them: row t of sequence b is at the position that its key has in the
 * cache.  k is not rounded to bfloat16 before it is quantised: with 8 bits the
 * code is nearest(127 x / max |x|) of the fp32 products.  A vector in which a
 * NaN or an infinity stands or arises reads back as NaN (8 bits).
 * q: [q_heads][128] a row (NULL with q_heads 0: none), k and v:
 * [num_heads][128] a row, bfloat16, rows q_stride, k_stride, v_stride elements
 * apart (as above, even), so that they can be parts of one projection's rows.
 * q_out: bfloat16, [T][q_heads][128] contiguous; it may be q itself where that
 * is.  q_heads is any number up to 2^17.  Rows of a skipped sequence are 0 in
 * q_out; a bad page does not keep queries from being turned. */
qdr_status qdr_kv_write_rotary(qdr_kv *kv, qdr_rotary *rotary, const int32_t *pages, int32_t max_pages,
                               const int32_t *cu, const int32_t *context, int32_t n, int32_t T, const uint16_t *q,
                               int64_t q_stride, int32_t q_heads, uint16_t *q_out, const uint16_t *k,
                               int64_t k_stride, const uint16_t *v, int64_t v_stride, void *stream);

/* ---- pages ---- */

/* Copy page src_pages[i] of `from` to page dst_pages[i] of `to`, for i < m.
 * The two may be the same cache, or two of the same page_tokens, num_heads,
 * kind and device.  A pair with -1 on either side is skipped; another number
 * outside its cache sets QDR_DEVERR_PAGE there and the pair is skipped.  A page
 * that is written may not stand in another pair (the pairs run in any order). */
qdr_status qdr_kv_copy(qdr_kv *from, const int32_t *src_pages, qdr_kv *to, const int32_t *dst_pages, int32_t m,
                       void *stream);
/* The same for the slots of a pool: every head's stored state as it is.  A
 * number outside [-1, num_slots) sets QDR_DEVERR_SLOT. */
qdr_status qdr_slot_copy(qdr_pool *pool, const int32_t *src_slots, const int32_t *dst_slots, int32_t m, void *stream);

/* Page tables of the next step from those of this one.
 *
 * A cache in use is described by page tables and contexts (qdr_mixer.h) and by
 * refs, int32 [num_pages]: how many rows of tables hold each page, plus what
 * the program itself holds; 0: the page is free.  The cache keeps none of
 * these.  Pages are shared by rows that have tokens in common, except that a
 * row's last page, where it is not full, has to be that row's alone.
 *
 * The n rows of `pages` [n][max_pages] and `context` [n] are given up, and the m
 * rows of `new_pages` [m][max_pages] and `new_context` [m] take their place.  Row
 * j begins with the kept = min(context[a], context[a] + add[j]) first tokens of
 * row a = parent[j] (-1: with none) and has room for context[a] + add[j] of them:
 * so a row goes on by add tokens, is taken back by -add tokens, forks (several
 * rows with one parent), ends (no row with it as parent) or begins (parent -1).
 *   - Its full pages (kept / page_tokens of them) are the parent's.
 *   - A last page in part is the parent's for the first row (lowest j) that
 *     keeps it in part, where no row keeps it as a full page and the program
 *     does not hold it; other rows get a copy of its tokens (in whole blocks of
 *     32) in a free page.  (Rows count here that then run out of pages.)
 *   - Then come free pages for the rest.  Rows get free pages in the order of j
 *     and of their tokens, lowest first; pages given up by this call are free
 *     in the next.
 *   - Entries behind a row's last page are -1.
 * new_refs [num_pages] is refs less what the n rows held and more what the m
 * rows hold.  parent, add: int32 [m].
 *
 * Rows for which the free pages do not suffice (that is, row j where the rows
 * up to j need more than there are, and j any) set QDR_DEVERR_FULL; a parent
 * outside [-1, n), a context below 0, above max_pages*page_tokens or above 2^30,
 * before or after, sets QDR_DEVERR_LENGTH.  Such a row is empty afterwards:
 * context 0, pages -1, nothing held.  A page of the old tables outside the cache
 * sets QDR_DEVERR_PAGE and is held by nobody (-1 as a full page, a free page
 * without a copy as the last one).
 * No input is written, so a call that ran out of pages can be made again with
 * fewer rows; the new arrays may not overlap the old ones.  UNSUPPORTED for a
 * cache of more than 2^26 pages. */
qdr_status qdr_kv_assign_workspace(const qdr_kv *kv, int32_t m, size_t *bytes);
qdr_status qdr_kv_assign(qdr_kv *kv, const int32_t *pages, const int32_t *context, int32_t n, int32_t max_pages,
                         const int32_t *parent, const int32_t *add, int32_t m, const int32_t *refs,
                         int32_t *new_pages, int32_t *new_context, int32_t *new_refs, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Move the pages in use together: with L of them (refs not 0), the k-th of
 * those numbered L and above goes to the k-th free page below L, and all
 * numbers from L on are free.  moved [num_pages]: a page's new number (-1 for a
 * free one), new_refs [num_pages]: refs by new numbers, new_pages [n][max_pages]:
 * the tables by new numbers (-1 for entries outside the cache and of free
 * pages).  n may be 0.  Inputs, and contents of pages that are not moved onto,
 * are left as they are; the new arrays may not overlap the old ones.  UNSUPPORTED
 * for a cache of more than 2^26 pages. */
qdr_status qdr_kv_compact_workspace(const qdr_kv *kv, size_t *bytes);
qdr_status qdr_kv_compact(qdr_kv *kv, const int32_t *refs, const int32_t *pages, int32_t n, int32_t max_pages,
                          int32_t *moved, int32_t *new_refs, int32_t *new_pages, void *workspace,
                          size_t workspace_bytes, void *stream);

/* ---- attention behind shared prefixes ---- */

/* qdr_kv_attend where sequences share their first tokens, whose keys and values
 * can then be read once a group instead of once a sequence (see below).  group_cu: int32
 * [groups+1], the sequences of group i are group_cu[i] .. group_cu[i+1]-1; a
 * sequence in no group shares nothing.  shared: int32 [groups]: the cache holds
 * the same at positions below shared[i] for every sequence of the group (the
 * library reads them from the pages of any), and these are older than every
 * row of it: shared[i] <= context[b] - rows of b.  A sequence with fewer sets
 * QDR_DEVERR_LENGTH and is skipped; where it is the group's first, or shared[i]
 * is below 0 or above max_pages*page_tokens, the whole group is.  A pair of
 * group_cu that decreases or leaves [0, n] sets QDR_DEVERR_LENGTH, and the
 * results are then unspecified (what is read and written stays inside the
 * arrays).
 * Whether shared keys are read once a group is decided by what that can save.
 * The call does so where (n - groups) x num_heads x (blocks of 32 tokens that
 * max_pages pages have) is 12288 or more: empty groups, as in arrays of a fixed
 * shape, count against it, and sequences in no group and tables wider than the
 * prefix for it.  Then a group goes together that has two sequences or more and
 * whose sequences bring fewer tokens on average than 128 / (q_heads / num_heads)
 * (rounded down, at least 1).  Elsewhere each sequence reads the shared keys by
 * itself, as in qdr_kv_attend.  The results are the same but for rounding: the
 * weights of shared keys that a group reads together have two parts (2^-16) if the
 * group's rows (tokens x q_heads / num_heads) are up to 16 and one (2^-8) if they
 * are more, all others those that qdr_kv_attend gives the sequence.  T x q_heads
 * has to be below 2^26.  Everything else is as in qdr_kv_attend. */
qdr_status qdr_kv_attend_shared_workspace(const qdr_kv *kv, int32_t n, int32_t T, int32_t groups, int32_t q_heads,
                                          int32_t max_pages, size_t *bytes);
qdr_status qdr_kv_attend_shared(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                                const int32_t *context, int32_t n, int32_t T, const int32_t *group_cu,
                                const int32_t *shared, int32_t groups, int32_t q_heads, const uint16_t *q,
                                float scale, uint16_t *o, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* QDR_CACHE_H */
