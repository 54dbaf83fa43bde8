/*
 * qdr_mixer.h -- C ABI of the token mixers beside the quantised decode step:
 * the prompt form of the recurrences that qdr_decode_step and
 * qdr_linear_step take token by token, the additive recurrence's step, and a
 * paged key/value cache (8-bit or bfloat16) with the attention of new tokens
 * over it, for stacks that keep softmax-attention layers between their
 * recurrent ones.
 *
 * The conventions of qdr.h hold for every entry point here: device pointers
 * to contiguous arrays owned by the caller (4-byte aligned), asynchronous
 * work on `stream`, host-side argument errors before anything is enqueued,
 * no C++ exception across the ABI, QDR_DIM = 128 channels a head.  Calls
 * that only enqueue can be captured into a HIP graph.  Handles belong to the
 * device they were created on: that device has to be current in every call
 * (QDR_E_INVAL otherwise), and `stream` has to be one of its streams.
 *
 * Token counts.  A call over n sequences takes `cu`, int32 [n+1]: the tokens
 * of sequence b are rows cu[b] .. cu[b+1]-1 of the token arrays, whose first
 * dimension is T >= cu[n].  Rows from cu[n] on, and before cu[0], are neither
 * read nor written.  A sequence may have no tokens.  A pair of counts that
 * decreases or leaves [0, T] sets QDR_DEVERR_LENGTH, and that sequence is
 * skipped; the other sequences' results are then unspecified as well (what
 * is read and written stays inside the arrays).
 *
 * Sizes.  n and T are at most 2^30.  A call that would take 2^24 workgroups (of
 * 256 threads) or more in one launch is refused with QDR_E_INVAL: cut it up.
 *
 * Workspaces.  A call that takes one uses it until the work it enqueued has
 * finished.  Calls that may run at the same time (other streams, other
 * captured graphs) need workspaces of their own.  16-byte aligned.  What a call
 * needs does not grow with its counts: a smaller one may cut its sequences or
 * keys into pieces where a larger one does not, and need more.  A workspace for
 * several shapes has the most bytes that any of them is said to need.
 */
#ifndef QDR_MIXER_H
#define QDR_MIXER_H

#include "qdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the device error words. */
#define QDR_DEVERR_LENGTH 2u   /* token counts out of order or out of range */
#define QDR_DEVERR_PAGE 4u     /* a page number outside the cache           */

/* The recurrence of a prompt: the gated delta rule of qdr_decode_step, or
 * linear attention with a decay (the same without its correction):
 *   DELTA  u_t = beta_t (v_t - alpha_t S_{t-1}^T k_t)
 *   SUM    u_t = v_t
 *   S_t = alpha_t S_{t-1} + k_t u_t^T,   o_t = S_t^T q_t                   */
enum { QDR_RULE_DELTA = 0, QDR_RULE_SUM = 1 };

/* Bytes of the workspace of a prompt call over n sequences and T rows, for just
 * these counts (fewer can need more). */
qdr_status qdr_prompt_workspace(const qdr_pool *pool, int32_t n, int32_t T, size_t *bytes);

/* The prompt form: n sequences of any lengths, taken 64 tokens at a time on
 * the matrix cores, end in the pool's slots.  For every b < n with
 * slots[b] >= 0 and every head: S_0 is the state restored from slot slots[b]
 * where carry[b] != 0 and zero otherwise (carry NULL: zero for every b); the
 * rows of sequence b go through the recurrence in fp32; S of the last row is
 * quantised into the slot as qdr_pack does.  Inside the prompt the state is
 * not quantised.  A sequence without tokens that carries leaves its slot as
 * it is; one that does not carry resets it to S = 0.
 * q, k, v, o: [T][H][128] bfloat16 bit patterns, o rounded to nearest even;
 * beta: [T][H] fp32, required for DELTA and ignored for SUM; gate: [T][H]
 * fp32, linear alpha in [0, 1] (0 forgets the state exactly).  Slots as in
 * qdr_decode_step (-1: the sequence is skipped and its o rows are 0).
 * Non-finite inputs reach only rows of their own (sequence, head), from the
 * first token of their 64-token chunk on.  A gate below 0 gives NaN there.
 * QDR_E_UNSUPPORTED for a pool with QDR_GATE_DIAG or more than 2^17 heads. */
qdr_status qdr_prompt(qdr_pool *pool, int32_t rule, const int32_t *slots, const int32_t *carry,
                      const int32_t *cu, int32_t n, int32_t T, const uint16_t *q, const uint16_t *k,
                      const uint16_t *v, const float *beta, const float *gate, uint16_t *o,
                      void *workspace, size_t workspace_bytes, void *stream);

/* One token of the SUM rule for B requests, in place in an uncompressed pool
 * (every head QDR_K_FP32, QDR_GATE_SCALAR; QDR_E_UNSUPPORTED otherwise).
 * q, k, v, o: [B][H][128] fp32; gate: [B][H] fp32, any value.  Slots, errors
 * and non-finite inputs as in qdr_decode_step. */
qdr_status qdr_linear_step(qdr_pool *pool, const int32_t *slots, int32_t B, const float *q,
                           const float *k, const float *v, const float *gate, float *o, void *stream);
/* The same with bfloat16 q, k, v and o (o rounded to nearest even). */
qdr_status qdr_linear_step_bf16(qdr_pool *pool, const int32_t *slots, int32_t B, const uint16_t *q,
                                const uint16_t *k, const uint16_t *v, const float *gate, uint16_t *o,
                                void *stream);

/* ---- paged key/value cache ---- */

typedef struct qdr_kv qdr_kv;   /* opaque; owned by the library */

/* Storage of keys and values.  INT8: symmetric codes z in [-127, 127] with
 * one fp32 scale per (token, head) and for K and V apart: r = max |x| (1 if
 * below 2^-126), z = nearest-even(127 x / r), the stored value is z (r/127)
 * (a vector that holds NaN or infinity reads back as NaN).  BF16: the
 * bfloat16 values themselves. */
enum { QDR_KV_INT8 = 8, QDR_KV_BF16 = 16 };

typedef struct {
  int32_t num_pages;     /* pages of the cache                              */
  int32_t page_tokens;   /* tokens of a page: 32, 64, 128, 256, 512 or 1024 */
  int32_t num_heads;     /* key/value heads                                 */
  int32_t d;             /* must be 128                                     */
  int32_t kind;          /* QDR_KV_*                                        */
} qdr_kv_desc;

/* Device bytes of the cache (pure host computation).  QDR_E_INVAL where they
 * do not fit 63 bits. */
qdr_status qdr_kv_bytes(const qdr_kv_desc *desc, size_t *bytes);
/* Create a cache on the current HIP device.  dev_mem as in qdr_pool_create
 * (at least qdr_kv_bytes, 256-byte aligned, outlives the cache; NULL: the
 * library allocates).  The memory is zero-filled.  Synchronises the device. */
qdr_status qdr_kv_create(const qdr_kv_desc *desc, void *dev_mem, size_t dev_bytes, qdr_kv **out);
/* Free the cache.  Synchronises its device first, which need not be current.
 * NULL is accepted. */
qdr_status qdr_kv_destroy(qdr_kv *kv);

/* Pages and contexts.  pages: int32 [n][max_pages], the page of tokens
 * i*page_tokens .. of sequence b at pages[b][i]; entries behind a sequence's
 * last page are not read.  context: int32 [n], the tokens of sequence b in
 * the cache, those of this call among them: its cu[b+1]-cu[b] rows are the
 * LAST of them, at positions context[b]-(cu[b+1]-cu[b]) .. context[b]-1.  A
 * context below a sequence's rows, above max_pages*page_tokens or above 2^30
 * sets QDR_DEVERR_LENGTH, and the sequence is skipped (rows to be returned
 * are 0).
 * A page outside [0, num_pages) sets QDR_DEVERR_PAGE: its tokens are not
 * written, read back as 0, and take no part in the attention. */

/* Write the rows of every sequence into the cache, quantised as its kind
 * says.  k, v: [T][num_heads][128] bfloat16.  A page may belong to several
 * sequences that read it, but the positions written in one call have to be
 * distinct. */
qdr_status qdr_kv_write(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                        const int32_t *context, int32_t n, int32_t T, const uint16_t *k,
                        const uint16_t *v, void *stream);
/* Read rows back as bfloat16 (rounded to nearest even). */
qdr_status qdr_kv_read(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                       const int32_t *context, int32_t n, int32_t T, uint16_t *k, uint16_t *v,
                       void *stream);

/* Bytes of the workspace of an attention call of just these counts (0 is
 * possible, and fewer sequences or rows can need more). */
qdr_status qdr_kv_attend_workspace(const qdr_kv *kv, int32_t n, int32_t T, int32_t q_heads,
                                   int32_t max_pages, size_t *bytes);
/* Attention of new tokens over the cache, their own keys and values among it
 * (written before by qdr_kv_write on the same stream): for row t of sequence
 * b at position p and query head j, with key/value head j / (q_heads /
 * num_heads),   o = sum_{i <= p} softmax_i(scale q.k_i) v_i.   scale: any sign,
 * with scale log2(e) finite in fp32.
 * q, o: [T][q_heads][128] bfloat16; q_heads a multiple of num_heads.  One new
 * token a sequence, many, or both in one call.  Scores, the softmax and the
 * sums are fp32; the weights enter their product as bfloat16, in two parts
 * (2^-16) for a sequence that brings up to 16 rows a key/value head (tokens x
 * q_heads / num_heads; a single token always), whatever the others bring, in
 * one (2^-8) for a longer one.  Of a call of one sequence T counts as its
 * length.  A key or value that is not finite reaches the rows that see its
 * token, in its own head, and no others; the weighted values are summed in fp32
 * before they are divided (weights up to 2^8), so values have to stay that far
 * from its end.  Rows of a skipped sequence are 0, and so is a row that sees no
 * key or whose scores are all -infinity. */
qdr_status qdr_kv_attend(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                         const int32_t *context, int32_t n, int32_t T, int32_t q_heads,
                         const uint16_t *q, float scale, uint16_t *o, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Read and clear the cache's device error word.  Synchronises the device. */
qdr_status qdr_kv_poll_device_error(qdr_kv *kv, uint32_t *flags);

#ifdef __cplusplus
}
#endif
#endif /* QDR_MIXER_H */
