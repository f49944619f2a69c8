/*
 * qmv_serve.h - the operators between a quantized model's products, on one
 * MI355X (gfx950): the norm in front of a product, the heads' norm with the
 * position's rotation, a key/value cache held in 8 or in 4 bits, attention
 * over either, the log probabilities of the LM head's logits, and the next
 * token drawn from them.  Plain C ABI beside qmv.h, whose products take what these
 * calls give: the status codes, the meaning of `stream` and "device pointer"
 * are the ones of qmv.h.
 *
 * All calls check their arguments on the host, enqueue kernels on `stream`
 * and return; none allocates, synchronizes, sets memory by a library call or
 * keeps anything from one call for the next, so each can be captured into a
 * graph at once.  Calls that need scratch memory take it from the caller:
 * its contents on entry do not matter, and two calls may share it only if
 * one is done before the other starts (two graphs that are replayed at the
 * same time each need their own).  Pointers belong to the current device.
 * Outputs must not overlap inputs, but where stated.  Results do not depend
 * on the order in which the GPU runs its workgroups.
 */
#ifndef QMV_SERVE_H
#define QMV_SERVE_H

#include <stdint.h>

#include "qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the calls below that take `dtype`: float32, or bfloat16
 * bit patterns (uint16). */
enum { QMV_F32 = 0, QMV_BF16 = 1 };

/*
 * Root-mean-square norm of each row, with the residual's addition, in the
 * forms that the products take.  For each of `rows` rows of `cols` values,
 * in float32 operations that each round once:
 *   h = x + res                       (h = x where res is NULL)
 *   r = 1 / sqrt(sum h^2 / cols + eps), computed in 64 bits, then rounded
 *   y = (h * r) * w
 * and the outputs that are not NULL:
 *   sum    h, float32: the residual stream for the next layer.  May be res
 *          or x itself (updated in place).
 *   y      y, float32 (what qmv_gemv takes)
 *   y_bf16 y rounded to bfloat16 (what qmv_gemm takes)
 *   q, d   y quantized per block of 32 by the rule of qmv_quantize_q8, bit
 *          for bit (what qmv_gemm_q8 takes): int8 [rows][cols] and float32
 *          [rows][cols / 32].  A block that holds an infinite or NaN y gets
 *          d = NaN and q = 0, so that products with it are NaN.
 * x, res, sum, y: [rows][cols], w: float32 [cols]; device memory, 16-byte
 * aligned; cols a multiple of 32, at most 2^24; eps >= 0.
 * Errors: QMV_E_ARG (x or w NULL, no output at all, only one of q and d,
 * misaligned pointer, rows 0, eps negative, infinite or NaN), QMV_E_SHAPE (cols),
 * QMV_E_DEVICE.
 */
int qmv_rms_norm(const float *x, const float *res, const float *w, float eps, uint32_t rows,
                 uint32_t cols, float *sum, float *y, uint16_t *y_bf16, int8_t *q, float *d,
                 void *stream);

/*
 * A key/value cache in 8 bits: pages of QMV_KV_PAGE tokens; in a page each
 * key/value head has one scale for its keys and one for its values, a power
 * of two from 2^-126 to 2^121 or 0 (so that a stored value is exact in
 * float32 and in bfloat16).  All arrays are the caller's device memory,
 * 16-byte aligned:
 *   k        int8 [pages][kv_heads][64][head_dim]
 *   v        int8 [pages][kv_heads][head_dim][64]  (tokens last: the order
 *            in which the matrix cores take the values)
 *   k_scale, v_scale   float32 [pages][kv_heads]
 * head_dim is 64, 128 or 256.  A new cache needs no initialisation: a page
 * takes its scale from the call that writes its first token.
 */
enum { QMV_KV_PAGE = 64 };
typedef struct qmv_kv_cache {
    int8_t *k;
    int8_t *v;
    float *k_scale;
    float *v_scale;
    uint32_t pages, kv_heads, head_dim;
} qmv_kv_cache;

/*
 * Which tokens a call is about: for each of `seqs` sequences its last
 * tokens, consecutive rows of the call's arrays.
 *   table  int32 [seqs][table_stride]: page ids; token t of sequence i lives
 *          in page table[i][t / 64] at place t % 64
 *   len    int32 [seqs]: tokens of the sequence, the call's included
 *   start  int32 [seqs + 1], not decreasing: sequence i has the rows
 *          start[i] .. start[i+1] - 1, which are its positions
 *          len[i] - (start[i+1] - start[i]) .. len[i] - 1
 * in device memory, 4-byte aligned, read by the kernels alone.  rows: rows
 * of the call's arrays; start is held to 0 .. rows, and rows of no sequence
 * are neither read nor written.  max_new, max_len: the largest count of rows
 * and the largest len among the sequences as far as the host knows; they
 * shape the launch: results are right whatever they are, and the same bits
 * for the same ones.  A max_len far above the lengths, or one length far above
 * the others, leaves much of the GPU idle in qmv_kv_attend.
 * A position below 0 (more rows than len), past the table or in a page whose
 * id is outside [0, pages) has no place: nothing is written for it, it reads
 * as zero, and attention leaves it out.
 */
typedef struct qmv_kv_seqs {
    const int32_t *table;
    const int32_t *len;
    const int32_t *start;
    uint32_t seqs, table_stride, rows, max_new, max_len;
} qmv_kv_seqs;

/*
 * Writes the rows of k and v ([rows][kv_heads][head_dim], dtype) into the
 * cache.  For each page, head and array that new tokens fall into, with amax
 * the largest magnitude of the new values there: need = the least power of
 * two d from 2^-126 with amax <= 127 d (0 if amax is 0; at most 2^121, where
 * codes end at 127); the scale becomes need if the page's first token is among
 * the new ones, else the larger of the old scale and need; earlier tokens'
 * codes become code * old / scale, and the new codes x / scale, both rounded
 * to the nearest whole number, halves to even.  A growing scale at least
 * doubles, so whatever the order of the writes every stored value stays within
 * one scale of what was written (half a scale if its page's scale did not grow
 * after it).  An infinite or NaN value makes the scale of its page, head and
 * array NaN: everything read from there is NaN until the page is begun anew.
 * A call must not write into one page twice, for two sequences or two places
 * of one table.  A page's first token is written before or with its others
 * (what is read of a page that was never begun is whatever its memory holds).
 * Errors: QMV_E_ARG (a NULL or misaligned pointer, pages, kv_heads, seqs,
 * table_stride or rows 0, dtype unknown), QMV_E_SHAPE (head_dim, or a size that
 * a launch cannot hold: kv_heads above 65535, seqs * kv_heads above 2^22,
 * pages * kv_heads or seqs * table_stride of 2^31 or more, rows above
 * 2^31 - 2^16), QMV_E_DEVICE.
 */
int qmv_kv_write(const qmv_kv_cache *cache, const qmv_kv_seqs *seqs, uint32_t dtype, const void *k,
                 const void *v, void *stream);

/*
 * Reads the rows' tokens back into k and v ([rows][kv_heads][head_dim],
 * dtype): code * scale, rounded once to dtype.  Either of k and v may be
 * NULL.  Errors: as qmv_kv_write (QMV_E_ARG if both are NULL).
 */
int qmv_kv_read(const qmv_kv_cache *cache, const qmv_kv_seqs *seqs, uint32_t dtype, void *k,
                void *v, void *stream);

/*
 * Attention of the rows over the cache: for row t at position p of its
 * sequence and query head h, with key/value head h / (heads / kv_heads) and
 * the stored keys k_j and values v_j of the positions j <= p (with window >
 * 0: p - window < j <= p),
 *   out[t][h] = sum_j e^(s_j) v_j / sum_j e^(s_j),  s_j = scale * q[t][h] . k_j.
 * q, out: [rows][heads][head_dim], dtype, 16-byte aligned; out may be q.
 * A row that sees no token gets zeros.  The rows' own tokens have to be in
 * the cache (qmv_kv_write before this call on the stream).  Scores, the
 * softmax's maximum and sums and the output sums are float32 or exact
 * integers.  Queries and probabilities enter the products as whole numbers
 * of up to 127 2^16 (a row's largest magnitude, a page's largest
 * probability), or, where bfloat16 queries are many (at least 16384 / head_dim
 * rows and heads to a sequence and key/value head, in a call of enough work,
 * by max_new and max_len), as float16: queries exactly down to 2^-31 of their
 * row's largest (below it to 2^-39 of that), probabilities rounded to 11 bits
 * (below 2^-28 of the largest: to 0).  A query, or a page and head that is seen,
 * with a NaN or infinity gives NaN for the rows that see it and touches no
 * other.  Scores past float32's range may give NaN; values below
 * 2^63 in magnitude never leave it.  Values below 2^-96, or below 2^-96 of the
 * largest of their sequence and head, may lose low bits or count as 0.  Scales
 * of the cache are taken to be powers of two, 0 or NaN, as qmv_kv_write makes
 * them.
 * workspace: device memory of at least qmv_kv_attend_workspace bytes (may be
 * NULL where that is 0), 16-byte aligned.
 * Errors: QMV_E_ARG (as qmv_kv_write; scale not finite; workspace too small),
 * QMV_E_SHAPE (as qmv_kv_write; heads 0, above 2^24 or no multiple of
 * kv_heads; rows * heads above 2^31 - 2^16), QMV_E_DEVICE.
 */
int qmv_kv_attend_workspace(const qmv_kv_cache *cache, const qmv_kv_seqs *seqs, uint32_t dtype,
                            uint32_t heads, uint32_t window, uint64_t *bytes);
int qmv_kv_attend(const qmv_kv_cache *cache, const qmv_kv_seqs *seqs, uint32_t dtype,
                  uint32_t heads, float scale, uint32_t window, const void *q, void *out,
                  void *workspace, uint64_t workspace_bytes, void *stream);

/*
 * Norm of query and key heads, with the position's rotation in the same pass.
 * For each of `rows` rows and each head x of head_dim values, with n =
 * head_dim, in float32 (squares are summed in 64 bits):
 *   y = (x r) w, r = 1 / sqrt(sum x^2 / n + eps)   (y = x where w is NULL)
 * and then, for i < rot / 2, with the angle pos[row] freq[i] taken in 64 bits,
 * c and s its cosine and sine times mscale, each pair (a, b) of y becomes
 *   (a c - b s, b c + a s);
 * pairs are (y[i], y[i + rot / 2]), or with neighbours != 0 (y[2 i], y[2 i +
 * 1]).  Channels from rot on stay as they are.  Any frequency scheme is a
 * choice of freq and mscale.  The result is rounded once to out_dtype.
 * q, k: the heads of the queries and of the keys; either may be NULL.
 *   x, y        dtype and out_dtype, [rows][heads][head_dim], rows x_stride
 *               and y_stride elements apart: slices of one array of all
 *               projections, say.  y may be x itself (the same stride and type).
 *   w           float32 [head_dim], or NULL: no norm
 * pos: int32 [rows], any value.  freq: float32 [rot / 2] (may be NULL if rot
 * is 0).  Device memory; x, y, w 16-byte aligned, pos and freq 4-byte aligned;
 * head_dim a multiple of 8, at most 512; rot a multiple of 16, at most
 * head_dim; strides multiples of 8, at least heads * head_dim.
 * Errors: QMV_E_ARG (q and k NULL, a NULL or misaligned pointer, a dtype
 * unknown, rows or heads 0, eps negative, infinite or NaN, mscale infinite or
 * NaN, y is x with another stride or type), QMV_E_SHAPE (head_dim, rot, strides,
 * heads above 2^20, rows above 2^31 - 2^16, strides above 2^40), QMV_E_DEVICE.
 */
typedef struct qmv_heads {
    const void *x;
    void *y;
    const float *w;
    uint64_t x_stride, y_stride;
    uint32_t heads;
} qmv_heads;
int qmv_qk_rotate(const qmv_heads *q, const qmv_heads *k, uint32_t rows, uint32_t head_dim,
                  uint32_t dtype, uint32_t out_dtype, float eps, const int32_t *pos,
                  const float *freq, uint32_t rot, uint32_t neighbours, float mscale, void *stream);

/*
 * A key/value cache in 4 bits: pages of QMV_KV_PAGE tokens; each block of 32
 * channels of one token and head has a scale byte b and 32 codes of 4 bits, a
 * sign (8) above an index into 0, .5, 1, 1.5, 2, 3, 4, 6: a stored value is
 * that times 2^(b - 127), exact in float32 and in bfloat16.  4.25 bits a
 * value.  All arrays are the caller's device memory, 16-byte aligned:
 *   k, v               uint8 [pages][kv_heads][64 * head_dim / 2]
 *   k_scale, v_scale   uint8 [pages][kv_heads][64 * head_dim / 32]
 * head_dim is 64, 128 or 256.  Within a page and head, token t keeps (two
 * codes a byte, the lower channel in the lower half; all byte offsets)
 *   channel c of its key      at t * head_dim / 2 + c / 2
 *   block b's scale of it     at ((t % 16) * (head_dim / 32) + b) * 4 + t / 16
 *   channel c of its value    at ((t / 4 * 16 + c / e) * 4 + t % 4) * e / 2 + c % e / 2,
 *                             e = head_dim / 16
 *   block b's scale of it     at ((t / 4 % 4 * (head_dim / 32) + b) * 4 + t / 16) * 4 + t % 4
 * A new cache needs no initialisation.  A token's bytes depend on that token
 * alone; pages may be copied as they are.
 */
typedef struct qmv_kv4_cache {
    uint8_t *k;
    uint8_t *v;
    uint8_t *k_scale;
    uint8_t *v_scale;
    uint32_t pages, kv_heads, head_dim;
} qmv_kv4_cache;

/*
 * Writes the rows of k and v ([rows][kv_heads][head_dim], dtype) into the
 * cache: for each block, with amax its largest magnitude, d the least power of
 * two from 2^-125 to 2^125 with amax <= 7 d (the ends where there is none), and
 * codes of x / d to the nearest value, halves to the even code, at most 6 (so
 * a stored value is within d / 4 of values below 2 d, d / 2 below 4 d, d above).
 * An infinite or NaN value makes its token's keys and values of that head NaN
 * (key scale bytes 255, values 0) until the token is written again.
 * A call must not write one place twice.  seqs as for qmv_kv_write.
 * Errors: as qmv_kv_write.
 */
int qmv_kv4_write(const qmv_kv4_cache *cache, const qmv_kv_seqs *seqs, uint32_t dtype,
                  const void *k, const void *v, void *stream);

/*
 * Reads the rows' tokens back into k and v ([rows][kv_heads][head_dim],
 * dtype), exactly.  Either of k and v may be NULL.  Errors: as qmv_kv_read.
 */
int qmv_kv4_read(const qmv_kv4_cache *cache, const qmv_kv_seqs *seqs, uint32_t dtype, void *k,
                 void *v, void *stream);

/*
 * Attention of the rows over the cache: as qmv_kv_attend, with its arguments,
 * positions, window and zero rows.  Scores, the softmax's statistics and the
 * output sums are float32.  Queries enter the products exactly; probabilities
 * exactly with float32, with 16 bits or, where bfloat16 queries are many (as
 * there), 11 bits (fewer below 2^-16 of the largest, those below 2^-27 as 0);
 * then values of blocks whose scale is below 2^-13 of their page's and head's
 * largest scale are off by up to 2^-15 of that scale, and values below 2^-80 of
 * the largest of their sequence and head may count as 0.  A query, or a token
 * and head that is seen, with a NaN or infinity gives NaN for the rows that see
 * it and touches no other.  Scores past float32's range may give NaN; values
 * below 2^62 in magnitude never leave it.  Values below 2^-96 may lose low bits
 * or count as 0.
 * A sequence's pages are cut into pieces by its own length beside the others',
 * so one long sequence among short ones uses the whole GPU; max_new and max_len
 * only choose the kernel and how many pieces there are in all.
 * workspace: device memory of at least qmv_kv4_attend_workspace bytes (may be
 * NULL where that is 0), 16-byte aligned.  Errors: as qmv_kv_attend.
 */
int qmv_kv4_attend_workspace(const qmv_kv4_cache *cache, const qmv_kv_seqs *seqs, uint32_t dtype,
                             uint32_t heads, uint32_t window, uint64_t *bytes);
int qmv_kv4_attend(const qmv_kv4_cache *cache, const qmv_kv_seqs *seqs, uint32_t dtype,
                   uint32_t heads, float scale, uint32_t window, const void *q, void *out,
                   void *workspace, uint64_t workspace_bytes, void *stream);

/*
 * Log probabilities of given tokens, with the distribution's entropy and its
 * top alternatives, from logits [rows][vocab] (float32, as qmv_gemv writes
 * an LM head's).  With p = softmax of a row:
 *   lp[row][i] = ln p[ids[row][i]], i < n_ids; 0 for an id outside [0, vocab)
 *   entropy[row] = - sum p ln p
 *   top_ids, top_lp [row][n]: the `top` largest logits' indexes and ln p,
 *   the largest first, equal ones by the lower index.
 * ids: int32 [rows][n_ids].  lp, entropy may be NULL (ids too if lp is);
 * top_ids and top_lp are given together, or NULL with top 0.  A logit of
 * -infinity is a token of probability 0.  A row that holds a NaN or
 * +infinity, or nothing but -infinity, gets NaN for lp, entropy and top_lp;
 * its top_ids are then some indexes of the row.  Sums are float32, of at
 * most 32 terms in each thread and then pairwise, relative to the largest
 * logit.
 * logits 4-byte aligned, the others 4-byte aligned; workspace: 16-byte
 * aligned, at least qmv_logprobs_workspace bytes.
 * Errors: QMV_E_ARG (logits NULL, no output, lp without ids or with n_ids 0,
 * top_ids or top_lp without the other or with top 0, misaligned pointer,
 * rows or vocab 0, workspace NULL or too small), QMV_E_SHAPE (vocab above 2^24, top
 * above 32 or above vocab, rows above 2^22), QMV_E_DEVICE.
 */
int qmv_logprobs_workspace(uint32_t rows, uint32_t vocab, uint32_t top, uint64_t *bytes);
int qmv_logprobs(const float *logits, uint32_t rows, uint32_t vocab, const int32_t *ids,
                 uint32_t n_ids, uint32_t top, float *lp, float *entropy, int32_t *top_ids,
                 float *top_lp, void *workspace, uint64_t workspace_bytes, void *stream);

/*
 * The next token of each row, drawn from logits [rows][vocab] (float32, as
 * qmv_gemv writes an LM head's) with a given random number.  For a row with
 * temperature T, tokens in the order of their logits x, the largest first,
 * equal ones by the lower index, and weights w = e^((x - x_max) / T):
 *   top_k  k > 0: the first k tokens stay (k <= 0: all)
 *   top_p  p < 1: of these, a token stays if the weights before it sum to
 *          less than p times the sum of all of these; the first always stays
 *   min_p  of these, a token stays if w >= m; the first always stays
 * and ids[row] is the first token, by index, at which the sum of the weights
 * of the tokens that stayed exceeds u times their total.  lp[row] = ln of that
 * token's weight over the total.  T = 0 takes the first token in the order
 * (lp 0).  u outside [0, 1) counts as the nearer end, NaN as 0.  A row that
 * holds a NaN or +infinity, or nothing but -infinity, or whose T is negative,
 * infinite or NaN, gets the id -1 and lp NaN.  A NaN in top_p or min_p turns
 * that filter off; p below 0 counts as 0, m above 1 as 1.
 * Weights are whole multiples of 2^-39 of the largest, right to about 2^-22 of
 * themselves; sums are whole numbers, but the total of a whole row (no filter, or
 * top_p without top_k), which is right to about 2^-20.  A row's result depends on
 * that row alone and is the same in every call.  Rows from whose likely tokens
 * the answer cannot be told (a nucleus past about 2500 tokens; top_k now and
 * then from 800 or 1000 on, always from about 2000; more than 256 likely tokens
 * among 1024 neighbours), and vocabularies above 2^19, take one workgroup 0.4 to
 * 0.7 ms a row of 250000.
 * u, temperature, top_p, min_p: float32 [rows], top_k: int32 [rows]; each of
 * the last four may be NULL (T = 1, or no such filter).  ids: int32 [rows];
 * lp: float32 [rows], may be NULL.  All 4-byte aligned device memory;
 * workspace: 16-byte aligned, at least qmv_sample_workspace bytes.
 * Errors: QMV_E_ARG (logits, u or ids NULL, misaligned pointer, rows or vocab
 * 0, workspace NULL or too small), QMV_E_SHAPE (vocab above 2^24, rows above
 * 2^22), QMV_E_DEVICE.
 */
int qmv_sample_workspace(uint32_t rows, uint32_t vocab, uint64_t *bytes);
int qmv_sample(const float *logits, uint32_t rows, uint32_t vocab, const float *u,
               const float *temperature, const int32_t *top_k, const float *top_p,
               const float *min_p, int32_t *ids, float *lp, void *workspace,
               uint64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QMV_SERVE_H */
