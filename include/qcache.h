/*
 * qcache.h - C ABI of the paged cache of quantised keys and values (part of libfq.so), sm_103a.
 *
 * Beside the FibQuant store (fq.h), which holds rows at 0.19 to 4 bits per coordinate behind a
 * shared codebook, this cache holds them at 8 or 4 bits behind a scale per row: what the newest
 * tokens of a sequence, or a cache that must be appended to in a microsecond, want. Four operators
 * make up a decoding step of one layer around it: the heads' norm and position rotation
 * (qc_norm_rope), the quantised write (qc_write), the read back (qc_read) and the attention of a
 * sequence's drafted tokens over its cached ones (qc_attend).
 *
 * Conventions are those of fq.h: caller-owned device buffers, asynchronous calls on a stream
 * (void* cudaStream_t, NULL = legacy default stream) that validate on the host and return FQ_*
 * codes, the current device left as it was, one host thread per context. Conditions only the
 * device can see set sticky bits that qc_status() reads and clears; nothing traps.
 *
 * Formats. A row is the d elements of one token and head; A is its largest magnitude.
 *   QC_INT8: s = A / 127, code = round(x (127 / A)), value = code s.
 *   QC_E4M3: s = A / 448, code = e4m3(x (448 / A)), value = code s.
 *   QC_E2M1: s = A / 2688; per block of 16 elements with largest magnitude a: sb = e4m3(a (448 / A));
 *            code = e2m1(x ((2688 / A) / sb)), value = (code sb) s. Blocks with sb = 0 hold zeros.
 * All in float32, each operation rounded to nearest even, as are the conversions to a code; values
 * beyond a code's range take its largest. Rows with A < 2^-100 hold zeros and s = 0.
 *
 * Pages. The cache is an array of n_pages pages of page_tokens tokens; token slot i is token
 * i mod page_tokens of page i / page_tokens. A page holds, head by head, one run of bytes:
 *   keys' codes [page_tokens][row bytes], values' codes (the same), keys' scales float32
 *   [page_tokens], values' scales, and for QC_E2M1 the keys' block scales [page_tokens][d / 16]
 *   (e4m3 bytes), then the values'.
 * Row bytes are d (8 bits) or d / 2 (4 bits; the element of even index in the low half). In a run
 * of codes the 16-byte piece p counted from the run's start lies at piece p ^ ((p >> 3) & 7): a
 * page copied to shared memory as it lies is then read by rows and by columns without bank conflicts.
 */
#ifndef FQ_QCACHE_H
#define FQ_QCACHE_H

#include <stdint.h>

#include "fq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qc_ctx qc_ctx;

/* Formats of the cache, and types of the rows that go in and come out. */
enum { QC_INT8 = 0, QC_E4M3 = 1, QC_E2M1 = 2 };
enum { QC_F16 = 0, QC_BF16 = 1, QC_F32 = 2 };

/* Sticky device flags returned by qc_status(). */
enum {
    QC_FLAG_RANGE = 1u,      /* a slot, position, page number, length or node count was out of range */
    QC_FLAG_NONFINITE = 2u,  /* a written row had a NaN or Inf: the cache holds zeros for it */
    QC_FLAG_TIMEOUT = 4u     /* a bounded device-side wait gave up: that call's output is invalid */
};

/*
 * qc_create - a context for caches of one geometry on `device`.
 *   format      : QC_INT8, QC_E4M3 or QC_E2M1.
 *   d           : head dimension, 64 or 128.
 *   n_heads     : key/value heads, 1 .. 1024.
 *   page_tokens : 16, 32, 64, 128 or 256.
 * Returns FQ_OK and *out, or FQ_EINVAL / FQ_ENOMEM / FQ_ECUDA / FQ_ENODEV and *out = NULL.
 */
int qc_create(qc_ctx **out, int format, int d, int n_heads, int page_tokens, int device);

/* Bytes of one page: n_heads * 2 page_tokens (row bytes + 4 [+ d / 16]). -1 for a NULL context. */
int64_t qc_page_bytes(const qc_ctx *ctx);

/*
 * qc_norm_rope - norm of each query and key head and its rotation by position, in one pass:
 *   y = x / sqrt(mean(x^2) + eps) * w;  for i < rot / 2 the pair (a, b) of elements i and i + rot / 2
 *   (interleaved: 2 i and 2 i + 1) becomes (a cos - b sin, b cos + a sin).
 * Sums and products are float32; each result is rounded once, to `type`.
 *   type        : QC_F16, QC_BF16 or QC_F32, of q, k and the outputs.
 *   q, k        : device [n][heads][d], d contiguous, token and head strides in elements; either may
 *                 have 0 heads. hq, hk <= 1024.
 *   wq, wk      : device float32 [d], 16-byte aligned; NULL: no norm, the rotation alone.
 *   pos         : device int64 [n]; a position outside [0, max_pos) gives zero rows and QC_FLAG_RANGE.
 *   table       : device float32 [max_pos][rot], 16-byte aligned: cosines [rot / 2], then sines.
 *   rot         : rotated elements, a multiple of 16, 0 <= rot <= d. 0: the norm alone (pos and table
 *                 are not read).
 *   q_out, k_out: as q and k with strides of their own; they may be q and k themselves.
 * Every row starts on a 16-byte boundary (FQ_EALIGN). eps is finite and >= 0, n <= 2^32.
 */
int qc_norm_rope(qc_ctx *ctx, int type, int64_t n, const void *q, int hq, int64_t q_token, int64_t q_head,
                 const float *wq, const void *k, int hk, int64_t k_token, int64_t k_head, const float *wk, float eps,
                 const int64_t *pos, const float *table, int64_t max_pos, int rot, int interleaved, void *q_out,
                 int64_t qo_token, int64_t qo_head, void *k_out, int64_t ko_token, int64_t ko_head, void *stream);

/*
 * qc_write - quantise the keys and values of n tokens into their slots.
 *   k, v   : device [n][n_heads][d] of `type`, strides as above.
 *   slots  : device int64 [n], all different; -1 skips the token; any other slot outside
 *            [0, n_pages * page_tokens) skips it and sets QC_FLAG_RANGE.
 *   pages  : device bytes [n_pages][qc_page_bytes], 16-byte aligned. Bytes of other tokens are not
 *            written.
 * n <= 2^32 and n * n_heads <= 2^35, here and in qc_read.
 */
int qc_write(qc_ctx *ctx, int type, int64_t n, const void *k, int64_t k_token, int64_t k_head, const void *v,
             int64_t v_token, int64_t v_head, const int64_t *slots, void *pages, int64_t n_pages, void *stream);

/*
 * qc_read - the values that the cache holds of the tokens in n slots, in any order.
 *   k_out, v_out : device [n][n_heads][d] of `type`, contiguous, 16-byte aligned; either may be NULL.
 *   slots        : device int64 [n]; -1 gives zero rows; any other slot out of range too, and sets
 *                  QC_FLAG_RANGE.
 */
int qc_read(qc_ctx *ctx, int type, int64_t n, const int64_t *slots, const void *pages, int64_t n_pages, void *k_out,
            void *v_out, void *stream);

/*
 * qc_attend - softmax attention of the drafted tokens ("nodes") of n_seq sequences over the cache.
 * Sequence b holds lens[b] cached tokens, its prefix, at places 0 .. lens[b] - 1, and its node j at
 * place lens[b] + j (written there by qc_write, seen by others or not); place t is slot
 * table[b][t / page_tokens] * page_tokens + t % page_tokens. Node i < nodes[b] sees the whole prefix
 * and the nodes that its bits name. For query head h and the key/value head h / (n_q_heads / n_heads):
 *   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(s_t - max s),  s_t = scale * q . k_t,
 *   lse = log sum_t exp(s_t),  t over the places seen.
 * A row that sees nothing, and every row of a node i >= nodes[b], has out = 0 and lse = -inf.
 * A row that sees a place and whose query holds a NaN or an infinity, or a score above float32's range, has
 * out = NaN and lse = NaN (scores below it weigh nothing).
 * n_nodes = 1 is the single-token step of a decoder.
 *   type      : QC_F16 or QC_BF16, of q and out.
 *   n_nodes   : 1 .. 1024 nodes per sequence, that of the longest.
 *   n_q_heads : a multiple of n_heads, at most 64 times it.
 *   q         : device [n_seq][n_nodes][n_q_heads][d], d contiguous, the other strides in elements;
 *               every row on a 16-byte boundary.
 *   table     : device int32 [n_seq], rows table_stride apart, of table_stride >=
 *               ceil((max_len + n_nodes) / page_tokens) page numbers. Only the entries of places up to
 *               lens[b] + nodes[b] are read. Tokens of a page outside [0, n_pages) are not seen and set
 *               QC_FLAG_RANGE.
 *   lens      : device int32 [n_seq], 0 <= lens[b] <= max_len; nodes: device int32 [n_seq], 0 <=
 *               nodes[b] <= n_nodes, or NULL for n_nodes each. Others are clamped and set QC_FLAG_RANGE.
 *   tree      : device uint32 [n_seq][n_nodes][ceil(n_nodes / 32)]: bit j % 32 of word j / 32 says that
 *               the row's node sees node j. NULL: node i sees nodes 0 .. i.
 *   out       : device [n_seq][n_nodes][n_q_heads][d], 16-byte aligned; lse: device float32
 *               [n_seq][n_nodes][n_q_heads], or NULL.
 *   workspace : device, 16-byte aligned, at least qc_attend_workspace() bytes, used by one call at a
 *               time; its contents do not matter and mean nothing afterwards.
 * Products take the codes as they are, exactly, and q as it is, but for elements of a QC_BF16 row below 2^-30 of its
 * largest, which are off by up to 2^-38 of that (float16's range); sums are float32. The products p s of a weight and
 * its value row's scale are rounded to 11 bits (one float16) for QC_BF16 and to 22 (two) for QC_F16. Above 32 query rows
 * (n_nodes * n_q_heads / n_heads) and from 1,024 places (max_len + n_nodes) on, those that are light beside the row's
 * largest are held to 2^-29 of it instead, so that an element which is zero wherever p s is large may lose that much
 * a place. Below, rows whose values are small beside others of the sequence are summed in float32, and an element that
 * is zero in a row's heavy places may lose 2^-20 of the row's largest element for each light one. Products p s
 * below 2^-90 of the row's heaviest weight times the largest scale of its sequence lose bits, down to none.
 * n_seq <= 65,535, and n_seq * n_nodes * n_q_heads < 2^31. Results do not depend on timing.
 */
int qc_attend(qc_ctx *ctx, int type, int64_t n_seq, int n_nodes, int n_q_heads, const void *q, int64_t q_seq,
              int64_t q_node, int64_t q_head, const int32_t *table, int64_t table_stride, const int32_t *lens,
              const int32_t *nodes, const uint32_t *tree, const void *pages, int64_t n_pages, float scale,
              int64_t max_len, void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace that qc_attend wants for these sizes: enough for calls with fewer of each, too. -1 on bad
 * arguments. */
int64_t qc_attend_workspace(const qc_ctx *ctx, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len);

/* qc_status - reads and clears the context's sticky QC_FLAG_* bits in one atomic exchange on the device
 * (as fq_status), then synchronises `stream`. */
int qc_status(qc_ctx *ctx, void *stream, uint32_t *flags);

/* qc_destroy - frees the context. Synchronises its device. NULL is a no-op. */
void qc_destroy(qc_ctx *ctx);

#ifdef __cplusplus
}
#endif

#endif /* FQ_QCACHE_H */
