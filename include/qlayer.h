/*
 * qlayer.h - C ABI of what stands between a decoder layer's compressed
 * projections (qgemv.h) and its KV cache (qcache.h) on MI355X (gfx950): the
 * low-rank adapters of many requests beside one shared projection, the norms
 * of query and key heads with the position rotation, and attention over whole
 * prompts.  Part of libqgemv; status codes, dtypes, ownership, streams and
 * error rules are those of qgemv.h (device pointers owned by the caller, no
 * device allocation, calls asynchronous on the caller's stream and capturable,
 * Q_OK or a negative status, nothing launched when validation fails,
 * reentrant).
 *
 * Rows: T rows of a batch of B sequences (or requests).  starts[B+1]
 * (nondecreasing, starts[B] <= T, device): sequence b owns rows starts[b] .. starts[b+1]-1.
 * Rows that no sequence owns (below starts[0], at or behind starts[B]) are
 * left as they were.  Everything that depends on device data is read on the
 * device, so a captured call follows it.
 */
#ifndef QLAYER_H
#define QLAYER_H

#include "qcache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --------------------------------------------------------- low-rank adapters
 * A set of n adapters of one projection with K inputs and N outputs, each of
 * rank r at most: out = y + scale[a] * B_a (A_a x). */
typedef struct qadapters {
  int64_t n;                 /* 1 .. 2^20 */
  int64_t K, N;              /* K a multiple of 8, below 2^23; N below 2^25 */
  int rank;                  /* r, a multiple of 8, 8 .. 128 */
  const void* A;             /* [n][r][K] bf16, 16-byte aligned */
  const void* B;             /* [n][N][r] bf16, 16-byte aligned */
  const float* scales;       /* [n] */
  const int32_t* ranks;      /* [n] each adapter's own rank, 0 .. r (others count as these bounds), or NULL: all r.
                                What lies behind it in A and B may be anything. */
} qadapters;

/* Workspace bytes of qadapt (host only; reads n, K, N and rank).  Fewer rows may
 * need more (A_a x is divided further), so a workspace for calls of several sizes
 * has the largest of their values. */
int qadapt_ws(const qadapters* a, int64_t B, int64_t T, size_t* ws_bytes);

/* out[t][:] = y[t][:] + scale[a] * B_a (A_a x[t][:]) with a = ids[b] for the
 * rows of request b; starts = NULL means one row each (T = B).  A request whose
 * id lies outside [0, n) has no adapter: out = y.  x bf16, y and out fp32 or
 * bf16 (y_dtype, both); out may be y itself (the same pointer and stride), and
 * otherwise overlaps no input.  ids: [B] int32, device.  1 <= T <= 2^27, and with
 * starts 1 <= B <= 65536.  Strides in elements from row to row;
 * x 16-byte aligned and its stride a multiple of 8, below 2^24; y and out aligned
 * to their elements.
 * Precision: sums in fp32; A_a x enters the second product in bf16 parts, all of
 * it where y is fp32 and 16 bits and more where it is bf16 (sums of 2^128 - 2^119
 * or more as infinities).  Values of x and A that are not finite come out as the
 * formula has them; an infinity in B or in a scale may come out as NaN.  A row's
 * result depends neither on the other rows' values nor on when the call runs, its
 * last bits on how many rows and requests there are and on which adapters they
 * name.
 * Speed: which kernels run is chosen on the host from B and T, so a long request
 * among many single rows (fewer than 16 rows each on average) is faster in a call
 * of its own.
 * ws: device, 16-byte aligned, >= the qadapt_ws value; calls that may overlap
 * need one each. */
int qadapt(const qadapters* a, int64_t B, int64_t T, const int32_t* ids, const int32_t* starts, const void* x,
           int64_t x_stride, const void* y, int64_t y_stride, void* out, int64_t o_stride, int y_dtype, void* ws,
           size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------- head norms and rotation
 * For every row x of every query and key head, head_dim = 64 or 128 values:
 *   n_i = x_i * w_i / sqrt(mean_j x_j^2 + eps)   (weight NULL: n = x)
 * and of the first rot values the pairs (n_i, n_{i + rot/2}), i < rot/2, or
 * with `pairs` (n_2i, n_{2i+1}), turned by position * freqs[i] radians:
 *   (a cos - b sin, b cos + a sin).
 * The angle is formed in fp64 and reduced to a part of a turn before its sine
 * and cosine, which are fp32.  The rest is fp32, rounded once. */
typedef struct qrope {
  int head_dim, q_heads, kv_heads;   /* heads >= 0, together 1 .. 65536 */
  int rot;                   /* a multiple of 16, 0 .. head_dim */
  int pairs;                 /* 0: halves, 1: neighbours */
  const double* freqs;       /* [rot/2], device; may be NULL for rot = 0 */
  const void* q_weight;      /* [head_dim], device, 16-byte aligned, or NULL: no norm */
  const void* k_weight;
  int w_dtype;               /* Q_BF16 or Q_F32 */
  float eps;                 /* 1e-20 or more, finite; not read where both weights are NULL */
  int64_t offset;            /* added to every position (a shared prefix's length), |offset| < 2^31 */
} qrope;

/* Rows of Q [T][q_heads][head_dim] and K [T][kv_heads][head_dim] (in_dtype
 * Q_BF16 or Q_F32) to Qo and Ko (out_dtype Q_BF16 or Q_F32).  Row starts[b] + i
 * of a sequence with n new rows has position lens[b] - n + i + offset, as in
 * qcache_write; a negative one turns the other way.  starts = NULL means one
 * row for each sequence (T = B).  Strides in elements from one token's rows to
 * the next one's; all four pointers 16-byte aligned and the strides a multiple
 * of 16 bytes.  An output may be its input itself (the same pointer, stride
 * and dtype), and otherwise overlaps no input.  Q may be NULL where q_heads = 0,
 * K where kv_heads = 0.  1 <= T <= 2^27, and 1 <= B <= 65536 with starts. */
int qnorm_rope(const qrope* p, int64_t B, int64_t T, const int32_t* lens, const int32_t* starts, const void* Q,
               int64_t q_stride, const void* K, int64_t k_stride, int in_dtype, void* Qo, int64_t qo_stride, void* Ko,
               int64_t ko_stride, int out_dtype, hipStream_t stream);

/* --------------------------------------------------------- whole prompts
 * Causal attention of B packed prompts over their own, unquantized keys and
 * values: for row t of a sequence that begins at row s,
 *   out[t][hq][:] = sum_{j = s..t} softmax_j(scale <Q[t][hq][:], K[j][hk][:]>) V[j][hk][:],
 * hk = hq / (q_heads / kv_heads); q_heads a multiple of kv_heads, at most 64
 * times it, kv_heads at most 1024, head_dim 64 or 128.  starts = NULL means one
 * sequence of T rows (B = 1).  Q, K, V bf16, out bf16 or fp32 (out_dtype); rows
 * of one token contiguous, strides in elements between tokens, 16-byte aligned
 * and a multiple of 16 bytes.  out overlaps no input.  scale is finite and of
 * magnitude 2^45 at most (else Q_EUNSUPPORTED); |scale| sum_i |Q_i K_i| has to
 * stay below 2^120, sum_i |Q_i K_i| below 2^126, and |V| times the keys of a
 * sequence below 2^118.  1 <= B <= 65536,
 * 1 <= T <= 2^27, T * q_heads / kv_heads at most 2^30.
 * A row that sees a logit of NaN or +inf is NaN; a logit of -inf weighs nothing,
 * and a row that sees no other is NaN.  A row that sees a value that is not
 * finite comes out as NaN or infinite, in that component at least.  The rows
 * before such keys and values do not change.
 * Precision: products of bf16 values in fp32, sums, maxima and the softmax
 * statistics fp32, weights rounded to bf16 before they meet V, also where the
 * output is fp32.  No workspace: calls may overlap.
 * Speed: how a tile's keys are shared is chosen on the host from T and B, so one
 * long prompt is faster in a call of its own than among many short or empty ones. */
int qprompt_attend(int head_dim, int q_heads, int kv_heads, int64_t B, int64_t T, const int32_t* starts, const void* Q,
                   int64_t q_stride, const void* K, int64_t k_stride, const void* V, int64_t v_stride, float scale,
                   void* out, int64_t o_stride, int out_dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QLAYER_H */
