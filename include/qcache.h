/*
 * qcache.h - C ABI of the quantized, paged KV cache of the MI355X (gfx950)
 * compressed-weight library: write, read back, attend.  Part of libqgemv;
 * status codes, dtypes, ownership, streams and error rules are those of
 * qgemv.h (device pointers owned by the caller, no device allocation, calls
 * asynchronous on the caller's stream and capturable, Q_OK or a negative
 * status, nothing launched when validation fails, reentrant).
 *
 * A cache holds the K and V rows of `heads` KV heads for n_pages pages of
 * page_size tokens (16, 32, 64, 128 or 256).  A row is one token of one head,
 * head_dim = 64 or 128 values, stored by the group round-to-nearest of
 * qpack_group with the whole row as its group and bits = 4 or 8: fp16 scale s
 * and offset o, w_hat = s*q + o.
 *   codes  [page][head][slot][head_dim*bits/8] bytes; 8 bits: one byte per
 *          value, 4 bits: value 2i in the low and 2i+1 in the high half of
 *          byte i (the format-1 code layout of 4-bit groups).
 *   meta   [page][head][slot] u32: bits 0..15 fp16 s, bits 16..31 fp16 o.
 * K and V have a codes and a meta buffer each, 16-byte aligned.
 *
 * Constants: o = largest fp16 <= min, s = smallest fp16 >= (max - o)/(2^b - 1)
 * (fp64), q = rint((x - o)/s) in fp64, ties to even.  Values beyond +-65280
 * are stored as +-65280, so that no level leaves fp16.  A row that holds an
 * infinity or a NaN gets s = o = NaN and codes 0: it reads back as NaN, and an
 * attention row that sees it comes out as NaN.  Buffers that are filled by
 * other means have to keep to the same range: in every row that holds a token
 * o and s*(2^b - 1) + o lie within +-65504, or s and o are NaN (qcache_attend
 * forms values in fp16, and one beyond it would reach rows that do not see its
 * token).  Rows that hold no token may be anything.
 *
 * Sequences: every call takes the batch as a qseqs.  Rows of K, V, Q and the
 * outputs are ragged: sequence b owns rows starts[b] .. starts[b+1]-1, its
 * newest tokens.  With n = starts[b+1] - starts[b], row starts[b] + i is the
 * token at position lens[b] - n + i, and position p lives in slot p % page_size
 * of page pages[b][p / page_size].  starts = NULL means one row for each
 * sequence (T = B).  lens counts the tokens of the sequence with the new rows.
 * A row without a place (a negative position, one behind the page table, a
 * page outside [0, n_pages)) is not written, reads as zeros, and is seen by
 * no attention row.  Rows that no sequence owns (below starts[0], at or
 * behind starts[B]) are left as they were.  A page may appear in several
 * tables as long as no two rows of one qcache_write land in the same slot
 * (the slot's contents are then one of the rows', codes and constants not
 * necessarily of the same one).
 */
#ifndef QCACHE_H
#define QCACHE_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qcache {
  int64_t n_pages;
  int page_size, heads, head_dim, bits;
  void* k_codes;
  void* k_meta;
  void* v_codes;
  void* v_meta;
} qcache;

typedef struct qseqs {
  int64_t B;                 /* sequences, 1 .. 65536 */
  int64_t T;                 /* rows of K, V, Q and the outputs, 1 .. 2^27, starts[B] <= T */
  int64_t max_pages;         /* width of the page table, max_pages * page_size <= 2^30 */
  const int32_t* pages;      /* [B][max_pages], device */
  const int32_t* lens;       /* [B], device; positions behind the table have no place */
  const int32_t* starts;     /* [B+1] nondecreasing, device, or NULL */
} qseqs;

/* Byte sizes of one codes and one meta buffer (host only).  n_pages >= 1,
 * 1 <= heads <= 1024. */
int qcache_sizes(int64_t n_pages, int page_size, int heads, int head_dim, int bits,
                 size_t* codes_bytes, size_t* meta_bytes);

/* Quantize rows K[t][h][:], V[t][h][:] (dtype Q_BF16 or Q_F32) into the cache.
 * k_stride, v_stride: elements from one token's rows to the next one's (at
 * least heads * head_dim; a slice of a fused projection is fine); the rows of
 * one token are contiguous.  K, V 16-byte aligned and the strides a multiple
 * of 16 bytes. */
int qcache_write(const qcache* c, const qseqs* s, const void* K, int64_t k_stride, const void* V,
                 int64_t v_stride, int dtype, hipStream_t stream);

/* Rows of the cache as values: K[t][h][:] = s*q + o (fp32, and rounded once
 * more to nearest even for Q_BF16).  Strides and alignment as qcache_write. */
int qcache_read(const qcache* c, const qseqs* s, void* K, int64_t k_stride, void* V, int64_t v_stride,
                int dtype, hipStream_t stream);

/* Workspace bytes of qcache_attend (prefix_len = 0) and of
 * qcache_attend_shared (host only; reads B, T and max_pages of s). */
int qcache_attend_ws(const qcache* c, const qseqs* s, int q_heads, int64_t prefix_len, size_t* ws_bytes);

/* out[t][hq][:] = sum_j softmax_j(scale <Q[t][hq][:], k_j>) v_j over the
 * positions j of the row's own sequence up to the row's own position, KV head
 * hq / (q_heads / heads); q_heads a multiple of heads, at most 64 times it.
 * scale is finite (else Q_EINVAL) and of magnitude 2^45 at most (else
 * Q_EUNSUPPORTED); |scale| sum_i |Q_i k_i| has to stay below 2^120.  Q is bf16,
 * of magnitudes below 2^63 (2^-57 and less may count as 0), out bf16 or fp32
 * (out_dtype); rows of one token contiguous, q_stride and o_stride elements
 * between tokens; Q and out 16-byte aligned, strides a multiple of 16 bytes.
 * A row that sees nothing is zero.
 * Precision: sums, maxima and the softmax statistics are fp32.  Let R be
 * ceil(T / B) * q_heads / heads, the rows of a KV head and sequence on average
 * (T * q_heads / heads for the prefix's keys of qcache_attend_shared).  For
 * R <= 32 keys and values enter as they are and weights with 16 bits; beyond,
 * keys, values and weights are rounded to 11 bits and queries to 2^-25 of their
 * row's largest, also where the output is fp32.  So a row's last bits depend on
 * the other rows of the call, but not on when or how often it runs.
 * Speed: which kernels run is chosen on the host from B, T and max_pages (the
 * lengths stay on the device), so a page table no wider than the longest
 * sequence can become is the fastest, and decode steps and chunks of prompts
 * are faster in a call each than in one together.
 * ws: device, 16-byte aligned, >= the qcache_attend_ws value; calls that may
 * overlap need one each. */
int qcache_attend(const qcache* c, const qseqs* s, const void* Q, int64_t q_stride, int q_heads, float scale,
                  void* out, int64_t o_stride, int out_dtype, void* ws, size_t ws_bytes, hipStream_t stream);

/* The same with a prefix that every row of the call sees before its own
 * sequence: prefix_len tokens (>= 1) in the pages prefix_pages (device,
 * ceil(prefix_len / page_size) entries).  Its rows are read once for every 256
 * attention rows of a KV head (T * q_heads / heads in all), not once for every
 * sequence.  lens, starts and pages describe each sequence's own tokens only,
 * and lens[b] = 0 is a sequence that so far is the prefix alone. */
int qcache_attend_shared(const qcache* c, const qseqs* s, const int32_t* prefix_pages, int64_t prefix_len,
                         const void* Q, int64_t q_stride, int q_heads, float scale, void* out,
                         int64_t o_stride, int out_dtype, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QCACHE_H */
