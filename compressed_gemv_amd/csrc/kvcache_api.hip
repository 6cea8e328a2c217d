// C ABI of the quantized, paged KV cache (declared in include/qcache.h):
// argument validation, size queries, dispatch to the kernels.  Validation
// runs on the host before any HIP call.
#include "qcache.h"

#include "kvcache.hpp"

#include <math.h>
#include <stdint.h>

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? Q_OK : Q_EHIP; }

int dims_ok(int64_t n_pages, int page_size, int heads, int head_dim, int bits) {
  if (n_pages < 1 || heads < 1) return Q_EINVAL;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return Q_EINVAL;
  if (bits != 4 && bits != 8) return Q_EINVAL;
  if (head_dim != 64 && head_dim != 128) return head_dim < 1 ? Q_EINVAL : Q_EUNSUPPORTED;
  // page numbers are 32-bit, and a cache row index times 128 bytes stays far inside 64 bits
  if (heads > 1024 || n_pages > INT32_MAX) return Q_EUNSUPPORTED;
  return Q_OK;
}

int cache_ok(const qcache* c) {
  if (!c) return Q_EINVAL;
  const int st = dims_ok(c->n_pages, c->page_size, c->heads, c->head_dim, c->bits);
  if (st != Q_OK) return st;
  if (!c->k_codes || !c->k_meta || !c->v_codes || !c->v_meta) return Q_EINVAL;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_meta, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_meta, 16))
    return Q_EALIGN;
  return Q_OK;
}

// sizes alone: what the workspace query reads
int seq_sizes_ok(const qcache* c, const qseqs* s) {
  if (!s || s->B < 1 || s->B > 65536 || s->T < 1 || s->max_pages < 1) return Q_EINVAL;
  // rows and positions are 32-bit, and a grid of 256 threads for 16 rows stays below 2^32 threads
  if (s->T > (1 << 27) || s->max_pages > ((int64_t)1 << 30) / c->page_size) return Q_EUNSUPPORTED;
  return Q_OK;
}

int seqs_ok(const qcache* c, const qseqs* s) {
  const int st = seq_sizes_ok(c, s);
  if (st != Q_OK) return st;
  if (!s->pages || !s->lens || (!s->starts && s->T != s->B)) return Q_EINVAL;
  if (!aligned(s->pages, 4) || !aligned(s->lens, 4) || !aligned(s->starts, 4)) return Q_EALIGN;
  return Q_OK;
}

// rows of `width` elements of es bytes at stride `stride`
int rows_ok(const void* p, int64_t stride, int64_t width, int es) {
  if (!p || stride < width) return Q_EINVAL;
  if (stride > ((int64_t)1 << 30)) return Q_EUNSUPPORTED;
  return aligned(p, 16) && stride * es % 16 == 0 ? Q_OK : Q_EALIGN;
}

qg::KvView view(const qcache* c) {
  qg::KvView v;
  v.codes[0] = static_cast<uint8_t*>(c->k_codes);
  v.codes[1] = static_cast<uint8_t*>(c->v_codes);
  v.meta[0] = static_cast<uint32_t*>(c->k_meta);
  v.meta[1] = static_cast<uint32_t*>(c->v_meta);
  v.n_pages = (int)c->n_pages;
  v.page_shift = __builtin_ctz((unsigned)c->page_size);
  v.heads = c->heads;
  return v;
}

qg::SeqView view(const qseqs* s) {
  return qg::SeqView{s->pages, s->lens, s->starts, (int)s->B, (int)s->T, (int)s->max_pages};
}

int attend_heads_ok(const qcache* c, int q_heads) {
  if (q_heads < 1 || q_heads % c->heads) return Q_EINVAL;
  return q_heads / c->heads <= 64 ? Q_OK : Q_EUNSUPPORTED;
}

int attend(const qcache* c, const qseqs* s, const int32_t* prefix_pages, int64_t prefix_len, const void* Q,
           int64_t q_stride, int q_heads, float scale, void* out, int64_t o_stride, int out_dtype, void* ws,
           size_t ws_bytes, hipStream_t stream) {
  int st = cache_ok(c);
  if (st != Q_OK) return st;
  if ((st = seqs_ok(c, s)) != Q_OK) return st;
  size_t need = 0;
  if ((st = qcache_attend_ws(c, s, q_heads, prefix_len, &need)) != Q_OK) return st;
  if (!isfinite(scale) || (out_dtype != Q_BF16 && out_dtype != Q_F32)) return Q_EINVAL;
  // the kernel for few rows holds scale * log2(e) * 2^69 * s in fp32, s at most 8734 (a 4-bit row over +-65504)
  if (fabsf(scale) > 0x1p45f) return Q_EUNSUPPORTED;
  const int64_t width = (int64_t)q_heads * c->head_dim;
  if ((st = rows_ok(Q, q_stride, width, 2)) != Q_OK) return st;
  if ((st = rows_ok(out, o_stride, width, out_dtype == Q_F32 ? 4 : 2)) != Q_OK) return st;
  if (!ws || ws_bytes < need) return Q_EWORKSPACE;
  if (!aligned(ws, 16)) return Q_EALIGN;
  qg::KvAttend a;
  a.c = view(c);
  a.s = view(s);
  a.Q = static_cast<const uint16_t*>(Q);
  a.q_stride = q_stride;
  a.o_stride = o_stride;
  a.group = q_heads / c->heads;
  a.scale = scale;
  a.out = out;
  a.out_f32 = out_dtype == Q_F32;
  a.prefix_pages = prefix_pages;
  a.prefix_len = (int)prefix_len;
  return hip_status(qg::launch_kv_attend(a, c->head_dim, c->bits, ws, stream));
}

}  // namespace

extern "C" {

int qcache_sizes(int64_t n_pages, int page_size, int heads, int head_dim, int bits, size_t* codes_bytes,
                 size_t* meta_bytes) {
  const int st = dims_ok(n_pages, page_size, heads, head_dim, bits);
  if (st != Q_OK) return st;
  const int64_t rows = n_pages * heads * page_size;
  if (codes_bytes) *codes_bytes = (size_t)(rows * (head_dim * bits / 8));
  if (meta_bytes) *meta_bytes = (size_t)(rows * 4);
  return Q_OK;
}

int qcache_write(const qcache* c, const qseqs* s, const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                 int dtype, hipStream_t stream) {
  int st = cache_ok(c);
  if (st != Q_OK) return st;
  if ((st = seqs_ok(c, s)) != Q_OK) return st;
  if (dtype != Q_BF16 && dtype != Q_F32) return Q_EINVAL;
  const int64_t width = (int64_t)c->heads * c->head_dim;
  const int es = dtype == Q_F32 ? 4 : 2;
  if ((st = rows_ok(K, k_stride, width, es)) != Q_OK) return st;
  if ((st = rows_ok(V, v_stride, width, es)) != Q_OK) return st;
  return hip_status(qg::launch_kv_write(view(c), view(s), c->head_dim, c->bits, K, k_stride, V, v_stride,
                                        dtype == Q_F32, stream));
}

int qcache_read(const qcache* c, const qseqs* s, void* K, int64_t k_stride, void* V, int64_t v_stride, int dtype,
                hipStream_t stream) {
  int st = cache_ok(c);
  if (st != Q_OK) return st;
  if ((st = seqs_ok(c, s)) != Q_OK) return st;
  if (dtype != Q_BF16 && dtype != Q_F32) return Q_EINVAL;
  const int64_t width = (int64_t)c->heads * c->head_dim;
  const int es = dtype == Q_F32 ? 4 : 2;
  if ((st = rows_ok(K, k_stride, width, es)) != Q_OK) return st;
  if ((st = rows_ok(V, v_stride, width, es)) != Q_OK) return st;
  return hip_status(qg::launch_kv_read(view(c), view(s), c->head_dim, c->bits, K, k_stride, V, v_stride,
                                       dtype == Q_F32, stream));
}

int qcache_attend_ws(const qcache* c, const qseqs* s, int q_heads, int64_t prefix_len, size_t* ws_bytes) {
  if (!c || !ws_bytes) return Q_EINVAL;
  int st = dims_ok(c->n_pages, c->page_size, c->heads, c->head_dim, c->bits);
  if (st != Q_OK) return st;
  if ((st = seq_sizes_ok(c, s)) != Q_OK) return st;
  if ((st = attend_heads_ok(c, q_heads)) != Q_OK) return st;
  if (prefix_len < 0) return Q_EINVAL;
  if (prefix_len > ((int64_t)1 << 30)) return Q_EUNSUPPORTED;
  // rows of one KV head are counted in 32 bits
  const int64_t rows = s->T * (q_heads / c->heads);
  if (rows > (1 << 30)) return Q_EUNSUPPORTED;
  // weights of the line of work times 512 pieces stay below 2^52: half a weight for a key of a tile of 8 rows or more
  if ((double)(rows / 8 + s->B) * (double)((s->max_pages * c->page_size + prefix_len) / 2 + 512) * 512.0 > 4e15)
    return Q_EUNSUPPORTED;
  *ws_bytes = qg::kv_attend_ws_bytes(s->B, s->T, s->max_pages, __builtin_ctz((unsigned)c->page_size), c->heads,
                                     q_heads / c->heads, c->head_dim, prefix_len);
  return Q_OK;
}

int qcache_attend(const qcache* c, const qseqs* s, const void* Q, int64_t q_stride, int q_heads, float scale, void* out,
                  int64_t o_stride, int out_dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  return attend(c, s, nullptr, 0, Q, q_stride, q_heads, scale, out, o_stride, out_dtype, ws, ws_bytes, stream);
}

int qcache_attend_shared(const qcache* c, const qseqs* s, const int32_t* prefix_pages, int64_t prefix_len, const void* Q,
                         int64_t q_stride, int q_heads, float scale, void* out, int64_t o_stride, int out_dtype,
                         void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!prefix_pages || prefix_len < 1) return Q_EINVAL;
  if (!aligned(prefix_pages, 4)) return Q_EALIGN;
  return attend(c, s, prefix_pages, prefix_len, Q, q_stride, q_heads, scale, out, o_stride, out_dtype, ws, ws_bytes,
                stream);
}

}  // extern "C"
