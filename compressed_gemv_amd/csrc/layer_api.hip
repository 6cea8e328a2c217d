// C ABI of the steps between a layer's projections and its KV cache (declared
// in include/qlayer.h): argument validation, size queries, dispatch.  Validation
// runs on the host before any HIP call.
#include "qlayer.h"

#include "layer.hpp"

#include <math.h>
#include <stdint.h>

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 27, kMaxSeqs = 65536;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? Q_OK : Q_EHIP; }
bool float_dtype(int dt) { return dt == Q_F32 || dt == Q_BF16; }
int size_of(int dt) { return dt == Q_F32 ? 4 : 2; }

// rows of `width` elements of es bytes at stride `stride`
int rows_ok(const void* p, int64_t stride, int64_t width, int es) {
  if (!p || stride < width) return Q_EINVAL;
  if (stride > ((int64_t)1 << 30)) return Q_EUNSUPPORTED;
  return aligned(p, 16) && stride * es % 16 == 0 ? Q_OK : Q_EALIGN;
}

// the same where only elements have to be aligned
int loose_rows_ok(const void* p, int64_t stride, int64_t width, int es) {
  if (!p || stride < width) return Q_EINVAL;
  if (stride > ((int64_t)1 << 30)) return Q_EUNSUPPORTED;
  return aligned(p, es) ? Q_OK : Q_EALIGN;
}

int adapters_ok(const qadapters* a) {
  if (!a || a->n < 1 || a->K < 1 || a->N < 1 || a->rank < 1) return Q_EINVAL;
  if (a->K % 8 || a->rank % 8) return Q_EINVAL;
  // a workgroup's part of A and an offset into it stay below 2^31 bytes, N over 1024 below 2^16
  if (a->n > (1 << 20) || a->K >= (1 << 23) || a->N >= (1 << 25) || a->rank > 128) return Q_EUNSUPPORTED;
  return Q_OK;
}

int batch_ok(int64_t B, int64_t T) {
  if (B < 1 || T < 1) return Q_EINVAL;
  return T > kMaxRows ? Q_EUNSUPPORTED : Q_OK;
}

int heads_ok(int head_dim, int q_heads, int kv_heads) {
  if (head_dim < 1 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads) return Q_EINVAL;
  if ((head_dim != 64 && head_dim != 128) || kv_heads > 1024 || q_heads / kv_heads > 64) return Q_EUNSUPPORTED;
  return Q_OK;
}

}  // namespace

extern "C" {

int qadapt_ws(const qadapters* a, int64_t B, int64_t T, size_t* ws_bytes) {
  int st = adapters_ok(a);
  if (st != Q_OK) return st;
  if (!ws_bytes) return Q_EINVAL;
  if ((st = batch_ok(B, T)) != Q_OK) return st;
  if (B > T && B > kMaxSeqs) return Q_EINVAL;
  *ws_bytes = qg::adapt_ws_bytes(B, T, a->K, a->rank);
  return Q_OK;
}

int qadapt(const qadapters* a, int64_t B, int64_t T, const int32_t* ids, const int32_t* starts, const void* x,
           int64_t x_stride, const void* y, int64_t y_stride, void* out, int64_t o_stride, int y_dtype, void* ws,
           size_t ws_bytes, hipStream_t stream) {
  size_t need = 0;
  int st = qadapt_ws(a, B, T, &need);
  if (st != Q_OK) return st;
  if (!a->A || !a->B || !a->scales || !ids || (starts ? B > kMaxSeqs : B != T) || !float_dtype(y_dtype)) return Q_EINVAL;
  if (!aligned(a->A, 16) || !aligned(a->B, 16) || !aligned(a->scales, 4) || !aligned(a->ranks, 4) || !aligned(ids, 4) ||
      !aligned(starts, 4))
    return Q_EALIGN;
  if ((st = rows_ok(x, x_stride, a->K, 2)) != Q_OK) return st;
  if (x_stride >= (1 << 24)) return Q_EUNSUPPORTED;
  if ((st = loose_rows_ok(y, y_stride, a->N, size_of(y_dtype))) != Q_OK) return st;
  if ((st = loose_rows_ok(out, o_stride, a->N, size_of(y_dtype))) != Q_OK) return st;
  if (out == y && o_stride != y_stride) return Q_EINVAL;
  if (!ws || ws_bytes < need) return Q_EWORKSPACE;
  if (!aligned(ws, 16)) return Q_EALIGN;
  qg::Adapt p;
  p.A = static_cast<const uint16_t*>(a->A);
  p.B = static_cast<const uint16_t*>(a->B);
  p.scales = a->scales;
  p.ranks = a->ranks;
  p.n = (int)a->n;
  p.rank = a->rank;
  p.K = (int)a->K;
  p.N = (int)a->N;
  p.seqs = (int)B;
  p.T = (int)T;
  p.ids = ids;
  p.starts = starts;
  p.x = static_cast<const uint16_t*>(x);
  p.y = y;
  p.out = out;
  p.x_stride = x_stride;
  p.y_stride = y_stride;
  p.o_stride = o_stride;
  p.f32 = y_dtype == Q_F32;
  p.part = static_cast<float*>(ws);
  return hip_status(qg::launch_adapt(p, stream));
}

int qnorm_rope(const qrope* p, int64_t B, int64_t T, const int32_t* lens, const int32_t* starts, const void* Q,
               int64_t q_stride, const void* K, int64_t k_stride, int in_dtype, void* Qo, int64_t qo_stride, void* Ko,
               int64_t ko_stride, int out_dtype, hipStream_t stream) {
  if (!p || p->head_dim < 1 || p->q_heads < 0 || p->kv_heads < 0 || (int64_t)p->q_heads + p->kv_heads < 1) return Q_EINVAL;
  if (p->head_dim != 64 && p->head_dim != 128) return Q_EUNSUPPORTED;
  if ((int64_t)p->q_heads + p->kv_heads > 65536) return Q_EUNSUPPORTED;
  if (p->rot < 0 || p->rot > p->head_dim || p->rot % 2) return Q_EINVAL;
  if (p->rot % 16) return Q_EUNSUPPORTED;
  if (p->rot > 0 && !p->freqs) return Q_EINVAL;
  if (!float_dtype(in_dtype) || !float_dtype(out_dtype)) return Q_EINVAL;
  const bool normed = p->q_weight || p->k_weight;
  if (normed && (!float_dtype(p->w_dtype) || !(p->eps >= 1e-20f) || !isfinite(p->eps))) return Q_EINVAL;
  if (p->offset <= -((int64_t)1 << 31) || p->offset >= ((int64_t)1 << 31)) return Q_EUNSUPPORTED;
  int st = batch_ok(B, T);
  if (st != Q_OK) return st;
  if (B > kMaxSeqs && starts) return Q_EINVAL;
  if (!lens || (!starts && B != T)) return Q_EINVAL;
  if (!aligned(p->freqs, 8) || !aligned(p->q_weight, 16) || !aligned(p->k_weight, 16) || !aligned(lens, 4) || !aligned(starts, 4))
    return Q_EALIGN;
  qg::NormRope r;
  r.in[0] = Q;
  r.in[1] = K;
  r.out[0] = Qo;
  r.out[1] = Ko;
  r.in_stride[0] = q_stride;
  r.in_stride[1] = k_stride;
  r.out_stride[0] = qo_stride;
  r.out_stride[1] = ko_stride;
  for (int i = 0; i < 2; ++i) {
    const int64_t width = (int64_t)(i ? p->kv_heads : p->q_heads) * p->head_dim;
    if (width == 0) continue;
    if ((st = rows_ok(r.in[i], r.in_stride[i], width, size_of(in_dtype))) != Q_OK) return st;
    if ((st = rows_ok(r.out[i], r.out_stride[i], width, size_of(out_dtype))) != Q_OK) return st;
    if (r.in[i] == r.out[i] && (r.in_stride[i] != r.out_stride[i] || in_dtype != out_dtype)) return Q_EINVAL;
  }
  r.head_dim = p->head_dim;
  r.q_heads = p->q_heads;
  r.kv_heads = p->kv_heads;
  r.rot = p->rot;
  r.pairs = p->pairs != 0;
  r.freqs = p->freqs;
  r.weight[0] = p->q_weight;
  r.weight[1] = p->k_weight;
  r.w_f32 = p->w_dtype == Q_F32;
  r.eps = normed ? p->eps : 1.0f;
  r.offset = p->offset;
  r.lens = lens;
  r.starts = starts;
  r.B = (int)B;
  r.T = (int)T;
  r.in_f32 = in_dtype == Q_F32;
  r.out_f32 = out_dtype == Q_F32;
  return hip_status(qg::launch_norm_rope(r, stream));
}

int qprompt_attend(int head_dim, int q_heads, int kv_heads, int64_t B, int64_t T, const int32_t* starts, const void* Q,
                   int64_t q_stride, const void* K, int64_t k_stride, const void* V, int64_t v_stride, float scale,
                   void* out, int64_t o_stride, int out_dtype, hipStream_t stream) {
  int st = heads_ok(head_dim, q_heads, kv_heads);
  if (st != Q_OK) return st;
  if (B > kMaxSeqs) return Q_EINVAL;
  if ((st = batch_ok(B, T)) != Q_OK) return st;
  if (T * (q_heads / kv_heads) > ((int64_t)1 << 30)) return Q_EUNSUPPORTED;
  if ((!starts && B != 1) || !isfinite(scale) || !float_dtype(out_dtype)) return Q_EINVAL;
  if (fabsf(scale) > 0x1p45f) return Q_EUNSUPPORTED;
  if (!aligned(starts, 4)) return Q_EALIGN;
  const int64_t qw = (int64_t)q_heads * head_dim, kw = (int64_t)kv_heads * head_dim;
  if ((st = rows_ok(Q, q_stride, qw, 2)) != Q_OK) return st;
  if ((st = rows_ok(K, k_stride, kw, 2)) != Q_OK) return st;
  if ((st = rows_ok(V, v_stride, kw, 2)) != Q_OK) return st;
  if ((st = rows_ok(out, o_stride, qw, size_of(out_dtype))) != Q_OK) return st;
  qg::Prompt p;
  p.head_dim = head_dim;
  p.heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.B = (int)B;
  p.T = (int)T;
  p.starts = starts;
  p.Q = static_cast<const uint16_t*>(Q);
  p.K = static_cast<const uint16_t*>(K);
  p.V = static_cast<const uint16_t*>(V);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.o_stride = o_stride;
  p.scale = scale;
  p.out = out;
  p.out_f32 = out_dtype == Q_F32;
  return hip_status(qg::launch_prompt(p, stream));
}

}  // extern "C"
