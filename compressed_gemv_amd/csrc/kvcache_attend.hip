// Attention over the quantized, paged KV cache.
//
// One workgroup per (row, query head): the four waves take every fourth key,
// each lane holding D / 64 coordinates; online softmax per wave in fp32, the
// four joined in LDS.
#include "common.hpp"
#include "kvcache.hpp"

namespace qg {

template <int D, int BITS>
__global__ __launch_bounds__(256) void kv_attend_kernel(KvAttend a) {
  constexpr int E = D / 64;
  __shared__ float os[4][D], ms[4], ls[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / a.group;
  int b = t, seen;
  if (a.s.starts) {
    b = find_seq<64>(a.s.starts, a.s.B, t, lane, lane);
    const int s0 = a.s.starts[b], s1 = a.s.starts[b + 1];
    if (t < s0 || t >= s1) return;
    const int64_t n = (int64_t)a.s.lens[b] - (s1 - t) + 1;
    seen = n < 0 ? 0 : (int)n;
  } else {
    seen = a.s.lens[b] < 0 ? 0 : a.s.lens[b];
  }
  const int64_t cap = (int64_t)a.s.max_pages << a.c.page_shift;
  if (seen > cap) seen = (int)cap;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_bits_to_f32(a.Q[t * a.q_stride + (int64_t)hq * D + lane * E + e]) * a.scale;
    o[e] = 0.f;
  }
  auto code = [&](const uint8_t* base, int64_t row, int d) -> float {
    if (BITS == 8) return (float)base[row * D + d];
    const uint32_t w = base[row * (D / 2) + d / 2];
    return (float)((d & 1) ? w >> 4 : w & 15u);
  };
  auto key = [&](int64_t row) {
    const float ks = f16_lo(a.c.meta[0][row]), ko = f16_hi(a.c.meta[0][row]);
    float dot = 0.f;
    for (int e = 0; e < E; ++e) dot += q[e] * (ks * code(a.c.codes[0], row, lane * E + e) + ko);
    dot = wave_sum(dot);
    const float vs = f16_lo(a.c.meta[1][row]), vo = f16_hi(a.c.meta[1][row]);
    const float mn = dot > m ? dot : m;
    const float f = m == mn ? 1.f : __expf(m - mn), p = __expf(dot - mn);
    m = mn;
    l = l * f + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * (vs * code(a.c.codes[1], row, lane * E + e) + vo);
  };
  auto over = [&](const int32_t* pages, int n) {
    for (int j = wave; j < n; j += 4) {
      const int page = pages[j >> a.c.page_shift];
      if (page < 0 || page >= a.c.n_pages) continue;
      key((((int64_t)page * a.c.heads + h) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1)));
    }
  };
  if (a.prefix_len) over(a.prefix_pages, a.prefix_len);
  over(a.s.pages + (int64_t)b * a.s.max_pages, seen);
  for (int e = 0; e < E; ++e) os[wave][lane * E + e] = o[e];
  if (lane == 0) { ms[wave] = m; ls[wave] = l; }
  __syncthreads();
  float mm = -INFINITY;
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ms[w]);
  float ll = 0.f, acc = 0.f;
  const int d = threadIdx.x;
  if (d >= D) return;
  for (int w = 0; w < 4; ++w)
    if (ls[w] != 0.f) {
      const float f = __expf(ms[w] - mm);
      ll += ls[w] * f;
      acc += os[w][d] * f;
    }
  acc = ll != 0.f ? acc / ll : 0.f;
  const int64_t at = t * a.o_stride + (int64_t)hq * D + d;
  if (a.out_f32) static_cast<float*>(a.out)[at] = acc;
  else static_cast<uint16_t*>(a.out)[at] = (uint16_t)(cvt_pk_bf16(acc, 0.f) & 0xFFFFu);
}

size_t kv_attend_ws_bytes(int64_t, int64_t, int, int, int, int64_t) { return 16; }

hipError_t launch_kv_attend(const KvAttend& a, int head_dim, int bits, void*, hipStream_t st) {
  const dim3 grid((unsigned)a.s.T, (unsigned)(a.c.heads * a.group));
  if (head_dim == 128) {
    if (bits == 8) hipLaunchKernelGGL((kv_attend_kernel<128, 8>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((kv_attend_kernel<128, 4>), grid, dim3(256), 0, st, a);
  } else {
    if (bits == 8) hipLaunchKernelGGL((kv_attend_kernel<64, 8>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((kv_attend_kernel<64, 4>), grid, dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace qg
