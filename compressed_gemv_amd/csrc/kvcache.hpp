// Shared by the kernels of the quantized, paged KV cache: the views a launch
// passes by value, and the search for a row's sequence.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace qg {

struct KvView {
  uint8_t* codes[2];          // K, V
  uint32_t* meta[2];
  int n_pages, page_shift, heads;
};
struct SeqView {
  const int32_t* pages;
  const int32_t* lens;
  const int32_t* starts;      // or null: one row per sequence
  int B, T, max_pages;
};

hipError_t launch_kv_write(const KvView& c, const SeqView& s, int head_dim, int bits, const void* K, int64_t k_stride,
                           const void* V, int64_t v_stride, bool f32, hipStream_t st);
hipError_t launch_kv_read(const KvView& c, const SeqView& s, int head_dim, int bits, void* K, int64_t k_stride, void* V,
                          int64_t v_stride, bool f32, hipStream_t st);
struct KvAttend {
  KvView c;
  SeqView s;
  const uint16_t* Q;
  int64_t q_stride, o_stride;
  int group;                  // query heads per KV head
  float scale;
  void* out;
  bool out_f32;
  const int32_t* prefix_pages;
  int prefix_len;
};
hipError_t launch_kv_attend(const KvAttend& a, int head_dim, int bits, void* ws, hipStream_t st);
size_t kv_attend_ws_bytes(int64_t B, int64_t T, int64_t max_pages, int page_shift, int heads, int group, int head_dim,
                          int64_t prefix_len);

// Largest b in [0, B) with starts[b] <= t, searched by the LPR lanes of a row
// group together: every step probes LPR evenly spaced entries at once, so B
// <= LPR^2 takes two loads.  starts need not be sorted for safety: the result
// is in range whatever it holds, and the caller checks that b owns t.
template <int LPR>
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ starts, int B, int t, int sub, int lane) {
  int lo = 0, n = B;                                     // answer in [lo, lo + n)
  while (n > 1) {
    const int step = (n + LPR - 1) / LPR;
    const int i = lo + sub * step;
    const bool le = sub * step < n && starts[i] <= t;
    const uint64_t m = __ballot(le) >> (lane & ~(LPR - 1));
    const int cnt = __popcll(LPR == 64 ? m : m & ((1ull << (LPR & 63)) - 1ull));
    const int k = cnt > 0 ? cnt - 1 : 0;
    lo += k * step;
    n = n - k * step < step ? n - k * step : step;
    if (n < 1) n = 1;
  }
  return lo;
}

// The slot (page * page_size + offset) of row t, or -1 with *owned telling
// whether some sequence owns the row.
template <int LPR>
__device__ __forceinline__ int64_t slot_of_row(const KvView& c, const SeqView& s, int t, int sub, int lane, bool* owned) {
  *owned = false;
  int b = t;
  int64_t pos;
  if (s.starts) {
    b = find_seq<LPR>(s.starts, s.B, t, sub, lane);
    const int s0 = s.starts[b], s1 = s.starts[b + 1];
    if (t < s0 || t >= s1) return -1;
    pos = (int64_t)s.lens[b] - (s1 - t);
  } else {
    pos = (int64_t)s.lens[b] - 1;
  }
  *owned = true;
  const int64_t ps = pos >> c.page_shift;
  if (pos < 0 || ps >= s.max_pages) return -1;
  const int page = s.pages[(int64_t)b * s.max_pages + ps];
  if (page < 0 || page >= c.n_pages) return -1;
  return ((int64_t)page << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// Row index (page, head, slot) of a cache slot for one head.
__device__ __forceinline__ int64_t cache_row(const KvView& c, int64_t slot, int h) {
  const int64_t page = slot >> c.page_shift, off = slot & ((1 << c.page_shift) - 1);
  return ((page * c.heads + h) << c.page_shift) + off;
}

}  // namespace qg
