// What the attention kernels over the paged cache share: the launch's
// arguments, an item's rows and keys, and the layout of partial results.
#pragma once

#include "kvcache_plan.hpp"

namespace qg {

struct AttendArgs {
  KvAttend a;
  SplitRule rule;
  Partials part;
  bool shared;                // a prefix part exists: results always go through the partials
  // prefix launch: all T rows against the prefix's keys in host-known chunks
  bool prefix;
  int prefix_cu, prefix_chunks;
};

// Wave-uniform description of what one workgroup does.
struct Work {
  int b;                      // < 0: nothing
  int slot;                   // partial slot of this item
  int row0, rows;             // first row (token * group + g) of the tile and rows of the sequence in all
  int t0, vis0;
  int k0, k1;                 // keys of the chunk that some row of the tile may see
  int need;                   // keys the sequence's last row sees
  bool causal, direct;
  const int32_t* pages;
  int max_pages;
};

__device__ __forceinline__ Work work_of(const AttendArgs& x, int item, int lane) {
  const KvAttend& a = x.a;
  Work w{};
  w.b = -1;
  int tile, chunk, cu;
  if (x.prefix) {
    tile = item / x.prefix_chunks;
    chunk = item % x.prefix_chunks;
    cu = x.prefix_cu;
    w.b = 0;
    w.t0 = 0;
    w.rows = a.s.T * a.group;
    w.vis0 = w.need = a.prefix_len;
    w.causal = false;
    w.direct = false;
    w.pages = a.prefix_pages;
    w.max_pages = (a.prefix_len + (1 << a.c.page_shift) - 1) >> a.c.page_shift;
  } else {
    cu = split_units(a.s, x.rule, lane);
    const Item it = find_item(a.s, x.rule, cu, item, lane);
    if (it.b < 0) return w;
    tile = it.tile;
    chunk = it.chunk;
    w.b = it.b;
    w.t0 = it.r.t0;
    w.rows = it.r.count * a.group;
    w.vis0 = it.r.vis0;
    w.need = it.r.need;
    w.causal = true;
    w.direct = it.chunks == 1 && !x.shared;
    w.pages = a.s.pages + (int64_t)it.b * a.s.max_pages;
    w.max_pages = a.s.max_pages;
  }
  w.slot = item;
  if (!w.direct && item >= x.part.slots) {
    w.b = -1;
    return w;
  }
  w.row0 = tile * x.rule.rt;
  // the last row of the tile sees the most
  int last = w.row0 + x.rule.rt - 1;
  if (last >= w.rows) last = w.rows - 1;
  int vis = w.need;
  if (w.causal) {
    const int v = w.vis0 + last / a.group;
    vis = v < 0 ? 0 : (v < w.need ? v : w.need);
  }
  const int64_t len = (int64_t)cu * x.rule.ku, k0 = chunk * len, k1 = k0 + len;
  w.k0 = k0 < vis ? (int)k0 : vis;
  w.k1 = k1 < vis ? (int)k1 : vis;
  return w;
}

// Keys that row R (an index of the sequence's rows) sees.
__device__ __forceinline__ int row_sees(const Work& w, int token) {
  if (!w.causal) return w.need;
  const int v = w.vis0 + token;
  return v < 0 ? 0 : (v < w.need ? v : w.need);
}

template <int D>
__device__ __forceinline__ float* part_o(const AttendArgs& x, int slot, int h, int row) {
  return x.part.o + (((int64_t)slot * x.a.c.heads + h) * x.rule.rt + row) * D;
}
__device__ __forceinline__ float* part_ml(const AttendArgs& x, int slot, int h, int row) {
  return x.part.ml + (((int64_t)slot * x.a.c.heads + h) * x.rule.rt + row) * 2;
}

// Four neighbouring outputs of a row.
__device__ __forceinline__ void store_out4(const KvAttend& a, int64_t at, const f32x4_t& v) {
  if (a.out_f32) {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + at) = v;
  } else {
    uint2 p;
    p.x = cvt_pk_bf16(v[0], v[1]);
    p.y = cvt_pk_bf16(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = p;
  }
}

hipError_t launch_kv_rows(const AttendArgs& x, int head_dim, int bits, int64_t items, hipStream_t st);
hipError_t launch_kv_tiles(const AttendArgs& x, int head_dim, int bits, int64_t items, hipStream_t st);

}  // namespace qg
