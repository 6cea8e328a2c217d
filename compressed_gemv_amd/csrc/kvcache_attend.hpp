// What the attention kernels over the paged cache share: the launch's
// arguments, an item's rows and keys, and the layout of partial results.
#pragma once

#include "kvcache_plan.hpp"

namespace qg {

struct AttendArgs {
  KvAttend a;
  SeqView s;                   // a.s, or the prefix as one sequence that owns all rows
  SplitRule rule;
  Partials part;
  bool keep;                   // every result goes through the partials (a shared prefix joins in)
  Line line;                   // of a shared prefix, known on the host
  // decoded keys and values, one image for each step of keys and KV head, or null
  uint8_t* image;
  int64_t images;              // steps of keys there is room for
};

// Wave-uniform description of one tile's part in one piece.
struct Work {
  int slot;                    // partial slot, of a tile that is not direct
  int row0, rows;              // first row (token * group + g) of the tile and rows of the sequence in all
  int t0, vis0;
  int k0, k1;                  // keys of this part that some row of the tile may see
  int need;                    // keys the sequence's last row sees
  bool causal, direct;
  const int32_t* pages;
  int max_pages;
  int64_t steps;               // images: of the sequences before this one
};

// Steps through the tiles of a workgroup's piece.
struct Pieces {
  Line line;
  int piece;
  int64_t x, end;              // weights still to do
  TileAt t;                    // the last tile; b < 0: none yet
  Cursor from;
};

template <bool SPREAD = false>
__device__ __forceinline__ Pieces pieces_of(const AttendArgs& x, int piece, int lane) {
  Pieces p;
  p.from = Cursor{};
  if (!SPREAD && x.rule.single) {                     // found without a look at the other sequences' weights
    p.line = Line{};
    p.piece = piece;
    p.x = (int64_t)piece * kSub;
    p.end = p.x + kSub;
    p.t.b = -1;
    return p;
  }
  p.line = x.s.lens ? line_of(x.s, x.rule, lane) : x.line;
  p.piece = piece;
  p.x = p.end = 0;
  p.t.b = -1;
  if constexpr (SPREAD) {
    p.end = piece < p.line.N ? 1 : 0;      // one tile
  } else if (piece < p.line.N) {
    p.x = p.line.cut(piece);
    p.end = p.line.cut(piece + 1);
  }
  return p;
}

// ADVANCE: from tile to tile of a sequence without a search, for which a piece
// of many tiles keeps more state (a prompt's tiles 267 -> 251 us; the kernel for
// few rows, whose tiles are mostly sequences, is 1 % slower with it).
// SPREAD: for rules that say so.
template <bool ADVANCE, bool STEPS = false, bool SPREAD = false>
__device__ __forceinline__ bool next_work(const AttendArgs& x, Pieces& p, Work& w, int lane) {
  // the tile's rows and the steps of keys that its last row, which sees the most, needs
  auto tile = [&](const TileAt& t) {
    w.t0 = t.r.t0;
    w.rows = t.r.count * x.a.group;
    w.vis0 = t.r.vis0;
    w.need = t.r.need;
    w.causal = x.s.lens != nullptr;
    w.pages = x.s.pages + (int64_t)t.b * x.s.max_pages;
    w.max_pages = x.s.max_pages;
    w.row0 = t.tile * x.rule.rt;
    int last = w.row0 + x.rule.rt - 1;
    if (last >= w.rows) last = w.rows - 1;
    int vis = w.need;
    if (w.causal) {
      const int v = w.vis0 + last / x.a.group;
      vis = v < 0 ? 0 : (v < w.need ? v : w.need);
    }
    return vis;
  };
  auto keys = [&](int u0, int u1, int vis) {
    w.k0 = u0 * x.rule.ku;
    w.k1 = u1 * x.rule.ku < vis ? u1 * x.rule.ku : vis;
    if (w.k0 > w.k1) w.k0 = w.k1;
  };
  if constexpr (SPREAD) {
    if (p.x >= p.end) return false;
    p.x = p.end;
    const PartAt a = part_at(x.s, x.rule, p.line, p.piece, lane);
    if (a.t.b < 0) return false;
    const int vis = tile(a.t), units = (vis + x.rule.ku - 1) / x.rule.ku, c = p.piece - a.first;
    keys((int)((int64_t)units * c / a.parts), (int)((int64_t)units * (c + 1) / a.parts), vis);
    w.steps = 0;
    w.direct = a.parts == 1;
    w.slot = 2 * p.piece;
    return w.direct || w.slot < x.part.slots;
  }
  while (p.x < p.end) {
    if (!ADVANCE || p.t.b < 0 || !p.t.advance()) p.t = tile_at<false, STEPS>(x.s, x.rule, p.x, lane, p.from);
    const TileAt& t = p.t;
    if (t.b < 0 || t.hi <= p.x) return false;              // (weights that overflow under starts that make no sense)
    w.steps = t.steps;
    const int64_t from = p.x;
    const bool whole = t.lo >= from && t.hi <= p.end;
    w.direct = whole && !x.keep;
    const int vis = tile(t);
    // the cuts, from weights to whole steps of the tile's keys
    const int units = (vis + x.rule.ku - 1) / x.rule.ku;
    const double per = (double)units / (double)(t.hi - t.lo);
    const int u0 = from <= t.lo ? 0 : __builtin_amdgcn_readfirstlane((int)((double)(from - t.lo) * per));
    const int u1 = p.end >= t.hi ? units : __builtin_amdgcn_readfirstlane((int)((double)(p.end - t.lo) * per));
    keys(u0, u1, vis);
    p.x = t.hi;
    if (w.direct) return true;
    const int64_t slot = slot_of(p.line, t, p.piece, x.keep);
    w.slot = (int)slot;
    if (slot < x.part.slots) return true;
  }
  return false;
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
template <bool F32>
__device__ __forceinline__ void store_out4(const KvAttend& a, int64_t at, const f32x4_t& v) {
  if constexpr (F32) {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + at) = v;
  } else {
    uint2 p;
    p.x = cvt_pk_bf16(v[0], v[1]);
    p.y = cvt_pk_bf16(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = p;
  }
}
__device__ __forceinline__ void store_out4(const KvAttend& a, int64_t at, const f32x4_t& v) {
  if (a.out_f32) store_out4<true>(a, at, v);
  else store_out4<false>(a, at, v);
}

// y: a second set of tiles of the same height in the same launch, or null
hipError_t launch_kv_rows(const AttendArgs& x, const AttendArgs* y, int head_dim, int bits, hipStream_t st);
hipError_t launch_kv_tiles(const AttendArgs& x, int head_dim, int bits, hipStream_t st);
hipError_t launch_kv_images(const AttendArgs& x, int head_dim, int bits, hipStream_t st);
// Bytes of one image (128 keys of one KV head): the LDS rows of the keys, those
// of the values' coordinates, and 1 KB whose first word has a bit for every 16
// keys whose page is not in the cache.
constexpr int64_t kv_image_bytes(int head_dim) { return 128 * (2 * head_dim + 16) + head_dim * (2 * 128 + 16) + 1024; }

}  // namespace qg
