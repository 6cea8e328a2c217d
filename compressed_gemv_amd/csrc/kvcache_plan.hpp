// How an attention launch over the paged cache divides its work, computed by
// every wave from the device's lens and starts (so a captured launch follows
// the sequences as they grow).
//
// A KV head's rows of one sequence are its tokens times `group` query heads,
// row = token * group + g; they are cut into tiles of RT rows.  Tile t of a
// sequence weighs A + S t, about the keys it sees in steps of KU / 64 (later
// tokens see more, so S > 0 where a tile holds a good part of a step) and what
// starting and ending a tile costs.  All
// tiles of the batch form one line of U weights per KV head, which is cut into
// N equal pieces, one per workgroup, wherever the cuts fall: no workgroup has
// more to do than another, however unequal the sequences are.  A tile that a
// cut goes through leaves partial results, which the join adds up.  Where there
// are few tiles the line is spread instead: every tile gets pieces of its own,
// about its share of them.  All of it in integers and in fp64 products that are
// the same everywhere, so every wave of every kernel finds the same cuts.
#pragma once

#include "common.hpp"
#include "kvcache.hpp"

namespace qg {

constexpr int kSub = 64;       // weight of KU keys

struct SplitRule {
  int group, rt, ku;           // query heads per KV head, rows per tile, keys per step
  int wgs;                     // workgroups per KV head in the grid
  int cap;                     // positions the page table holds
  bool whole;                  // tiles are never cut: each weighs one step
  bool single;                 // and there is a workgroup for every tile there can be: piece i is tile i
  bool sloped;                 // weigh a sequence's tiles by what each sees
  bool spread;                 // no piece holds parts of two tiles
  int extra;                   // weight of what a tile costs beside its keys
};

struct SeqRows {
  int t0, count;               // rows of Q that the sequence owns
  int vis0;                    // keys that row t0 sees (may be <= 0); each later row sees one more
  int need;                    // keys that its last row sees, 0 .. cap
};

__device__ __forceinline__ SeqRows seq_rows(const SeqView& s, int b, int cap) {
  SeqRows r{0, 0, 0, 0};
  if (b >= s.B) return r;
  if (!s.lens) return SeqRows{0, s.T, cap, cap};        // a shared prefix: every row sees all of it
  const int64_t len = s.lens[b];                        // on its way beside the starts
  int64_t s0 = b, s1 = b + 1;
  if (s.starts) { s0 = s.starts[b]; s1 = s.starts[b + 1]; }
  const int64_t end = s1 < s.T ? s1 : s.T, t0 = s0 < 0 ? 0 : s0;
  if (end <= t0) return r;
  r.t0 = (int)t0;
  r.count = (int)(end - t0);
  const int64_t low = -((int64_t)1 << 30);
  const int64_t v0 = len - (s1 - t0) + 1, v1 = len - (s1 - end);
  r.vis0 = (int)(v0 < low ? low : (v0 > cap ? cap : v0));
  r.need = (int)(v1 < 0 ? 0 : (v1 > cap ? cap : v1));
  return r;
}

__device__ __forceinline__ int steps_of(const SplitRule& p, const SeqRows& r) { return (r.need + p.ku - 1) / p.ku; }

// Weights of a sequence: W(t) = A t + S t (t - 1) / 2 before tile t.
struct Weights {
  int tiles;
  int A, S;
  __device__ __forceinline__ int64_t before(int64_t t) const { return A * t + S * (t * (t - 1) / 2); }
};

__device__ __forceinline__ Weights weights_of(const SplitRule& p, const SeqRows& r) {
  Weights w;
  w.tiles = (int)(((int64_t)r.count * p.group + p.rt - 1) / p.rt);
  const int step = p.ku / kSub;
  const int full = (r.need + p.ku - 1) / p.ku * kSub;     // of a tile that sees all
  w.A = full < kSub || p.whole ? kSub : full;
  w.S = 0;
  if (p.sloped && w.tiles > 1) {
    const int s = p.rt / p.group / step;
    const int64_t first = w.A - (int64_t)s * (w.tiles - 1);
    if (first >= kSub) { w.S = s; w.A = (int)first; }
    else { w.S = (w.A - kSub) / (w.tiles - 1); w.A -= w.S * (w.tiles - 1); }
  }
  w.A += p.extra;
  return w;
}

// Inclusive sums over the lanes of a wave: DPP shifts inside the rows of 16,
// then lane 15 of a row added to the next one, lane 31 to the upper half.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t dpp_i64(int64_t v) {
  const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xF, false);
  return ((int64_t)hi << 32) | (uint32_t)lo;
}
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
  v += dpp_i64<0x111, 0xF>(v);     // row_shr:1
  v += dpp_i64<0x112, 0xF>(v);
  v += dpp_i64<0x114, 0xF>(v);
  v += dpp_i64<0x118, 0xF>(v);
  v += dpp_i64<0x142, 0xA>(v);     // row_bcast:15
  v += dpp_i64<0x143, 0xC>(v);     // row_bcast:31
  return v;
}
__device__ __forceinline__ int64_t lane_i64(int64_t v, int l) {
  return ((int64_t)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32) | (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}

// fp64 results live in vector registers; equal in all lanes, they go back to scalar ones.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return ((int64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// The cut line.  Quotients go through fp64: with all products below 2^52 the
// rounded quotient never reaches the next integer.
struct Line {
  int64_t U;                   // in grains: kSub where tiles are not cut, else 1
  int N, grain;
  double rate;                 // spread: pieces for a weight beside one for each tile
  // spread: the first piece of what begins at weight x as tile number `tile`.
  // Pieces of a tile: 1 + about its share of the N - T left over, so each has
  // at most U / (N - T) to do.
  __device__ __forceinline__ int first(int64_t x, int64_t tile) const { return (int)(tile + (int64_t)((double)x * rate)); }
  __device__ __forceinline__ int64_t cut(int i) const {
    return uniform((int64_t)((double)i * (double)U / (double)N)) * grain;
  }
  // the piece that weight x lies in
  __device__ __forceinline__ int piece(int64_t x) const {
    const int64_t y = grain == 1 ? x : x / kSub;
    return __builtin_amdgcn_readfirstlane((int)(((double)(y + 1) * (double)N - 1.0) / (double)U));
  }
};

__device__ __forceinline__ Line line_of(const SeqView& s, const SplitRule& p, int lane) {
  int64_t u = 0, tiles = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const Weights w = weights_of(p, seq_rows(s, b0 + lane, p.cap));
    u += w.before(w.tiles);
    tiles += w.tiles;
  }
  Line l;
  u = lane_i64(wave_scan(u), 63);
  l.grain = p.whole ? kSub : 1;
  l.U = p.whole ? u / kSub : u;
  const int64_t n = u / kSub;                              // a piece is a step of keys at least
  l.N = n < p.wgs ? (int)n : p.wgs;
  if (l.N < 1) l.N = 1;
  l.rate = 0.;
  if (p.spread) {
    tiles = lane_i64(wave_scan(tiles), 63);
    if (tiles < l.N) l.rate = (double)(l.N - tiles) / (double)u;
  }
  return l;
}

// Where a search begins: the 64 sequences that the one before ended in, and
// what lies before them.
struct Cursor {
  int b0;
  int64_t carry, tiles, steps; // weights, tiles, steps of keys
};

// The tile that weight x of the line lies in, or (BY_INDEX) tile number x of
// it; b < 0: none.
struct TileAt {
  int b, tile;
  int64_t index;               // of the tile in the whole line
  int64_t lo, hi;              // its weights
  int64_t steps;               // steps of keys of the sequences before b
  SeqRows r;
  Weights v;                   // of the sequence
  int64_t base;                // weight before it
  __device__ __forceinline__ bool advance() {              // to the sequence's next tile
    if (tile + 1 >= v.tiles) return false;
    ++tile;
    ++index;
    lo = hi;
    hi = base + v.before(tile + 1);
    return true;
  }
};

template <bool BY_INDEX = false, bool STEPS = false>
__device__ __forceinline__ TileAt tile_at(const SeqView& s, const SplitRule& p, int64_t x, int lane, Cursor& at) {
  TileAt a{};
  a.b = -1;
  int64_t carry = at.carry, tiles = at.tiles, steps = at.steps;
  for (int b0 = at.b0; b0 < s.B; b0 += 64) {
    const SeqRows r = seq_rows(s, b0 + lane, p.cap);
    const Weights w = weights_of(p, r);
    const int k = steps_of(p, r);
    const int64_t kinc = STEPS ? wave_scan((int64_t)k) : 0;
    const int64_t u = w.before(w.tiles), inc = wave_scan(u), tinc = wave_scan((int64_t)w.tiles);
    const uint64_t m = __ballot(BY_INDEX ? tiles + tinc > x : carry + inc > x);
    if (m) {
      const int l = __ffsll((unsigned long long)m) - 1;
      Weights& v = a.v;
      v.tiles = __builtin_amdgcn_readlane(w.tiles, l);
      v.A = __builtin_amdgcn_readlane(w.A, l);
      v.S = __builtin_amdgcn_readlane(w.S, l);
      const int64_t base = carry + lane_i64(inc, l) - lane_i64(u, l), first = tiles + lane_i64(tinc, l) - v.tiles;
      a.base = base;
      int lo = 0;
      if (BY_INDEX) {
        lo = (int)(x - first);
      } else {
        int n = v.tiles;                                   // last tile that begins at or before x
        while (n > 1) {
          const int half = n >> 1;
          if (base + v.before(lo + half) <= x) { lo += half; n -= half; }
          else n = half;
        }
      }
      at = Cursor{b0, carry, tiles, steps};
      a.b = b0 + l;
      a.tile = lo;
      a.steps = STEPS ? steps + lane_i64(kinc, l) - __builtin_amdgcn_readlane(k, l) : 0;
      a.index = first + lo;
      a.lo = base + v.before(lo);
      a.hi = base + v.before(lo + 1);
      a.r.t0 = __builtin_amdgcn_readlane(r.t0, l);
      a.r.count = __builtin_amdgcn_readlane(r.count, l);
      a.r.vis0 = __builtin_amdgcn_readlane(r.vis0, l);
      a.r.need = __builtin_amdgcn_readlane(r.need, l);
      return a;
    }
    carry += lane_i64(inc, 63);
    tiles += lane_i64(tinc, 63);
    if (STEPS) steps += lane_i64(kinc, 63);
  }
  return a;
}

template <bool BY_INDEX = false>
__device__ __forceinline__ TileAt tile_at(const SeqView& s, const SplitRule& p, int64_t x, int lane) {
  Cursor from{};
  return tile_at<BY_INDEX>(s, p, x, lane, from);
}

// The tile that piece number `piece` of a spread line belongs to, its first
// piece and its number of pieces; t.b < 0: none.
struct PartAt {
  TileAt t;
  int first, parts;
};

__device__ __forceinline__ PartAt part_at(const SeqView& s, const SplitRule& p, const Line& line, int piece, int lane) {
  PartAt a{};
  a.t.b = -1;
  int64_t carry = 0, tiles = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const SeqRows r = seq_rows(s, b0 + lane, p.cap);
    const Weights w = weights_of(p, r);
    const int64_t u = w.before(w.tiles), inc = wave_scan(u), tinc = wave_scan((int64_t)w.tiles);
    const uint64_t m = __ballot(line.first(carry + inc, tiles + tinc) > piece);
    if (m) {
      const int l = __ffsll((unsigned long long)m) - 1;
      Weights& v = a.t.v;
      v.tiles = __builtin_amdgcn_readlane(w.tiles, l);
      v.A = __builtin_amdgcn_readlane(w.A, l);
      v.S = __builtin_amdgcn_readlane(w.S, l);
      a.t.base = carry + lane_i64(inc, l) - lane_i64(u, l);
      const int64_t first = tiles + lane_i64(tinc, l) - v.tiles;
      auto begin = [&](int tile) {
        return __builtin_amdgcn_readfirstlane(line.first(a.t.base + v.before(tile), first + tile));
      };
      int lo = 0, n = v.tiles;                             // last tile that begins at or before the piece
      while (n > 1) {
        const int half = n >> 1;
        if (begin(lo + half) <= piece) { lo += half; n -= half; }
        else n = half;
      }
      a.t.tile = lo;
      a.t.index = first + lo;
      a.first = begin(lo);
      a.parts = begin(lo + 1) - a.first;
      // (starts that overlap can make more tiles than there are numbers)
      if (a.first < 0 || a.first > piece || piece - a.first >= a.parts) return a;
      a.t.b = b0 + l;
      a.t.r.t0 = __builtin_amdgcn_readlane(r.t0, l);
      a.t.r.count = __builtin_amdgcn_readlane(r.count, l);
      a.t.r.vis0 = __builtin_amdgcn_readlane(r.vis0, l);
      a.t.r.need = __builtin_amdgcn_readlane(r.need, l);
      return a;
    }
    carry += lane_i64(inc, 63);
    tiles += lane_i64(tinc, 63);
  }
  return a;
}

// Step x of all the sequences' steps of keys; b < 0: none.
struct StepAt {
  int b, step, need;
};

__device__ __forceinline__ StepAt step_at(const SeqView& s, const SplitRule& p, int64_t x, int lane) {
  int64_t carry = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const SeqRows r = seq_rows(s, b0 + lane, p.cap);
    const int k = steps_of(p, r);
    const int64_t inc = wave_scan((int64_t)k);
    const uint64_t m = __ballot(carry + inc > x);
    if (m) {
      const int l = __ffsll((unsigned long long)m) - 1;
      return StepAt{b0 + l, (int)(x - carry - lane_i64(inc, l)) + __builtin_amdgcn_readlane(k, l),
                    __builtin_amdgcn_readlane(r.need, l)};
    }
    carry += lane_i64(inc, 63);
  }
  return StepAt{-1, 0, 0};
}

// Partial results: slots of RT rows, per row the unnormalised sum of D values,
// its maximum (log2 domain) and its sum of weights.  A piece has at most two
// tiles that a cut goes through, its first and its last; where everything is
// kept (a shared prefix joins in), piece + tile index numbers the parts; in a
// spread line piece i has slot 2 i.
struct Partials {
  float* o;                    // [slot][head][rt][D]
  float* ml;                   // [slot][head][rt][2]
  int slots;                   // starts that overlap could ask for more, which are left out
};

__device__ __forceinline__ int64_t slot_of(const Line& line, const TileAt& t, int piece, bool keep_all) {
  return keep_all ? piece + t.index : 2 * (int64_t)piece + (t.lo > line.cut(piece) ? 1 : 0);
}

}  // namespace qg
