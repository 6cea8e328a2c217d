// How an attention launch over the paged cache divides its work, computed by
// every wave from the device's lens and starts (so a captured launch follows
// the sequences as they grow).
//
// A KV head's rows of one sequence are its tokens times `group` query heads,
// row = token * group + g; they are cut into tiles of RT rows, and the keys a
// tile sees into chunks of `cu` units of KU keys.  An item is one (sequence,
// row tile, chunk).  cu is the least that leaves about `target` items per KV
// head, one number for the whole batch, so items cost about the same however
// unequal the sequences are; with `target` row tiles or more nothing is split.
#pragma once

#include "common.hpp"
#include "kvcache.hpp"

namespace qg {

constexpr int kNoSplit = 1 << 30;

struct SeqRows {
  int t0, count;              // rows of Q that the sequence owns
  int vis0;                   // keys that row t0 sees (may be <= 0); each later row sees one more
  int need;                   // keys that its last row sees, 0 .. cap
};

__device__ __forceinline__ SeqRows seq_rows(const SeqView& s, int b, int cap) {
  SeqRows r{0, 0, 0, 0};
  if (b >= s.B) return r;
  int64_t s0 = b, s1 = b + 1;
  if (s.starts) { s0 = s.starts[b]; s1 = s.starts[b + 1]; }
  const int64_t end = s1 < s.T ? s1 : s.T, t0 = s0 < 0 ? 0 : s0;
  if (end <= t0) return r;
  r.t0 = (int)t0;
  r.count = (int)(end - t0);
  const int64_t len = s.lens[b];
  int64_t v0 = len - (s1 - t0) + 1, v1 = len - (s1 - end);
  v0 = v0 < -(int64_t)kNoSplit ? -(int64_t)kNoSplit : (v0 > cap ? cap : v0);
  v1 = v1 < 0 ? 0 : (v1 > cap ? cap : v1);
  r.vis0 = (int)v0;
  r.need = (int)v1;
  return r;
}

struct SplitRule { int group, rt, ku, target, min_units, cap; };

__device__ __forceinline__ int tiles_of(const SplitRule& p, const SeqRows& r) {
  return (int)(((int64_t)r.count * p.group + p.rt - 1) / p.rt);
}
__device__ __forceinline__ int chunks_of(const SplitRule& p, const SeqRows& r, int cu) {
  const int units = (r.need + p.ku - 1) / p.ku;
  return units <= cu ? 1 : (units + cu - 1) / cu;
}

// The batch's chunk length in units.  Wave-uniform; all lanes take part.
__device__ __forceinline__ int split_units(const SeqView& s, const SplitRule& p, int lane) {
  float w = 0.f;
  int64_t tiles = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const SeqRows r = seq_rows(s, b0 + lane, p.cap);
    const int rt = tiles_of(p, r);
    w += (float)rt * (float)((r.need + p.ku - 1) / p.ku);
    tiles += rt;
  }
  w = wave_sum(w);
  const float tf = wave_sum((float)tiles);
  if (tf >= (float)p.target) return kNoSplit;
  const float c = w / (float)p.target;
  const int cu = c < 1e9f ? (int)c + 1 : kNoSplit;
  return cu < p.min_units ? p.min_units : cu;
}

// Inclusive sum over the lanes of a wave: DPP shifts inside the rows of 16,
// then lane 15 of a row added to the next one, lane 31 to the upper half.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31
  return v;
}

// One item of the launch, wave-uniform; b < 0: there is none.
struct Item {
  int b, tile, chunk, chunks;
  SeqRows r;
};

__device__ __forceinline__ Item find_item(const SeqView& s, const SplitRule& p, int cu, int item, int lane) {
  Item it{-1, 0, 0, 1, {0, 0, 0, 0}};
  int carry = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const SeqRows r = seq_rows(s, b0 + lane, p.cap);
    const int ch = chunks_of(p, r, cu), n = tiles_of(p, r) * ch;
    const int inc = wave_scan(n);
    const uint64_t m = __ballot(carry + inc > item);
    if (m) {
      const int l = __ffsll((unsigned long long)m) - 1;
      const int k = item - carry - (__builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(n, l));
      it.chunks = __builtin_amdgcn_readlane(ch, l);
      it.b = b0 + l;
      it.tile = k / it.chunks;
      it.chunk = k % it.chunks;
      it.r.t0 = __builtin_amdgcn_readlane(r.t0, l);
      it.r.count = __builtin_amdgcn_readlane(r.count, l);
      it.r.vis0 = __builtin_amdgcn_readlane(r.vis0, l);
      it.r.need = __builtin_amdgcn_readlane(r.need, l);
      return it;
    }
    carry += __builtin_amdgcn_readlane(inc, 63);
  }
  return it;
}

// Items of the sequences before b.
__device__ __forceinline__ int items_before(const SeqView& s, const SplitRule& p, int cu, int b, int lane) {
  int sum = 0;
  for (int b0 = 0; b0 < b; b0 += 64) {
    const SeqRows r = seq_rows(s, b0 + lane, p.cap);
    if (b0 + lane < b) sum += tiles_of(p, r) * chunks_of(p, r, cu);
  }
  return __builtin_amdgcn_readlane(wave_scan(sum), 63);
}

// Partial results of one part of the keys: item slots of RT rows, per row the
// unnormalised sum of D values, its maximum (log2 domain) and its sum of weights.
struct Partials {
  float* o;                   // [slot][rt][D]
  float* ml;                  // [slot][rt][2]
  int slots;                  // per KV head; starts that overlap could ask for more, which are left out
};

}  // namespace qg
