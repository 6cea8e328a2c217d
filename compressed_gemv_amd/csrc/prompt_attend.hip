// Causal attention of whole, packed prompts over their own bf16 keys and values,
// with grouped heads.
//
// A KV head's rows of one sequence are its tokens times `group` query heads,
// row = token * group + g; a workgroup takes a tile of 256 of them (128 or 64
// where there are few tiles) and walks the keys that its last token sees, 128 at
// a time.  Tiles go to workgroups in the order of what they cost, the long ones
// first, so no workgroup is left with a long one at the end.
//
// Bound by what a SIMD's one wave issues.  Measured on several cards (8 KV heads
// of 128, 8 query heads each): 0.98 to 1.06 PFLOP/s for one prompt of 16000 (3.95
// to 4.28 ms; a large matrix product reaches 1.2 here), 0.70 to 0.78 for three of
// 999 .. 2500 (216 to 243 us).  In copies of the kernel with parts left out, 16000
// tokens took 11 % less without the fetches of the next keys, 4 % less without
// exponentials, 2 % without the maximum and nothing less without the reads from
// LDS; other orders of the products and more vector instructions between them cost
// 1 to 2 %.
//
// Weights meet V as bf16: the products' operands are of one type, V's is bf16, and
// a second part of each weight would take half as many products again.  It leaves
// 2^-8 of a weight at most, what a bf16 output's own rounding does; the sum of the
// weights is of the unrounded ones, in fp32.
#include <type_traits>

#include "common.hpp"
#include "layer.hpp"

namespace qg {

namespace {

// Keys and values lie in LDS as they come from memory, 1 KB a wave and
// instruction: 4 keys of 128 values (8 of 64), of which four lanes fetch 64
// bytes in a row.  Those 64 bytes of four neighbouring keys follow each other, so
// that a transposing read of 4 keys and 32 coordinates takes 256 bytes in a row,
// and 16 (32) bytes between the KBs let a piece of 16 neighbouring keys lie in
// all banks once; every address of the inner loop is one register plus a
// constant.  (64: the second four keys of a KB swap neighbouring pieces.)
template <int D>
struct Image {
  static constexpr int KPB = 512 / D;                       // keys in a KB
  static constexpr int PITCH = D == 128 ? 1024 + 16 : 1024 + 32;
  static constexpr int bytes(int keys) { return keys / KPB * PITCH; }
  // of a key and its 16-byte piece c; 16 keys or 2 pieces (S, even c) more are a constant
  static __device__ __forceinline__ int at(int key, int c) {
    const int q = D == 128 ? 0 : (key >> 2) & 1;
    return key / KPB * PITCH + q * 512 + c / 4 * 256 + (key & 3) * 64 + ((c & 3) ^ q) * 16;
  }
  static constexpr int two(int s) { return s / 2 * 256 + s % 2 * 32; }
  // the key and piece that a lane of a KB holds
  static __device__ __forceinline__ int key_of(int lane) { return (D == 128 ? 0 : 4 * (lane >> 5)) + ((lane >> 2) & 3); }
  static __device__ __forceinline__ int piece_of(int lane) {
    return D == 128 ? 4 * (lane >> 4) + (lane & 3) : 4 * ((lane >> 4) & 1) + ((lane & 3) ^ (lane >> 5));
  }
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr float kLag = 8.0f;               // the running maximum may lag so far: weights up to 2^8
constexpr float kFar = 1024.0f;            // a maximum (times log2 e) beyond which exponents are formed in two steps
constexpr int kNoLoads = 0x0F70;           // s_waitcnt vmcnt(0), the other counters as they are

__device__ __forceinline__ int wave_sum_i32(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return __builtin_amdgcn_readlane(v, 63);
}

struct PromptTile {
  int s0, rows;                            // first token and rows of the sequence; rows = 0: no tile
  int row0;
};

__device__ __forceinline__ void bounds_of(const Prompt& p, int b, int& s0, int& s1) {
  s0 = 0;
  s1 = p.T;
  if (p.starts) {
    const int a = p.starts[b], e = p.starts[b + 1];
    s0 = a < 0 ? 0 : a;
    s1 = e > p.T ? p.T : e;
    if (s1 < s0) s1 = s0;
  }
}

// Tile number j of the call, the costly ones first: those of up to 256 sequences
// by the keys they see, of more sequences each one's own in that order.
// Wave-uniform.
template <int RT>
__device__ __forceinline__ PromptTile tile_of(const Prompt& p, int64_t j, int lane) {
  PromptTile t{0, 0, 0};
  int s0, s1, k;
  if (p.B <= 256) {
    int tiles[4], most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 64 * i + lane;
      tiles[i] = 0;
      if (64 * i < p.B && b < p.B) {
        bounds_of(p, b, s0, s1);
        tiles[i] = (int)(((int64_t)(s1 - s0) * p.group + RT - 1) / RT);
      }
      most = tiles[i] > most ? tiles[i] : most;
    }
    // tiles of index k and more
    auto above = [&](int k) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) n += tiles[i] > k ? tiles[i] - k : 0;
      return wave_sum_i32(n);
    };
    if (j >= above(0)) return t;
    int b = 0;
    if (p.B == 1) {
      k = __builtin_amdgcn_readlane(tiles[0], 0) - 1 - (int)j;
    } else {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_xor(most, d);
        most = o > most ? o : most;
      }
      k = 0;                               // the largest k with above(k) > j
      for (int n = __builtin_amdgcn_readfirstlane(most); n > 1;) {
        const int half = n >> 1;
        if (above(k + half) > j) { k += half; n -= half; }
        else n = half;
      }
      int r = (int)j - above(k + 1);       // the r-th sequence with more than k tiles
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t m = __ballot(tiles[i] > k);
        const int n = __popcll(m);
        if (r >= 0 && r < n) {
          const uint64_t hit = __ballot(((m >> lane) & 1u) && __popcll(m & ((1ull << lane) - 1ull)) == r);
          b = 64 * i + __ffsll((unsigned long long)hit) - 1;
        }
        r -= n;
      }
    }
    bounds_of(p, b, s0, s1);
  } else {
    int b = 0, n = p.B;                    // the last b with starts[b] * group / RT + b <= j
    while (n > 1) {
      const int half = n >> 1;
      int64_t s = p.starts[b + half];
      s = s < 0 ? 0 : s;
      if (s * p.group / RT + b + half <= j) { b += half; n -= half; }
      else n = half;
    }
    bounds_of(p, b, s0, s1);
    const int64_t i = j - ((int64_t)s0 * p.group / RT + b), tiles = ((int64_t)(s1 - s0) * p.group + RT - 1) / RT;
    if (i < 0 || i >= tiles) return t;
    k = (int)(tiles - 1 - i);
  }
  t.s0 = __builtin_amdgcn_readfirstlane(s0);
  t.rows = __builtin_amdgcn_readfirstlane((s1 - s0) * p.group);
  t.row0 = __builtin_amdgcn_readfirstlane(k * RT);
  return t;
}

// The order of a turn's instructions: after each product the vector work of one
// logit and a read or two from LDS, so that the vector unit has work while a
// product runs.
template <int READS>
__device__ __forceinline__ void sched_turn(int products) {
#pragma unroll
  for (int i = 0; i < products; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
  }
}

// A workgroup: four waves of 64 rows (two blocks of 32), one wave per SIMD with
// all its registers; 128 keys a step, two LDS buffers.  S^T = K Q^T on
// 32x32x16 products puts a row's logits of 16 keys into one lane; the weights go
// back in as the other operand of O^T = V^T P^T without leaving the lane.  The
// two blocks take turns, the products of one running while the vector unit does
// the softmax of the other:
//   turn 1 of 32 keys:  products  O_A += V P_A (the keys before), S_A (these)
//                       vector    softmax of S_B (the keys before)
//   turn 2:             products  O_B += V P_B (the keys before), S_B (these)
//                       vector    softmax of S_A (these)
//
// KS: that many waves share 64 rows, each with its part of every step's keys, and
// add up in LDS at the end: a tile's time is that of one wave's keys, and where
// there are few tiles nothing else fills the card.
//
// PER_CU: workgroups a CU holds at once.  Two, with half the registers each, for
// heads of 64 and many tiles: one starts and ends its tiles while the other works.
template <int D, int KS, int PER_CU>
__global__ __launch_bounds__(256, PER_CU) void prompt_kernel(Prompt p, int64_t tiles) {
  constexpr int NW = 4, KT = 32 * NW, KBS = NW / KS, RT = 64 * NW / KS;
  constexpr int STEPS = D / 16, DT = D / 32;
  using Im = Image<D>;
  constexpr int BUF = Im::bytes(KT), KB32 = Im::bytes(32), KB16 = KB32 / 2, KB8 = KB32 / 4;
  constexpr int LOADS = KT * D * 2 / 1024;                  // KBs of a step's keys
  __shared__ __align__(16) uint8_t lds[4 * BUF];
  uint8_t* const ksh = lds;
  uint8_t* const vsh = lds + 2 * BUF;
  __shared__ uint32_t bad[2][NW];                           // of masked steps: keys whose values are not finite
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hh = lane >> 5;
  const int part = wave % KS, row_wave = wave / KS;         // the wave's share of the keys, and its rows
  const int h = blockIdx.x % p.heads;
  for (int64_t j = blockIdx.x / p.heads; j < tiles; j += gridDim.x / p.heads) {
  const PromptTile w = tile_of<RT>(p, j, lane);
  if (w.rows == 0) continue;
  const int last_row = w.row0 + RT < w.rows ? w.row0 + RT - 1 : w.rows - 1;
  const int k1 = last_row / p.group + 1;                    // keys the tile needs
  const int sure = w.row0 / p.group + 1;                    // keys that all its rows see

  const uint16_t* const kp = p.K + (int64_t)w.s0 * p.k_stride + (int64_t)h * D + Im::piece_of(lane) * 8;
  const uint16_t* const vp = p.V + (int64_t)w.s0 * p.v_stride + (int64_t)h * D + Im::piece_of(lane) * 8;
  // The wave's KBs `from` .. `to` - 1 of a step's keys and values.  They are fetched
  // in four parts over the step before: 16 loads at once hold up the products
  // behind them (16000 tokens: 4017 -> 3986 us).
  constexpr int SHARE = LOADS / NW;
  auto fetch = [&](int key0, int buf, int from, int to) {
    auto put = [&](const void* from, uint8_t* to) {
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                       (__attribute__((address_space(3))) void*)to, 16, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < SHARE; ++i) {
      if (i < from || i >= to) continue;
      const int kb = wave + i * NW;
      int key = key0 + kb * Im::KPB + Im::key_of(lane);
      key = key < k1 ? key : k1 - 1;                        // behind the last key it is repeated, and masked
      put(kp + (int64_t)key * p.k_stride, ksh + buf * BUF + kb * Im::PITCH);
      put(vp + (int64_t)key * p.v_stride, vsh + buf * BUF + kb * Im::PITCH);
    }
  };
  // Values of keys that some row must not see: a weight of zero does not undo an
  // infinity or a NaN, so they become zeros, and their key's logit NaN for the
  // rows that do see it.
  auto clean = [&](int buf) {
    if (tid < NW) bad[buf ^ 1][tid] = 0;
    for (int i = tid; i < KT * D / 8; i += 64 * NW) {
      u32x4_t* at = reinterpret_cast<u32x4_t*>(vsh + buf * BUF + i / 64 * Im::PITCH + i % 64 * 16);
      u32x4_t v = *at;
      bool off = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((v[e] & 0x7F80u) == 0x7F80u) { v[e] &= 0xFFFF0000u; off = true; }
        if ((v[e] & 0x7F800000u) == 0x7F800000u) { v[e] &= 0xFFFFu; off = true; }
      }
      if (off) {
        *at = v;
        const int key = i / 64 * Im::KPB + Im::key_of(i % 64);
        atomicOr(&bad[buf][key / 32], 1u << (key % 32));
      }
    }
  };
  if (tid < 2 * NW) bad[tid / NW][tid % NW] = 0;
  fetch(0, 0, 0, SHARE);

  bf16x8_t qf[2][STEPS];
  int lim[2], limmin = k1;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    int row = w.row0 + row_wave * 64 + n * 32 + col;
    row = row < w.rows ? row : w.rows - 1;                  // behind the last row it is repeated, and not stored
    const int tok = row / p.group, g = row - tok * p.group;
    const uint16_t* q = p.Q + (int64_t)(w.s0 + tok) * p.q_stride + (int64_t)(h * p.group + g) * D + 8 * hh;
    lim[n] = tok + 1;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) qf[n][s] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(q + 16 * s));
  }
  {
    int row = w.row0 + row_wave * 64;                       // the wave's first row sees least
    row = row < w.rows ? row : w.rows - 1;
    limmin = row / p.group + 1;
  }
  if (p.scale < 0.f) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        u32x4_t v = __builtin_bit_cast(u32x4_t, qf[n][s]);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] ^= 0x80008000u;
        qf[n][s] = __builtin_bit_cast(bf16x8_t, v);
      }
  }
  // Positive also for a scale of 0, so that -inf stays -inf: the least there is, by
  // which logits below 2^126 are 2^-23 at most and all weights 1.
  const float cq = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 0x1p-149f);
  // The queries never change and only products read them: accumulation
  // registers hold them, the vector unit's stay free.
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int s = 0; s < STEPS; ++s) asm volatile("" : "+a"(qf[n][s]));

  f32x16_t acc[2][DT], z[2];
  float m[2], l[2], mx[2];
  // of exponents, and what a logit passes before the maximum is looked at: m and m + kLag, or beyond kFar 0 and -inf
  float base[2], lim_m[2];
  u32x4_t pw[2][2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][t][i] = 0.f;
    // before the first keys: weights of zero, logits that add nothing
#pragma unroll
    for (int i = 0; i < 16; ++i) z[n][i] = -INFINITY;
    mx[n] = m[n] = lim_m[n] = -INFINITY;
    base[n] = 0.f;
    l[n] = 0.f;
    pw[n][0] = pw[n][1] = u32x4_t{0u, 0u, 0u, 0u};
  }

  // a lane's keys: row col of 32, values 16 s + 8 hh .. + 7
  const uint8_t* const kread = ksh + part * KBS * KB32 + Im::at(col, hh);
  // a transposing read: 16 lanes take 4 keys and 16 coordinates; lane i brings 8
  // bytes of key i / 4 and gets coordinate i of all four.  Its 4 coordinates are
  // chosen so that a lane's results are runs of 8 (see the stores).
  const int li = lane & 15, dh = (lane >> 4) & 1;
  const uint8_t* const vread = vsh + part * KBS * KB32 + Im::at(4 * hh + (li >> 2), 2 * dh + (li & 1)) + ((li >> 1) & 1) * 8;
  bf16x8_t kf[STEPS], vf[2][DT];
  auto read_k = [&](int buf, int kb) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) kf[s] = *reinterpret_cast<const bf16x8_t*>(kread + buf * BUF + kb * KB32 + Im::two(s));
  };
  auto tr = [&](const uint8_t* at) {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)at));
  };
  auto read_v = [&](int buf, int kb) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const uint8_t* at = vread + buf * BUF + kb * KB32 + s * KB16 + t * 256;
        const uint2 a = tr(at), b = tr(at + KB8);
        vf[s][t] = __builtin_bit_cast(bf16x8_t, u32x4_t{a.x, a.y, b.x, b.y});
      }
  };
  auto max_of = [&](const f32x16_t& v) {
    float r = v[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) r = fmaxf(r, v[i]);
    return r;
  };
  // masks, and the running maximum moved where it has to be (keys key .. key + 31)
  auto bounds = [&](auto blk, int key, uint32_t nan) {
    constexpr int n = decltype(blk)::value;
    if (__builtin_expect(key + 32 > limmin || nan, 0)) {
      asm volatile("");                    // a branch: the selects must not run in every step
#pragma unroll
      for (int i = 0; i < 16; ++i) z[n][i] = key + 8 * (i / 4) + 4 * hh + i % 4 < lim[n] ? z[n][i] : -INFINITY;
      if (nan) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = 8 * (i / 4) + 4 * hh + i % 4;
          if (key + at < lim[n] && ((nan >> at) & 1u)) z[n][i] = NAN;
        }
      }
      mx[n] = max_of(z[n]);
    }
    if (__builtin_expect(__ballot(mx[n] * cq > lim_m[n]) != 0, 0)) {
      float v = mx[n] * cq;
      v = fmaxf(v, __shfl_xor(v, 32));
      v = v > m[n] + kLag ? v : m[n];      // a row's maximum moves by its own logits only
      const float f = v == m[n] ? 1.0f : __builtin_amdgcn_exp2f(m[n] - v);
      m[n] = v;
      l[n] *= f;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[n][t][i] *= f;
      // An exponent z cq - m of one rounding is off by half a step of m: beyond 2^24
      // the largest logit's own would leave 0 and take every weight with it.  The
      // rounded product minus m is 0 there; it goes on as a z for a base of 0.
      const bool far = fabsf(v) > kFar && v != -INFINITY;
      lim_m[n] = far ? -INFINITY : v + kLag;
      base[n] = fabsf(v) > kFar ? 0.f : v;  // where nothing is seen yet too
      if (__builtin_expect(__ballot(far) != 0, 0)) {
        const float up = 1.0f / cq;        // finite: logits below 2^126 pass kFar by a cq above 2^-116 only
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float e = z[n][i] * cq;
          asm volatile("" : "+v"(e));      // rounded
          z[n][i] = far ? (e - v) * up : z[n][i];
        }
      }
    }
  };
  // One turn: the softmax of block n against the products of the other block,
  // logits first, so that their maximum is there when the turn ends.
  auto turn = [&](auto soft, auto reads, auto&& after_s, auto&& after_pv) {
    constexpr int n = decltype(soft)::value, o = 1 - n;
    float pv[16];
    f32x16_t zn;
#pragma unroll
    for (int i = 0; i < 16; ++i) zn[i] = 0.f;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) zn = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[s], qf[o][s], zn, 0, 0, 0);
    after_s();
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < DT; ++t)
        acc[o][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[s][t], __builtin_bit_cast(bf16x8_t, pw[o][s]), acc[o][t], 0, 0, 0);
    after_pv();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      pv[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[n][i], cq, -base[n]));
    }
    // 16 weights are added up before they meet the sum, as in the products: by
    // itself a weight below 2^-24 of the sum would be lost there and not here
    float ps[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) ps[i] = pv[2 * i] + pv[2 * i + 1];
    l[n] += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
#pragma unroll
    for (int e = 0; e < 8; ++e) pw[n][e / 4][e % 4] = cvt_pk_bf16(pv[2 * e], pv[2 * e + 1]);
    z[o] = zn;
    mx[o] = max_of(zn);
    // the weights and the maximum are made here, not where they are used
    asm volatile("" : "+v"(pw[n][0]), "+v"(pw[n][1]), "+v"(l[n]), "+v"(mx[o]));
    sched_turn<decltype(reads)::value>(STEPS + 2 * DT);
    __builtin_amdgcn_sched_barrier(0);
  };
  using A = std::integral_constant<int, 0>;
  using B = std::integral_constant<int, 1>;
  auto none = [] {};

  __builtin_amdgcn_s_waitcnt(kNoLoads);
  __syncthreads();
  if (KT > sure) {
    clean(0);
    __syncthreads();
  }
  read_k(0, 0);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int t = 0; t < DT; ++t) vf[s][t] = bf16x8_t{};
  int buf = 0, prev = 0;                   // prev: the first of the 32 keys before
  uint32_t before = 0;                     // those of them whose values are not finite
  for (int key = 0; key < k1; key += KT, buf ^= 1) {
    const bool more = key + KT < k1;
    uint32_t nans[KBS];
#pragma unroll
    for (int i = 0; i < KBS; ++i) nans[i] = 0;
    if (key + KT > sure) {
#pragma unroll
      for (int i = 0; i < KBS; ++i) nans[i] = __builtin_amdgcn_readfirstlane(bad[buf][part * KBS + i]);
    }
#pragma unroll
    for (int kb = 0; kb < KBS; ++kb) {
      const int k = key + 32 * (part * KBS + kb);
      if ((KS > 1 || kb > 0) && k >= k1) break;             // the last step's keys may end early
      if (more) fetch(key + KT, buf ^ 1, kb * SHARE / KBS, (kb + 1) * SHARE / KBS);
      bounds(B{}, prev, before);
      before = nans[kb];
      prev = k;
      turn(B{}, std::integral_constant<int, 1>{}, none, none);
      bounds(A{}, k, before);
      turn(A{}, std::integral_constant<int, 2>{}, [&] { if (kb + 1 < KBS) read_k(buf, kb + 1); }, [&] { read_v(buf, kb); });
    }
    __builtin_amdgcn_s_waitcnt(kNoLoads);
    __syncthreads();
    if (more) {
      if (key + 2 * KT > sure) {
        clean(buf ^ 1);
        __syncthreads();
      }
      read_k(buf ^ 1, 0);
    }
  }
  // what is left: the last keys' products and block B's softmax
  bounds(B{}, prev, before);
  turn(B{}, std::integral_constant<int, 1>{}, none, none);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int t = 0; t < DT; ++t)
      acc[1][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[s][t], __builtin_bit_cast(bf16x8_t, pw[1][s]), acc[1][t], 0, 0, 0);

  if constexpr (KS > 1) {
    // every lane adds what the same lane of the waves that share its rows holds
    constexpr int LANE = 2 * DT * 4, WAVE = (LANE + 1) * 1024;   // 16-byte pieces of a lane, bytes of a wave
    static_assert(NW / KS * (KS - 1) * WAVE <= 4 * BUF, "the sums fit where the keys were");
    auto at = [&](int o) { return lds + (row_wave * (KS - 1) + o - 1) * WAVE + lane * 16; };
    if (part > 0) {                        // the last step's barrier has freed the LDS
      uint8_t* to = at(part);
#pragma unroll
      for (int i = 0; i < LANE; ++i) {
        const f32x16_t& v = acc[i / (4 * DT)][i / 4 % DT];
        *reinterpret_cast<f32x4_t*>(to + i * 1024) = f32x4_t{v[4 * (i % 4)], v[4 * (i % 4) + 1], v[4 * (i % 4) + 2], v[4 * (i % 4) + 3]};
      }
      *reinterpret_cast<f32x4_t*>(to + LANE * 1024) = f32x4_t{m[0], m[1], l[0], l[1]};
    }
    __syncthreads();
    if (part == 0) {
      for (int o = 1; o < KS; ++o) {
        const uint8_t* from = at(o);
        const f32x4_t ml = *reinterpret_cast<const f32x4_t*>(from + LANE * 1024);
        float fa[2], fb[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float M = fmaxf(m[n], ml[n]);
          fa[n] = m[n] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[n] - M);
          fb[n] = ml[n] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[n] - M);
          m[n] = M;
          l[n] = l[n] * fa[n] + ml[2 + n] * fb[n];          // a NaN sum (a NaN key was seen) stays one
        }
#pragma unroll
        for (int i = 0; i < LANE; ++i) {
          const f32x4_t u = *reinterpret_cast<const f32x4_t*>(from + i * 1024);
          f32x16_t& v = acc[i / (4 * DT)][i / 4 % DT];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[4 * (i % 4) + e] = v[4 * (i % 4) + e] * fa[i / (4 * DT)] + u[e] * fb[i / (4 * DT)];
        }
      }
    }
    __syncthreads();
    if (part > 0) continue;
  }
  // Register i of tile t is the tile's row 8 (i / 4) + 4 hh + i % 4, which holds
  // coordinate 32 t + 16 (i / 8) + 8 hh + i % 8 by the choice above.
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    l[n] += __shfl_xor(l[n], 32);
    const int row = w.row0 + row_wave * 64 + n * 32 + col;
    if (row >= w.rows) continue;
    const int tok = row / p.group, g = row - tok * p.group;
    const float inv = 1.0f / l[n];          // every logit -inf: 0 / 0
    const int64_t at = (int64_t)(w.s0 + tok) * p.o_stride + (int64_t)(h * p.group + g) * D + 8 * hh;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = acc[n][t][8 * e + i] * inv;
        const int d = 32 * t + 16 * e;
        if (p.out_f32) {
          f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at + d);
          o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
          o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
        } else {
          u32x4_t u;
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = cvt_pk_bf16(v[2 * i], v[2 * i + 1]);
          *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.out) + at + d) = u;
        }
      }
  }
  // the last step's barrier has freed the LDS for the next tile
  }
}

}  // namespace

namespace {

// How many waves share a tile's rows, from sizes alone (the lengths are the
// device's): the one with the least time by what was measured, in us: starting
// and ending a tile, 8, 10 and 13 for 1, 2 and 4 waves, once for every 256
// workgroups; and a step of 128 keys, 4.2 (2.1 for heads of 64), over the waves
// for the longest tile, or all tiles' over the card.  8 heads, 1 / 2 / 4 waves:
// one prompt of 77 tokens, group 8, 11.7 / 12.6 / 13.4; of 300 19.3 / 17.7 / 26.0;
// of 2000 95 / 116 / 182; of 4096, group 1, 133 / 81 / 73.  The host knows the mean
// length only: a long prompt among many short ones is shared as if all were short.
int sharers(const Prompt& p, double tiles, double len) {
  const double step = p.head_dim == 128 ? 4.2 : 2.1, spread = tiles * len / (256.0 * 256.0);
  const double fixed[3] = {8, 10, 13};
  int best = 0;
  double least = 0;
  for (int i = 0; i < 3; ++i) {
    const double wgs = tiles * (1 << i), longest = len / (128 << i);
    const double t = fixed[i] * (wgs > 256 ? wgs / 256 : 1) + step * (longest > spread ? longest : spread);
    if (i == 0 || t < least) { best = i; least = t; }
  }
  return 1 << best;
}

}  // namespace

hipError_t launch_prompt(const Prompt& p, hipStream_t st) {
  const double about = ((double)p.T * p.group / 256 + 0.5 * p.B) * p.heads, len = (double)p.T / p.B;
  const int ks = sharers(p, about, len);
  // Two workgroups a CU against one, heads of 64, us (in brackets `about`): 64
  // prompts of 1 .. 100 (328) 12.5 against 15.9, 32 of 1 .. 333 (397) 16.6 against
  // 20.2, 32 of 1 .. 500 (564) 25.5 against 31.6, one of 8000 (1004) 298 against
  // 328; but 16 of 1 .. 1000 (266) 29.4 against 28.2, one of 3000 (379) 68.3 against
  // 63.4, 8 of 500 .. 1100 (415) 31.7 against 30.6.  One of 4096 is either's: 8 KV
  // heads (516) 101 against 104, 4 (514) 99 against 96, 32 (528) 103 against 102.
  const bool two = p.head_dim == 64 && ks == 1 && (about > 512 || (about > 256 && len <= 256));
  const int64_t tiles = (int64_t)p.T * p.group / (256 / ks) + p.B;
  const int64_t most = (1 << 22) / p.heads;
  const dim3 grid((unsigned)((tiles < most ? tiles : most) * p.heads));
#define GO(D, KS, N) hipLaunchKernelGGL((prompt_kernel<D, KS, N>), grid, dim3(256), 0, st, p, tiles)
#define GO_D(D)                   \
  do {                            \
    if (ks == 1) GO(D, 1, 1);      \
    else if (ks == 2) GO(D, 2, 1); \
    else GO(D, 4, 1);              \
  } while (0)
  if (p.head_dim == 128) GO_D(128);
  else if (two) GO(64, 1, 2);
  else GO_D(64);
#undef GO_D
#undef GO
  return hipGetLastError();
}

}  // namespace qg
