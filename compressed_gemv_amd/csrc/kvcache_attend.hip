// Attention over the quantized, paged KV cache: few rows against many keys
// (one token or a few drafted tokens per sequence), and the joining of partial
// results.
//
// Softmax in one pass over the keys with a running maximum; log2 domain.  The
// cache's codes are operands of the matrix cores as they lie in memory: a code
// zero-extended to 16 bits is a bf16 subnormal, q * 2^-133 exactly, so one byte
// permute (8 bits) or one shift and mask (4 bits) makes a pair of operands, and
// no code is ever converted or scaled one by one.  The other operand carries
// 2^64 (exact: only exponents move), so products stay far from fp32's ends.
//   logits   <x, k_j> = s_j sum_i x_i q_ij + o_j sum_i x_i
//   output   sum_j p_j v_j = sum_j (p_j s_j) q_j + sum_j p_j o_j
// The weights p_j s_j enter as bf16 hi + lo (two products): with one rounding
// to 8 bits the offset form would lose three times what a plain bf16
// probability does, since codes count from the row's minimum.
//
// Measured (8 KV heads of 128, 8 query heads each): 32 sequences of 1000 .. 8000
// tokens at 8 bits 58 us, 5.2 TB/s of codes and constants, 6.4 over 32000 each,
// bound by memory; 4 of 100000 .. 131072 at 4 bits 96 us, 5.2 TB/s, where
// decoding, products and softmax are 270 vector instructions for 32 keys
// (counted), 58 us of a SIMD's issue at 4 clocks each and 2.1 GHz, beside the 71
// us that a plain read would take.  A third step in flight was no faster there.
// One sequence of 517 tokens takes 11 us, nearly all of it latency: lens,
// page table, codes and the join of the waves one after the other.
#include "common.hpp"
#include "kvcache_attend.hpp"

namespace qg {

constexpr float kFar = 0x1p20f;                     // maxima (times log2 e) beyond it are taken off first
constexpr float kUp = 0x1p64f, kDown = 0x1p-64f;   // scale of the query and weight operands
constexpr float kCode = 0x1p69f;                   // product of a scaled operand and a code, undone

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// fp16 times fp32 in one instruction (v_fma_mix_f32; a plain product would convert first)
__device__ __forceinline__ float mix_mul(float h, float x) { return __builtin_fmaf(h, x, 0.f); }

// bf16 pair times a power of two
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, float f) {
  const float lo = bf16_lo_to_f32(w) * f, hi = bf16_hi_to_f32(w) * f;
  return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xFFFF0000u);
}

template <typename V>
__device__ __forceinline__ V ld_nt(const uint8_t* base, uint32_t off) {
  return __builtin_nontemporal_load(reinterpret_cast<const V*>(base + off));
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// A workgroup goes through the tiles (RT rows) of its piece; its four waves
// take a quarter of a tile's keys each, 32 keys a step.  Lane l, r = l % 16, kg = l / 16:
//   K operand: key r, a quarter kg of the coordinates, straight from memory
//   logits:    query r, keys 4 kg .. 4 kg + 3 of both halves of the step
//   V operand: coordinates r D/16 .. of exactly those eight keys (the order of
//              the contraction is free), so the weights never leave their lane
// A lane brings in the constants of one key (K's in lanes 0 .. 31, V's in the
// others); they go round through 256 bytes of LDS while the logits are formed.
// RT = 8 (one token of a group of up to 8 heads): both halves of the 16 columns
// hold the same rows, one with the high and one with the low parts of the
// weights, so that one product does for two.
template <int D, int BITS, int RT, bool SPREAD = false>
__device__ __forceinline__ void rows_body(const AttendArgs& x, unsigned block) {
  constexpr int NT = RT > 16 ? 2 : 1;
  constexpr bool PACK = RT == 8;
  constexpr int ROWB = D * BITS / 8;       // bytes of a cache row
  constexpr int KB = ROWB / 4;             // bytes of a K row per lane
  constexpr int KW = KB / 4;
  constexpr int VB = ROWB / 16;            // bytes of a V row per lane
  constexpr int VW = VB < 4 ? 1 : VB / 4;
  constexpr int TILES = D / 16, STEPS = D / 32;
  constexpr int PITCH = D + 4;
  __shared__ __align__(16) float os[4][RT][PITCH];
  __shared__ float ms[4][RT], ls[4][RT];
  __shared__ __align__(16) uint32_t consts[4][64];
  const KvAttend& a = x.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kg = lane >> 4;
  const int heads = a.c.heads, h = block % heads;
  Pieces pieces = pieces_of<SPREAD>(x, block / heads, lane);
  Work w;
  while (next_work<false, false, SPREAD>(x, pieces, w, lane)) {
  f32x4_t acc[NT][TILES];
  float m[NT], l[NT], po[NT];              // maximum, sum of weights, sum of weights times offsets
  // of exponents, and what a logit passes before the maximum moves: m - 64 and m + 8, or beyond kFar -64 and -inf
  float base[NT], lim_m[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[n][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    m[n] = lim_m[n] = -INFINITY;
    base[n] = 0.f;
    l[n] = po[n] = 0.f;
  }

  const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
  const int per = (w.k1 - w.k0 + 127) / 128 * 32;
  const int ks = w.k0 + wave * per;
  const int ke = ks + per < w.k1 ? ks + per : w.k1;

  // page numbers of the next 64 pages, one per lane; -1: not in the cache
  int pbase = 0, ids = -1;
  auto refill = [&](int first) {
    pbase = first;
    const int p = first + lane;
    int id = -1;
    if (p < w.max_pages && p <= (w.k1 - 1) >> shift) id = w.pages[p];
    ids = id >= 0 && id < a.c.n_pages ? id : -1;
  };

  struct Raw {
    uint32_t k[2][KW];
    uint32_t v[8][VW];
    uint32_t mt;                           // constants of K's key lane, of V's key lane - 32
    int bad;                               // halves whose page is not in the cache
  };
  auto load = [&](int key, Raw& w_) {
    if (((key + 16) >> shift) - pbase >= 64) refill(key >> shift);
    w_.bad = 0;
    int64_t rows[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int kk = key + 16 * hf;
      const int id = __builtin_amdgcn_readlane(ids, (kk >> shift) - pbase);
      if (id < 0) w_.bad |= 1 << hf;
      const int64_t row = (((int64_t)(id < 0 ? 0 : id) * heads + h) << shift) + (kk & pmask);
      rows[hf] = row;
      const uint8_t* kc = a.c.codes[0] + row * ROWB;
      const uint8_t* vc = a.c.codes[1] + row * ROWB;
      if constexpr (KB == 32) {
        const u32x4_t p0 = ld_nt<u32x4_t>(kc, r * ROWB + kg * 16), p1 = ld_nt<u32x4_t>(kc, r * ROWB + 64 + kg * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) { w_.k[hf][e] = p0[e]; w_.k[hf][(4 + e) % KW] = p1[e]; }
      } else if constexpr (KB == 16) {
        const u32x4_t p0 = ld_nt<u32x4_t>(kc, r * ROWB + kg * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) w_.k[hf][e % KW] = p0[e];
      } else {
        const u32x2_t p0 = ld_nt<u32x2_t>(kc, r * ROWB + kg * 8);
        w_.k[hf][0] = p0[0];
        w_.k[hf][1 % KW] = p0[1];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t off = (4 * kg + i) * ROWB + r * VB;
        if constexpr (VB == 8) {
          const u32x2_t p = ld_nt<u32x2_t>(vc, off);
          w_.v[4 * hf + i][0] = p[0];
          w_.v[4 * hf + i][1 % VW] = p[1];
        } else if constexpr (VB == 4) {
          w_.v[4 * hf + i][0] = ld_nt<uint32_t>(vc, off);
        } else {
          w_.v[4 * hf + i][0] = ld_nt<uint16_t>(vc, off);
        }
      }
    }
    const uint32_t* mp = lane < 32 ? a.c.meta[0] : a.c.meta[1];
    w_.mt = mp[((lane & 16) ? rows[1] : rows[0]) + r];
  };

  // the first keys are on their way while the queries are made ready
  Raw ra, rb;
  if (ks < ke) {
    refill(ks >> shift);
    load(ks, ra);
  }
  __builtin_amdgcn_sched_barrier(0);

  // queries: operand registers, sums, and what each row sees
  u32x4_t qf[NT][STEPS];
  float qs[NT];
  int lim[NT];
  int limmin = w.k1;
  const float c0 = a.scale * 1.4426950408889634f, c1 = c0 * kCode;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = w.row0 + (PACK ? r % 8 : 16 * n + r);
    const bool ok = row < w.rows;
    const int tok = ok ? row / a.group : 0, g = ok ? row - tok * a.group : 0;
    const uint16_t* q = a.Q + (int64_t)(w.t0 + tok) * a.q_stride + (int64_t)(h * a.group + g) * D;
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int d0 = BITS == 8 ? (D == 128 ? 64 * (s / 2) + 16 * kg + 8 * (s % 2) : 16 * kg + 8 * s)
                               : 2 * KB * kg + 8 * s;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (ok) v = *reinterpret_cast<const u32x4_t*>(q + d0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum += bf16_lo_to_f32(v[e]) + bf16_hi_to_f32(v[e]);
        v[e] = scale_pair(v[e], kUp);
      }
      if constexpr (BITS == 4) {           // pairs (j, j + 4), as a nibble mask leaves them; odd nibbles
        const u32x4_t t = v;               // stay where they are, as 16 times their code
        v[0] = __builtin_amdgcn_perm(t[2], t[0], 0x05040100u);
        v[1] = __builtin_amdgcn_perm(t[2], t[0], 0x07060302u);
        v[2] = __builtin_amdgcn_perm(t[3], t[1], 0x05040100u);
        v[3] = __builtin_amdgcn_perm(t[3], t[1], 0x07060302u);
        v[1] = scale_pair(v[1], 0x1p-4f);
        v[3] = scale_pair(v[3], 0x1p-4f);
      }
      qf[n][s] = v;
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    qs[n] = sum * c0;
    lim[n] = ok ? row_sees(w, tok) : w.k1;
    int lo = lim[n];
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) { const int o = __shfl_xor(lo, d); lo = o < lo ? o : lo; }
    limmin = lo < limmin ? lo : limmin;
  }
  limmin = __builtin_amdgcn_readfirstlane(limmin);

  const float low = r < 8 ? 0.f : -1.f;    // PACK: which part of the weights this lane's column holds
  auto compute = [&](int key, const Raw& w_) {
    u32x4_t km[2], vmr[2];                 // of this lane's keys 4 kg .. + 3 of both halves
    consts[wave][lane] = w_.mt;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      km[hf] = *reinterpret_cast<const u32x4_t*>(&consts[wave][16 * hf + 4 * kg]);
      vmr[hf] = *reinterpret_cast<const u32x4_t*>(&consts[wave][32 + 16 * hf + 4 * kg]);
    }
    f32x4_t z[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) z[n][hf] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        u32x4_t f;
        if constexpr (BITS == 8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[2 * e] = __builtin_amdgcn_perm(0u, w_.k[hf][2 * s + e], 0x0C010C00u);
            f[2 * e + 1] = __builtin_amdgcn_perm(0u, w_.k[hf][2 * s + e], 0x0C030C02u);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = (w_.k[hf][s] >> (8 * (e / 2))) & (e % 2 ? 0x00F000F0u : 0x000F000Fu);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
          z[n][hf] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f),
                                                             __builtin_bit_cast(bf16x8_t, qf[n][s]), z[n][hf], 0, 0, 0);
      }
    // logits; where some row of the tile does not see all of the step, what it does not see is -inf
    float t[NT][8];
    const bool masked = key + 32 > limmin || w_.bad;
    auto seen = [&](int n, int j) {
      return key + 16 * (j / 4) + 4 * kg + j % 4 < lim[n] && !((w_.bad >> (j / 4)) & 1);
    };
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t kc = km[j / 4][j % 4];
        t[n][j] = __builtin_fmaf(z[n][j / 4][j % 4], mix_mul(f16_lo(kc), c1), mix_mul(f16_hi(kc), qs[n]));
      }
      if (masked) {
        asm volatile("");                  // a branch: the selects must not run in every step
#pragma unroll
        for (int j = 0; j < 8; ++j) t[n][j] = seen(n, j) ? t[n][j] : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = fmaxf(mx, t[n][j]);
      grow |= mx > lim_m[n];
      z[n][0][0] = mx;
    }
    // The maximum may lag by 8 (weights up to 2^8): it moves only when some
    // lane's logits pass it by more, one vote per step instead of a reduction.
    if (__ballot(grow)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float mx = z[n][0][0];
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        mx = fmaxf(mx, m[n]);
        const float f = mx == m[n] ? 1.0f : exp2_hw(m[n] - mx);
        m[n] = mx;
        l[n] *= f;
        po[n] *= f;
#pragma unroll
        for (int q = 0; q < TILES; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][q][i] *= f;
        // far from zero m - 64 is not 64 below m: the weights' factor would be 2^128, or 1
        const bool far = fabsf(mx) > kFar && mx != -INFINITY;
        lim_m[n] = far ? -INFINITY : mx + 8.0f;
        base[n] = far ? -64.0f : (mx == -INFINITY ? 0.f : mx - 64.0f);
        if (__builtin_expect(__ballot(far) != 0, 0)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) t[n][j] = far ? t[n][j] - mx : t[n][j];
        }
      }
    }
    u32x4_t wh[NT], wl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t vm[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) vm[j] = vmr[j / 4][j % 4];
      if (masked) {                        // constants of slots that are not seen may be anything
        asm volatile("");
#pragma unroll
        for (int j = 0; j < 8; ++j) vm[j] = seen(n, j) ? vm[j] : 0u;
      }
      float wv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = exp2_hw(t[n][j] - base[n]);   // 2^64 times the weight
        wv[j] = mix_mul(f16_lo(vm[j]), p);
        po[n] = __builtin_fmaf(f16_hi(vm[j]), p, po[n]);
        l[n] += p;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        wh[n][e] = cvt_pk_bf16(wv[2 * e], wv[2 * e + 1]);
        if constexpr (PACK)                // columns 8 .. 15: what the high part leaves
          wh[n][e] = cvt_pk_bf16(__builtin_fmaf(low, bf16_lo_to_f32(wh[n][e]), wv[2 * e]),
                                 __builtin_fmaf(low, bf16_hi_to_f32(wh[n][e]), wv[2 * e + 1]));
        else
          wl[n][e] = cvt_pk_bf16(wv[2 * e] - bf16_lo_to_f32(wh[n][e]), wv[2 * e + 1] - bf16_hi_to_f32(wh[n][e]));
      }
    }
    u32x4_t pair = {0u, 0u, 0u, 0u};       // 4 bits: the halves of the current four coordinates
#pragma unroll
    for (int q = 0; q < TILES; ++q) {
      u32x4_t f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (BITS == 8) {
          const uint32_t sel = (uint32_t)(q % 4) | 0x0C000C00u | ((4u + q % 4) << 16);
          f[e] = __builtin_amdgcn_perm(w_.v[2 * e + 1][q / 4], w_.v[2 * e][q / 4], sel);
        } else {
          if (q % 4 == 0)
            pair[e] = __builtin_amdgcn_perm(w_.v[2 * e + 1][0], w_.v[2 * e][0], q == 0 ? 0x05040100u : 0x07060302u);
          f[e] = (pair[e] >> (8 * (q % 4 / 2))) & (q % 2 ? 0x00F000F0u : 0x000F000Fu);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[n][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f),
                                                            __builtin_bit_cast(bf16x8_t, wh[n]), acc[n][q], 0, 0, 0);
        if constexpr (!PACK)
          acc[n][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f),
                                                              __builtin_bit_cast(bf16x8_t, wl[n]), acc[n][q], 0, 0, 0);
      }
    }
  };

  if (ks < ke) {
    int key = ks;
    while (true) {
      if (key + 32 < ke) load(key + 32, rb);
      __builtin_amdgcn_sched_barrier(0);
      compute(key, ra);
      key += 32;
      if (key >= ke) break;
      if (key + 32 < ke) load(key + 32, ra);
      __builtin_amdgcn_sched_barrier(0);
      compute(key, rb);
      key += 32;
      if (key >= ke) break;
    }
  }

  // join the four waves
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] += __shfl_xor(l[n], 16);
    l[n] += __shfl_xor(l[n], 32);
    po[n] += __shfl_xor(po[n], 16);
    po[n] += __shfl_xor(po[n], 32);
    if constexpr (PACK) {                  // high and low parts meet
#pragma unroll
      for (int q = 0; q < TILES; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][q][i] += dpp_f32<0x128>(acc[n][q][i]);   // row_ror:8
    }
    if (kg == 0 && (!PACK || r < 8)) ms[wave][16 * n + r] = m[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (PACK && r >= 8) continue;
    const int row = 16 * n + r;
    const float mm = fmaxf(fmaxf(ms[0][row], ms[1][row]), fmaxf(ms[2][row], ms[3][row]));
    const float f = m[n] == -INFINITY ? 0.f : exp2_hw(m[n] - mm);
    if (kg == 0) ls[wave][row] = l[n] * kDown * f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < TILES; q += 4) {
        f32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (acc[n][q + e][i] * (BITS == 4 && e % 2 ? kCode / 16 : kCode) + po[n] * kDown) * f;
        *reinterpret_cast<f32x4_t*>(&os[wave][row][TILES * (4 * kg + i) + q]) = v;
      }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < RT * (D / 4); e += 256) {
    const int row = e / (D / 4), d = 4 * (e % (D / 4)), R = w.row0 + row;
    if (R >= w.rows) continue;
    const f32x4_t o0 = *reinterpret_cast<const f32x4_t*>(&os[0][row][d]), o1 = *reinterpret_cast<const f32x4_t*>(&os[1][row][d]);
    const f32x4_t o2 = *reinterpret_cast<const f32x4_t*>(&os[2][row][d]), o3 = *reinterpret_cast<const f32x4_t*>(&os[3][row][d]);
    const float lt = (ls[0][row] + ls[1][row]) + (ls[2][row] + ls[3][row]);
    f32x4_t v;
    for (int i = 0; i < 4; ++i) v[i] = (o0[i] + o1[i]) + (o2[i] + o3[i]);
    if (w.direct) {
      const int tok = R / a.group, g = R - tok * a.group;
      const float inv = lt == 0.f ? 0.f : 1.0f / lt;
      for (int i = 0; i < 4; ++i) v[i] *= inv;
      store_out4(a, (int64_t)(w.t0 + tok) * a.o_stride + (int64_t)(h * a.group + g) * D + d, v);
    } else {
      *reinterpret_cast<f32x4_t*>(part_o<D>(x, w.slot, h, row) + d) = v;
      if (d == 0) {
        float* ml = part_ml(x, w.slot, h, row);
        ml[0] = fmaxf(fmaxf(ms[0][row], ms[1][row]), fmaxf(ms[2][row], ms[3][row]));
        ml[1] = lt;
      }
    }
  }
  __syncthreads();                         // LDS is free for the next tile
  }
}

constexpr int rows_wgs_per_cu(int d, int rt) { return (rt > 16 ? 2 : 1) * d > 128 ? 1 : 2; }

template <int D, int BITS, int RT>
__global__ __launch_bounds__(256, rows_wgs_per_cu(D, RT)) void kv_rows_kernel(AttendArgs x) {
  rows_body<D, BITS, RT>(x, blockIdx.x);
}

// For few tiles: no piece holds parts of two.  A kernel of its own, since the
// second way to find work costs the other 1 %.
template <int D, int BITS, int RT>
__global__ __launch_bounds__(256, rows_wgs_per_cu(D, RT)) void kv_rows_spread_kernel(AttendArgs x) {
  rows_body<D, BITS, RT, true>(x, blockIdx.x);
}

// Two sets of tiles of one height, a short prefix's and the sequences' own:
// one launch of both is 22 -> 17 us for 6 sequences of 40 behind 701 tokens.
// A kernel of its own, since the choice costs the other 4 % of 131072 keys.
template <int D, int BITS, int RT>
__global__ __launch_bounds__(256, rows_wgs_per_cu(D, RT)) void kv_rows_pair_kernel(AttendArgs one, AttendArgs two,
                                                                                  unsigned split) {
  AttendArgs x;
  unsigned block = blockIdx.x;
  if (block < split) {
    x = one;
  } else {
    x = two;
    block -= split;
  }
  rows_body<D, BITS, RT>(x, block);
}

// ------------------------------------------------------------------- join
// out = sum_c 2^(m_c - M) o_c over sum_c 2^(m_c - M) l_c, c the parts of a row.
// All latency: D / 4 lanes hold a row, and a lane group takes its parts in
// batches of 8 (or 4) with all their loads in flight at once.
struct RowSum {
  float M, L;
  f32x4_t acc;
};

__device__ __forceinline__ void join2(RowSum& a, float M2, float L2, const f32x4_t& a2) {
  const float mm = fmaxf(a.M, M2);
  const float f = a.M == -INFINITY ? 0.f : exp2_hw(a.M - mm), f2 = M2 == -INFINITY ? 0.f : exp2_hw(M2 - mm);
  a.L = a.L * f + L2 * f2;
#pragma unroll
  for (int k = 0; k < 4; ++k) a.acc[k] = a.acc[k] * f + a2[k] * f2;
  a.M = mm;
}

// Parts first, first + step, ... below n of one row; at(c): the partials and slot of part c, and the row in it.
template <int D, int BATCH, typename AT>
__device__ __forceinline__ RowSum sum_parts(AT at, int first, int step, int n, int h, int sub) {
  RowSum s{-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
  for (int c0 = first; c0 < n; c0 += step * BATCH) {
    float mc[BATCH], lc[BATCH];
    f32x4_t o[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int c = c0 + i * step;
      mc[i] = -INFINITY;
      lc[i] = 0.f;
      o[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (c < n) {
        const AttendArgs* x;
        int slot, row;
        at(c, x, slot, row);
        const float2 v = *reinterpret_cast<const float2*>(part_ml(*x, slot, h, row));
        mc[i] = v.x;
        lc[i] = v.y;
        o[i] = *reinterpret_cast<const f32x4_t*>(part_o<D>(*x, slot, h, row) + 4 * sub);
      }
    }
    float mb = s.M;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) mb = fmaxf(mb, mc[i]);
    const float f0 = s.M == -INFINITY ? 0.f : exp2_hw(s.M - mb);
    s.L *= f0;
#pragma unroll
    for (int k = 0; k < 4; ++k) s.acc[k] *= f0;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const float f = mc[i] == -INFINITY ? 0.f : exp2_hw(mc[i] - mb);
      s.L += lc[i] * f;                    // a NaN sum (a NaN key was seen) stays one
#pragma unroll
      for (int k = 0; k < 4; ++k) s.acc[k] = __builtin_fmaf(o[i][k], f, s.acc[k]);
    }
    s.M = mb;
  }
  return s;
}

// Joins the lane groups of a wave; every lane then holds the wave's sum.
template <int D>
__device__ __forceinline__ void join_groups(RowSum& s) {
#pragma unroll
  for (int d = D / 4; d < 64; d <<= 1) {
    f32x4_t a2;
#pragma unroll
    for (int k = 0; k < 4; ++k) a2[k] = __shfl_xor(s.acc[k], d);
    join2(s, __shfl_xor(s.M, d), __shfl_xor(s.L, d), a2);
  }
}

template <int D>
__device__ __forceinline__ void store_row(const KvAttend& a, const SeqRows& r, int R, int h, int sub, const RowSum& s) {
  const int tok = R / a.group, g = R - tok * a.group;
  const float inv = s.L == 0.f ? 0.f : 1.0f / s.L;
  f32x4_t v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = s.acc[k] * inv;
  store_out4(a, (int64_t)(r.t0 + tok) * a.o_stride + (int64_t)(h * a.group + g) * D + 4 * sub, v);
}

// The tiles that cuts go through: one workgroup per cut and KV head, the cuts
// of one tile share its rows.  With few parts a lane group joins a row; with
// many (few rows then, one long sequence) all four waves do.
template <int D>
__global__ __launch_bounds__(256) void kv_join_cuts_kernel(AttendArgs x) {
  constexpr int LPR = D / 4, GRP = 64 / LPR;
  __shared__ __align__(16) float os[4][D];
  __shared__ float mls[4][2];
  const KvAttend& a = x.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPR;
  const int h = blockIdx.x % a.c.heads, i = blockIdx.x / a.c.heads + 1;
  const Line line = line_of(x.s, x.rule, lane);
  if (i >= line.N) return;
  TileAt t;
  int i0, parts, slot0;
  if (x.rule.spread) {
    const PartAt p = part_at(x.s, x.rule, line, i, lane);
    if (p.t.b < 0 || p.first == i) return;
    t = p.t;
    i0 = p.first;
    parts = p.parts;
    slot0 = 2 * i0;
  } else {
    const int64_t cut = line.cut(i);
    t = tile_at(x.s, x.rule, cut, lane);
    if (t.b < 0 || t.lo == cut) return;
    i0 = line.piece(t.lo);
    parts = line.piece(t.hi - 1) - i0 + 1;
    slot0 = (int)slot_of(line, t, i0, false);
  }
  if (2 * (i0 + parts) > x.part.slots) return;
  const int row0 = t.tile * x.rule.rt, rows = t.r.count * a.group - row0, n = rows < x.rule.rt ? rows : x.rule.rt;
  // the tile's rows go round the workgroups of its cuts, gridDim.y of them each
  const int k = (i - i0 - 1) * gridDim.y + blockIdx.y, sharers = (parts - 1) * gridDim.y;
  if (parts >= 16) {
    for (int row = k; row < n; row += sharers) {           // workgroup-uniform
      auto at = [&](int c, const AttendArgs*& px, int& slot, int& r) {
        px = &x;
        slot = c == 0 ? slot0 : 2 * (i0 + c);
        r = row;
      };
      RowSum s = sum_parts<D, 8>(at, wave * GRP + lane / LPR, 4 * GRP, parts, h, sub);
      join_groups<D>(s);
      if (lane < LPR) *reinterpret_cast<f32x4_t*>(&os[wave][4 * sub]) = s.acc;
      if (lane == 0) { mls[wave][0] = s.M; mls[wave][1] = s.L; }
      __syncthreads();
      if (wave == 0 && lane < LPR) {
#pragma unroll
        for (int w = 1; w < 4; ++w) join2(s, mls[w][0], mls[w][1], *reinterpret_cast<const f32x4_t*>(&os[w][4 * sub]));
        store_row<D>(a, t.r, row0 + row, h, sub, s);
      }
      __syncthreads();
    }
  } else {                                 // a lane group for each row
    for (int row = (4 * k + wave) * GRP + lane / LPR; row < n; row += 4 * sharers * GRP) {
      auto at = [&](int c, const AttendArgs*& px, int& slot, int& r) {
        px = &x;
        slot = c == 0 ? slot0 : 2 * (i0 + c);
        r = row;
      };
      const RowSum s = sum_parts<D, 4>(at, 0, 1, parts, h, sub);
      store_row<D>(a, t.r, row0 + row, h, sub, s);
    }
  }
}

// Every row's own parts and its prefix's: `rpw` rows of a tile and KV head are
// a unit, a wave takes a row.
template <int D>
__global__ __launch_bounds__(256) void kv_join_prefix_kernel(AttendArgs own, AttendArgs pre, int rpw, int64_t units) {
  constexpr int LPR = D / 4, GRP = 64 / LPR;
  const KvAttend& a = own.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPR;
  const int per_tile = own.rule.rt / rpw;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int h = (int)(unit % a.c.heads);
    const int64_t u = unit / a.c.heads;
    const TileAt t = tile_at<true>(own.s, own.rule, u / per_tile, lane);
    if (t.b < 0) return;
    const int row0 = t.tile * own.rule.rt, rows = t.r.count * a.group;
    const int first = row0 + (int)(u % per_tile) * rpw;
    if (first >= rows) continue;
    const Line line = line_of(own.s, own.rule, lane), pline = pre.line;
    const int i0 = line.piece(t.lo), parts = line.piece(t.hi - 1) - i0 + 1;
    const int slot0 = (int)(i0 + t.index);
    if (slot0 + parts > own.part.slots) continue;
    const int64_t A = (int64_t)(pre.a.prefix_len + pre.rule.ku - 1) / pre.rule.ku * kSub;   // weight of a tile of the prefix
    const int last = first + rpw < rows ? first + rpw : rows;
    for (int R = first + wave; R < last; R += 4) {
      const int64_t P = (int64_t)t.r.t0 * a.group + R;
      const int pt = (int)(P / pre.rule.rt), prow = (int)(P % pre.rule.rt);
      const int p0 = pline.piece(A * pt), np = pline.piece(A * (pt + 1) - 1) - p0 + 1;
      if (p0 + pt + np > pre.part.slots) continue;
      auto at = [&](int c, const AttendArgs*& px, int& slot, int& r) {
        const bool p = c < np;
        px = p ? &pre : &own;
        slot = p ? p0 + pt + c : slot0 + c - np;
        r = p ? prow : R - row0;
      };
      RowSum s = sum_parts<D, 8>(at, lane / LPR, GRP, np + parts, h, sub);
      join_groups<D>(s);
      if (lane < LPR) store_row<D>(a, t.r, R, h, sub, s);
    }
  }
}

// ------------------------------------------------------------------ launch
hipError_t launch_kv_rows(const AttendArgs& x, const AttendArgs* y, int head_dim, int bits, hipStream_t st) {
  const unsigned split = (unsigned)(x.rule.wgs * x.a.c.heads);
  const dim3 grid(split + (y ? (unsigned)(y->rule.wgs * y->a.c.heads) : 0u));
#define ROWS(D, B, R)                                                                                         \
  do {                                                                                                        \
    if (y) hipLaunchKernelGGL((kv_rows_pair_kernel<D, B, R>), grid, dim3(256), 0, st, x, *y, split);          \
    else if (x.rule.spread) hipLaunchKernelGGL((kv_rows_spread_kernel<D, B, R>), grid, dim3(256), 0, st, x);  \
    else hipLaunchKernelGGL((kv_rows_kernel<D, B, R>), grid, dim3(256), 0, st, x);                            \
  } while (0)
#define ROWS_N(D, B)                          \
  do {                                        \
    if (x.rule.rt == 8) ROWS(D, B, 8);        \
    else if (x.rule.rt == 16) ROWS(D, B, 16); \
    else ROWS(D, B, 32);                      \
  } while (0)
  if (head_dim == 128) {
    if (bits == 8) ROWS_N(128, 8);
    else ROWS_N(128, 4);
  } else {
    if (bits == 8) ROWS_N(64, 8);
    else ROWS_N(64, 4);
  }
#undef ROWS_N
#undef ROWS
  return hipGetLastError();
}

namespace {

// Workgroups in all: as many as are resident at once on 256 CUs, two of the
// kernel for few rows (four: 66 -> 78 us for 32 sequences of 8000), one of the
// kernel for tiles of 256 rows, two for those of 128.
constexpr int kRowWorkgroups = 512;
constexpr int kTileWorkgroups = 256;
// Page tables of up to so many positions leave their tiles whole, each with one
// workgroup: a second launch to join parts costs more than an even division
// saves.  8 heads, whole against cut: 1 / 8 sequences of 1000 keys 14.3 / 15.0
// against 15.4 / 18.3 us, 1 / 8 / 24 / 65 of 1500 keys 18.4 / 19.6 / 22 / 56
// against 17.0 / 20.8 / 30 / 52 us.  Tiles of 32 rows take twice as long for a
// key (2 sequences of 1500, 32 rows, 4 bits: 26 against 18 us), so half as many.
constexpr int kWholeKeys = 1536;
// What a tile costs beside its keys, in steps of keys / kSub: one step of the
// kernel for few rows (32 sequences of 8000: 63.4 us with 0 and with 64, 64.7
// with 128), one and a half of the other's 4 us (prompts of 999 .. 2500: 289 us
// with 0, 268 with 64, 266 with 96, 271 with 192).
constexpr int kRowsExtra = 64, kTileExtra = 96;
// Keys are decoded beforehand where at least this many rows of a sequence meet
// them (8 tiles) and the images, sized for full page tables, fit this many
// bytes.  8 heads, with images against without: 4 x 1120 rows on 4000 keys
// 150 against 141 us, 4 x 2048 rows on 4000 keys 211 against 215, 2 x 4096 rows
// on 8000 keys 318 against 343, 8192 rows on 8000 keys 320 against 357.
constexpr int64_t kImageRows = 2048;
constexpr int64_t kImageBytes = (int64_t)1 << 30;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Everything the host decides about one call, from sizes alone.
struct CallPlan {
  SplitRule own, pre;
  int64_t own_slots, pre_slots;      // per KV head
  bool shared, join;
  bool pair;                         // prefix and own keys in one launch
  int64_t images;                    // steps of keys to decode beforehand
  Line pre_line;
  size_t o_own, ml_own, o_pre, ml_pre, image, bytes;
};

// Tile height by the rows a KV head has against one run of keys.  Up to 8 rows
// share a product's 16 columns with their low parts (32 sequences of 8000, 8
// bits: 66 us either way; 4 of 131072, 4 bits: 105 against 112 us).  33 .. 64
// rows cost the same in tiles of 32 and of 128 (16 sequences of 3000, 48 rows:
// 64 us); 96 rows 58 us in tiles of 128 and 66 in tiles of 256, 200 rows 73 us
// in tiles of 256 and 89 in tiles of 128 (8 sequences of 4000).
int tile_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256; }

// The division of tiles of rt rows of `seqs` sequences with at most cap keys each.
SplitRule rule_for(int rt, int64_t total_rows, int64_t seqs, int group, int heads, int cap, bool must_cut,
                   bool keep) {
  SplitRule r{};
  r.group = group;
  r.rt = rt;
  r.ku = 128;
  r.cap = cap;
  r.sloped = r.rt > 32;
  r.whole = !must_cut && cap <= (r.rt <= 16 ? kWholeKeys : r.rt <= 32 ? kWholeKeys / 2 : r.ku);
  r.extra = r.whole || must_cut ? 0 : r.rt <= 32 ? kRowsExtra : kTileExtra;
  const int64_t most = (total_rows / r.rt + seqs) * (r.whole ? 1 : ceil_div(cap > 0 ? cap : 1, r.ku));   // steps of keys, at most
  int64_t n = (r.rt == 256 ? kTileWorkgroups : kRowWorkgroups) / heads;
  r.single = r.whole && n >= most;
  if (n > most) n = most;
  r.wgs = (int)(n < 1 ? 1 : n);
  // Few tiles of few keys, four or more pieces each: a piece with parts of two
  // tiles takes 4 us longer than the others, and pieces of one tile only have up
  // to N / (N - T) of an even share of the keys, which is more where there are
  // many (5 rows of 8 sequences of 200 .. 3001, 4 bits: 25.2 -> 20.4 us; 7 of 3008
  // 26.6 -> 23.9; but 3 of 20000, 15 steps by this count, 35 -> 38).
  const int64_t tiles = total_rows / rt + seqs;
  r.spread = r.rt <= 32 && !r.whole && !must_cut && !keep && tiles * 4 <= r.wgs && tiles * ceil_div(cap, r.ku) <= 6 * r.wgs;
  return r;
}

CallPlan plan_call(int64_t B, int64_t T, int64_t max_pages, int page_shift, int heads, int group, int head_dim,
                   int64_t prefix_len) {
  CallPlan p{};
  const int64_t cap = max_pages << page_shift;
  p.shared = prefix_len > 0;
  int rt = tile_rows(ceil_div(T, B) * group);
  const int pre_rt = tile_rows(T * group);
  p.pair = p.shared && pre_rt <= 32 && cap <= kWholeKeys / 2;
  if (p.pair) rt = pre_rt;
  p.own = rule_for(rt, T * group, B, group, heads, (int)cap, false, p.shared);
  const int64_t tiles = T * group / rt + B;                 // at most, over all sequences
  p.own_slots = p.shared ? p.own.wgs + tiles : 2 * p.own.wgs;
  p.join = p.shared || (!p.own.whole && p.own.wgs > 1);
  if (!p.join) p.own_slots = 0;
  if (p.shared) {
    p.pre = rule_for(pre_rt, T * group, 1, group, heads, (int)prefix_len, true, true);
    p.pre.sloped = false;                                   // every row sees all of it
    p.pre_slots = p.pre.wgs + ceil_div(T * group, pre_rt);
    p.pre_line = Line{ceil_div(T * group, pre_rt) * ceil_div(prefix_len, p.pre.ku) * kSub, p.pre.wgs, 1};
    if (p.pre_line.U / kSub < p.pre_line.N) p.pre_line.N = (int)(p.pre_line.U / kSub);
  }
  if (p.own.rt == 256 && ceil_div(T, B) * group >= kImageRows) {
    p.images = B * ceil_div(cap, 128);
    if (p.images > kImageBytes / (heads * kv_image_bytes(head_dim))) p.images = 0;
  }
  size_t at = 0;
  auto take = [&](int64_t floats) {
    const size_t here = at;
    at += ((size_t)floats * 4 + 255) / 256 * 256;
    return here;
  };
  p.o_own = take(p.own_slots * heads * p.own.rt * head_dim);
  p.ml_own = take(p.own_slots * heads * p.own.rt * 2);
  p.o_pre = take(p.pre_slots * heads * p.pre.rt * head_dim);
  p.ml_pre = take(p.pre_slots * heads * p.pre.rt * 2);
  p.image = take(p.images * heads * kv_image_bytes(head_dim) / 4);
  p.bytes = at > 16 ? at : 16;
  return p;
}

}  // namespace

size_t kv_attend_ws_bytes(int64_t B, int64_t T, int64_t max_pages, int page_shift, int heads, int group, int head_dim,
                          int64_t prefix_len) {
  return plan_call(B, T, max_pages, page_shift, heads, group, head_dim, prefix_len).bytes;
}

hipError_t launch_kv_attend(const KvAttend& a, int head_dim, int bits, void* ws, hipStream_t st) {
  const CallPlan p =
      plan_call(a.s.B, a.s.T, a.s.max_pages, a.c.page_shift, a.c.heads, a.group, head_dim, a.prefix_len);
  char* base = static_cast<char*>(ws);
  auto at = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  const int pre_pages = (a.prefix_len + (1 << a.c.page_shift) - 1) >> a.c.page_shift;
  const SeqView prefix{a.prefix_pages, nullptr, nullptr, 1, a.s.T, pre_pages};
  const AttendArgs own{a, a.s, p.own, Partials{at(p.o_own), at(p.ml_own), (int)p.own_slots}, p.shared, Line{},
                       p.images ? reinterpret_cast<uint8_t*>(base + p.image) : nullptr, p.images};
  const AttendArgs pre{a, prefix, p.pre, Partials{at(p.o_pre), at(p.ml_pre), (int)p.pre_slots}, true, p.pre_line, nullptr, 0};
  hipError_t e;
  auto launch = [&](const AttendArgs& x) {
    return x.rule.rt > 32 ? launch_kv_tiles(x, head_dim, bits, st) : launch_kv_rows(x, nullptr, head_dim, bits, st);
  };
  if (p.pair) {
    if ((e = launch_kv_rows(pre, &own, head_dim, bits, st)) != hipSuccess) return e;
  } else {
    if (p.shared && (e = launch(pre)) != hipSuccess) return e;
    if (own.image && (e = launch_kv_images(own, head_dim, bits, st)) != hipSuccess) return e;
    if ((e = launch(own)) != hipSuccess) return e;
  }
  if (!p.join) return hipSuccess;
  if (p.shared) {
    const int rpw = own.rule.rt <= 32 ? 8 : 16;
    const int64_t tiles = p.own_slots - p.own.wgs;
    const int64_t units = tiles * (own.rule.rt / rpw) * a.c.heads;
    const dim3 grid((unsigned)(units < (1 << 20) ? units : 1 << 20));
    if (head_dim == 128) hipLaunchKernelGGL((kv_join_prefix_kernel<128>), grid, dim3(256), 0, st, own, pre, rpw, units);
    else hipLaunchKernelGGL((kv_join_prefix_kernel<64>), grid, dim3(256), 0, st, own, pre, rpw, units);
  } else {
    const dim3 grid((unsigned)((p.own.wgs - 1) * a.c.heads), (unsigned)ceil_div(own.rule.rt, 64));
    if (head_dim == 128) hipLaunchKernelGGL((kv_join_cuts_kernel<128>), grid, dim3(256), 0, st, own);
    else hipLaunchKernelGGL((kv_join_cuts_kernel<64>), grid, dim3(256), 0, st, own);
  }
  return hipGetLastError();
}

}  // namespace qg
