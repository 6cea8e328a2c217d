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
#include "common.hpp"
#include "kvcache_attend.hpp"

namespace qg {

constexpr float kUp = 0x1p64f, kDown = 0x1p-64f;   // scale of the query and weight operands
constexpr float kCode = 0x1p69f;                   // product of a scaled operand and a code, undone

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// fp16 times fp32 in one instruction (v_fma_mix_f32; a plain product would convert first)
__device__ __forceinline__ float mix_mul(float h, float x) { return __builtin_fmaf(h, x, 0.f); }

// bf16 pair times 2^64
__device__ __forceinline__ uint32_t up_pair(uint32_t w) {
  const float lo = bf16_lo_to_f32(w) * kUp, hi = bf16_hi_to_f32(w) * kUp;
  return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xFFFF0000u);
}

template <typename V>
__device__ __forceinline__ V ld_nt(const uint8_t* base, uint32_t off) {
  return __builtin_nontemporal_load(reinterpret_cast<const V*>(base + off));
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// One workgroup: one item of 16 NT rows.  Its four waves take a quarter of the
// chunk's keys each, 32 keys a step.  Lane l, r = l % 16, kg = l / 16:
//   K operand: key r, a quarter kg of the coordinates, straight from memory
//   logits:    query r, keys 4 kg .. 4 kg + 3 of both halves of the step
//   V operand: coordinates r D/16 .. of exactly those eight keys (the order of
//              the contraction is free), so the weights never leave their lane
// The row constants of a lane's eight keys come with four 16-byte loads.
template <int D, int BITS, int NT>
__global__ __launch_bounds__(256) void kv_rows_kernel(AttendArgs x) {
  constexpr int RT = 16 * NT;
  constexpr int ROWB = D * BITS / 8;       // bytes of a cache row
  constexpr int KB = ROWB / 4;             // bytes of a K row per lane
  constexpr int KW = KB / 4;
  constexpr int VB = ROWB / 16;            // bytes of a V row per lane
  constexpr int VW = VB < 4 ? 1 : VB / 4;
  constexpr int TILES = D / 16, STEPS = D / 32;
  constexpr int PITCH = D + 4;
  __shared__ __align__(16) float os[4][RT][PITCH];
  __shared__ float ms[4][RT], ls[4][RT];
  const KvAttend& a = x.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kg = lane >> 4;
  const int heads = a.c.heads, h = blockIdx.x % heads, item = blockIdx.x / heads;
  const Work w = work_of(x, item, lane);
  if (w.b < 0) return;

  f32x4_t acc[NT][TILES];
  float m[NT], l[NT], po[NT];              // maximum, sum of weights, sum of weights times offsets
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[n][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    m[n] = -INFINITY;
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
    u32x4_t km[2], vm[2];
    int bad;                               // halves whose page is not in the cache
  };
  auto load = [&](int key, Raw& w_) {
    if (((key + 16) >> shift) - pbase >= 64) refill(key >> shift);
    w_.bad = 0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int kk = key + 16 * hf;
      const int id = __builtin_amdgcn_readlane(ids, (kk >> shift) - pbase);
      if (id < 0) w_.bad |= 1 << hf;
      const int64_t row = (((int64_t)(id < 0 ? 0 : id) * heads + h) << shift) + (kk & pmask);
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
      w_.km[hf] = *reinterpret_cast<const u32x4_t*>(a.c.meta[0] + row + 4 * kg);
      w_.vm[hf] = *reinterpret_cast<const u32x4_t*>(a.c.meta[1] + row + 4 * kg);
    }
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
    const int row = w.row0 + 16 * n + r;
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
        v[e] = up_pair(v[e]);
      }
      if constexpr (BITS == 4) {           // pairs (j, j + 4), as a nibble mask leaves them
        const u32x4_t t = v;
        v[0] = __builtin_amdgcn_perm(t[2], t[0], 0x05040100u);
        v[1] = __builtin_amdgcn_perm(t[2], t[0], 0x07060302u);
        v[2] = __builtin_amdgcn_perm(t[3], t[1], 0x05040100u);
        v[3] = __builtin_amdgcn_perm(t[3], t[1], 0x07060302u);
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

  auto compute = [&](int key, const Raw& w_) {
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
          for (int e = 0; e < 4; ++e) f[e] = (w_.k[hf][s] >> (4 * e)) & 0x000F000Fu;
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
        const uint32_t km = w_.km[j / 4][j % 4];
        t[n][j] = __builtin_fmaf(z[n][j / 4][j % 4], mix_mul(f16_lo(km), c1), mix_mul(f16_hi(km), qs[n]));
      }
      if (masked) {
        asm volatile("");                  // a branch: the selects must not run in every step
#pragma unroll
        for (int j = 0; j < 8; ++j) t[n][j] = seen(n, j) ? t[n][j] : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = fmaxf(mx, t[n][j]);
      grow |= mx > m[n] + 8.0f;
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
      }
    }
    u32x4_t wh[NT], wl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float base = m[n] == -INFINITY ? 0.f : m[n] - 64.0f;
      uint32_t vm[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) vm[j] = w_.vm[j / 4][j % 4];
      if (masked) {                        // constants of slots that are not seen may be anything
        asm volatile("");
#pragma unroll
        for (int j = 0; j < 8; ++j) vm[j] = seen(n, j) ? vm[j] : 0u;
      }
      float wv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = exp2_hw(t[n][j] - base);   // 2^64 times the weight
        wv[j] = mix_mul(f16_lo(vm[j]), p);
        po[n] = __builtin_fmaf(f16_hi(vm[j]), p, po[n]);
        l[n] += p;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        wh[n][e] = cvt_pk_bf16(wv[2 * e], wv[2 * e + 1]);
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
          f[e] = (pair[e] >> (4 * (q % 4))) & 0x000F000Fu;
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[n][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f),
                                                            __builtin_bit_cast(bf16x8_t, wh[n]), acc[n][q], 0, 0, 0);
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
    if (kg == 0) ms[wave][16 * n + r] = m[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
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
        for (int e = 0; e < 4; ++e) v[e] = (acc[n][q + e][i] * kCode + po[n] * kDown) * f;
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
}

// ------------------------------------------------------------------- join
// out = sum_c 2^(m_c - M) o_c over sum_c 2^(m_c - M) l_c, c the chunks of the
// prefix (if any) and of the row's own keys.  All latency: D / 4 lanes hold a
// row, and a lane group takes its chunks in batches of 8 with all their loads
// in flight at once.  WAVES waves work on one (row, query head): 4 where there
// are few rows, each with many chunks, 1 where there are many.
template <int D, int WAVES>
__global__ __launch_bounds__(256) void kv_join_kernel(AttendArgs own, AttendArgs pre) {
  constexpr int LPR = D / 4, GRP = 64 * WAVES / LPR, BATCH = 8;
  __shared__ __align__(16) float os[WAVES][D];
  __shared__ float mls[WAVES][2];
  const KvAttend& a = own.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cu = split_units(a.s, own.rule, lane);
  if (!own.shared && cu == kNoSplit) return;
  const int Hq = a.c.heads * a.group;
  const int grp = (WAVES == 4 ? threadIdx.x : lane) / LPR, sub = lane % LPR;
  const int64_t step = (int64_t)gridDim.x * (4 / WAVES);
  for (int64_t idx = (int64_t)blockIdx.x * (4 / WAVES) + (WAVES == 4 ? 0 : wave); idx < (int64_t)a.s.T * Hq; idx += step) {
    // uniform over the WAVES waves of the row
    const int t = (int)(idx / Hq), hq = (int)(idx % Hq), h = hq / a.group, g = hq - h * a.group;
    int b = t;
    if (a.s.starts) b = find_seq<64>(a.s.starts, a.s.B, t, lane, lane);
    const SeqRows r = seq_rows(a.s, b, own.rule.cap);
    if (t < r.t0 || t >= r.t0 + r.count) continue;
    const int chunks = chunks_of(own.rule, r, cu);
    if (!own.shared && chunks == 1) continue;
    const int R = (t - r.t0) * a.group + g;
    const int slot = items_before(a.s, own.rule, cu, b, lane) + R / own.rule.rt * chunks, row = R % own.rule.rt;
    if (slot + chunks > own.part.slots) continue;
    const int P = t * a.group + g, np = own.shared ? pre.prefix_chunks : 0;
    const int pslot = own.shared ? P / pre.rule.rt * np : 0, prow = own.shared ? P % pre.rule.rt : 0;
    const int n = np + chunks;
    float M = -INFINITY, L = 0.f;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = grp; c0 < n; c0 += GRP * BATCH) {
      float mc[BATCH], lc[BATCH];
      f32x4_t o[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int c = c0 + i * GRP;
        mc[i] = -INFINITY;
        lc[i] = 0.f;
        o[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (c < n) {
          const bool p = c < np;
          const float* ml = p ? part_ml(pre, pslot + c, h, prow) : part_ml(own, slot + c - np, h, row);
          const float* src = p ? part_o<D>(pre, pslot + c, h, prow) : part_o<D>(own, slot + c - np, h, row);
          const float2 v = *reinterpret_cast<const float2*>(ml);
          mc[i] = v.x;
          lc[i] = v.y;
          o[i] = *reinterpret_cast<const f32x4_t*>(src + 4 * sub);
        }
      }
      float mb = M;
#pragma unroll
      for (int i = 0; i < BATCH; ++i) mb = fmaxf(mb, mc[i]);
      const float f0 = M == -INFINITY ? 0.f : exp2_hw(M - mb);
      L *= f0;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] *= f0;
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float f = mc[i] == -INFINITY ? 0.f : exp2_hw(mc[i] - mb);
        L += lc[i] * f;                    // a NaN sum (a NaN key was seen) stays one
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(o[i][k], f, acc[k]);
      }
      M = mb;
    }
    // the groups of the wave, then the waves
    auto join2 = [&](float M2, float L2, const f32x4_t& a2) {
      const float mm = fmaxf(M, M2);
      const float f = M == -INFINITY ? 0.f : exp2_hw(M - mm), f2 = M2 == -INFINITY ? 0.f : exp2_hw(M2 - mm);
      L = L * f + L2 * f2;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = acc[k] * f + a2[k] * f2;
      M = mm;
    };
#pragma unroll
    for (int d = LPR; d < 64; d <<= 1) {
      f32x4_t a2;
#pragma unroll
      for (int k = 0; k < 4; ++k) a2[k] = __shfl_xor(acc[k], d);
      join2(__shfl_xor(M, d), __shfl_xor(L, d), a2);
    }
    if constexpr (WAVES > 1) {
      if (lane < LPR) *reinterpret_cast<f32x4_t*>(&os[wave][4 * sub]) = acc;
      if (lane == 0) { mls[wave][0] = M; mls[wave][1] = L; }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int w2 = 1; w2 < WAVES; ++w2)
          join2(mls[w2][0], mls[w2][1], *reinterpret_cast<const f32x4_t*>(&os[w2][4 * sub]));
      }
      __syncthreads();
    }
    if (lane < LPR && (WAVES == 1 || wave == 0)) {
      const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] *= inv;
      store_out4(a, (int64_t)t * a.o_stride + (int64_t)hq * D + 4 * sub, acc);
    }
  }
}

// ------------------------------------------------------------------ launch
hipError_t launch_kv_rows(const AttendArgs& x, int head_dim, int bits, int64_t items, hipStream_t st) {
  const dim3 grid((unsigned)(items * x.a.c.heads));
#define ROWS(D, B, N) hipLaunchKernelGGL((kv_rows_kernel<D, B, N>), grid, dim3(256), 0, st, x)
#define ROWS_N(D, B)                   \
  do {                                 \
    if (x.rule.rt == 16) ROWS(D, B, 1); \
    else ROWS(D, B, 2);                \
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

constexpr int kWorkgroups = 1024;   // items aimed at in all: 4 workgroups of 4 waves for each of 256 CUs
constexpr int kTileWorkgroups = 512;
constexpr int kJoinGrid = 4096;      // workgroups of the join at most; each takes rows in turn
constexpr int kJoinFew = 1024;       // rows up to which a whole workgroup joins one row

// How one call is cut: everything the host decides, from sizes alone.
struct CallPlan {
  SplitRule own, pre;
  int pre_cu, pre_chunks;
  int64_t own_items, own_slots, pre_items;   // per KV head
  bool shared, join;
  size_t o_own, ml_own, o_pre, ml_pre, bytes;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tile height and splitting by the rows a KV head has against one run of keys.
SplitRule rule_for(int64_t rows, int group, int heads, int cap) {
  const bool tiles = rows > 32;
  const int wgs = tiles ? kTileWorkgroups : kWorkgroups;
  return SplitRule{group, rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256, 128,
                   wgs / heads > 1 ? wgs / heads : 1, 1, cap};
}

CallPlan plan_call(int64_t B, int64_t T, int64_t max_pages, int page_shift, int heads, int group, int head_dim,
                   int64_t prefix_len) {
  CallPlan p{};
  const int64_t cap = max_pages << page_shift;
  const int64_t rows = ceil_div(T, B) * group;            // of one sequence, on average
  p.own = rule_for(rows, group, heads, (int)cap);
  const int64_t tiles = T * group / p.own.rt + B;         // at most, over all sequences
  const int64_t most_chunks = ceil_div(ceil_div(cap, p.own.ku), p.own.min_units);
  p.shared = prefix_len > 0;
  const int target = p.own.target;
  p.own_items = most_chunks == 1 ? tiles : tiles + target + 8;
  if (tiles * most_chunks < p.own_items) p.own_items = tiles * most_chunks;
  // a launch with `target` tiles or more splits nothing
  p.own_slots = p.own_items < 2 * target + 8 ? p.own_items : 2 * target + 8;
  if (p.shared) p.own_slots = p.own_items;
  else if (most_chunks == 1) p.own_slots = 0;
  p.join = p.shared || p.own_slots > 0;
  if (p.shared) {
    p.pre = rule_for(T * group, group, heads, 0);
    const int64_t pt = ceil_div(T * group, p.pre.rt), units = ceil_div(prefix_len, p.pre.ku);
    int64_t cu = ceil_div(pt * units, p.pre.target);
    if (cu < p.pre.min_units) cu = p.pre.min_units;
    if (cu > units) cu = units;
    p.pre_cu = (int)cu;
    p.pre_chunks = (int)ceil_div(units, cu);
    p.pre_items = pt * p.pre_chunks;
  }
  size_t at = 0;
  auto take = [&](int64_t floats) {
    const size_t here = at;
    at += ((size_t)floats * 4 + 255) / 256 * 256;
    return here;
  };
  p.o_own = take(p.own_slots * heads * p.own.rt * head_dim);
  p.ml_own = take(p.own_slots * heads * p.own.rt * 2);
  p.o_pre = take(p.pre_items * heads * p.pre.rt * head_dim);
  p.ml_pre = take(p.pre_items * heads * p.pre.rt * 2);
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
  AttendArgs own{a, p.own, Partials{at(p.o_own), at(p.ml_own), (int)p.own_slots}, p.shared, false, 0, 0};
  AttendArgs pre{a, p.pre, Partials{at(p.o_pre), at(p.ml_pre), (int)p.pre_items}, true, true, p.pre_cu, p.pre_chunks};
  hipError_t e;
  auto launch = [&](const AttendArgs& x, int64_t items) {
    return x.rule.rt > 32 ? launch_kv_tiles(x, head_dim, bits, items, st) : launch_kv_rows(x, head_dim, bits, items, st);
  };
  if (p.shared && (e = launch(pre, p.pre_items)) != hipSuccess) return e;
  if ((e = launch(own, p.own_items)) != hipSuccess) return e;
  if (!p.join) return hipSuccess;
  const int64_t rows = (int64_t)a.s.T * a.c.heads * a.group;
  const bool few = rows <= kJoinFew;
  const int64_t wgs = few ? rows : ceil_div(rows, 4);
  const dim3 grid((unsigned)(wgs < kJoinGrid ? wgs : kJoinGrid));
  if (head_dim == 128) {
    if (few) hipLaunchKernelGGL((kv_join_kernel<128, 4>), grid, dim3(256), 0, st, own, pre);
    else hipLaunchKernelGGL((kv_join_kernel<128, 1>), grid, dim3(256), 0, st, own, pre);
  } else {
    if (few) hipLaunchKernelGGL((kv_join_kernel<64, 4>), grid, dim3(256), 0, st, own, pre);
    else hipLaunchKernelGGL((kv_join_kernel<64, 1>), grid, dim3(256), 0, st, own, pre);
  }
  return hipGetLastError();
}

}  // namespace qg
