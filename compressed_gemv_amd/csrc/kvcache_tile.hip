// Attention over the quantized, paged KV cache with many rows per KV head: a
// chunk or a whole prompt, or a batch in front of a shared prefix.
//
// Bound by the matrix cores and, next to them, by the softmax's vector work,
// so a cached row is decoded once per workgroup and used by all its rows:
// codes become fp16 values s q + o in LDS (one rounding to 11 bits; s and o are
// multiples of 2^-24 below fp16's normal range, so small rows stay exact), keys
// row by row, values transposed.  fp16 and not bf16 for values and weights: the
// roundings of both then stay an eighth of the output's own.
#include "common.hpp"
#include "kvcache_attend.hpp"

namespace qg {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t pk_add(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, a) + __builtin_bit_cast(f16x2_t, b));
}
__device__ __forceinline__ uint32_t pk_fma(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, a), __builtin_bit_cast(f16x2_t, b),
                                                                __builtin_bit_cast(f16x2_t, c)));
}
__device__ __forceinline__ uint32_t cvt_pk_f16(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

constexpr uint32_t k1024 = 0x64006400u, kM1024 = 0xE400E400u;   // fp16 pairs 1024, -1024

// 16-byte chunk c of row `row` in a tile whose rows hold CH chunks, swizzled so
// that 16 neighbouring rows' reads of one chunk cover all banks.
template <int CH>
__device__ __forceinline__ int k_at(int row, int c) {
  return row * CH + (CH == 16 ? c ^ (row & 15) : c ^ ((row >> 1) & 7));
}
__device__ __forceinline__ int v_at(int dim, int c) { return dim * 8 + (c ^ (((dim >> 1) ^ (dim >> 3)) & 7)); }

}  // namespace

// A workgroup: RT = 128 RB rows, each wave 32 RB of them; 64 keys a step, two
// LDS buffers, one barrier a step.  Waves 0 and 1 decode the keys, 2 and 3 the
// values of the next step.  S^T = K Q^T on 32x32x16 products puts a row's
// logits of 16 keys into one lane; the weights go back in as the other operand
// of O^T = V^T P^T without leaving the lane, because V's columns are stored in
// the order in which the lanes hold them.
template <int D, int BITS, int RB>
__global__ __launch_bounds__(256) void kv_tile_kernel(AttendArgs x) {
  constexpr int ROWB = D * BITS / 8;
  constexpr int CH = D / 8;                // 16-byte chunks of a decoded key
  constexpr int STEPS = D / 16, DT = D / 32;
  constexpr int KL = ROWB / 2 / 16;        // 16-byte loads per K thread (half a row)
  constexpr int VB = ROWB / 16;            // bytes of a value row per V thread
  constexpr int VW = VB < 4 ? 1 : VB / 4;
  constexpr int DPT = D / 16;              // coordinates per V thread
  constexpr int CW = 4 * KL > 8 * VW ? 4 * KL : 8 * VW;
  __shared__ __align__(16) u32x4_t ksh[2][64 * CH];
  __shared__ __align__(16) u32x4_t vsh[2][D * 8];
  __shared__ uint32_t gone[2][4];          // per 16 keys: not in the cache
  const KvAttend& a = x.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hh = lane >> 5;
  const int heads = a.c.heads, h = blockIdx.x % heads, item = blockIdx.x / heads;
  const Work w = work_of(x, item, lane);
  if (w.b < 0) return;

  // queries: rows scaled by a power of two to a largest value in [1, 2) (exact
  // up to 2^-25 of it), what each row sees, and the factor back
  f16x8_t qf[RB][STEPS];
  float cq[RB];
  int lim[RB], limmin = w.k1, limmax = 0;
  const float c0 = fabsf(a.scale) * 1.4426950408889634f;
#pragma unroll
  for (int n = 0; n < RB; ++n) {
    const int row = w.row0 + (wave * RB + n) * 32 + col;
    const bool ok = row < w.rows;
    const int tok = ok ? row / a.group : 0, g = ok ? row - tok * a.group : 0;
    const uint16_t* q = a.Q + (int64_t)(w.t0 + tok) * a.q_stride + (int64_t)(h * a.group + g) * D;
    u32x4_t raw[STEPS];
    uint32_t big = 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      raw[s] = u32x4_t{0u, 0u, 0u, 0u};
      if (ok) raw[s] = *reinterpret_cast<const u32x4_t*>(q + 16 * s + 8 * hh);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = raw[s][e] & 0x7F80u, hi = (raw[s][e] >> 16) & 0x7F80u;
        big = lo > big ? lo : big;
        big = hi > big ? hi : big;
      }
    }
    const uint32_t other = (uint32_t)__shfl_xor((int)big, 32);
    big = other > big ? other : big;
    int ex = (int)(big >> 7) - 127;
    ex = ex < -126 ? -126 : (ex > 126 ? 126 : ex);
    const float down = ldexpf(a.scale < 0.f ? -1.f : 1.f, -ex);
    cq[n] = ldexpf(c0, ex);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      u32x4_t v;
      if constexpr (BITS == 4) {           // pairs (j, j + 4), as a nibble mask leaves the keys
        const u32x4_t t = raw[s];
        raw[s][0] = __builtin_amdgcn_perm(t[2], t[0], 0x05040100u);
        raw[s][1] = __builtin_amdgcn_perm(t[2], t[0], 0x07060302u);
        raw[s][2] = __builtin_amdgcn_perm(t[3], t[1], 0x05040100u);
        raw[s][3] = __builtin_amdgcn_perm(t[3], t[1], 0x07060302u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = cvt_pk_f16(bf16_lo_to_f32(raw[s][e]) * down, bf16_hi_to_f32(raw[s][e]) * down);
      qf[n][s] = __builtin_bit_cast(f16x8_t, v);
    }
    lim[n] = ok ? row_sees(w, tok) : w.k1;
    int lo = lim[n], hi = ok ? lim[n] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_xor(lo, d), v = __shfl_xor(hi, d);
      lo = u < lo ? u : lo;
      hi = v > hi ? v : hi;
    }
    limmin = lo < limmin ? lo : limmin;
    limmax = hi > limmax ? hi : limmax;
  }
  limmin = __builtin_amdgcn_readfirstlane(limmin);
  limmax = __builtin_amdgcn_readfirstlane(limmax);

  f32x16_t acc[RB][DT];
  float m[RB], l[RB];
#pragma unroll
  for (int n = 0; n < RB; ++n) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][t][i] = 0.f;
    m[n] = -INFINITY;
    l[n] = 0.f;
  }

  // ---- what this thread decodes: half a key row, or 8 values of DPT coordinates
  const bool is_k = wave < 2;
  const int dt = tid & 127;
  const int kkey = dt >> 1, khalf = dt & 1;
  const int vchunk = dt >> 4, vdim = (dt & 15) * DPT;
  const int vkey = 16 * (vchunk >> 1) + 4 * (vchunk & 1);   // keys vkey .. + 3 and vkey + 8 .. + 3
  const int mykey = is_k ? kkey : vkey;
  const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
  auto page_of = [&](int key0) -> int {    // page of this thread's keys of the step at key0
    const int key = key0 + (is_k ? kkey : vkey & ~15);
    if (key >= w.k1 || (key >> shift) >= w.max_pages) return -1;
    const int id = w.pages[key >> shift];
    return id < a.c.n_pages ? id : -1;
  };
  struct Codes {
    uint32_t c[CW];
    uint32_t meta[8];                      // K: own key's constants of K and V; V: those of the 8 keys
    int page;
  };
  auto load = [&](int key0, int page, Codes& r) {
    r.page = page;
    const int64_t row = (((int64_t)(page < 0 ? 0 : page) * heads + h) << shift) + ((key0 + mykey) & pmask);
    if (is_k) {
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(a.c.codes[0] + row * ROWB + khalf * (ROWB / 2));
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const u32x4_t v = p[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) r.c[4 * i + e] = v[e];
      }
      r.meta[0] = a.c.meta[0][row];
      r.meta[1] = a.c.meta[1][row];
    } else {
      const uint8_t* p = a.c.codes[1] + row * ROWB + vdim * BITS / 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t* pj = p + ((j & 3) + 8 * (j >> 2)) * ROWB;
        if constexpr (VB == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(pj);
          r.c[2 * j] = v.x;
          r.c[(2 * j + 1) % CW] = v.y;
        } else if constexpr (VB == 4) {
          r.c[j] = *reinterpret_cast<const uint32_t*>(pj);
        } else {
          r.c[j] = *reinterpret_cast<const uint16_t*>(pj);
        }
      }
      const u32x4_t m0 = *reinterpret_cast<const u32x4_t*>(a.c.meta[1] + row), m1 = *reinterpret_cast<const u32x4_t*>(a.c.meta[1] + row + 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) { r.meta[e] = m0[e]; r.meta[4 + e] = m1[e]; }
    }
  };
  // A value row that is NaN is decoded as zeros and makes its key NaN instead,
  // so it reaches exactly the rows whose mask lets them see it; constants of
  // keys that no row sees become zero.
  auto nan_meta = [](uint32_t mt) { return (mt & 0x7C00u) == 0x7C00u; };
  auto decode = [&](int key0, const Codes& r, int buf) {
    if (is_k) {
      uint32_t mt = r.page < 0 || key0 + kkey >= w.k1 ? 0u : (nan_meta(r.meta[1]) ? 0x7E007E00u : r.meta[0]);
      const uint32_t s2 = __builtin_amdgcn_perm(mt, mt, 0x01000100u), o2 = __builtin_amdgcn_perm(mt, mt, 0x03020302u);
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        u32x4_t v;
        if constexpr (BITS == 8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            v[2 * e] = __builtin_amdgcn_perm(k1024, r.c[2 * i + e], 0x05010500u);
            v[2 * e + 1] = __builtin_amdgcn_perm(k1024, r.c[2 * i + e], 0x05030502u);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = ((r.c[i] >> (4 * e)) & 0x000F000Fu) | k1024;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pk_fma(pk_add(v[e], kM1024), s2, o2);
        ksh[buf][k_at<CH>(kkey, khalf * (CH / 2) + i)] = v;
      }
      if (khalf == 0 && (kkey & 15) == 0) gone[buf][kkey >> 4] = r.page < 0 ? 1u : 0u;
    } else {
      uint32_t s2[4], o2[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t mt[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 2 * p + e;
          const uint32_t t = r.meta[j];
          mt[e] = r.page < 0 || key0 + vkey + (j & 3) + 8 * (j >> 2) >= w.k1 || nan_meta(t) ? 0u : t;
        }
        s2[p] = __builtin_amdgcn_perm(mt[1], mt[0], 0x05040100u);
        o2[p] = __builtin_amdgcn_perm(mt[1], mt[0], 0x07060302u);
      }
      uint32_t half[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int d = 0; d < DPT; ++d) {
        u32x4_t v;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint32_t u;
          if constexpr (BITS == 8) {
            const uint32_t sel = (uint32_t)(d % 4) | 0x0C000C00u | ((4u + d % 4) << 16);
            u = __builtin_amdgcn_perm(r.c[(2 * p + 1) * VW + d / 4], r.c[2 * p * VW + d / 4], sel);
          } else {
            if (d % 4 == 0) half[p] = __builtin_amdgcn_perm(r.c[2 * p + 1], r.c[2 * p], d == 0 ? 0x05040100u : 0x07060302u);
            u = (half[p] >> (4 * (d % 4))) & 0x000F000Fu;
          }
          v[p] = pk_fma(pk_add(u | k1024, kM1024), s2[p], o2[p]);
        }
        vsh[buf][v_at(vdim + d, vchunk)] = v;
      }
    }
  };

  auto compute = [&](int key0, int buf) {
    const uint32_t holes = gone[buf][0] | (gone[buf][1] << 1) | (gone[buf][2] << 2) | (gone[buf][3] << 3);
    const bool masked = key0 + 64 > limmin || __builtin_amdgcn_readfirstlane(holes) != 0u;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x16_t z[RB];
#pragma unroll
      for (int n = 0; n < RB; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) z[n][i] = 0.f;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const f16x8_t kf = __builtin_bit_cast(f16x8_t, ksh[buf][k_at<CH>(32 * kb + col, 2 * s + hh)]);
#pragma unroll
        for (int n = 0; n < RB; ++n) z[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[n][s], z[n], 0, 0, 0);
      }
      if (masked) {
#pragma unroll
        for (int n = 0; n < RB; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int k = 32 * kb + 8 * (i / 4) + 4 * hh + i % 4;
            const bool vis = key0 + k < lim[n] && !((holes >> (k >> 4)) & 1u);
            z[n][i] = vis ? z[n][i] : -INFINITY;
          }
      }
      bool grow = false;
      float mx[RB];
#pragma unroll
      for (int n = 0; n < RB; ++n) {
        float v = z[n][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) v = fmaxf(v, z[n][i]);
        mx[n] = v == -INFINITY ? v : v * cq[n];          // a scale of 0 must not turn -inf into NaN
        grow |= mx[n] > m[n] + 8.0f;
      }
      if (__ballot(grow)) {                // the maximum may lag by 8, as in the kernel for few rows
#pragma unroll
        for (int n = 0; n < RB; ++n) {
          float v = fmaxf(mx[n], __shfl_xor(mx[n], 32));
          v = fmaxf(v, m[n]);
          const float f = v == m[n] ? 1.0f : __builtin_amdgcn_exp2f(m[n] - v);
          m[n] = v;
          l[n] *= f;
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[n][t][i] *= f;
        }
      }
      u32x4_t p[RB][2];
#pragma unroll
      for (int n = 0; n < RB; ++n) {
        const float base = m[n] == -INFINITY ? 0.f : m[n];
        float pv[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          pv[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[n][i], cq[n], -base));
          if (masked) pv[i] = z[n][i] == -INFINITY ? 0.f : pv[i];
          l[n] += pv[i];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) p[n][e / 4][e % 4] = cvt_pk_f16(pv[2 * e], pv[2 * e + 1]);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          const f16x8_t vf = __builtin_bit_cast(f16x8_t, vsh[buf][v_at(32 * t + col, 4 * kb + 2 * s + hh)]);
#pragma unroll
          for (int n = 0; n < RB; ++n)
            acc[n][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, __builtin_bit_cast(f16x8_t, p[n][s]), acc[n][t], 0, 0, 0);
        }
    }
  };

  if (w.k0 < w.k1) {                       // workgroup-uniform
    Codes r;
    load(w.k0, page_of(w.k0), r);
    int next = page_of(w.k0 + 64);
    decode(w.k0, r, 0);
    __syncthreads();
    int buf = 0;
    for (int key = w.k0; key < w.k1; key += 64) {
      const bool more = key + 64 < w.k1;
      if (more) {
        load(key + 64, next, r);
        next = page_of(key + 128);
      }
      if (key < limmax) compute(key, buf);
      if (more) decode(key + 64, r, buf ^ 1);
      __syncthreads();
      buf ^= 1;
    }
  }

  // lane (col, hh) holds coordinates 32 t + 8 (i / 4) + 4 hh + i % 4 of its rows
#pragma unroll
  for (int n = 0; n < RB; ++n) {
    l[n] += __shfl_xor(l[n], 32);
    const int trow = (wave * RB + n) * 32 + col, row = w.row0 + trow;
    if (row >= w.rows) continue;
    if (w.direct) {
      const int tok = row / a.group, g = row - tok * a.group;
      const float inv = l[n] == 0.f ? 0.f : 1.0f / l[n];
      const int64_t at = (int64_t)(w.t0 + tok) * a.o_stride + (int64_t)(h * a.group + g) * D + 4 * hh;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f32x4_t v;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = acc[n][t][4 * e + i] * inv;
          store_out4(a, at + 32 * t + 8 * e, v);
        }
    } else {
      float* o = part_o<D>(x, w.slot, h, trow) + 4 * hh;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f32x4_t v;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = acc[n][t][4 * e + i];
          *reinterpret_cast<f32x4_t*>(o + 32 * t + 8 * e) = v;
        }
      if (hh == 0) {
        float* ml = part_ml(x, w.slot, h, trow);
        ml[0] = m[n];
        ml[1] = l[n];
      }
    }
  }
}

hipError_t launch_kv_tiles(const AttendArgs& x, int head_dim, int bits, int64_t items, hipStream_t st) {
  const dim3 grid((unsigned)(items * x.a.c.heads));
#define TILE(D, B, N) hipLaunchKernelGGL((kv_tile_kernel<D, B, N>), grid, dim3(256), 0, st, x)
#define TILE_N(D, B)                     \
  do {                                   \
    if (x.rule.rt == 128) TILE(D, B, 1); \
    else TILE(D, B, 2);                  \
  } while (0)
  if (head_dim == 128) {
    if (bits == 8) TILE_N(128, 8);
    else TILE_N(128, 4);
  } else {
    if (bits == 8) TILE_N(64, 8);
    else TILE_N(64, 4);
  }
#undef TILE_N
#undef TILE
  return hipGetLastError();
}

}  // namespace qg
