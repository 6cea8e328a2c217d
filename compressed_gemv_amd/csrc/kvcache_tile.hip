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

}  // namespace

// A workgroup: NW waves of 32 rows; 16 NW keys a step, two LDS buffers, one
// barrier a step.  The first half of the waves decode the keys of the next
// step, the others its values.  S^T = K Q^T on 32x32x16 products puts a row's
// logits of 16 keys into one lane; the weights go back in as the other operand
// of O^T = V^T P^T without leaving the lane, because V's columns are stored in
// the order in which the lanes hold them.  LDS rows are padded by 16 bytes: 16
// neighbouring rows then cover all banks, and every address of the inner loop
// is one register plus a constant.  Coordinate DPT g + q of V lies in row
// 16 q + g, so that the lanes that write it (q fixed) write neighbouring rows.
template <int D, int BITS, int NW>
__global__ __launch_bounds__(64 * NW, 2) void kv_tile_kernel(AttendArgs x) {
  constexpr int KT = 16 * NW;              // keys per step
  constexpr int ROWB = D * BITS / 8;
  constexpr int STEPS = D / 16, DT = D / 32;
  constexpr int KP = D * 2 + 16, VP = KT * 2 + 16;   // pitch of a key's and of a coordinate's LDS row
  constexpr int KBUF = KT * KP, VBUF = D * VP;
  constexpr int KL = ROWB / 2 / 16;        // 16-byte loads per K thread (half a row)
  constexpr int VB = ROWB / 16;            // bytes of a value row per V thread
  constexpr int VW = VB < 4 ? 1 : VB / 4;
  constexpr int DPT = D / 16;              // coordinates per V thread
  constexpr int CW = 4 * KL > 8 * VW ? 4 * KL : 8 * VW;
  __shared__ __align__(16) uint8_t ksh[2 * KBUF];
  __shared__ __align__(16) uint8_t vsh[2 * VBUF];
  __shared__ uint32_t gone[2][NW];         // per 16 keys: 1 << (their place) where they are not in the cache
  const KvAttend& a = x.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hh = lane >> 5;
  const int heads = a.c.heads, h = blockIdx.x % heads, item = blockIdx.x / heads;
  const Work w = work_of(x, item, lane);
  if (w.b < 0) return;

  // queries: rows scaled by a power of two to a largest value in [1, 2) (exact
  // up to 2^-25 of it), what each row sees, and the factor back
  f16x8_t qf[STEPS];
  const float c0 = fabsf(a.scale) * 1.4426950408889634f;
  const int trow = wave * 32 + col, row = w.row0 + trow;
  const bool ok = row < w.rows;
  const int tok = ok ? row / a.group : 0, g = ok ? row - tok * a.group : 0;
  float cq;
  {
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
    cq = fmaxf(ldexpf(c0, ex), 1e-37f);    // positive also for a scale of 0: -inf times it stays -inf
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
      qf[s] = __builtin_bit_cast(f16x8_t, v);
    }
  }
  const int lim = ok ? row_sees(w, tok) : w.k1;
  int limmin = lim, limmax = ok ? lim : 0; // over the wave's rows
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_xor(limmin, d), v = __shfl_xor(limmax, d);
    limmin = u < limmin ? u : limmin;
    limmax = v > limmax ? v : limmax;
  }
  limmin = __builtin_amdgcn_readfirstlane(limmin);
  limmax = __builtin_amdgcn_readfirstlane(limmax);

  f32x16_t acc[DT];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;

  // ---- what this thread decodes: half a key row, or 8 values of DPT coordinates
  const bool is_k = wave < NW / 2;
  const int dt = tid & (32 * NW - 1);
  const int kkey = dt >> 1, khalf = dt & 1;
  const int vchunk = dt >> 4;              // 8 keys
  const int vkey = 16 * (vchunk >> 1) + 4 * (vchunk & 1);   // keys vkey .. + 3 and vkey + 8 .. + 3
  const int mykey = is_k ? kkey : vkey;
  const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
  // byte offsets inside a page: this head's rows, this thread's part of a row
  const uint32_t page_rows = (uint32_t)heads << shift;
  const uint32_t head_row = (uint32_t)h << shift;
  const uint32_t my_off = is_k ? khalf * (ROWB / 2) : (dt & 15) * VB;
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
    const uint32_t in_page = head_row + ((uint32_t)(key0 + mykey) & (uint32_t)pmask);
    const uint64_t prow = (uint64_t)(uint32_t)(page < 0 ? 0 : page) * page_rows + in_page;
    if (is_k) {
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(a.c.codes[0] + prow * ROWB + my_off);
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const u32x4_t v = p[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) r.c[4 * i + e] = v[e];
      }
      r.meta[0] = a.c.meta[0][prow];
      r.meta[1] = a.c.meta[1][prow];
    } else {
      const uint8_t* p = a.c.codes[1] + prow * ROWB + my_off;
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
      const uint32_t* mp = a.c.meta[1] + prow;
      const u32x4_t m0 = *reinterpret_cast<const u32x4_t*>(mp), m1 = *reinterpret_cast<const u32x4_t*>(mp + 8);
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
      for (int i = 0; i < D / 16; ++i) {
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
        *reinterpret_cast<u32x4_t*>(ksh + buf * KBUF + kkey * KP + khalf * D + i * 16) = v;
      }
      if (khalf == 0 && (kkey & 15) == 0) gone[buf][kkey >> 4] = r.page < 0 ? 1u << (kkey >> 4) : 0u;
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
      uint8_t* vout = vsh + buf * VBUF + (dt & 15) * VP + vchunk * 16;
#pragma unroll
      for (int d = 0; d < DPT; ++d) {
        u32x4_t v;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint32_t u;
          if constexpr (BITS == 8) {       // two coordinates of both keys, then one with the exponent of 1024
            if (d % 2 == 0)
              half[p] = __builtin_amdgcn_perm(r.c[(2 * p + 1) * VW + d / 4], r.c[2 * p * VW + d / 4],
                                              d % 4 == 0 ? 0x05010400u : 0x07030602u);
            u = __builtin_amdgcn_perm(k1024, half[p], d % 2 == 0 ? 0x05010500u : 0x05030502u);
          } else {
            if (d % 4 == 0) half[p] = __builtin_amdgcn_perm(r.c[2 * p + 1], r.c[2 * p], d == 0 ? 0x05040100u : 0x07060302u);
            u = ((half[p] >> (4 * (d % 4))) & 0x000F000Fu) | k1024;
          }
          v[p] = pk_fma(pk_add(u, kM1024), s2[p], o2[p]);
        }
        *reinterpret_cast<u32x4_t*>(vout + 16 * d * VP) = v;
      }
    }
  };

  const uint8_t* kread = ksh + col * KP + hh * 16;
  const uint8_t* vread = vsh + col * VP + hh * 16;
  auto compute = [&](int key0, int buf, uint32_t holes) {
    const bool masked = key0 + KT > limmin || holes;
    const uint8_t* kp = kread + buf * KBUF;
    const uint8_t* vp = vread + buf * VBUF;
    f16x8_t kf[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) kf[s] = *reinterpret_cast<const f16x8_t*>(kp + s * 32);
#pragma unroll
    for (int kb = 0; kb < KT / 32; ++kb) {
      f32x16_t z;
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = 0.f;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) z = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[s], qf[s], z, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      // operands of the products to come, read while the softmax runs
      f16x8_t vf[DT];
#pragma unroll
      for (int t = 0; t < DT; ++t) vf[t] = *reinterpret_cast<const f16x8_t*>(vp + t * 32 * VP + 4 * kb * 16);
      if (kb + 1 < KT / 32) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) kf[s] = *reinterpret_cast<const f16x8_t*>(kp + (kb + 1) * 32 * KP + s * 32);
      }
      if (masked) {
        asm volatile("");                  // a branch: the selects must not run in every step
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = 32 * kb + 8 * (i / 4) + 4 * hh + i % 4;
          const bool vis = key0 + k < lim && !((holes >> (2 * kb + i / 8)) & 1u);
          z[i] = vis ? z[i] : -INFINITY;
        }
      }
      float mx = z[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) mx = fmaxf(mx, z[i]);
      mx *= cq;
      if (__ballot(mx > m + 8.0f)) {       // the maximum may lag by 8, as in the kernel for few rows
        float v = fmaxf(mx, __shfl_xor(mx, 32));
        v = fmaxf(v, m);
        const float f = v == m ? 1.0f : __builtin_amdgcn_exp2f(m - v);
        m = v;
        l *= f;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[t][i] *= f;
      }
      const float base = m == -INFINITY ? 0.f : m;
      float pv[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        pv[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[i], cq, -base));
        l += pv[i];
      }
      u32x4_t p[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e / 4][e % 4] = cvt_pk_f16(pv[2 * e], pv[2 * e + 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[t], __builtin_bit_cast(f16x8_t, p[s]), acc[t], 0, 0, 0);
          if (s == 0) vf[t] = *reinterpret_cast<const f16x8_t*>(vp + t * 32 * VP + (4 * kb + 2) * 16);
        }
    }
  };

  if (w.k0 < w.k1) {                       // workgroup-uniform
    Codes r;
    load(w.k0, page_of(w.k0), r);
    int next = page_of(w.k0 + KT);
    decode(w.k0, r, 0);
    __syncthreads();
    int buf = 0;
    for (int key = w.k0; key < w.k1; key += KT) {
      const bool more = key + KT < w.k1;
      if (more) {
        load(key + KT, next, r);
        next = page_of(key + 2 * KT);
      }
      if (key < limmax) {
        uint32_t holes = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) holes |= gone[buf][i];
        holes = __builtin_amdgcn_readfirstlane(holes);
        compute(key, buf, holes);
      }
      if (more) decode(key + KT, r, buf ^ 1);
      __syncthreads();
      buf ^= 1;
    }
  }

  // Register i of tile t is LDS row 32 t + 8 (i / 4) + 4 hh + i % 4 of V: with
  // i = 4 e + j, coordinate DPT (8 (e % 2) + 4 hh + j) + 2 t + e / 2.  For one
  // (e % 2, j) a lane holds DPT neighbouring coordinates.
  l += __shfl_xor(l, 32);
  if (!ok) return;
  const float inv = w.direct ? (l == 0.f ? 0.f : 1.0f / l) : 1.0f;
  const int64_t at = (int64_t)(w.t0 + tok) * a.o_stride + (int64_t)(h * a.group + g) * D;
  float* po = w.direct ? nullptr : part_o<D>(x, w.slot, h, trow);
#pragma unroll
  for (int e0 = 0; e0 < 2; ++e0)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d0 = DPT * (8 * e0 + 4 * hh + j);
#pragma unroll
      for (int q = 0; q < DPT; q += 4) {
        f32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = acc[(q + i) / 2][4 * (e0 + 2 * ((q + i) % 2)) + j] * inv;
        if (w.direct) store_out4(a, at + d0 + q, v);
        else *reinterpret_cast<f32x4_t*>(po + d0 + q) = v;
      }
    }
  if (!w.direct && hh == 0) {
    float* ml = part_ml(x, w.slot, h, trow);
    ml[0] = m;
    ml[1] = l;
  }
}

hipError_t launch_kv_tiles(const AttendArgs& x, int head_dim, int bits, int64_t items, hipStream_t st) {
  const dim3 grid((unsigned)(items * x.a.c.heads));
#define TILE(D, B, N) hipLaunchKernelGGL((kv_tile_kernel<D, B, N>), grid, dim3(64 * N), 0, st, x)
#define TILE_N(D, B)                     \
  do {                                   \
    if (x.rule.rt == 128) TILE(D, B, 4); \
    else TILE(D, B, 8);                  \
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
