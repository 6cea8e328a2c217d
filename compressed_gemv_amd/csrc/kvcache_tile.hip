// Attention over the quantized, paged KV cache with many rows per KV head: a
// chunk or a whole prompt, or a batch in front of a shared prefix.
//
// Bound by what a SIMD's one wave issues, products and the softmax's vector
// work, so a cached row is decoded once per workgroup and used by all its rows:
// codes become fp16 values s q + o in LDS (one rounding to 11 bits; s and o are
// multiples of 2^-24 below fp16's normal range, so small rows stay exact), keys
// row by row, values transposed.  fp16 and not bf16 for values and weights: the
// roundings of both then stay an eighth of the output's own.
//
// Measured (8 KV heads of 128, 8 query heads each): 1.07 PFLOP/s for 1024 tokens
// that see 33000 cached ones (0.99 over the call; a large matrix product reaches
// 1.2 here).  A product then takes 68 clocks of its SIMD, of which the matrix core
// works 32 (counted: 49 % busy).  A prompt of 16000 0.93 over the call.  Shorter
// calls pay for starting and ending a tile, 7 us or so: 0.83 for chunks of 700 ..
// 1024 behind 4500 .. 6001, 0.65 for prompts of 999 .. 2500.
#include <type_traits>

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

// The order of a turn's instructions: after each product the vector work of one
// logit (a fused multiply-add, an exponential, a sum, half a conversion) and a
// read from LDS, so that the vector unit has work while a product runs.
#define KV_SCHED                                          \
  _Pragma("unroll") for (int i_ = 0; i_ < 16; ++i_) {     \
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);    \
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    \
    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);    \
  }

// Weights are held times 2^9, with a maximum that may lag by 6: at most 2^15, so
// inside fp16, whose subnormals then begin at 2^-23 of the largest weight and
// lose 2^-34 of it for a key.  With plain weights and a lag of 8, thousands of
// keys of weight 2^-25 would count as nothing; that was 1 to 2 % faster.  A lag
// of 2 moves the maximum often: prompts of 999 .. 2500 281 us, against 263.
constexpr float kLift = 9.0f, kLag = 6.0f;
constexpr float kFar = 1024.0f;            // a maximum (times log2 e) beyond which exponents are formed in two steps
constexpr int kNoLoads = 0x0F70;           // s_waitcnt vmcnt(0), the other counters as they are
constexpr uint32_t k1024 = 0x64006400u, kM1024 = 0xE400E400u;   // fp16 pairs 1024, -1024

}  // namespace

// Decoding of KT = NT / 2 keys by NT threads: half a key row and D / 16
// coordinates of 8 values each.  ks, vs: LDS or an image in memory.
template <int D, int BITS, int NT>
struct Decoder {
  static constexpr int KT = NT / 2;
  static constexpr int ROWB = D * BITS / 8;
  static constexpr int KP = D * 2 + 16, VP = KT * 2 + 16;   // pitch of a key's and of a coordinate's row
  static constexpr int KBUF = KT * KP, VBUF = D * VP;
  static constexpr int KL = ROWB / 2 / 16;        // 16-byte loads of a thread's half key row
  static constexpr int VB = ROWB / 16;            // bytes of a value row per thread
  static constexpr int VW = VB < 4 ? 1 : VB / 4;
  static constexpr int DPT = D / 16;              // coordinates per thread of 8 values
  struct Codes {
    u32x4_t k[KL];
    uint32_t v[8][VW];
    uint32_t km, kvm;                      // the key's constants of K and of V
    u32x4_t vm[2];
    int kpage, vpage;
  };
  const KvView& c;
  const int32_t* pages;
  int max_pages, k1;                       // keys behind k1 are nobody's
  int kkey, khalf, vchunk, vg, vkey;       // values vkey .. + 3 and vkey + 8 .. + 3
  uint32_t pmask, page_rows, head_row;
  int kpage, vpage;                        // of the step to be loaded next

  __device__ __forceinline__ Decoder(const KvView& c_, int h, int tid) : c(c_) {
    kkey = tid >> 1;
    khalf = tid & 1;
    vchunk = tid >> 4;
    vg = tid & 15;
    vkey = 16 * (vchunk >> 1) + 4 * (vchunk & 1);
    pmask = (1u << c.page_shift) - 1u;
    page_rows = (uint32_t)c.heads << c.page_shift;
    head_row = (uint32_t)h << c.page_shift;
  }
  __device__ __forceinline__ int page_of(int key) const {
    if (key >= k1 || (key >> c.page_shift) >= max_pages) return -1;
    const int id = pages[key >> c.page_shift];
    return id < c.n_pages ? id : -1;
  }
  __device__ __forceinline__ void find_pages(int key0) {
    kpage = page_of(key0 + kkey);
    vpage = page_of(key0 + (vkey & ~15));
  }
  __device__ __forceinline__ void load(int key0, Codes& r) {
    r.kpage = kpage;
    r.vpage = vpage;
    const uint64_t krow = (uint64_t)(uint32_t)(kpage < 0 ? 0 : kpage) * page_rows + (head_row + ((uint32_t)(key0 + kkey) & pmask));
    const uint64_t vrow = (uint64_t)(uint32_t)(vpage < 0 ? 0 : vpage) * page_rows + (head_row + ((uint32_t)(key0 + vkey) & pmask));
    const u32x4_t* kp = reinterpret_cast<const u32x4_t*>(c.codes[0] + krow * ROWB + khalf * (ROWB / 2));
#pragma unroll
    for (int i = 0; i < KL; ++i) r.k[i] = kp[i];
    r.km = c.meta[0][krow];
    r.kvm = c.meta[1][krow];
    const uint8_t* vp = c.codes[1] + vrow * ROWB + vg * VB;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t* pj = vp + ((j & 3) + 8 * (j >> 2)) * ROWB;
      if constexpr (VB == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(pj);
        r.v[j][0] = v.x;
        r.v[j][1 % VW] = v.y;
      } else if constexpr (VB == 4) {
        r.v[j][0] = *reinterpret_cast<const uint32_t*>(pj);
      } else {
        r.v[j][0] = *reinterpret_cast<const uint16_t*>(pj);
      }
    }
    const uint32_t* mp = c.meta[1] + vrow;
    r.vm[0] = *reinterpret_cast<const u32x4_t*>(mp);
    r.vm[1] = *reinterpret_cast<const u32x4_t*>(mp + 8);
  }
  // A value row that is NaN is decoded as zeros and makes its key NaN instead,
  // so it reaches exactly the rows whose mask lets them see it; constants of
  // keys that no row sees become zero.
  static __device__ __forceinline__ bool nan_meta(uint32_t mt) { return (mt & 0x7C00u) == 0x7C00u; }
  __device__ __forceinline__ void keys(int key0, const Codes& r, uint8_t* ks, uint32_t* gone) const {
    const uint32_t mt = r.kpage < 0 || key0 + kkey >= k1 ? 0u : (nan_meta(r.kvm) ? 0x7E007E00u : r.km);
    const uint32_t s2 = __builtin_amdgcn_perm(mt, mt, 0x01000100u), o2 = __builtin_amdgcn_perm(mt, mt, 0x03020302u);
    uint8_t* out = ks + kkey * KP + khalf * D;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      u32x4_t v;
      if constexpr (BITS == 8) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t c = r.k[(2 * i + e) / 4][(2 * i + e) % 4];
          v[2 * e] = __builtin_amdgcn_perm(k1024, c, 0x05010500u);
          v[2 * e + 1] = __builtin_amdgcn_perm(k1024, c, 0x05030502u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ((r.k[i / 4][i % 4] >> (4 * e)) & 0x000F000Fu) | k1024;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = pk_fma(pk_add(v[e], kM1024), s2, o2);
      *reinterpret_cast<u32x4_t*>(out + i * 16) = v;
    }
    if (khalf == 0 && (kkey & 15) == 0) gone[kkey >> 4] = r.kpage < 0 ? 1u << (kkey >> 4) : 0u;
  }
  __device__ __forceinline__ void values(int key0, const Codes& r, uint8_t* vs) const {
    uint32_t s2[4], o2[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t mt[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 2 * q + e;
        const uint32_t t = r.vm[j / 4][j % 4];
        mt[e] = r.vpage < 0 || key0 + vkey + (j & 3) + 8 * (j >> 2) >= k1 || nan_meta(t) ? 0u : t;
      }
      s2[q] = __builtin_amdgcn_perm(mt[1], mt[0], 0x05040100u);
      o2[q] = __builtin_amdgcn_perm(mt[1], mt[0], 0x07060302u);
    }
    uint32_t half[4] = {0u, 0u, 0u, 0u};
    uint8_t* out = vs + vg * VP + vchunk * 16;
#pragma unroll
    for (int d = 0; d < DPT; ++d) {
      u32x4_t v;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t u;
        if constexpr (BITS == 8) {         // two coordinates of both keys, then one with the exponent of 1024
          if (d % 2 == 0)
            half[q] = __builtin_amdgcn_perm(r.v[2 * q + 1][d / 4], r.v[2 * q][d / 4], d % 4 == 0 ? 0x05010400u : 0x07030602u);
          u = __builtin_amdgcn_perm(k1024, half[q], d % 2 == 0 ? 0x05010500u : 0x05030502u);
        } else {
          if (d % 4 == 0) half[q] = __builtin_amdgcn_perm(r.v[2 * q + 1][0], r.v[2 * q][0], d == 0 ? 0x05040100u : 0x07060302u);
          u = ((half[q] >> (4 * (d % 4))) & 0x000F000Fu) | k1024;
        }
        v[q] = pk_fma(pk_add(u, kM1024), s2[q], o2[q]);
      }
      *reinterpret_cast<u32x4_t*>(out + 16 * d * VP) = v;
    }
  }
};

// A workgroup: NW waves of 64 rows (two blocks of 32), one wave per SIMD with
// all its registers; 32 NW keys a step, two LDS buffers, one barrier a step.
// S^T = K Q^T on 32x32x16 products puts a row's logits of 16 keys into one
// lane; the weights go back in as the other operand of O^T = V^T P^T without
// leaving the lane, because V's columns are stored in the order in which the
// lanes hold them.  64 rows per wave halve the LDS reads per product, which
// otherwise cost as much time as the products; the two blocks take turns, the
// products of one running while the vector unit does the softmax of the other:
//   turn 1 of 32 keys:  products  O_A += V P_A (the keys before), S_A (these)
//                       vector    softmax of S_B (the keys before)
//   turn 2:             products  O_B += V P_B (the keys before), S_B (these)
//                       vector    softmax of S_A (these)
// LDS rows are padded by 16 bytes: 16 neighbouring rows then cover all banks,
// and every address of the inner loop is one register plus a constant.
// Coordinate DPT g + q of V lies in row 16 q + g, so that the lanes that write
// it (q fixed) write neighbouring rows.
template <int D, int BITS, int NW, bool IMAGE>
__global__ __launch_bounds__(64 * NW, 1) void kv_tile_kernel(AttendArgs x) {
  constexpr int KT = 32 * NW;              // keys per step
  constexpr int KBS = KT / 32;
  constexpr int STEPS = D / 16, DT = D / 32, DPT = D / 16;
  using Dec = Decoder<D, BITS, 64 * NW>;
  constexpr int KP = Dec::KP, VP = Dec::VP, KBUF = Dec::KBUF, VBUF = Dec::VBUF;
  __shared__ __align__(16) uint8_t ksh[2 * KBUF];
  __shared__ __align__(16) uint8_t vsh[2 * VBUF];
  // per 16 keys: 1 << (their place) where they are not in the cache (an image brings 1 KB)
  __shared__ __align__(16) uint32_t gone[2][IMAGE ? 256 : KT / 16];
  const KvAttend& a = x.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hh = lane >> 5;
  const int heads = a.c.heads, h = blockIdx.x % heads;
  Pieces pieces = pieces_of(x, blockIdx.x / heads, lane);
  Work w;
  while (next_work<true, IMAGE>(x, pieces, w, lane)) {
  Dec dec(a.c, h, tid);
  dec.pages = w.pages;
  dec.max_pages = w.max_pages;
  dec.k1 = w.k1;

  // An image is copied to LDS as it lies, 1 KB a wave and instruction, without
  // passing through registers; each wave waits for its own copies before the
  // barrier, which by itself waits for what the wave did in LDS only.
  auto fetch = [&](int key0, int buf) {
    const int64_t step = w.steps + key0 / KT;
    const uint8_t* src = x.image + (step * heads + h) * kv_image_bytes(D) + lane * 16;
    auto put = [&](const uint8_t* from, uint8_t* to) {
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                       (__attribute__((address_space(3))) void*)to, 16, 0, 0);
    };
    for (int i = wave; i < KBUF / 1024; i += NW) put(src + i * 1024, ksh + buf * KBUF + i * 1024);
    for (int i = wave; i < VBUF / 1024; i += NW) put(src + KBUF + i * 1024, vsh + buf * VBUF + i * 1024);
    if (wave == 0) put(src + KBUF + VBUF, reinterpret_cast<uint8_t*>(gone[buf]));
  };
  // the first keys are on their way while the queries come
  typename Dec::Codes r;
  if (w.k0 < w.k1) {                       // workgroup-uniform
    if constexpr (IMAGE) {
      fetch(w.k0, 0);
    } else {
      dec.find_pages(w.k0);
      dec.load(w.k0, r);
      dec.find_pages(w.k0 + KT);
    }
  }

  // queries: rows scaled by a power of two to a largest value in [1, 2) (exact
  // up to 2^-25 of it), what each row sees, and the factor back
  f16x8_t qf[2][STEPS];
  u32x4_t raw[2][STEPS];
  float cq[2];
  int lim[2], limmin = w.k1;
  const float c0 = fabsf(a.scale) * 1.4426950408889634f;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    int row = w.row0 + wave * 64 + n * 32 + col;
    row = row < w.rows ? row : w.rows - 1; // behind the last row it is repeated, and not stored
    const int tok = row / a.group, g = row - tok * a.group;
    const uint16_t* q = a.Q + (int64_t)(w.t0 + tok) * a.q_stride + (int64_t)(h * a.group + g) * D + 8 * hh;
    lim[n] = row_sees(w, tok);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) raw[n][s] = *reinterpret_cast<const u32x4_t*>(q + 16 * s);
  }
  __builtin_amdgcn_sched_barrier(0);       // all of them under way before the first is used
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    uint32_t big = 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = raw[n][s][e] & 0x7F80u, hi = (raw[n][s][e] >> 16) & 0x7F80u;
        big = lo > big ? lo : big;
        big = hi > big ? hi : big;
      }
    const uint32_t other = (uint32_t)__shfl_xor((int)big, 32);
    big = other > big ? other : big;
    int ex = (int)(big >> 7) - 127;
    ex = ex < -126 ? -126 : (ex > 126 ? 126 : ex);
    const float down = ldexpf(a.scale < 0.f ? -1.f : 1.f, -ex);
    cq[n] = fmaxf(ldexpf(c0, ex), 1e-37f); // positive also for a scale of 0: -inf times it stays -inf
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      u32x4_t v;
      if constexpr (BITS == 4) {           // pairs (j, j + 4), as a nibble mask leaves the keys
        const u32x4_t t = raw[n][s];
        raw[n][s][0] = __builtin_amdgcn_perm(t[2], t[0], 0x05040100u);
        raw[n][s][1] = __builtin_amdgcn_perm(t[2], t[0], 0x07060302u);
        raw[n][s][2] = __builtin_amdgcn_perm(t[3], t[1], 0x05040100u);
        raw[n][s][3] = __builtin_amdgcn_perm(t[3], t[1], 0x07060302u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = cvt_pk_f16(bf16_lo_to_f32(raw[n][s][e]) * down, bf16_hi_to_f32(raw[n][s][e]) * down);
      qf[n][s] = __builtin_bit_cast(f16x8_t, v);
    }
    int lo = lim[n];                       // the least of the wave's rows
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_xor(lo, d);
      lo = u < lo ? u : lo;
    }
    limmin = lo < limmin ? lo : limmin;
  }
  limmin = __builtin_amdgcn_readfirstlane(limmin);
  // The queries never change and only products read them: accumulation
  // registers hold them, the vector unit's stay free.
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int s = 0; s < STEPS; ++s) asm volatile("" : "+a"(qf[n][s]));

  f32x16_t acc[2][DT], z[2];
  float m[2], l[2];
  // of exponents, and what a logit passes before the maximum is looked at: m - kLift and m + kLag, or beyond kFar
  // -kLift and -inf
  float base[2], lim_m[2];
  u32x4_t p[2][2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][t][i] = 0.f;
    m[n] = lim_m[n] = -INFINITY;
    base[n] = l[n] = 0.f;
    p[n][0] = p[n][1] = u32x4_t{0u, 0u, 0u, 0u};
  }

  const uint8_t* kread = ksh + col * KP + hh * 16;
  const uint8_t* vread = vsh + col * VP + hh * 16;
  f16x8_t kf[STEPS], vf[2][DT];
  auto read_k = [&](int buf, int kb) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) kf[s] = *reinterpret_cast<const f16x8_t*>(kread + buf * KBUF + kb * 32 * KP + s * 32);
  };
  auto read_v = [&](int buf, int kb) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < DT; ++t)
        vf[s][t] = *reinterpret_cast<const f16x8_t*>(vread + buf * VBUF + t * 32 * VP + (4 * kb + 2 * s) * 16);
  };
  float mx[2];                             // of a block's logits, its lane's
  auto max_of = [&](const f32x16_t& v) {
    float r = v[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) r = fmaxf(r, v[i]);
    return r;
  };
  // masks, and the running maximum moved where it has to be (keys key .. key + 31)
  auto bounds = [&](auto blk, int key, uint32_t holes) {
    constexpr int n = decltype(blk)::value;
    if (__builtin_expect(key + 32 > limmin || holes, 0)) {
      asm volatile("");                    // a branch: the selects must not run in every step
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool vis = key + 8 * (i / 4) + 4 * hh + i % 4 < lim[n] && !((holes >> (i / 8)) & 1u);
        z[n][i] = vis ? z[n][i] : -INFINITY;
      }
      mx[n] = max_of(z[n]);
    }
    if (__builtin_expect(__ballot(mx[n] * cq[n] > lim_m[n]) != 0, 0)) {
      float v = mx[n] * cq[n];
      v = fmaxf(v, __shfl_xor(v, 32));
      v = fmaxf(v, m[n]);
      const float f = v == m[n] ? 1.0f : __builtin_amdgcn_exp2f(m[n] - v);
      m[n] = v;
      l[n] *= f;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[n][t][i] *= f;
      // An exponent z cq - m of one rounding is off by half a step of m: beyond 2^24
      // the largest logit's own would leave 0 and take every weight with it.  The
      // rounded product minus m is 0 there; it goes on as a z.
      const bool far = fabsf(v) > kFar && v != -INFINITY;
      lim_m[n] = far ? -INFINITY : v + kLag;
      base[n] = far ? -kLift : (v == -INFINITY ? 0.f : v - kLift);
      if (__builtin_expect(__ballot(far) != 0, 0)) {
        const float up = 1.0f / cq[n];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float e = z[n][i] * cq[n];
          asm volatile("" : "+v"(e));      // rounded
          z[n][i] = far ? (e - v) * up : z[n][i];
        }
      }
    }
  };
  // One turn: the softmax of block n against the products of the other block,
  // logits first, so that their maximum is there when the turn ends.
  auto turn = [&](auto soft, auto&& after_s, auto&& after_pv) {
    constexpr int n = decltype(soft)::value, o = 1 - n;
    float pv[16];
    f32x16_t zn;
#pragma unroll
    for (int i = 0; i < 16; ++i) zn[i] = 0.f;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) zn = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[s], qf[o][s], zn, 0, 0, 0);
    after_s();
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < DT; ++t)
        acc[o][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[s][t], __builtin_bit_cast(f16x8_t, p[o][s]), acc[o][t], 0, 0, 0);
    after_pv();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      pv[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[n][i], cq[n], -base[n]));
      l[n] += pv[i];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) p[n][e / 4][e % 4] = cvt_pk_f16(pv[2 * e], pv[2 * e + 1]);
    z[o] = zn;
    mx[o] = max_of(zn);
    // the weights and the maximum are made here, not where they are used
    asm volatile("" : "+v"(p[n][0]), "+v"(p[n][1]), "+v"(l[n]), "+v"(mx[o]));
    KV_SCHED
    __builtin_amdgcn_sched_barrier(0);
  };
  using A = std::integral_constant<int, 0>;
  using B = std::integral_constant<int, 1>;
  auto none = [] {};

  if (w.k0 < w.k1) {
    if constexpr (IMAGE) {
      __builtin_amdgcn_s_waitcnt(kNoLoads);
    } else {
      dec.keys(w.k0, r, ksh, gone[0]);
      dec.values(w.k0, r, vsh);
      if (w.k0 + KT < w.k1) {
        dec.load(w.k0 + KT, r);
        dec.find_pages(w.k0 + 2 * KT);
      }
    }
    __syncthreads();
    // before the first keys: weights of zero, logits that add nothing
#pragma unroll
    for (int i = 0; i < 16; ++i) z[0][i] = z[1][i] = -INFINITY;
    mx[0] = mx[1] = -INFINITY;
    read_k(0, 0);
    read_v(0, 0);
    int buf = 0;
    uint32_t before = 0;                   // holes of the 32 keys before
    for (int key = w.k0; key < w.k1; key += KT, buf ^= 1) {
      uint32_t holes = 0;
#pragma unroll
      for (int i = 0; i < KT / 16; ++i) holes |= gone[buf][i];
      holes = __builtin_amdgcn_readfirstlane(holes);
      const bool more = key + KT < w.k1;
      if constexpr (IMAGE) {
        if (more) fetch(key + KT, buf ^ 1);
      }
#pragma unroll
      for (int kb = 0; kb < KBS; ++kb) {
        const int k = key + 32 * kb;
        if (kb > 0 && k >= w.k1) break;    // the last step's keys may end early
        bounds(B{}, k - 32, before);
        before = (holes >> (2 * kb)) & 3u;
        turn(B{}, none, none);             // softmax B (before); O_A, S_A
        bounds(A{}, k, before);
        turn(A{}, [&] { if (kb + 1 < KBS) read_k(buf, kb + 1); }, [&] { read_v(buf, kb); });
        if constexpr (!IMAGE) {
          if (kb == KBS - 2 && more) dec.keys(key + KT, r, ksh + (buf ^ 1) * KBUF, gone[buf ^ 1]);
          if (kb == KBS - 1 && more) {
            dec.values(key + KT, r, vsh + (buf ^ 1) * VBUF);
            if (key + 2 * KT < w.k1) {
              dec.load(key + 2 * KT, r);
              dec.find_pages(key + 3 * KT);
            }
          }
        }
      }
      if constexpr (IMAGE) __builtin_amdgcn_s_waitcnt(kNoLoads);
      __syncthreads();
      if (more) read_k(buf ^ 1, 0);
    }
    // what is left: the last keys' products and block B's softmax
    bounds(B{}, w.k0 + (w.k1 - w.k0 + 31) / 32 * 32 - 32, before);
    turn(B{}, none, none);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < DT; ++t)
        acc[1][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[s][t], __builtin_bit_cast(f16x8_t, p[1][s]), acc[1][t], 0, 0, 0);
  }

  // Register i of tile t is LDS row 32 t + 8 (i / 4) + 4 hh + i % 4 of V: with
  // i = 4 e + j, coordinate DPT (8 (e % 2) + 4 hh + j) + 2 t + e / 2.  For one
  // (e % 2, j) a lane holds DPT neighbouring coordinates.
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    l[n] += __shfl_xor(l[n], 32);
    const int trow = wave * 64 + n * 32 + col, row = w.row0 + trow;
    if (row >= w.rows) continue;
    const int tok = row / a.group, g = row - tok * a.group;
    const float inv = w.direct ? (l[n] == 0.f ? 0.f : 1.0f / l[n]) : 1.0f;
    auto each = [&](auto&& put) {
#pragma unroll
      for (int e0 = 0; e0 < 2; ++e0)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int d0 = DPT * (8 * e0 + 4 * hh + j);
#pragma unroll
          for (int q = 0; q < DPT; q += 4) {
            f32x4_t v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = acc[n][(q + i) / 2][4 * (e0 + 2 * ((q + i) % 2)) + j] * inv;
            put(d0 + q, v);
          }
        }
    };
    if (w.direct) {
      const int64_t at = (int64_t)(w.t0 + tok) * a.o_stride + (int64_t)(h * a.group + g) * D;
      if (a.out_f32) each([&](int d, const f32x4_t& v) { store_out4<true>(a, at + d, v); });
      else each([&](int d, const f32x4_t& v) { store_out4<false>(a, at + d, v); });
    } else {
      float* po = part_o<D>(x, w.slot, h, trow);
      each([&](int d, const f32x4_t& v) { *reinterpret_cast<f32x4_t*>(po + d) = v; });
    }
    if (!w.direct && hh == 0) {
      float* ml = part_ml(x, w.slot, h, trow);
      ml[0] = m[n] - kLift;                // of which l is the sum
      ml[1] = l[n];
    }
  }
  // the last step's barrier has freed the LDS for the next tile
  }
}

// Images of the decoded keys and values, one workgroup for 128 keys of one KV
// head at a time: where many row tiles meet the same keys, each key is decoded
// once and not once for every tile, and the tile kernel's vector unit, which
// shares its issue slots with the products, is left to the softmax.
template <int D, int BITS>
__global__ __launch_bounds__(256) void kv_image_kernel(AttendArgs x) {
  using Dec = Decoder<D, BITS, 256>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int heads = x.a.c.heads;
  for (int64_t i = blockIdx.x; i < x.images * heads; i += gridDim.x) {
    const int h = (int)(i % heads);
    const StepAt at = step_at(x.s, x.rule, i / heads, lane);
    if (at.b < 0) return;
    Dec dec(x.a.c, h, tid);
    dec.pages = x.s.pages + (int64_t)at.b * x.s.max_pages;
    dec.max_pages = x.s.max_pages;
    dec.k1 = at.need;
    typename Dec::Codes r;
    const int key0 = at.step * 128;
    dec.find_pages(key0);
    dec.load(key0, r);
    uint8_t* out = x.image + i * kv_image_bytes(D);
    dec.keys(key0, r, out, reinterpret_cast<uint32_t*>(out + Dec::KBUF + Dec::VBUF));
    dec.values(key0, r, out + Dec::KBUF);
  }
}

hipError_t launch_kv_images(const AttendArgs& x, int head_dim, int bits, hipStream_t st) {
  const int64_t n = x.images * x.a.c.heads;
  const dim3 grid((unsigned)(n < 8192 ? n : 8192));
  if (head_dim == 128) {
    if (bits == 8) hipLaunchKernelGGL((kv_image_kernel<128, 8>), grid, dim3(256), 0, st, x);
    else hipLaunchKernelGGL((kv_image_kernel<128, 4>), grid, dim3(256), 0, st, x);
  } else {
    if (bits == 8) hipLaunchKernelGGL((kv_image_kernel<64, 8>), grid, dim3(256), 0, st, x);
    else hipLaunchKernelGGL((kv_image_kernel<64, 4>), grid, dim3(256), 0, st, x);
  }
  return hipGetLastError();
}

hipError_t launch_kv_tiles(const AttendArgs& x, int head_dim, int bits, hipStream_t st) {
  const dim3 grid((unsigned)(x.rule.wgs * x.a.c.heads));
#define TILE(D, B, N, I) hipLaunchKernelGGL((kv_tile_kernel<D, B, N, I>), grid, dim3(64 * N), 0, st, x)
#define TILE_N(D, B)                             \
  do {                                           \
    if (x.rule.rt == 128) TILE(D, B, 2, false);  \
    else if (!x.image) TILE(D, B, 4, false);     \
    else TILE(D, B, 4, true);                    \
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
