// Writing the quantized KV cache and reading it back.
//
// A row of D values is held by D / 8 neighbouring lanes, 8 values each, so one
// 16-byte load per lane brings it in, the row's minimum and maximum are DPP
// reductions inside those lanes, and each lane stores its 8 codes with one
// store.  No contraction here: the codes come out bit-identical to any other
// IEEE implementation of the definition.
//
// Measured (8 heads of 128): four prompts of 517 .. 4096 tokens at 4 bits are
// written in 18 us, in which a SIMD issues 6800 vector instructions (counted),
// 13 us at 4 clocks each and 2.1 GHz, beside 10 us of memory at a copy's rate,
// and read back in 10.6 (4.5 TB/s read and written).  16 sequences of 300 .. 4000
// tokens at 8 bits are read back in 47 us, 4.5 TB/s next to a plain copy's 4.8,
// or in 39 into a block that was just written (the last-level cache takes the
// stores).  16 single tokens take 3.6 us either way, a launch's own time.
#pragma clang fp contract(off)

#include "common.hpp"
#include "kvcache.hpp"

namespace qg {

constexpr float kKvMax = 65280.0f;   // largest stored magnitude: s*q + o stays below fp16's largest value

// min or max over the LPR (8 or 16) lanes of a row group
template <int LPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : fminf(a, b); };
  v = op(v, dpp_f32<0xB1>(v));                    // quad_perm [1,0,3,2]
  v = op(v, dpp_f32<0x4E>(v));                    // quad_perm [2,3,0,1]
  v = op(v, dpp_f32<0x141>(v));                   // row_half_mirror
  if constexpr (LPR == 16) v = op(v, dpp_f32<0x140>(v));   // row_mirror
  return v;
}

// The next fp16 above / below h (finite, and not the largest in that direction).
__device__ __forceinline__ uint32_t f16_up(uint32_t h) { return (h & 0x8000u) ? h - 1u : h + 1u; }
__device__ __forceinline__ uint32_t f16_down(uint32_t h) {
  return (h & 0x7FFFu) == 0u ? 0x8001u : ((h & 0x8000u) ? h + 1u : h - 1u);
}

// 8 values of a lane as they come from memory.
template <bool F32>
struct Raw8 {
  u32x4_t w[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw8<F32> load8(const void* p, int64_t elem) {
  Raw8<F32> r;
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(p) + elem * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.w[i] = q[i];
  return r;
}

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// Constants and packed codes of a row, r the lane's 8 values of it.  The codes
// are the fp64 definition's: t = (x - o) / s is formed in fp32 with an error
// below 255 * 2^-22 < 2^-13, and a lane with a t closer than 2^-12 to a
// half-way point takes its codes in fp64.  Bound by the vector unit until it
// was cut to about 15 instructions a value: the checks for values that are not
// finite or too large look at packed bits and leave the clamp to a branch, the
// codes go from fp32 to bytes in one instruction each (4 bits: two codes make
// one byte in fp32 first), and (max - o) / L is a product with 1 / L whose
// rounding is put right by comparing s L with max - o, both exact in fp64.
template <int LPR, int BITS, bool F32>
__device__ __forceinline__ void quant_row(const Raw8<F32>& r, int lane, uint32_t (&q)[BITS / 4], uint32_t* meta) {
  constexpr float L = (float)((1 << BITS) - 1);
  float x[8];
  uint32_t big;                                   // largest magnitude, as bits; bf16: in the upper half
  if constexpr (F32) {
    big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = r.w[i / 4][i % 4], m = u & 0x7FFFFFFFu;
      x[i] = __uint_as_float(u);
      big = m > big ? m : big;
    }
  } else {
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, r.w[0][i] & 0x7FFF7FFFu));
      x[2 * i] = bf16_lo_to_f32(r.w[0][i]);
      x[2 * i + 1] = bf16_hi_to_f32(r.w[0][i]);
    }
    big = (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
  }
  if (__ballot(big > 0x477F0000u)) {              // 65280: in some row of the wave
    const uint64_t rowmask = ((1ull << LPR) - 1ull) << (lane & ~(LPR - 1));
    if (__ballot(big >= 0x7F800000u) & rowmask) {
#pragma unroll
      for (int i = 0; i < BITS / 4; ++i) q[i] = 0;
      *meta = 0x7E007E00u;                        // s = o = NaN
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -kKvMax), kKvMax);
  }
  float mn = fminf(x[0], x[1]), mx = fmaxf(x[0], x[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) { mn = fminf(mn, x[i]); mx = fmaxf(mx, x[i]); }
  mn = row_reduce<LPR, false>(mn);
  mx = row_reduce<LPR, true>(mx);
  uint32_t ob = __builtin_bit_cast(uint16_t, (_Float16)mn);
  if (f16_bits_to_f32(ob) > mn) ob = f16_down(ob);
  if ((ob & 0x7FFFu) == 0u) ob = 0u;
  const float o = f16_bits_to_f32(ob);
  const double d = (double)mx - (double)o;        // >= 0
  // three roundings, but the result lies within half a step (and a bit) of
  // d / L on either side, so at most one step up reaches the smallest fp16 >= d / L
  uint32_t sb = __builtin_bit_cast(uint16_t, (_Float16)(float)(d * (1.0 / L))) & 0x7FFFu;   // -0 becomes 0
  if ((double)(f16_bits_to_f32(sb) * L) < d) sb = f16_up(sb);
  const float s = f16_bits_to_f32(sb);
  *meta = sb | (ob << 16);
  const float rs = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;
  float n[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = (x[i] - o) * rs;              // 0 .. L
    n[i] = __builtin_rintf(t);
    far = fmaxf(far, fabsf(t - n[i]));
  }
  if (far > 0.5f - 0x1p-12f && s > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      n[i] = fminf((float)__builtin_rint(((double)x[i] - (double)o) / (double)s), L);
  }
#pragma unroll
  for (int i = 0; i < BITS / 4; ++i) q[i] = 0;
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i / 4] = __builtin_amdgcn_cvt_pk_u8_f32(n[i], i % 4, q[i / 4]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[0] = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_fmaf(n[2 * i + 1], 16.f, n[2 * i]), i, q[0]);
  }
}

// Grid (row groups, head groups): a workgroup takes 256 / LPR tokens and hpw
// heads of each, K and V, so a token's place is looked up once for 2 hpw rows.
template <int D, int BITS, bool F32>
__global__ __launch_bounds__(256) void kv_write_kernel(KvView c, SeqView sv, const void* __restrict__ K, int64_t k_stride,
                                                       const void* __restrict__ V, int64_t v_stride, int hpw) {
  constexpr int LPR = D / 8;
  const int lane = threadIdx.x & 63, sub = threadIdx.x % LPR;
  const int t = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (t >= sv.T) return;                           // whole row groups leave together
  const int h0 = blockIdx.y * hpw, h1 = h0 + hpw < c.heads ? h0 + hpw : c.heads;
  // the rows are on their way while the token's place is looked up, and the
  // next head's while this one's codes are made
  auto rows = [&](int h, Raw8<F32> (&x)[2]) {
    x[0] = load8<F32>(K, t * k_stride + h * D + sub * 8);
    x[1] = load8<F32>(V, t * v_stride + h * D + sub * 8);
  };
  Raw8<F32> next[2];
  rows(h0, next);
  bool owned;
  const int64_t slot = slot_of_row<LPR>(c, sv, t, sub, lane, &owned);
  if (slot < 0) return;
  for (int h = h0; h < h1; ++h) {
    const Raw8<F32> x[2] = {next[0], next[1]};
    if (h + 1 < h1) rows(h + 1, next);
    const int64_t row = cache_row(c, slot, h);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t q[BITS / 4], meta;
      quant_row<LPR, BITS, F32>(x[kv], lane, q, &meta);
      if constexpr (BITS == 8) *reinterpret_cast<uint2*>(c.codes[kv] + row * D + sub * 8) = uint2{q[0], q[1]};
      else *reinterpret_cast<uint32_t*>(c.codes[kv] + row * (D / 2) + sub * 4) = q[0];
      if (sub == 0) c.meta[kv][row] = meta;
    }
  }
}

// The same shape as the write: codes and constants of a row in one load each,
// s q + o with one rounding in fp32, 8 values a lane; bound by memory.  A row
// without a place is zeros.
template <int D, int BITS, bool F32>
__global__ __launch_bounds__(256) void kv_read_kernel(KvView c, SeqView sv, void* __restrict__ K, int64_t k_stride,
                                                      void* __restrict__ V, int64_t v_stride, int hpw) {
  constexpr int LPR = D / 8;
  const int lane = threadIdx.x & 63, sub = threadIdx.x % LPR;
  const int t = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (t >= sv.T) return;
  bool owned;
  const int64_t slot = slot_of_row<LPR>(c, sv, t, sub, lane, &owned);
  if (!owned) return;
  const int h0 = blockIdx.y * hpw, h1 = h0 + hpw < c.heads ? h0 + hpw : c.heads;
  for (int h = h0; h < h1; ++h) {
    const int64_t row = slot < 0 ? 0 : cache_row(c, slot, h);
    uint32_t w[2][2] = {{0u, 0u}, {0u, 0u}}, meta[2] = {0u, 0u};
    if (slot >= 0) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if constexpr (BITS == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(c.codes[kv] + row * D + sub * 8);
          w[kv][0] = v.x; w[kv][1] = v.y;
        } else {
          w[kv][0] = *reinterpret_cast<const uint32_t*>(c.codes[kv] + row * (D / 2) + sub * 4);
        }
        meta[kv] = c.meta[kv][row];
      }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float s = f16_lo(meta[kv]), o = f16_hi(meta[kv]);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t q = BITS == 8 ? (w[kv][i / 4] >> (8 * (i % 4))) & 255u : (w[kv][0] >> (4 * i)) & 15u;
        x[i] = __builtin_fmaf(s, (float)q, o);
      }
      void* out = kv ? V : K;
      const int64_t at = t * (kv ? v_stride : k_stride) + h * D + sub * 8;
      if constexpr (F32) {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        f[0] = float4{x[0], x[1], x[2], x[3]};
        f[1] = float4{x[4], x[5], x[6], x[7]};
      } else {
        u32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = cvt_pk_bf16(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + at) = v;
      }
    }
  }
}

// Heads per workgroup: as many as leave about 2048 workgroups (8 per CU; four
// prompts written and read back 28.8 us, with a quarter of the workgroups 32,
// with four times as many 29.4).
static int heads_per_wg(int64_t row_groups, int heads) {
  const int64_t n = row_groups * heads / 2048;
  return n < 1 ? 1 : (n > heads ? heads : (int)n);
}

#define KV_DISPATCH(NAME, ...)                                                                        \
  do {                                                                                                \
    const int64_t rg = (s.T + 2048 / head_dim - 1) / (2048 / head_dim);                               \
    const int hpw = heads_per_wg(rg, c.heads);                                                        \
    const dim3 grid((unsigned)rg, (unsigned)((c.heads + hpw - 1) / hpw));                             \
    if (head_dim == 128) {                                                                            \
      if (bits == 8) {                                                                                \
        if (f32) hipLaunchKernelGGL((NAME<128, 8, true>), grid, dim3(256), 0, st, __VA_ARGS__, hpw);  \
        else hipLaunchKernelGGL((NAME<128, 8, false>), grid, dim3(256), 0, st, __VA_ARGS__, hpw);     \
      } else {                                                                                        \
        if (f32) hipLaunchKernelGGL((NAME<128, 4, true>), grid, dim3(256), 0, st, __VA_ARGS__, hpw);  \
        else hipLaunchKernelGGL((NAME<128, 4, false>), grid, dim3(256), 0, st, __VA_ARGS__, hpw);     \
      }                                                                                               \
    } else {                                                                                          \
      if (bits == 8) {                                                                                \
        if (f32) hipLaunchKernelGGL((NAME<64, 8, true>), grid, dim3(256), 0, st, __VA_ARGS__, hpw);   \
        else hipLaunchKernelGGL((NAME<64, 8, false>), grid, dim3(256), 0, st, __VA_ARGS__, hpw);      \
      } else {                                                                                        \
        if (f32) hipLaunchKernelGGL((NAME<64, 4, true>), grid, dim3(256), 0, st, __VA_ARGS__, hpw);   \
        else hipLaunchKernelGGL((NAME<64, 4, false>), grid, dim3(256), 0, st, __VA_ARGS__, hpw);      \
      }                                                                                               \
    }                                                                                                 \
  } while (0)

hipError_t launch_kv_write(const KvView& c, const SeqView& s, int head_dim, int bits, const void* K, int64_t k_stride,
                           const void* V, int64_t v_stride, bool f32, hipStream_t st) {
  KV_DISPATCH(kv_write_kernel, c, s, K, k_stride, V, v_stride);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvView& c, const SeqView& s, int head_dim, int bits, void* K, int64_t k_stride, void* V,
                          int64_t v_stride, bool f32, hipStream_t st) {
  KV_DISPATCH(kv_read_kernel, c, s, K, k_stride, V, v_stride);
  return hipGetLastError();
}
#undef KV_DISPATCH

}  // namespace qg
