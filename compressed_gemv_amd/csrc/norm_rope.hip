// RMS norm of every query and key head and the rotation by its position, in
// one pass: n = x w / sqrt(mean x^2 + eps), then pairs of n turned by position *
// freq.  Every value is read and written once; bound by memory, and by a
// launch's own time for single tokens.
//
// A wave takes one token, whose angles all heads share: lane j forms angle j in
// fp64 (a far position's turns lose their fraction in fp32), and the lanes of a
// head fetch the eight they need by permutes.  A head's row lies in D / 16
// lanes, 16 values each, in two runs of 8 that hold both values of a pair: run i
// and run i + rot / 16 of halves, runs 2i and 2i + 1 of neighbours (and of what
// is not rotated).  So neither the rotation nor the norm needs more than one
// reduction over D / 16 lanes.
#include "kvcache.hpp"
#include "layer.hpp"

namespace qg {

namespace {

// Sum over groups of LPR (4 or 8) neighbouring lanes.
template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp_f32<0xB1>(v);                   // quad_perm [1,0,3,2]
  v += dpp_f32<0x4E>(v);                   // quad_perm [2,3,0,1]
  if (LPR == 8) v += dpp_f32<0x141>(v);    // row_half_mirror
  return v;
}

template <bool F32>
struct Run {                               // 8 values as they lie in memory
  u32x4_t v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* row, int at) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(row) + at * (F32 ? 4 : 2));
    v[0] = p[0];
    if constexpr (F32) v[1] = p[1];
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (F32) return __uint_as_float(v[j / 4][j % 4]);
    else return (j & 1) ? bf16_hi_to_f32(v[0][j / 2]) : bf16_lo_to_f32(v[0][j / 2]);
  }
};

template <bool F32>
__device__ __forceinline__ void store_run(void* row, int at, const float (&x)[8]) {
  if constexpr (F32) {
    f32x4_t* p = reinterpret_cast<f32x4_t*>(static_cast<float*>(row) + at);
    p[0] = f32x4_t{x[0], x[1], x[2], x[3]};
    p[1] = f32x4_t{x[4], x[5], x[6], x[7]};
  } else {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = cvt_pk_bf16(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(row) + at) = v;
  }
}

template <int D, bool IN32, bool OUT32>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRope p, int splits, int64_t units) {
  constexpr int LPR = D / 16, RPW = 64 / LPR;
  constexpr int IB = IN32 ? 4 : 2, OB = OUT32 ? 4 : 2;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane % LPR, row = lane / LPR;
  const int heads = p.q_heads + p.kv_heads, passes = (heads + RPW - 1) / RPW;
  const int half = p.rot / 2;
  const bool turns = i < p.rot / 16;
  int at[2];                               // where the lane's runs begin
  if (turns && !p.pairs) { at[0] = 8 * i; at[1] = half + 8 * i; }
  else { at[0] = 16 * i; at[1] = 16 * i + 8; }

  for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < units; u += (int64_t)gridDim.x * 4) {
    const int t = (int)(u / splits), first = (int)(u % splits);
    int b = t;
    int64_t pos;
    if (p.starts) {
      b = find_seq<64>(p.starts, p.B, t, lane, lane);
      const int s0 = p.starts[b], s1 = p.starts[b + 1];
      if (t < s0 || t >= s1) continue;     // nobody's row (wave-uniform)
      pos = (int64_t)p.lens[b] - ((int64_t)s1 - t);
    } else {
      pos = (int64_t)p.lens[b] - 1;
    }
    float sn = 0.f, cs = 1.f;
    if (lane < half) {
      // turns in fp64: position * freq / 2 pi, then the part behind the point
      const double w = (double)(pos + p.offset) * p.freqs[lane] * 0.15915494309189535;
      sincospif(2.0f * (float)(w - rint(w)), &sn, &cs);
    }
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = __shfl(cs, 8 * i + j);
      s[j] = __shfl(sn, 8 * i + j);
    }
    for (int g = first; g < passes; g += splits) {
      const int hd = g * RPW + row;
      const bool on = hd < heads;
      const int k = (on ? hd : heads - 1) >= p.q_heads ? 1 : 0;
      const int h = (on ? hd : heads - 1) - (k ? p.q_heads : 0);
      const char* in = static_cast<const char*>(p.in[k]) + ((int64_t)t * p.in_stride[k] + (int64_t)h * D) * IB;
      Run<IN32> r[2];
      r[0].load(in, at[0]);
      r[1].load(in, at[1]);
      float x[2][8];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[e][j] = r[e].get(j);
      const void* w = p.weight[k];
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(x[e][j], x[e][j], ss);
      ss = group_sum<LPR>(ss);
      float f = rsqrtf(ss * (1.0f / D) + p.eps), down = 1.0f;
      if (ss == INFINITY) {                // squares beyond fp32: once more of values times 2^-70
        float s2 = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = x[e][j] * 0x1p-70f;
            s2 = __builtin_fmaf(v, v, s2);
          }
        // only whole groups of lanes are in this branch
        f = rsqrtf(group_sum<LPR>(s2) * (1.0f / D));
        down = 0x1p-70f;
      }
      if (w) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float wv[8];
          if (p.w_f32) {
            Run<true> q;
            q.load(w, at[e]);
#pragma unroll
            for (int j = 0; j < 8; ++j) wv[j] = q.get(j);
          } else {
            Run<false> q;
            q.load(w, at[e]);
#pragma unroll
            for (int j = 0; j < 8; ++j) wv[j] = q.get(j);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) x[e][j] = x[e][j] * f * down * wv[j];
        }
      }
      if (turns) {
        if (p.pairs) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const float a = x[e][j], z = x[e][j + 1];
              x[e][j] = a * c[4 * e + j / 2] - z * s[4 * e + j / 2];
              x[e][j + 1] = z * c[4 * e + j / 2] + a * s[4 * e + j / 2];
            }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float a = x[0][j], z = x[1][j];
            x[0][j] = a * c[j] - z * s[j];
            x[1][j] = z * c[j] + a * s[j];
          }
        }
      }
      if (on) {
        char* out = static_cast<char*>(p.out[k]) + ((int64_t)t * p.out_stride[k] + (int64_t)h * D) * OB;
        store_run<OUT32>(out, at[0], x[0]);
        store_run<OUT32>(out, at[1], x[1]);
      }
    }
  }
}

}  // namespace

hipError_t launch_norm_rope(const NormRope& p, hipStream_t st) {
  const int passes = (p.q_heads + p.kv_heads + 64 / (p.head_dim / 16) - 1) / (64 / (p.head_dim / 16));
  // one token's heads over several waves where there are few tokens
  int64_t splits = 4096 / p.T;
  splits = splits < 1 ? 1 : (splits > passes ? passes : splits);
  const int64_t units = p.T * splits, wgs = (units + 3) / 4;
  const dim3 grid((unsigned)(wgs < (1 << 20) ? wgs : 1 << 20));
#define GO(D, I, O) hipLaunchKernelGGL((norm_rope_kernel<D, I, O>), grid, dim3(256), 0, st, p, (int)splits, units)
#define GO_D(D)                                          \
  do {                                                   \
    if (p.in_f32 && p.out_f32) GO(D, true, true);        \
    else if (p.in_f32) GO(D, true, false);               \
    else if (p.out_f32) GO(D, false, true);              \
    else GO(D, false, false);                            \
  } while (0)
  if (p.head_dim == 128) GO_D(128);
  else GO_D(64);
#undef GO_D
#undef GO
  return hipGetLastError();
}

}  // namespace qg
