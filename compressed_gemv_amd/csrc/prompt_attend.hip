// Causal attention of whole, packed prompts over their own bf16 keys and values,
// with grouped heads.
//
// A KV head's rows of one sequence are its tokens times `group` query heads,
// row = token * group + g; a workgroup of four waves takes a tile of 128 of them
// and walks the keys that its last token sees, 32 at a time.  S^T = K Q^T on
// 32x32x16 products puts a row's logits of 16 keys into one lane, and the
// weights go back in as the other operand of O^T = V^T P^T without leaving it.
// Tile k of sequence b is number starts[b] * group / 128 + b + k: numbers that
// need no sum over the sequences.
#include "kvcache.hpp"
#include "layer.hpp"

namespace qg {

namespace {

constexpr int kRows = 128, kKeys = 32;

template <int D>
__global__ __launch_bounds__(256) void prompt_kernel(Prompt p) {
  constexpr int STEPS = D / 16, DT = D / 32;
  constexpr int KP = D + 8, VP = kKeys + 8;                 // pitch of a key's and of a coordinate's row
  __shared__ __align__(16) uint16_t ks[kKeys * KP], vs[D * VP];
  __shared__ uint32_t bad;                                  // keys whose values are not finite
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, hh = lane >> 5;
  const int h = blockIdx.x % p.heads;
  const int64_t j = blockIdx.x / p.heads;
  // the tile's sequence
  int b = 0;
  int64_t s0 = 0, s1 = p.T;
  if (p.starts) {
    int n = p.B;
    while (n > 1) {
      const int half = n >> 1;
      int64_t s = p.starts[b + half];
      s = s < 0 ? 0 : s;
      if (s * p.group / kRows + b + half <= j) { b += half; n -= half; }
      else n = half;
    }
    s0 = p.starts[b];
    s1 = p.starts[b + 1];
    s0 = s0 < 0 ? 0 : s0;
    s1 = s1 > p.T ? p.T : s1;
  }
  const int64_t k = j - (s0 * p.group / kRows + b);
  const int64_t rows = (s1 - s0) * p.group, row0 = k * kRows;
  if (k < 0 || row0 >= rows) return;
  const int64_t last = (row0 + kRows < rows ? row0 + kRows : rows) - 1;
  const int keys = (int)(last / p.group) + 1;
  const int64_t row = row0 + wave * 32 + col < rows ? row0 + wave * 32 + col : rows - 1;
  const int tok = (int)(row / p.group), g = (int)(row % p.group);
  bf16x8_t q[STEPS];
  const uint16_t* qp = p.Q + (s0 + tok) * p.q_stride + (int64_t)(h * p.group + g) * D + 8 * hh;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    u32x4_t v = *reinterpret_cast<const u32x4_t*>(qp + 16 * s);
    if (p.scale < 0.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] ^= 0x80008000u;
    }
    q[s] = __builtin_bit_cast(bf16x8_t, v);
  }
  const float c = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-37f);   // positive also for a scale of 0
  f32x16_t acc[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int key0 = 0; key0 < keys; key0 += kKeys) {
    __syncthreads();
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * D / 8; i += 256) {
      const int kk = i / (D / 8), d = 8 * (i % (D / 8));
      const int key = key0 + kk < keys ? key0 + kk : keys - 1;
      const u32x4_t kv = *reinterpret_cast<const u32x4_t*>(p.K + (s0 + key) * p.k_stride + (int64_t)h * D + d);
      const u32x4_t vv = *reinterpret_cast<const u32x4_t*>(p.V + (s0 + key) * p.v_stride + (int64_t)h * D + d);
      *reinterpret_cast<u32x4_t*>(ks + kk * KP + d) = kv;
      // place of key kk among a product's operands: the order in which lanes hold the weights
      const int at = (kk & ~15) | ((kk & 4) << 1) | ((kk & 8) >> 1) | (kk & 3);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t v = (vv[e / 2] >> (16 * (e % 2))) & 0xFFFFu;
        if ((v & 0x7F80u) == 0x7F80u) {
          v = 0;
          atomicOr(&bad, 1u << kk);
        }
        vs[(d + e) * VP + at] = (uint16_t)v;
      }
    }
    __syncthreads();
    f32x16_t z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8_t*>(ks + col * KP + 16 * s + 8 * hh), q[s], z, 0, 0, 0);
    const uint32_t nan = bad;
    float mx = m;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int kk = 8 * (i / 4) + 4 * hh + i % 4;
      z[i] = key0 + kk <= tok ? ((nan >> kk) & 1u ? NAN : z[i] * c) : -INFINITY;
      mx = fmaxf(mx, z[i]);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float base = mx == -INFINITY ? 0.f : mx, f = m == mx ? 1.f : __builtin_amdgcn_exp2f(m - base);
    m = mx;
    l *= f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[t][i] *= f;
    u32x4_t w[2];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      z[i] = __builtin_amdgcn_exp2f(z[i] - base);
      l += z[i];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 4][e % 4] = cvt_pk_bf16(z[2 * e], z[2 * e + 1]);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < DT; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            *reinterpret_cast<const bf16x8_t*>(vs + (32 * t + col) * VP + 16 * s + 8 * hh), __builtin_bit_cast(bf16x8_t, w[s]),
            acc[t], 0, 0, 0);
  }
  l += __shfl_xor(l, 32);
  if (row0 + wave * 32 + col >= rows) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int64_t o = (s0 + tok) * p.o_stride + (int64_t)(h * p.group + g) * D;
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 32 * t + 8 * e + 4 * hh;
      f32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = acc[t][4 * e + i] * inv;
      if (p.out_f32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + o + d) = v;
      else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o + d) = make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
    }
}

}  // namespace

size_t prompt_ws_bytes(int head_dim, int heads, int group, int64_t B, int64_t T) { return 0; }

hipError_t launch_prompt(const Prompt& p, void* ws, hipStream_t st) {
  const int64_t tiles = (int64_t)p.T * p.group / kRows + p.B;
  const dim3 grid((unsigned)(tiles * p.heads));
  if (p.head_dim == 128) hipLaunchKernelGGL((prompt_kernel<128>), grid, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((prompt_kernel<64>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace qg
