// Launchers of the steps between a layer's projections and its KV cache
// (include/qlayer.h), called by the C ABI layer after argument validation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

struct NormRope {
  int head_dim, q_heads, kv_heads, rot;
  bool pairs;
  const double* freqs;
  const void* weight[2];       // q, k; null: no norm
  bool w_f32;
  float eps;
  int64_t offset;
  const int32_t* lens;
  const int32_t* starts;
  int B, T;
  const void* in[2];           // Q, K
  void* out[2];
  int64_t in_stride[2], out_stride[2];
  bool in_f32, out_f32;
};
hipError_t launch_norm_rope(const NormRope& p, hipStream_t st);

struct Adapt {
  const uint16_t* A;
  const uint16_t* B;
  const float* scales;
  const int32_t* ranks;
  int n, rank;
  int K;
  int N;
  int seqs, T;
  const int32_t* ids;
  const int32_t* starts;       // or null: one row for each request
  const uint16_t* x;
  const void* y;
  void* out;
  int64_t x_stride, y_stride, o_stride;
  bool f32;                    // y and out
  float* part;                 // workspace: [splits][T][rank padded to 16]
};
size_t adapt_ws_bytes(int64_t seqs, int64_t T, int64_t K, int rank);
hipError_t launch_adapt(const Adapt& p, hipStream_t st);

struct Prompt {
  int head_dim, heads, group;  // KV heads, query heads of each
  int B, T;
  const int32_t* starts;       // or null: one sequence of T rows
  const uint16_t* Q;
  const uint16_t* K;
  const uint16_t* V;
  int64_t q_stride, k_stride, v_stride, o_stride;
  float scale;
  void* out;
  bool out_f32;
};
hipError_t launch_prompt(const Prompt& p, hipStream_t st);

}  // namespace qg
