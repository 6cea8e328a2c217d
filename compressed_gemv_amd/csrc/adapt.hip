// Low-rank adapters of many requests beside a shared projection:
//   out[t] = y[t] + scale[a] * B_a (A_a x[t]).
//
// Two launches: `down` forms h = A_a x in fp32, split over K into partial sums;
// `up` adds them, in the order of the splits, and forms y + scale * B_a h.  Few
// rows are bound by reading A and B of each adapter once, many by reading x and y
// and writing out; the products are small beside either, so both run on
// v_mfma_f32_16x16x32_bf16 with operands straight from memory.  h goes in as bf16
// parts, each the rounded rest of those before: three where y is fp32, which hold
// all of it, and two where the result is rounded to bf16 (16 bits; one would lose
// 2^-8).  They multiply a product of depth `rank` only.
//
// Rows meet an adapter in tiles of up to 64.  With starts, tile k of request b is
// number starts[b] / 64 + b + k of T / 64 + B: numbers that need no sum over the
// requests, and of which at most B stay empty.  With a row for each request, a
// block of 64 rows is divided by the adapters it names: workgroup `slot` takes
// the slot-th of them (and every slots-th behind it), so an adapter that several
// rows name is read once for all of them.
#include "common.hpp"
#include "layer.hpp"

namespace qg {

namespace {

// y and out rows begin wherever N and the caller's strides put them; the
// hardware takes wide accesses at any element.
typedef f32x4_t f32x4_any __attribute__((aligned(4)));
typedef u32x4_t u32x4_any __attribute__((aligned(2)));

constexpr int kTile = 64;                  // rows of a tile
constexpr uint32_t kOut = 0x7FFFFFF0u;     // an offset behind every buffer: the load gives 0

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of a call and how its axes are cut, from sizes alone.
struct AdaptPlan {
  int64_t blocks;                          // tiles, or blocks of 64 rows
  int slots;
  int splits, kchunk;                      // of K, a multiple of 128
  int nchunk;                              // of N, a multiple of 256
  int R;                                   // rank padded to 16
};

AdaptPlan plan_adapt(bool segments, int64_t seqs, int64_t T, int64_t K, int64_t N, int rank) {
  AdaptPlan p{};
  p.R = (rank + 15) / 16 * 16;
  int64_t tiles;
  if (segments) {
    p.blocks = T / kTile + seqs;
    p.slots = 1;
    tiles = T / kTile + (seqs < 16 ? seqs : 16);
  } else {
    p.blocks = ceil_div(T, kTile);
    // A workgroup without an adapter costs 3 us of its place: 64 rows with 12
    // adapters take 49 us with 64 slots, 16 with 16.  Behind 1024 rows there are
    // blocks enough.
    p.slots = T <= 1024 ? (int)(T < 16 ? T : 16) : 4;
    tiles = p.blocks * p.slots;
  }
  const bool wide = segments && T >= 16 * seqs;
  int64_t s = ceil_div(1024, tiles);       // (5 prompts of 77 .. 1500 rows: 512 workgroups 164 us, 768 155, 1024 157)
  const int64_t most = ceil_div(K, 512);
  s = s > most ? most : s;
  s = s > 32 ? 32 : s;
  p.kchunk = (int)(ceil_div(ceil_div(K, s), wide ? 256 : 512) * (wide ? 256 : 512));
  p.splits = (int)ceil_div(K, p.kchunk);
  // every workgroup adds up h again (16 single rows, N = 28672: 256 outputs each 26 us,
  // 512 19.5, 1024 14.8; 5 prompts, N = 8192: 256 152 us, 768 149, 1024 160)
  int64_t c = ceil_div(N * tiles, segments ? 1024 : 512);
  c = ceil_div(c, 256) * 256;
  p.nchunk = (int)(c < 256 ? 256 : (c > 1024 ? 1024 : c));
  return p;
}

// The rows a workgroup works on.
struct Tile {
  int a;                                   // adapter; -1: none
  int row0;                                // of the tile or block
  int n;                                   // rows; 0: nothing to do
};

// Tile number j of a call with starts: wave-uniform.
__device__ __forceinline__ Tile segment_tile(const Adapt& p, int64_t j, int lane) {
  int lo = 0, n = p.seqs;                  // largest b with starts[b] / 64 + b <= j
  while (n > 1) {
    const int step = (n + 63) / 64, i = lo + lane * step;
    bool le = false;
    if (lane * step < n) {
      const int s = p.starts[i];
      le = (int64_t)((s < 0 ? 0 : s) / kTile) + i <= j;
    }
    const int cnt = __popcll(__ballot(le)), k = cnt > 0 ? cnt - 1 : 0;
    lo += k * step;
    n = n - k * step < step ? n - k * step : step;
    if (n < 1) n = 1;
  }
  int s0 = p.starts[lo], s1 = p.starts[lo + 1];
  s0 = s0 < 0 ? 0 : s0;
  s1 = s1 > p.T ? p.T : s1;
  const int64_t k = j - ((int64_t)(s0 / kTile) + lo);
  const int64_t row0 = s0 + k * kTile;
  Tile t{-1, 0, 0};
  if (k < 0 || row0 >= s1) return t;
  t.row0 = (int)row0;
  t.n = s1 - t.row0 < kTile ? s1 - t.row0 : kTile;
  t.a = p.ids[lo];
  return t;
}

// Walks a workgroup's tiles; rows[] (LDS) gets each tile's rows, relative to row0.
struct Tiles {
  uint64_t left = 0;                       // rows of the block not looked at
  int id = 0, index = 0;                   // a lane's row's adapter; adapters passed
  bool segment, done = false;
  __device__ __forceinline__ int own_id(const Adapt& p, int a) const {
    if (a < 0 || a >= p.n) return -1;
    return p.ranks && p.ranks[a] <= 0 ? -1 : a;
  }
  __device__ __forceinline__ Tiles(const Adapt& p, int64_t block, int lane) {
    segment = p.starts != nullptr;
    if (segment) return;
    const int64_t row = block * kTile + lane;
    const bool on = row < p.T;
    id = on ? own_id(p, p.ids[row]) : -1;
    left = __ballot(on);
  }
  // All waves of the workgroup call it together; behind it rows[] may be read.
  __device__ __forceinline__ bool next(const Adapt& p, int64_t block, int slot, int slots, int lane, uint8_t* rows, Tile& t) {
    __syncthreads();                       // the tile before is done with rows[]
    if (segment) {
      if (done) return false;
      done = true;
      t = segment_tile(p, block, lane);
      t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
      t.n = __builtin_amdgcn_readfirstlane(t.n);
      if (t.n == 0) return false;
      t.a = own_id(p, __builtin_amdgcn_readfirstlane(t.a));
      if (threadIdx.x < kTile) rows[threadIdx.x] = (uint8_t)threadIdx.x;
      __syncthreads();
      return true;
    }
    while (left) {
      const int a = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
      const uint64_t m = __ballot(id == a) & left;
      left &= ~m;
      if (index++ % slots != slot) continue;
      t.a = a;
      t.row0 = (int)(block * kTile);
      t.n = __popcll(m);
      if (threadIdx.x < kTile && ((m >> lane) & 1u)) rows[__popcll(m & ((1ull << lane) - 1ull))] = (uint8_t)lane;
      __syncthreads();
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ int rank_of(const Adapt& p, int a) {
  if (!p.ranks) return p.rank;
  const int k = p.ranks[a];
  return k < p.rank ? k : p.rank;
}

__device__ __forceinline__ bf16x8_t frag(u32x4_t v) { return __builtin_bit_cast(bf16x8_t, v); }
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
  return u32x4_t{v[0], v[1], v[2], v[3]};
}

// ------------------------------------------------------------------- down
// One workgroup: a tile, a range of K and up to 64 ranks (QT tiles of 16).  With
// more than 16 rows each wave takes 16 of them; otherwise the waves share the
// range of K and add up in LDS.  A lane's operands are 16 bytes: a rank's (a
// row's) 8 inputs from 8 (lane / 16) on.
template <int QT>
__global__ __launch_bounds__(256) void adapt_down_kernel(Adapt p, int slots, int kchunk, int R) {
  __shared__ uint8_t rows[kTile];
  __shared__ __align__(16) float red[3][64][QT][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t block = blockIdx.x / slots;
  const int slot = blockIdx.x % slots, rank0 = blockIdx.z * 64;
  const int k0 = blockIdx.y * kchunk, k1 = p.K - k0 < kchunk ? p.K : k0 + kchunk;
  const int r16 = lane & 15, g = lane >> 4;
  Tiles tiles(p, block, lane);
  Tile t;
  while (tiles.next(p, block, slot, slots, lane, rows, t)) {
    if (t.a < 0) continue;
    const int ranks = rank_of(p, t.a) - rank0;
    if (ranks <= 0) continue;
    const int held = ranks < 16 * QT ? ranks : 16 * QT;      // ranks of this workgroup
    const bool wide = t.n > 16;                              // workgroup-uniform
    const int at = wide ? wave * 16 + r16 : r16;             // the lane's place in the tile
    const int row = at < t.n ? rows[at] : -1;
    const int64_t xs = p.x_stride;
    const auto xb = make_rsrc(p.x + (int64_t)t.row0 * xs, (uint32_t)(((p.T - t.row0 < kTile ? p.T - t.row0 : kTile) - 1) * xs + p.K) * 2u);
    const auto ab = make_rsrc(p.A + ((int64_t)t.a * p.rank + rank0) * p.K, (uint32_t)held * (uint32_t)p.K * 2u);
    const uint32_t xrow = row < 0 ? kOut : (uint32_t)(row * xs + 8 * g) * 2u;
    uint32_t arow[QT];
#pragma unroll
    for (int q = 0; q < QT; ++q) arow[q] = (uint32_t)((16 * q + r16) * p.K + 8 * g) * 2u;
    f32x4_t acc[QT];
#pragma unroll
    for (int q = 0; q < QT; ++q) acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 4;                   // steps of 32 inputs under way at a time
    auto walk = [&](int from, int step) {
      for (int k = from; k < k1; k += U * step) {
        u32x4_t xv[U], av[U][QT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int kk = k + u * step;
          const bool in = kk + 8 * g < k1;                   // k1 is K, a multiple of 8, or of 32
          xv[u] = load16(xb, in && row >= 0 ? xrow + 2u * kk : kOut);
#pragma unroll
          for (int q = 0; q < QT; ++q) av[u][q] = load16(ab, in ? arow[q] + 2u * kk : kOut);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < QT; ++q)
            acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(av[u][q]), frag(xv[u]), acc[q], 0, 0, 0);
      }
    };
    if (wide) walk(k0, 32);
    else walk(k0 + 32 * wave, 128);
    if (!wide) {
      if (wave > 0) {
#pragma unroll
        for (int q = 0; q < QT; ++q) *reinterpret_cast<f32x4_t*>(red[wave - 1][lane][q]) = acc[q];
      }
      __syncthreads();
      if (wave > 0) continue;
#pragma unroll
      for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int q = 0; q < QT; ++q) acc[q] += *reinterpret_cast<const f32x4_t*>(red[w][lane][q]);
    }
    // lane: ranks 16 q + 4 g .. + 3 of its row
    if (row >= 0) {
      float* to = p.part + ((int64_t)blockIdx.y * p.T + t.row0 + row) * R + rank0 + 4 * g;
#pragma unroll
      for (int q = 0; q < QT; ++q)
        if (16 * q < held) *reinterpret_cast<f32x4_t*>(to + 16 * q) = acc[q];
    }
  }
}

// The same for requests of many rows.  A product's operands lie in 16 different
// rows, and fetched that way (four lanes, four lines) x arrives at 1.9
// TB/s; here four neighbouring lanes fetch 64 bytes of a row, and the operands
// pass through LDS, each wave's in a place of its own: no barrier.  The waves
// share the range of K, so A is fetched once for all 64 rows.  (5 prompts of 77 ..
// 1500 rows, 28672 inputs, rank 32: the call 206 -> 157 us.)
template <int QT>
__global__ __launch_bounds__(256) void adapt_down_tall_kernel(Adapt p, int kchunk, int R) {
  constexpr int U = 2, KW = 32 * U, STEP = 4 * KW;          // inputs a wave and a workgroup take at a time
  constexpr int STAGE = U * (4 + QT) * 1024;
  __shared__ uint8_t rows[kTile];
  __shared__ __align__(16) uint8_t stage[4 * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rank0 = blockIdx.z * 64;
  const int k0 = blockIdx.y * kchunk, k1 = p.K - k0 < kchunk ? p.K : k0 + kchunk;
  const int r16 = lane & 15, g = lane >> 4;
  Tiles tiles(p, blockIdx.x, lane);
  Tile t;
  if (!tiles.next(p, blockIdx.x, 0, 1, lane, rows, t) || t.a < 0) return;
  const int ranks = rank_of(p, t.a) - rank0;
  if (ranks <= 0) return;
  const int held = ranks < 16 * QT ? ranks : 16 * QT;
  const int rt = (t.n + 15) / 16, qt = (held + 15) / 16;    // tiles of rows and of ranks
  const uint16_t* const x = p.x + (int64_t)t.row0 * p.x_stride;
  const uint16_t* const A = p.A + ((int64_t)t.a * p.rank + rank0) * p.K;
  f32x4_t acc[QT][4];
#pragma unroll
  for (int q = 0; q < QT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[q][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // a 16 x 32 block: lane l fetches piece (l % 4) ^ (l / 16) of row l / 4, so that
  // reading piece g of 16 rows meets all banks once; rows behind the last one
  // (and ranks behind the adapter's own) repeat it, and are not used
  uint8_t* const mine = stage + wave * STAGE;
  const int lrow = lane >> 2, lpiece = (lane & 3) ^ (lane >> 4);
  const uint8_t* const read = mine + r16 * 64 + ((g ^ (r16 >> 2)) * 16);
  const uint16_t* xl[4];
  const uint16_t* al[QT];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 16 * i + lrow < t.n ? 16 * i + lrow : t.n - 1;
    xl[i] = x + row * p.x_stride + 8 * lpiece;
  }
#pragma unroll
  for (int q = 0; q < QT; ++q) {
    const int row = 16 * q + lrow < held ? 16 * q + lrow : held - 1;
    al[q] = A + (int64_t)row * p.K + 8 * lpiece;
  }
  auto put = [&](const uint16_t* from, uint8_t* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
  };
  int k = k0;
  for (; k + STEP <= k1; k += STEP) {
    const int kk = k + wave * KW;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < rt) put(xl[i] + kk + 32 * u, mine + (u * (4 + QT) + i) * 1024);
#pragma unroll
      for (int q = 0; q < QT; ++q)
        if (q < qt) put(al[q] + kk + 32 * u, mine + (u * (4 + QT) + 4 + q) * 1024);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);                     // vmcnt(0)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bf16x8_t av[QT];
#pragma unroll
      for (int q = 0; q < QT; ++q)
        if (q < qt) av[q] = *reinterpret_cast<const bf16x8_t*>(read + (u * (4 + QT) + 4 + q) * 1024);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= rt) continue;
        const bf16x8_t xv = *reinterpret_cast<const bf16x8_t*>(read + (u * (4 + QT) + i) * 1024);
#pragma unroll
        for (int q = 0; q < QT; ++q)
          if (q < qt) acc[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[q], xv, acc[q][i], 0, 0, 0);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);                     // lgkmcnt(0): read before it is written again
    asm volatile("" ::: "memory");
  }
  // what is left of K (of the last range only): operands straight from memory, zeros behind the end
  if (k < k1) {
    const int last = t.n - 1;
    const auto xb = make_rsrc(x, (uint32_t)(last * p.x_stride + p.K) * 2u);
    const auto ab = make_rsrc(A, (uint32_t)held * (uint32_t)p.K * 2u);
    for (int kk = k + 32 * wave; kk < k1; kk += 128) {
      const bool in = kk + 8 * g < k1;
      u32x4_t av[QT], xv[4];
#pragma unroll
      for (int q = 0; q < QT; ++q) av[q] = load16(ab, in ? (uint32_t)((16 * q + r16) * p.K + 8 * g + kk) * 2u : kOut);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xv[i] = load16(xb, in && 16 * i + r16 < t.n ? (uint32_t)((16 * i + r16) * p.x_stride + 8 * g + kk) * 2u : kOut);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < QT; ++q)
          acc[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(av[q]), frag(xv[i]), acc[q][i], 0, 0, 0);
    }
  }
  // the waves' sums: wave i adds up row tile i, in the waves' order
  float* const red = reinterpret_cast<float*>(stage);
  __syncthreads();
  for (int w = 0; w < 4; ++w) {            // one row tile at a time: 4 waves x QT KB
    if (w >= rt) break;
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      f32x4_t v = acc[q][0];
#pragma unroll
      for (int i = 1; i < 4; ++i) v = w == i ? acc[q][i] : v;
      *reinterpret_cast<f32x4_t*>(red + ((wave * QT + q) * 64 + lane) * 4) = v;
    }
    __syncthreads();
    const int at = 16 * w + r16;
    for (int q = wave; q < qt; q += 4) {
      f32x4_t v = *reinterpret_cast<const f32x4_t*>(red + (q * 64 + lane) * 4);
#pragma unroll
      for (int o = 1; o < 4; ++o) v += *reinterpret_cast<const f32x4_t*>(red + ((o * QT + q) * 64 + lane) * 4);
      if (at < t.n)
        *reinterpret_cast<f32x4_t*>(p.part + ((int64_t)blockIdx.y * p.T + t.row0 + at) * R + rank0 + 16 * q + 4 * g) = v;
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------------- up
// One workgroup: a tile and a range of N.  h (all splits added, times scale)
// lies in LDS as its bf16 parts: 32-deep blocks of the first, then those of the
// next, or for ranks up to 16 two parts in one block, so that one product does.
// A wave forms 64
// outputs of 16 rows at a time (of 32 with twice the registers: the call 149 -> 156
// us for 5 prompts of 77 .. 1500 rows): the four 16 x 16 products of a row tile give a
// lane four neighbouring outputs of a row each (fp32: 16-byte accesses), or,
// with the outputs of two products interleaved, eight (bf16).
template <bool F32>
constexpr int kParts = F32 ? 3 : 2;

struct UpRows {
  const uint8_t* rows;
  const uint16_t* h;
  int pitch, deep, blocks;                 // of h: values per row and per part, 32-deep blocks of a part
  int n, held;
};

// A wave's 64 outputs from n0 on: of B the first 32 ranks, fetched before h is there.
template <bool F32>
struct UpCols {
  __amdgpu_buffer_rsrc_t rsrc;
  int n0, n1, held;
  u32x4_t first[4];
  // outputs relative to n0: product c's row m is output perm(c, m)
  static __device__ __forceinline__ int perm(int c, int m) { return F32 ? 16 * c + m : 32 * (c / 2) + 8 * (m / 4) + 4 * (c % 2) + m % 4; }
  __device__ __forceinline__ void begin(const Adapt& p, const Tile& t, int n0_, int n1_, int held_, int lane) {
    n0 = n0_;
    n1 = n1_;
    held = held_;
    rsrc = make_rsrc(p.B + ((int64_t)t.a * p.N + n0) * p.rank, (uint32_t)(n1 - n0) * (uint32_t)p.rank * 2u);
    load(p.rank, 0, lane, first);
  }
  // ranks 32 J .. of B; a lane holds 8 (of ranks up to 16 the upper lanes the same again)
  __device__ __forceinline__ void load(int rank, int J, int lane, u32x4_t (&v)[4]) const {
    const int g = lane >> 4, j = held <= 16 ? 8 * (g & 1) : 32 * J + 8 * g;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = load16(rsrc, j < held ? (uint32_t)(perm(c, lane & 15) * rank + j) * 2u : kOut);
  }
  // what lies behind the adapter's own rank may be anything
  __device__ __forceinline__ void mask(int J, int lane, u32x4_t (&v)[4]) const {
    const int g = lane >> 4, c8 = held - (held <= 16 ? 8 * (g & 1) : 32 * J + 8 * g);
    if (c8 >= 8) return;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t m = c8 >= 2 * w + 2 ? 0xFFFFFFFFu : (c8 == 2 * w + 1 ? 0xFFFFu : 0u);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c][w] &= m;
    }
  }
};

template <bool F32>
__device__ __forceinline__ void up_tile(const Adapt& p, const Tile& t, const UpRows& u, const UpCols<F32>& b, int row_tile, int lane) {
  const int r16 = lane & 15, g = lane >> 4, n0 = b.n0, n1 = b.n1;
  const bool both = u.deep == 16;          // two parts in one block
  const int at = 16 * row_tile + r16;
  const bool on = at < u.n;
  const int64_t row = t.row0 + (on ? u.rows[at] : 0);
  const float* const yf = static_cast<const float*>(p.y) + (F32 ? row * p.y_stride + n0 : 0);
  const uint16_t* const yh = static_cast<const uint16_t*>(p.y) + (F32 ? 0 : row * p.y_stride + n0);
  // y comes while the products run
  f32x4_t y4[4];
  u32x4_t y8[2];
  if (on) {
    if constexpr (F32) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n0 + 16 * c + 4 * g + 4 <= n1) y4[c] = *reinterpret_cast<const f32x4_any*>(yf + 16 * c + 4 * g);
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (n0 + 32 * c + 8 * g + 8 <= n1) y8[c] = *reinterpret_cast<const u32x4_any*>(yh + 32 * c + 8 * g);
    }
  }
  f32x4_t acc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int J = 0; J < u.blocks; ++J) {
    u32x4_t bv[4];
    if (J == 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c) bv[c] = b.first[c];
    } else {
      b.load(p.rank, J, lane, bv);
    }
    b.mask(J, lane, bv);
    const uint16_t* hr = u.h + at * u.pitch + 32 * J + 8 * g;
#pragma unroll
    for (int part = 0; part < kParts<F32>; ++part) {
      if (both && part == 1) continue;
      u32x4_t h = {0u, 0u, 0u, 0u};        // both: the third part has nothing beside it
      if (!both || part == 0 || g < 2) h = *reinterpret_cast<const u32x4_t*>(hr + part * u.deep);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(bv[c]), frag(h), acc[c], 0, 0, 0);
    }
  }
  if (!on) return;
  const int64_t to = row * p.o_stride + n0;
  if constexpr (F32) {
    float* o = static_cast<float*>(p.out) + to;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int n = 16 * c + 4 * g;
      if (n0 + n + 4 <= n1) {
        *reinterpret_cast<f32x4_any*>(o + n) = y4[c] + acc[c];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n0 + n + k < n1) o[n + k] = yf[n + k] + acc[c][k];
      }
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + to;
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      const int n = 16 * c + 8 * g;
      if (n0 + n + 8 <= n1) {
        const u32x4_t v = y8[c / 2];
        u32x4_t w;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = cvt_pk_bf16(bf16_lo_to_f32(v[k]) + acc[c + k / 2][2 * (k % 2)], bf16_hi_to_f32(v[k]) + acc[c + k / 2][2 * (k % 2) + 1]);
        *reinterpret_cast<u32x4_any*>(o + n) = w;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (n0 + n + k < n1) o[n + k] = (uint16_t)cvt_pk_bf16(bf16_bits_to_f32(yh[n + k]) + acc[c + k / 4][k % 4], 0.f);
      }
    }
  }
}

template <bool F32>
__global__ __launch_bounds__(256) void adapt_up_kernel(Adapt p, int slots, int splits, int nchunk, int R) {
  __shared__ uint8_t rows[kTile];
  extern __shared__ __align__(16) uint16_t hbuf[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t block = blockIdx.x / slots;
  const int slot = blockIdx.x % slots;
  const int64_t first64 = (int64_t)blockIdx.y * nchunk;
  const int first = (int)first64, last = p.N - first64 < nchunk ? p.N : first + nchunk;
  const bool copies = p.out != p.y;
  Tiles tiles(p, block, lane);
  Tile t;
  while (tiles.next(p, block, slot, slots, lane, rows, t)) {
    if (t.a < 0) {                         // no adapter: y as it is
      if (!copies) continue;
      const int es = F32 ? 4 : 2;
      for (int i = wave; i < t.n; i += 4) {
        const int64_t row = t.row0 + rows[i];
        const char* y = static_cast<const char*>(p.y) + (row * p.y_stride + first) * es;
        char* o = static_cast<char*>(p.out) + (row * p.o_stride + first) * es;
        const int bytes = (last - first) * es;
        for (int b = lane * 16; b < bytes; b += 1024) {
          if (b + 16 <= bytes) *reinterpret_cast<u32x4_any*>(o + b) = *reinterpret_cast<const u32x4_any*>(y + b);
          else
            for (int k = b; k < bytes; k += 2) *reinterpret_cast<uint16_t*>(o + k) = *reinterpret_cast<const uint16_t*>(y + k);
        }
      }
      continue;
    }
    UpRows u;
    u.rows = rows;
    u.h = hbuf;
    u.n = t.n;
    u.held = rank_of(p, t.a);
    const bool both = u.held <= 16;
    const int deep = both ? 16 : (u.held + 31) / 32 * 32;
    u.deep = deep;
    u.blocks = both ? 1 : deep / 32;
    u.pitch = kParts<F32> * deep + 8;      // 16 bytes more: neighbouring rows in other banks
    const int tall = (t.n + 15) / 16 * 16, kept = (u.held + 15) / 16 * 16;   // down wrote so many ranks
    const float scale = p.scales[t.a];
    UpCols<F32> cols;
    const int mine = first + 64 * wave;
    if (mine < last) cols.begin(p, t, mine, last - mine < 64 ? last : mine + 64, u.held, lane);
    for (int i = threadIdx.x; i < tall * (deep / 4); i += 256) {
      const int at = i / (deep / 4), j = 4 * (i % (deep / 4));
      f32x4_t h = {0.f, 0.f, 0.f, 0.f};
      if (at < t.n && j < kept) {
        const float* from = p.part + ((int64_t)t.row0 + rows[at]) * R + j;
        for (int s = 0; s < splits; s += 8) {                // 8 loads under way, added in their order
          f32x4_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (s + e < splits) v[e] = *reinterpret_cast<const f32x4_t*>(from + (int64_t)(s + e) * p.T * R);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (s + e < splits) h += v[e];
        }
        h *= scale;
      }
      // ranks behind the adapter's own: infinities of x have made them NaN or infinite
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = j + k < u.held ? h[k] : 0.f;
#pragma unroll
      for (int part = 0; part < kParts<F32>; ++part) {
        uint32_t v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          v[k] = cvt_pk_bf16(h[2 * k], h[2 * k + 1]);
          const float a = bf16_lo_to_f32(v[k]), b = bf16_hi_to_f32(v[k]);
          // an infinity leaves nothing (its difference would be NaN)
          h[2 * k] = fabsf(a) < INFINITY ? h[2 * k] - a : 0.f;
          h[2 * k + 1] = fabsf(b) < INFINITY ? h[2 * k + 1] - b : 0.f;
        }
        *reinterpret_cast<uint2*>(hbuf + at * u.pitch + part * deep + j) = make_uint2(v[0], v[1]);
      }
    }
    __syncthreads();
    const int tiles16 = tall / 16;
    for (int n0 = mine; n0 < last; n0 += 256) {
      if (n0 != mine) cols.begin(p, t, n0, last - n0 < 64 ? last : n0 + 64, u.held, lane);
      for (int i = 0; i < tiles16; ++i) up_tile<F32>(p, t, u, cols, i, lane);
    }
  }
}

}  // namespace

size_t adapt_ws_bytes(int64_t seqs, int64_t T, int64_t K, int rank) {
  // with and without starts: the larger of both
  const AdaptPlan a = plan_adapt(true, seqs, T, K, 1, rank), b = plan_adapt(false, seqs, T, K, 1, rank);
  return (size_t)(a.splits > b.splits ? a.splits : b.splits) * T * a.R * 4;
}

hipError_t launch_adapt(const Adapt& p, hipStream_t st) {
  const AdaptPlan a = plan_adapt(p.starts != nullptr, p.seqs, p.T, p.K, p.N, p.rank);
  const dim3 down((unsigned)(a.blocks * a.slots), (unsigned)a.splits, (unsigned)((p.rank + 63) / 64));
  if (p.starts && p.T >= 16 * (int64_t)p.seqs) {
    if (p.rank <= 16) hipLaunchKernelGGL((adapt_down_tall_kernel<1>), down, dim3(256), 0, st, p, a.kchunk, a.R);
    else if (p.rank <= 32) hipLaunchKernelGGL((adapt_down_tall_kernel<2>), down, dim3(256), 0, st, p, a.kchunk, a.R);
    else hipLaunchKernelGGL((adapt_down_tall_kernel<4>), down, dim3(256), 0, st, p, a.kchunk, a.R);
  } else if (p.rank <= 16) hipLaunchKernelGGL((adapt_down_kernel<1>), down, dim3(256), 0, st, p, a.slots, a.kchunk, a.R);
  else if (p.rank <= 32) hipLaunchKernelGGL((adapt_down_kernel<2>), down, dim3(256), 0, st, p, a.slots, a.kchunk, a.R);
  else hipLaunchKernelGGL((adapt_down_kernel<4>), down, dim3(256), 0, st, p, a.slots, a.kchunk, a.R);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int deep = p.rank <= 16 ? 16 : (p.rank + 31) / 32 * 32;
  const int64_t tall = p.T < kTile ? ceil_div(p.T, 16) * 16 : kTile;
  const size_t lds = (size_t)tall * ((p.f32 ? kParts<true> : kParts<false>) * deep + 8) * 2;
  const dim3 up((unsigned)(a.blocks * a.slots), (unsigned)ceil_div(p.N, a.nchunk));
  if (p.f32) hipLaunchKernelGGL((adapt_up_kernel<true>), up, dim3(256), lds, st, p, a.slots, a.splits, a.nchunk, a.R);
  else hipLaunchKernelGGL((adapt_up_kernel<false>), up, dim3(256), lds, st, p, a.slots, a.splits, a.nchunk, a.R);
  return hipGetLastError();
}

}  // namespace qg
