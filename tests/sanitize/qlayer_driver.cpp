// Drives the entry points of include/qlayer.h on the host, with the library's
// host code built under the address and undefined-behaviour sanitizers and
// linked against the host-only HIP stand-in (fake_hip.cpp): accepted calls
// launch kernels within a launch's limits over sizes from one row to the
// largest the ABI takes, rejected ones launch nothing, and the size queries
// survive sizes of every magnitude.  Device pointers are fake addresses the
// host code never dereferences.
#include <cstdint>
#include <cstdio>

#include "fake_hip.h"
#include "qlayer.h"

namespace {

int g_fail = 0, g_checks = 0;

#define CHECK(cond, ...)                                        \
  do {                                                          \
    ++g_checks;                                                 \
    if (!(cond)) {                                              \
      ++g_fail;                                                 \
      std::fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__); \
      std::fprintf(stderr, __VA_ARGS__);                        \
      std::fprintf(stderr, "\n");                               \
    }                                                           \
  } while (0)

void* dp(int i) { return reinterpret_cast<void*>((uintptr_t)0x10000000u + (uintptr_t)i * 0x1000000u); }
template <class T>
T* dpt(int i) { return static_cast<T*>(dp(i)); }

uint64_t g_rng = 0x9E3779B97F4A7C15ull;
uint64_t next() {   // splitmix64
  uint64_t z = (g_rng += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
int64_t any_size() {   // of every magnitude, negative and zero included
  switch (next() % 8) {
    case 0: return -(int64_t)(next() % 1000);
    case 1: return (int64_t)(next() % 3);
    case 2: return INT64_MAX - (int64_t)(next() % 4);
    case 3: return ((int64_t)1 << (next() % 63)) + (int64_t)(next() % 3) - 1;
    default: return (int64_t)(next() >> (1 + next() % 63));
  }
}
int64_t upto(int64_t n) {   // 1 .. n, spread over its logarithm, the ends among them
  if (next() % 8 == 0) return n;
  int64_t v = (int64_t)(next() >> (1 + next() % 62));
  v = v % n + 1;
  const int cut = (int)(next() % 40);
  return (v >> cut) + (v >> cut == 0);
}

// A call that the library takes launches; one that it refuses does not.
template <class F>
void drive(const char* what, bool must, F&& call) {
  const long before = fake_hip_launches(), bad = fake_hip_bad_launches();
  const int st = call();
  CHECK(fake_hip_bad_launches() == bad, "%s: a launch outside the limits (%s)", what, fake_hip_last_kernel());
  CHECK((st == Q_OK) == (fake_hip_launches() > before), "%s: status %d, %ld launches", what, st, fake_hip_launches() - before);
  CHECK(!must || st == Q_OK, "%s: refused with %d", what, st);
}

void adapt(int64_t n, int64_t K, int64_t N, int rank, int64_t B, int64_t T, bool starts, bool must) {
  const qadapters a{n, K, N, rank, dp(1), dp(2), dpt<float>(3), nullptr};
  size_t ws = 0;
  const int st = qadapt_ws(&a, B, T, &ws);
  CHECK(!must || st == Q_OK, "qadapt_ws: %d", st);
  drive("qadapt", must, [&] {
    return qadapt(&a, B, T, dpt<int32_t>(4), starts ? dpt<int32_t>(5) : nullptr, dp(6), K, dp(7), N, dp(8), N,
                  next() % 2 ? Q_F32 : Q_BF16, dp(9), ws, nullptr);
  });
}

void norm(int D, int hq, int hk, int64_t B, int64_t T, bool starts, bool must) {
  const qrope p{D, hq, hk, D / 2, (int)(next() % 2), dpt<double>(1), dp(2), nullptr, Q_BF16, 1e-6f, 5};
  drive("qnorm_rope", must, [&] {
    return qnorm_rope(&p, B, T, dpt<int32_t>(3), starts ? dpt<int32_t>(4) : nullptr, dp(5), (int64_t)hq * D, dp(6), (int64_t)hk * D,
                      next() % 2 ? Q_F32 : Q_BF16, dp(7), (int64_t)hq * D, dp(8), (int64_t)hk * D, next() % 2 ? Q_F32 : Q_BF16, nullptr);
  });
}

void prompt(int D, int hq, int hk, int64_t B, int64_t T, bool starts, bool must) {
  drive("qprompt_attend", must, [&] {
    return qprompt_attend(D, hq, hk, B, T, starts ? dpt<int32_t>(1) : nullptr, dp(2), (int64_t)hq * D, dp(3), (int64_t)hk * D, dp(4),
                          (int64_t)hk * D, 0.1f, dp(5), (int64_t)hq * D, Q_BF16, nullptr);
  });
}

}  // namespace

int main() {
  for (int i = 0; i < 4000; ++i) {
    const int64_t K = 8 * upto((1 << 20) - 1), N = upto((1 << 25) - 1), T = upto(1 << 27);
    const int rank = 8 * (int)upto(16);
    adapt(upto(1 << 20), K, N, rank, upto(65536), T, true, true);
    adapt(upto(1 << 20), K, N, rank, T, T, false, true);
    const int D = next() % 2 ? 64 : 128, hk = (int)upto(1024), g = (int)upto(64);
    norm(D, hk * (g < 60 ? g : 60), hk < 1000 ? hk : 1000, upto(65536), T, true, (int64_t)hk * 60 + 1000 <= 65536);
    norm(D, 1 + (int)upto(60000), 1, T, T, false, true);
    const int64_t most = ((int64_t)1 << 30) / g;
    const int64_t Tp = T < most ? T : most;
    prompt(D, hk * g, hk, upto(65536), Tp, true, true);
    prompt(D, hk * g, hk, 1, Tp, false, true);
  }
  for (int i = 0; i < 20000; ++i) {
    adapt(any_size(), any_size(), any_size(), (int)any_size(), any_size(), any_size(), next() % 2, false);
    adapt(upto(100), 8 * upto(1000), any_size(), 8 * (int)upto(20), any_size(), any_size(), next() % 2, false);
    norm((int)any_size(), (int)any_size(), (int)any_size(), any_size(), any_size(), next() % 2, false);
    norm(64, (int)upto(100), (int)upto(100), any_size(), any_size(), next() % 2, false);
    prompt((int)any_size(), (int)any_size(), (int)any_size(), any_size(), any_size(), next() % 2, false);
    prompt(128, 8, 2, any_size(), any_size(), next() % 2, false);
  }
  CHECK(qadapt_ws(nullptr, 1, 1, nullptr) == Q_EINVAL, "null set");
  CHECK(qnorm_rope(nullptr, 1, 1, nullptr, nullptr, nullptr, 0, nullptr, 0, 0, nullptr, 0, nullptr, 0, 0, nullptr) == Q_EINVAL, "null");
  std::printf("%d checks, %d failed\n", g_checks, g_fail);
  return g_fail ? 1 : 0;
}
