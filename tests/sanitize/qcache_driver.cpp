// Drives the entry points of include/qcache.h on the host, with the library's
// host code built under the address and undefined-behaviour sanitizers and
// linked against the host-only HIP stand-in (fake_hip.cpp): accepted calls
// launch kernels within a launch's limits over sizes from one row to the
// largest the ABI takes, rejected ones launch nothing, and the size queries
// survive sizes of every magnitude.  Device pointers are fake addresses the
// host code never dereferences.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "fake_hip.h"
#include "qcache.h"

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
const hipStream_t S = nullptr;

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

qcache cache_of(int64_t n_pages, int page_size, int heads, int head_dim, int bits) {
  return qcache{n_pages, page_size, heads, head_dim, bits, dp(1), dp(2), dp(3), dp(4)};
}
qseqs seqs_of(int64_t B, int64_t T, int64_t max_pages, bool starts) {
  return qseqs{B, T, max_pages, static_cast<int32_t*>(dp(5)), static_cast<int32_t*>(dp(6)),
               starts ? static_cast<int32_t*>(dp(7)) : nullptr};
}

// every entry point with one set of sizes; all accepted or (attention only)
// refused as too large, all launches within the limits
void call_all(const qcache& c, const qseqs& s, int group, int64_t prefix) {
  const int64_t width = (int64_t)c.heads * c.head_dim;
  const int q_heads = c.heads * group;
  for (int dt : {(int)Q_BF16, (int)Q_F32}) {
    const long before = fake_hip_launches();
    CHECK(qcache_write(&c, &s, dp(8), width, dp(9), width + 8, dt, S) == Q_OK, "write");
    CHECK(qcache_read(&c, &s, dp(8), width, dp(9), width + 8, dt, S) == Q_OK, "read");
    CHECK(fake_hip_launches() == before + 2, "write and read launch one kernel each");
  }
  for (int64_t p : {(int64_t)0, prefix}) {
    size_t need = 0;
    const int st = qcache_attend_ws(&c, &s, q_heads, p, &need);
    CHECK(st == Q_OK || st == Q_EUNSUPPORTED, "ws query %d", st);
    if (st == Q_OK) CHECK(need > 0 && need % 16 == 0, "ws bytes %zu", need);
    for (int short_by : {0, 1}) {
      const long before = fake_hip_launches();
      const int got = p ? qcache_attend_shared(&c, &s, static_cast<int32_t*>(dp(10)), p, dp(8), width * group, q_heads,
                                               0.125f, dp(9), width * group, Q_BF16, dp(11), need - short_by, S)
                        : qcache_attend(&c, &s, dp(8), width * group, q_heads, 0.125f, dp(9), width * group, Q_F32,
                                        dp(11), need - short_by, S);
      if (st != Q_OK || short_by) {
        CHECK(got < 0 && fake_hip_launches() == before, "refused call: %d", got);
      } else {
        CHECK(got == Q_OK, "attend %d", got);
        CHECK(fake_hip_launches() > before && fake_hip_launches() <= before + (p ? 4 : 3), "%ld launches", fake_hip_launches() - before);
      }
    }
  }
}

}  // namespace

int main() {
  const int pages[] = {16, 32, 64, 128, 256};
  for (int i = 0; i < 20000; ++i) {
    const int head_dim = next() % 2 ? 64 : 128, bits = next() % 2 ? 4 : 8, page = pages[next() % 5];
    const int64_t B = upto(65536);
    const bool starts = next() % 2;
    const int64_t T = starts ? upto((int64_t)1 << 27) : B;
    const qcache c = cache_of(upto(INT32_MAX), page, (int)upto(64) * (next() % 4 ? 1 : 16), head_dim, bits);
    call_all(c, seqs_of(B, T, upto(((int64_t)1 << 30) / page), starts), (int)upto(64), upto((int64_t)1 << 30));
  }
  // the ends of every range
  for (int64_t B : {(int64_t)1, (int64_t)65536})
    for (int64_t T : {(int64_t)1, (int64_t)1 << 27})
      for (int heads : {1, 1024})
        for (int group : {1, 64})
          for (int64_t n : {(int64_t)1, (int64_t)1 << 26})
            call_all(cache_of(INT32_MAX, 16, heads, 64, 8), seqs_of(B, T, n, true), group, n * 16);
  // queries and calls with sizes of every magnitude: no overflow, no launch outside the limits
  for (int i = 0; i < 200000; ++i) {
    size_t a = 0, b = 0;
    const int page = next() % 3 ? pages[next() % 5] : (int)any_size(), dim = next() % 3 ? 64 : (int)any_size();
    const int heads = next() % 2 ? (int)upto(1024) : (int)any_size(), bits = next() % 4 ? 8 : (int)any_size();
    const int64_t n = any_size();
    const bool fits = qcache_sizes(n, page, heads, dim, bits, &a, &b) == Q_OK;
    if (fits) CHECK(a == (size_t)n * heads * page * (dim * bits / 8) && b == (size_t)n * heads * page * 4, "sizes");
    const qcache c = cache_of(n, page, heads, dim, bits);
    const qseqs s = seqs_of(any_size(), any_size(), any_size(), next() % 2);
    const int q_heads = next() % 2 ? heads : (int)any_size();
    const int64_t prefix = any_size();
    const long before = fake_hip_launches();
    if (qcache_attend_ws(&c, &s, q_heads, prefix, &a) != Q_OK) {
      const int st = qcache_attend_shared(&c, &s, static_cast<int32_t*>(dp(10)), prefix, dp(8), any_size(), q_heads, 1.f,
                                          dp(9), any_size(), Q_BF16, dp(11), (size_t)1 << 62, S);
      CHECK(st < 0 && fake_hip_launches() == before, "call accepted, its query was not");
    }
    qcache_write(&c, &s, dp(8), any_size(), dp(9), any_size(), Q_BF16, S);
    qcache_read(&c, &s, dp(8), any_size(), dp(9), any_size(), Q_F32, S);
  }
  std::printf("%d checks, %d failed, %ld launches recorded, %ld outside the limits\n", g_checks, g_fail,
              fake_hip_launches(), fake_hip_bad_launches());
  return g_fail == 0 && fake_hip_bad_launches() == 0 ? 0 : 1;
}
