// Host-side stress of the AdamW step's table builder for sanitizer builds.
// Test infrastructure only.
//
// Each worker draws seeded random tensor tables -- sizes from 0 up, both
// gradient types, with and without master, shard and scales, packed, shared,
// overlapping or misaligned addresses (none is dereferenced) -- and checks
// what wt_adamw_check says: an accepted table's counts follow from its sizes,
// and a table whose written ranges overlap by construction is refused.
//
// usage: adamw_stress ITERATIONS THREADS
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <thread>
#include <vector>

#include "wt.h"

namespace {

struct Rng {
  uint64_t s;
  explicit Rng(uint64_t seed) : s(seed * 0x9E3779B97F4A7C15ull + 1) {}
  uint64_t next() {
    s ^= s << 13, s ^= s >> 7, s ^= s << 17;
    return s;
  }
  int64_t in(int64_t lo, int64_t hi) { return lo + (int64_t)(next() % (uint64_t)(hi - lo + 1)); }
  bool p(int percent) { return (int)(next() % 100) < percent; }
};

int run(uint64_t first, uint64_t count) {
  int bad = 0;
  for (uint64_t i = first; i < first + count; ++i) {
    Rng r(i + 1);
    const int n = (int)r.in(1, 40);
    const bool s8 = r.p(50);
    std::vector<wt_adamw_tensor> t(n);
    uint64_t at = 0x100000;
    auto place = [&](uint64_t bytes, uint64_t align) {
      at = (at + align - 1) / align * align;
      const uint64_t p = at;
      at += bytes;
      return (void *)(uintptr_t)p;
    };
    int64_t elements = 0, blocks = 0, tensors = 0;
    for (auto &a : t) {
      std::memset(&a, 0, sizeof a);
      a.n = r.p(10) ? 0 : r.p(3) ? r.in(1, (int64_t)1 << 25) : r.in(1, 20000);
      a.grad_dtype = r.p(50) ? WT_DT_BF16 : WT_DT_F32;
      a.lr_mul = 1.0f;
      const uint64_t e = (uint64_t)a.n, nb = (e + 127) / 128, vec = r.p(50) ? 16 : 4;
      a.master = r.p(70) ? (float *)place(4 * e, vec) : nullptr;
      a.param = !a.master || r.p(80) ? place(2 * e, r.p(50) ? 8 : 2) : nullptr;
      a.grad = place((a.grad_dtype == WT_DT_BF16 ? 2 : 4) * e, vec);
      a.m = place((s8 ? 1 : 4) * e, s8 ? 1 : vec);
      a.v = place((s8 ? 1 : 4) * e, s8 ? 1 : vec);
      a.m_scale = (float *)place(4 * nb, 4);
      a.v_scale = (float *)place(4 * nb, 4);
      elements += a.n;
      blocks += (int64_t)nb;
      tensors += a.n > 0;
    }
    wt_adamw_options o;
    wt_adamw_options_init(&o);
    o.state_bits = s8 ? 8 : 32;
    wt_adamw_info info;
    const bool fits = blocks < ((int64_t)1 << 32);
    wt_status st = wt_adamw_check(t.data(), t.size(), &o, &info);
    if (fits != (st == WT_OK)) ++bad, std::fprintf(stderr, "seed %llu: status %d: %s\n", (unsigned long long)i, st,
                                                  wt_plan_last_error(nullptr));
    if (st == WT_OK && (info.n_elements != elements || info.n_blocks != blocks || info.n_tensors != tensors))
      ++bad, std::fprintf(stderr, "seed %llu: counts\n", (unsigned long long)i);
    // one tensor's m moved onto another range of the table
    const int k = (int)r.in(0, n - 1), j = (int)r.in(0, n - 1);
    if (st == WT_OK && t[k].n > 0 && t[j].n > 0) {
      std::vector<wt_adamw_tensor> u = t;
      const uint64_t target = (uint64_t)(uintptr_t)t[j].grad + 4 * (uint64_t)r.in(0, (t[j].n - 1) / 4);
      u[k].m = (void *)(uintptr_t)(target / 4 * 4);
      if (wt_adamw_check(u.data(), u.size(), &o, nullptr) != WT_E_OVERLAP)
        ++bad, std::fprintf(stderr, "seed %llu: overlap not seen\n", (unsigned long long)i);
    }
  }
  return bad;
}

}  // namespace

int main(int argc, char **argv) {
  const uint64_t iterations = argc > 1 ? std::strtoull(argv[1], nullptr, 10) : 100;
  const int threads = argc > 2 ? std::atoi(argv[2]) : 1;
  std::vector<int> bad(threads, 0);
  std::vector<std::thread> ts;
  for (int k = 0; k < threads; ++k)
    ts.emplace_back([&, k] { bad[k] = run(1000000ull * k, iterations); });
  for (auto &t : ts) t.join();
  int total = 0;
  for (int b : bad) total += b;
  if (total) return 1;
  std::printf("adamw stress ok\n");
  return 0;
}
