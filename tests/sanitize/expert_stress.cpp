// Random descriptions of experts' products, from several threads: each is refused
// with a message or becomes arguments whose extents the kernels can address. No
// GPU code. Usage: expert_stress <descriptions> <threads>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <thread>
#include <vector>

#include "expert.h"
#include "plan.h"

using namespace wt;

namespace {
int64_t pick(std::mt19937_64 &g, std::initializer_list<int64_t> of) { return *(of.begin() + g() % of.size()); }

int64_t size(std::mt19937_64 &g) {
  return pick(g, {1, 2, 7, 32, 1000, (int64_t)(g() % 5000), 1 << 24, (1 << 24) + 1, 0, -1, INT64_MAX, INT64_MIN});
}
int64_t stride(std::mt19937_64 &g, int64_t row) {
  return pick(g, {row, row, row < INT64_MAX / 2 ? row + 4 : row, (int64_t)1 << 40, 0, -8, INT64_MAX});
}

int run(uint64_t seed, int n) {
  std::mt19937_64 g(seed);
  int taken = 0;
  for (int i = 0; i < n; ++i) {
    wt_product_desc d;
    wt_product_desc_init(&d);
    auto address = [&] { return (void *)(uintptr_t)(g() % 10 ? 0x10000 + 2 * (g() % 64) : g() % 2); };
    const bool plain = g() % 2;
    d.n_rows = pick(g, {0, 1, 77, 1 << 27, (int64_t)(g() % 3000), -1, INT64_MAX});
    d.n_experts = (int32_t)pick(g, {1, 1, 5, 1024, 1025, 0});
    d.form = (int32_t)pick(g, {0, 1, 2, 2, 3});
    d.offsets = (const int32_t *)(g() % 2 ? (void *)0x20000 : nullptr);
    d.row_index = (const int32_t *)(g() % 4 ? nullptr : (void *)0x30000);
    d.n_index_rows = pick(g, {0, 5, INT32_MAX, (int64_t)1 << 31, -1});
    d.m = plain ? 64 : size(g);
    d.n = plain ? 96 : size(g);
    d.k = plain ? 128 : size(g);
    d.a = address(), d.b = address(), d.out = address();
    d.a_stride = stride(g, d.form == WT_PRODUCT_TN ? d.m : d.k);
    d.b_stride = stride(g, d.form == WT_PRODUCT_NT ? d.k : d.n);
    d.b_expert_stride = stride(g, 128 * 96);
    d.out_stride = stride(g, d.n);
    d.out_expert_stride = stride(g, 64 * 100);
    d.out_dtype = (int32_t)pick(g, {WT_DT_BF16, WT_DT_BF16, WT_DT_F32, 9});
    ProductArgs a;
    const Epilogue epi = d.form == WT_PRODUCT_NT && g() % 2 ? Epilogue::kGated : Epilogue::kPlain;
    const wt_status st = product_args("stress", &d, epi, nullptr, 0, &a);
    if (st == WT_OK) {
      ++taken;
      const bool direct = product_aligned(a, d.form, epi);
      if (a.n < 1 || (d.form == WT_PRODUCT_TN ? a.m : a.k) < 1) std::printf("a size was taken\n"), std::exit(1);
      if (direct && ((a.a | a.b) % 4 || a.a_stride % 4 || 256 * a.a_stride >= (int64_t)1 << 31 || 256 * a.b_stride >= (int64_t)1 << 31))
        std::printf("far or odd operands on the direct path\n"), std::exit(1);
    } else if (!wt_plan_last_error(nullptr)[0]) {
      std::printf("no message\n"), std::exit(1);
    }
    wt_mxfp4_product_desc x;
    wt_mxfp4_product_desc_init(&x);
    x.n_rows = d.n_rows, x.n_experts = d.n_experts, x.gated = (int32_t)(g() % 3), x.offsets = d.offsets;
    x.n = d.n, x.k = d.k;
    const int64_t nb = x.k > 0 && x.k < 1 << 30 ? (x.k + 31) / 32 : 1;
    x.a = x.b = (void *)0x10000, x.a_scales = x.b_scales = (void *)0x20000, x.out = address();
    x.a_stride = stride(g, 16 * nb), x.b_stride = stride(g, 16 * nb), x.b_expert_stride = stride(g, 16 * nb);
    x.a_scale_stride = stride(g, (nb + 3) / 4 * 4), x.b_scale_stride = stride(g, (nb + 3) / 4 * 4);
    x.out_stride = stride(g, x.n), x.out_dtype = d.out_dtype;
    if (mxfp4_product_args("stress", &x, &a) == WT_OK) ++taken;
    else if (!wt_plan_last_error(nullptr)[0]) std::printf("no message\n"), std::exit(1);
  }
  return taken;
}
}  // namespace

int main(int argc, char **argv) {
  const int n = argc > 1 ? std::atoi(argv[1]) : 1000, threads = argc > 2 ? std::atoi(argv[2]) : 2;
  std::vector<std::thread> t;
  std::vector<int> taken(threads);
  for (int i = 0; i < threads; ++i) t.emplace_back([&, i] { taken[i] = run(i + 1, n); });
  int all = 0;
  for (int i = 0; i < threads; ++i) t[i].join(), all += taken[i];
  if (all == 0) return std::printf("nothing was taken\n"), 1;
  std::printf("expert stress ok: %d taken\n", all);
  return 0;
}
