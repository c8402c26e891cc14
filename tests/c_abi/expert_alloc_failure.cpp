// The calls of the experts' products and of MXFP4 that a CPU can make (refusals and
// empty row spaces), with host allocations failing one after the other: a call has
// to return a status, not let an exception out. Test infrastructure only.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <new>

#include "wt.h"

namespace {
long g_left = -1;  // allocations before the first that fails; < 0: none fails
bool g_failed = false;

void *allocate(std::size_t n) {
  if (g_left == 0) {
    g_failed = true;
    throw std::bad_alloc();
  }
  if (g_left > 0) --g_left;
  if (void *p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}

int check(const char *name, const std::function<wt_status()> &call, wt_status refusal) {
  int bad = 0;
  for (long k = 0; k < 1000; ++k) {
    wt_status st = WT_OK;
    bool threw = false;
    g_failed = false;
    g_left = k;
    try {
      st = call();
    } catch (...) {
      threw = true;
    }
    g_left = -1;
    if (threw) std::printf("%s: an exception came out at allocation %ld\n", name, k), ++bad;
    else if (st != refusal && !(g_failed && st == WT_E_NOMEM))
      std::printf("%s: status %d at allocation %ld\n", name, (int)st, k), ++bad;
    else if (st != WT_OK && !wt_plan_last_error(nullptr)[0])
      std::printf("%s: no message at allocation %ld\n", name, k), ++bad;
    if (!g_failed) break;
  }
  return bad;
}
}  // namespace

void *operator new(std::size_t n) { return allocate(n); }
void *operator new[](std::size_t n) { return allocate(n); }
void operator delete(void *p) noexcept { std::free(p); }
void operator delete[](void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
void operator delete[](void *p, std::size_t) noexcept { std::free(p); }

int main() {
  int bad = 0;
  wt_product_desc d;
  wt_product_desc_init(&d);
  bad += check("wt_expert_product", [&] { return wt_expert_product(&d, nullptr); }, WT_E_INVAL);
  bad += check("wt_expert_product, NULL", [] { return wt_expert_product(nullptr, nullptr); }, WT_E_INVAL);
  bad += check("wt_gated_forward", [&] { return wt_gated_forward(&d, nullptr, 0, nullptr); }, WT_E_INVAL);
  bad += check("wt_gated_backward", [&] { return wt_gated_backward(&d, nullptr, 0, nullptr); }, WT_E_INVAL);
  wt_mxfp4_product_desc x;
  wt_mxfp4_product_desc_init(&x);
  bad += check("wt_mxfp4_product", [&] { return wt_mxfp4_product(&x, nullptr); }, WT_E_INVAL);
  x.n = x.k = 32;
  x.a_stride = x.b_stride = 24;
  x.a_scale_stride = x.b_scale_stride = x.out_stride = 32;
  bad += check("wt_mxfp4_product, alignment", [&] { return wt_mxfp4_product(&x, nullptr); }, WT_E_ALIGN);
  bad += check("wt_mxfp4_quantize",
               [] { return wt_mxfp4_quantize(nullptr, WT_DT_F32, -1, 1, 1, nullptr, 1, nullptr, 16, nullptr, 1, nullptr); }, WT_E_INVAL);
  bad += check("wt_mxfp4_quantize, nothing",
               [] { return wt_mxfp4_quantize(nullptr, WT_DT_F32, 0, 1, 1, nullptr, 0, nullptr, 16, nullptr, 1, nullptr); }, WT_OK);
  bad += check("wt_mxfp4_dequantize",
               [] { return wt_mxfp4_dequantize(nullptr, 16, nullptr, 1, 1, 1, nullptr, WT_DT_F32, 1, nullptr); }, WT_E_INVAL);
  std::printf(bad ? "%d failures\n" : "alloc failure ok\n", bad);
  return bad != 0;
}
