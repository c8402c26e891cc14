// Every call of the training-step operators that a CPU can make, with host
// allocations failing one after the other: a call has to return a status, not
// let an exception out. Test infrastructure only.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <new>

#include "wt.h"

namespace {
long g_left = -1;  // allocations before the first that fails; < 0: none fails
bool g_only_one = false, g_failed = false;

void *allocate(std::size_t n) {
  if (g_left == 0) {
    g_failed = true;
    if (g_only_one) g_left = -1;
    throw std::bad_alloc();
  }
  if (g_left > 0) --g_left;
  if (void *p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
}  // namespace

void *operator new(std::size_t n) { return allocate(n); }
void *operator new[](std::size_t n) { return allocate(n); }
void operator delete(void *p) noexcept { std::free(p); }
void operator delete[](void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
void operator delete[](void *p, std::size_t) noexcept { std::free(p); }

static int check(const char *name, const std::function<wt_status()> &call, wt_status refusal) {
  int bad = 0;
  for (int one = 0; one < 2; ++one)
    for (long k = 0; k < 1000; ++k) {
      // a message of another length than the call's own, so that each try allocates afresh
      size_t n = 0;
      (void)wt_dispatch_workspace_bytes(1, 0, 1, &n);
      wt_status st = WT_OK;
      bool threw = false;
      g_failed = false;
      g_only_one = one;
      g_left = k;
      try {
        st = call();
      } catch (...) {
        threw = true;
      }
      g_left = -1;
      if (threw) std::printf("%s: an exception came out at allocation %ld\n", name, k), ++bad;
      else if (g_failed ? st != WT_E_NOMEM && st != refusal : st != refusal)
        std::printf("%s: status %d at allocation %ld\n", name, (int)st, k), ++bad;
      else if (st != WT_OK && !wt_plan_last_error(nullptr)[0])
        std::printf("%s: no message at allocation %ld\n", name, k), ++bad;
      if (!g_failed) break;
    }
  return bad;
}

int main() {
  int bad = 0;
  wt_router_desc d;
  wt_router_desc_init(&d);
  size_t n = 0;
  wt_router_desc wrong = d;
  wrong.n_experts = 100000;
  bad += check("wt_router_workspace_bytes", [&] { return wt_router_workspace_bytes(&wrong, &n); }, WT_E_INVAL);
  bad += check("wt_router_workspace_bytes, NULL", [&] { return wt_router_workspace_bytes(nullptr, &n); }, WT_E_INVAL);
  bad += check("wt_router_forward",
               [&] { return wt_router_forward(&wrong, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr); },
               WT_E_INVAL);
  bad += check("wt_router_backward",
               [&] { return wt_router_backward(&wrong, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr); }, WT_E_INVAL);
  bad += check("wt_dispatch_workspace_bytes", [&] { return wt_dispatch_workspace_bytes(1, 1, 100000, &n); }, WT_E_INVAL);
  bad += check("wt_dispatch_rows",
               [&] {
                 return wt_dispatch_rows(nullptr, 1, 1, 100000, 1, 1, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr);
               },
               WT_E_INVAL);
  wt_adamw_tensor t[3];
  std::memset(t, 0, sizeof t);
  for (int i = 0; i < 3; ++i) {
    t[i].n = 10000;
    t[i].lr_mul = 1.0f;
    const uintptr_t at = 0x1000000 * (uintptr_t)(i + 1);
    t[i].param = (void *)at;
    t[i].grad = (void *)(at + 0x100000);
    t[i].m = (void *)(at + 0x200000);
    t[i].v = (void *)(at + 0x300000);
  }
  bad += check("wt_adamw_check", [&] { return wt_adamw_check(t, 3, nullptr, nullptr); }, WT_OK);
  t[2].v = t[0].m;
  bad += check("wt_adamw_check, overlap", [&] { return wt_adamw_check(t, 3, nullptr, nullptr); }, WT_E_OVERLAP);
  wt_adamw *h = nullptr;
  bad += check("wt_adamw_create, overlap", [&] { return wt_adamw_create(t, 3, nullptr, &h); }, WT_E_OVERLAP);
  std::printf(bad ? "%d failures\n" : "alloc failure ok\n", bad);
  return bad != 0;
}
