// adamw.cpp -- host side of the AdamW step that needs no GPU: defaults,
// validation of the tensor table and of a step's hyper values, and the work
// list. No HIP call is made here.
#include "adamw.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "plan.h"

namespace wt {
namespace {

struct Range {
  uint64_t lo, hi;
  bool written;
  size_t tensor;
  const char *what;
};

constexpr int64_t kMaxElements = (int64_t)1 << 46;
constexpr double kMaxFactor = 1e6;  // of learning rates and decays: their products stay far from infinity

uint64_t align256(uint64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

wt_adamw_options resolve_adamw_opts(const wt_adamw_options *o) {
  wt_adamw_options d;
  wt_adamw_options_init(&d);
  return o ? *o : d;
}

AdamOffsets adamw_offsets(const AdamLayout &L) {
  AdamOffsets o{};
  o.tensors = 0;
  o.items = align256(o.tensors + L.tensors.size() * sizeof(AdamTensor));
  o.grads = align256(o.items + L.items.size() * sizeof(AdamItem));
  o.partials = align256(o.grads + L.grads.size() * sizeof(AdamGradItem));
  o.norm = align256(o.partials + kAdamNormGrid * sizeof(double));
  o.bytes = align256(o.norm + sizeof(AdamNorm));
  return o;
}

wt_status build_adamw(const wt_adamw_tensor *t, size_t n, const wt_adamw_options &o, AdamLayout *L, std::string *err) {
  if (!t || n == 0) {
    *err = "empty tensor table";
    return WT_E_INVAL;
  }
  if (n > ((size_t)1 << 31)) {
    *err = "too many tensors";
    return WT_E_INVAL;
  }
  if (o.state_bits != 32 && o.state_bits != 8) {
    *err = "state_bits must be 32 or 8";
    return WT_E_INVAL;
  }
  L->state_bits = o.state_bits;
  const bool s8 = o.state_bits == 8;
  std::vector<Range> ranges;
  const uint64_t item = (uint64_t)adam_item(o.state_bits);
  uint64_t blocks = 0, items = 0;
  for (size_t i = 0; i < n; ++i) {
    const wt_adamw_tensor &a = t[i];
    const std::string at = "tensor " + std::to_string(i) + ": ";
    auto bad = [&](const char *m, wt_status st = WT_E_INVAL) {
      *err = at + m;
      return st;
    };
    if (a.n < 0 || a.n > kMaxElements) return bad("element count out of range");
    if (a.grad_dtype != WT_DT_F32 && a.grad_dtype != WT_DT_BF16) return bad("unknown gradient type");
    if (!(a.lr_mul >= 0 && a.lr_mul <= kMaxFactor)) return bad("lr_mul must lie in [0, 1e6]");
    if (!(a.weight_decay >= 0 && a.weight_decay <= kMaxFactor)) return bad("weight_decay must lie in [0, 1e6]");
    if (a.n == 0) continue;
    if (!a.param && !a.master) return bad("neither param nor master");
    if (!a.grad || !a.m || !a.v) return bad("NULL grad, m or v");
    if (s8 && (!a.m_scale || !a.v_scale)) return bad("NULL m_scale or v_scale");
    const uint64_t e = (uint64_t)a.n, nb = (e + kAdamBlock - 1) / kAdamBlock;
    const uint64_t gsize = a.grad_dtype == WT_DT_BF16 ? 2 : 4, ssize = s8 ? 1 : 4;
    auto add = [&](const void *p, uint64_t bytes, uint64_t align, bool written, const char *what) -> wt_status {
      if (!p) return WT_OK;
      const uint64_t lo = (uint64_t)(uintptr_t)p;
      if (lo % align) {
        *err = at + what + " misaligned";
        return WT_E_ALIGN;
      }
      if (lo > UINT64_MAX - bytes) {
        *err = at + what + " runs past the end of the address space";
        return WT_E_RANGE;
      }
      ranges.push_back({lo, lo + bytes, written, i, what});
      return WT_OK;
    };
    wt_status st = WT_OK;
    if (st == WT_OK) st = add(a.param, 2 * e, 2, true, "param");
    if (st == WT_OK) st = add(a.master, 4 * e, 4, true, "master");
    if (st == WT_OK) st = add(a.grad, gsize * e, gsize, false, "grad");
    if (st == WT_OK) st = add(a.m, ssize * e, ssize, true, "m");
    if (st == WT_OK) st = add(a.v, ssize * e, ssize, true, "v");
    if (st == WT_OK && s8) st = add(a.m_scale, 4 * nb, 4, true, "m_scale");
    if (st == WT_OK && s8) st = add(a.v_scale, 4 * nb, 4, true, "v_scale");
    if (st != WT_OK) return st;

    AdamTensor d{};
    d.param = (uint64_t)(uintptr_t)a.param;
    d.master = (uint64_t)(uintptr_t)a.master;
    d.grad = (uint64_t)(uintptr_t)a.grad;
    d.m = (uint64_t)(uintptr_t)a.m;
    d.v = (uint64_t)(uintptr_t)a.v;
    d.m_scale = s8 ? (uint64_t)(uintptr_t)a.m_scale : 0;
    d.v_scale = s8 ? (uint64_t)(uintptr_t)a.v_scale : 0;
    d.n = a.n;
    d.block0 = (uint32_t)blocks;
    d.lr_mul = a.lr_mul;
    d.weight_decay = a.weight_decay;
    if (a.grad_dtype == WT_DT_BF16) d.flags |= kAdamGradBf16;
    if (a.master) d.flags |= kAdamMaster;
    if (a.param) d.flags |= kAdamParam;
    const bool vec = (!a.param || d.param % 8 == 0) && (!a.master || d.master % 16 == 0) && d.grad % (4 * gsize) == 0 &&
                     d.m % (4 * ssize) == 0 && d.v % (4 * ssize) == 0;
    if (vec) d.flags |= kAdamVector, L->info.n_vector_tensors++;
    blocks += nb;
    items += (e + item - 1) / item;
    if (blocks >> 32 || (items * (item / 8)) >> 32) {  // numbers of blocks; threads of the launch, eight elements each
      *err = at + "the table holds too many elements";
      return WT_E_INVAL;
    }
    const uint32_t k = (uint32_t)L->tensors.size();
    for (uint64_t c = 0; c < (e + item - 1) / item; ++c) {
      const uint64_t first = c * item;
      L->items.push_back({k, (uint32_t)c});
      L->grads.push_back({d.grad + gsize * first, (uint32_t)std::min<uint64_t>(item, e - first), d.flags});
    }
    L->tensors.push_back(d);
    L->info.n_elements += a.n;
  }
  std::sort(ranges.begin(), ranges.end(), [](const Range &x, const Range &y) { return x.lo < y.lo; });
  // furthest end seen so far of any range, and of a written one
  uint64_t end_any = 0, end_written = 0;
  size_t last_any = 0, last_written = 0;
  for (size_t i = 0; i < ranges.size(); ++i) {
    const Range &r = ranges[i];
    const bool hit = r.written ? r.lo < end_any : r.lo < end_written;
    if (hit) {
      const Range &q = ranges[r.written ? last_any : last_written];
      *err = "tensor " + std::to_string(r.tensor) + ": " + r.what + " overlaps tensor " + std::to_string(q.tensor) +
             "'s " + q.what;
      return WT_E_OVERLAP;
    }
    if (r.hi > end_any) end_any = r.hi, last_any = i;
    if (r.written && r.hi > end_written) end_written = r.hi, last_written = i;
  }
  L->info.n_tensors = (int64_t)L->tensors.size();
  L->info.n_blocks = (int64_t)blocks;
  L->info.n_items = (int64_t)items;
  L->info.table_bytes = (int64_t)adamw_offsets(*L).bytes;
  return WT_OK;
}

wt_status check_adamw_hyper(const wt_adamw_hyper *h, std::string *err) {
  auto bad = [&](const char *m, wt_status st = WT_E_INVAL) {
    *err = m;
    return st;
  };
  if (!h) return bad("NULL hyper");
  if (!(h->lr >= 0 && h->lr <= kMaxFactor)) return bad("lr must lie in [0, 1e6]");
  if (!(h->beta1 >= 0 && h->beta1 < 1) || !(h->beta2 >= 0 && h->beta2 < 1)) return bad("betas must lie in [0, 1)");
  if (!(h->eps >= 1e-30) || !(h->eps <= 1e30)) return bad("eps must lie in [1e-30, 1e30]");
  if (!std::isfinite(h->grad_scale) || std::fabs(h->grad_scale) > 1e30) return bad("grad_scale out of range");
  if (!(h->max_norm >= 0) || !std::isfinite(h->max_norm)) return bad("max_norm must be finite and not negative");
  if (!h->step_dev && h->step < 1) return bad("step must be at least 1");
  if ((uintptr_t)h->step_dev % 8) return bad("step_dev not 8-byte aligned", WT_E_ALIGN);
  if ((uintptr_t)h->lr_dev % 4) return bad("lr_dev not 4-byte aligned", WT_E_ALIGN);
  if ((uintptr_t)h->norm_out % 4) return bad("norm_out not 4-byte aligned", WT_E_ALIGN);
  return WT_OK;
}

}  // namespace wt

using namespace wt;

extern "C" {

void wt_adamw_options_init(wt_adamw_options *opts) {
  if (!opts) return;
  std::memset(opts, 0, sizeof *opts);
  opts->state_bits = 32;
  opts->device = -1;
}

void wt_adamw_hyper_init(wt_adamw_hyper *hyper) {
  if (!hyper) return;
  std::memset(hyper, 0, sizeof *hyper);
  hyper->lr = 1e-3;
  hyper->beta1 = 0.9;
  hyper->beta2 = 0.999;
  hyper->eps = 1e-8;
  hyper->grad_scale = 1.0;
  hyper->step = 1;
}

wt_status wt_adamw_check(const wt_adamw_tensor *tensors, size_t n_tensors, const wt_adamw_options *opts,
                         wt_adamw_info *info) {
  try {
    AdamLayout L;
    std::string err;
    const wt_status st = build_adamw(tensors, n_tensors, resolve_adamw_opts(opts), &L, &err);
    if (st != WT_OK) {
      set_thread_error("wt_adamw: " + err);
      return st;
    }
    if (info) *info = L.info;
    return WT_OK;
  } catch (...) {
    return caught_status();
  }
}

}  // extern "C"
