// expert.hip -- entry points of the experts' BF16 products and the gated
// feed-forward block. The kernels of each form are compiled by a source of their own.
#include <hip/hip_runtime.h>

#include <string>

#include "expert.h"
#include "hip_util.h"
#include "plan.h"
#include "wt.h"

using namespace wt;

extern "C" {

wt_status wt_expert_product(const wt_product_desc *desc, void *stream) {
  const char *what = "wt_expert_product";
  try {
    ProductArgs a;
    const wt_status st = product_args(what, desc, Epilogue::kPlain, nullptr, 0, &a);
    if (st != WT_OK) return st;
    const StreamDevice on((hipStream_t)stream);
    if (desc->form == WT_PRODUCT_NT) return run_product<WT_PRODUCT_NT, Epilogue::kPlain>(what, a, (hipStream_t)stream);
    if (desc->form == WT_PRODUCT_NN) return run_product<WT_PRODUCT_NN, Epilogue::kPlain>(what, a, (hipStream_t)stream);
    return run_product<WT_PRODUCT_TN, Epilogue::kPlain>(what, a, (hipStream_t)stream);
  } catch (...) {
    return caught_status();
  }
}

wt_status wt_gated_forward(const wt_product_desc *desc, void *pre, int64_t pre_stride, void *stream) {
  const char *what = "wt_gated_forward";
  try {
    ProductArgs a;
    const wt_status st = product_args(what, desc, Epilogue::kGated, pre, pre_stride, &a);
    if (st != WT_OK) return st;
    const StreamDevice on((hipStream_t)stream);
    return run_product<WT_PRODUCT_NT, Epilogue::kGated>(what, a, (hipStream_t)stream);
  } catch (...) {
    return caught_status();
  }
}

wt_status wt_gated_backward(const wt_product_desc *desc, const void *pre, int64_t pre_stride, void *stream) {
  const char *what = "wt_gated_backward";
  try {
    ProductArgs a;
    const wt_status st = product_args(what, desc, Epilogue::kGatedBack, pre, pre_stride, &a);
    if (st != WT_OK) return st;
    const StreamDevice on((hipStream_t)stream);
    return run_product<WT_PRODUCT_NN, Epilogue::kGatedBack>(what, a, (hipStream_t)stream);
  } catch (...) {
    return caught_status();
  }
}

}  // extern "C"
