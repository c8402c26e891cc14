// expert.cpp -- the checks of the experts' products: a description is refused
// here or becomes the arguments of a kernel. No GPU call.
#include "expert.h"

#include <cstring>

#include "plan.h"

namespace wt {

wt_status operator_fail(const char *what, const std::string &m, wt_status st) {
  set_thread_error(std::string(what) + ": " + m);
  return st;
}

namespace {

// Row strides (in elements or bytes) with which the last of `rows` rows still has
// a 64-bit byte offset.
int64_t max_stride(int64_t rows) { return ((int64_t)1 << 59) / (rows > 1 ? rows : 1); }

bool stride_ok(int64_t stride, int64_t row, int64_t rows) { return stride >= row && stride <= max_stride(rows); }

bool size_ok(int64_t n) { return n >= 1 && n <= kProductMaxSize; }

wt_status check_rows(const char *what, int64_t n_rows, int32_t n_experts, const int32_t *offsets,
                     const int32_t *counts) {
  if (n_rows < 0 || n_rows > kProductMaxRows) return operator_fail(what, "n_rows out of range");
  if (n_experts < 1 || n_experts > kProductMaxExperts) return operator_fail(what, "n_experts out of range");
  if (!offsets && n_experts != 1) return operator_fail(what, "several experts without offsets");
  if (!offsets && counts) return operator_fail(what, "counts without offsets");
  if (((uintptr_t)offsets | (uintptr_t)counts) % 4) return operator_fail(what, "offsets or counts misaligned", WT_E_ALIGN);
  return WT_OK;
}

}  // namespace

wt_status product_args(const char *what, const wt_product_desc *d, Epilogue epi, const void *pre, int64_t pre_stride,
                       ProductArgs *a) {
  if (!d) return operator_fail(what, "NULL description");
  const wt_status st = check_rows(what, d->n_rows, d->n_experts, d->offsets, d->counts);
  if (st != WT_OK) return st;
  const int form = d->form;
  if (form != WT_PRODUCT_NT && form != WT_PRODUCT_NN && form != WT_PRODUCT_TN) return operator_fail(what, "unknown form");
  if (epi == Epilogue::kGated && form != WT_PRODUCT_NT) return operator_fail(what, "form must be WT_PRODUCT_NT");
  if (epi == Epilogue::kGatedBack && form != WT_PRODUCT_NN) return operator_fail(what, "form must be WT_PRODUCT_NN");
  const bool tn = form == WT_PRODUCT_TN;
  if (!size_ok(d->n) || (tn && !size_ok(d->m)) || (!tn && !size_ok(d->k))) return operator_fail(what, "m, n or k out of range");
  if (d->out_dtype != WT_DT_F32 && d->out_dtype != WT_DT_BF16) return operator_fail(what, "unknown out type");
  if (epi != Epilogue::kPlain && d->out_dtype != WT_DT_BF16) return operator_fail(what, "out must be BF16");
  if (epi != Epilogue::kPlain && d->act != WT_ACT_SILU && d->act != WT_ACT_GELU) return operator_fail(what, "unknown activation");
  if (d->row_index && (d->n_index_rows < 0 || d->n_index_rows >= (int64_t)1 << 31))
    return operator_fail(what, "n_index_rows out of range");
  if ((uintptr_t)d->row_index % 4) return operator_fail(what, "row_index misaligned", WT_E_ALIGN);

  const int64_t gathered = d->row_index ? d->n_index_rows : d->n_rows;
  const int64_t a_rows = tn ? d->n_rows : gathered, a_row = tn ? d->m : d->k;
  const int64_t b_rows = tn ? gathered : form == WT_PRODUCT_NT ? d->n * (epi == Epilogue::kGated ? 2 : 1) : d->k;
  const int64_t b_row = form == WT_PRODUCT_NT ? d->k : d->n;
  const int64_t out_rows = tn ? d->m : d->n_rows, out_row = d->n * (epi == Epilogue::kGatedBack ? 2 : 1);
  if (!stride_ok(d->a_stride, a_row, a_rows)) return operator_fail(what, "a_stride out of range");
  if (!stride_ok(d->b_stride, b_row, b_rows)) return operator_fail(what, "b_stride out of range");
  if (!stride_ok(d->out_stride, out_row, out_rows)) return operator_fail(what, "out_stride out of range");
  if (!tn && d->n_experts > 1 &&
      (d->b_expert_stride < 0 || d->b_expert_stride > max_stride(d->n_experts) / 2))
    return operator_fail(what, "b_expert_stride out of range");
  if (tn && d->n_experts > 1 &&
      (d->out_expert_stride < (d->m - 1) * d->out_stride + d->n || d->out_expert_stride > max_stride(d->n_experts)))
    return operator_fail(what, "out_expert_stride out of range");
  if (pre && !stride_ok(pre_stride, 2 * d->n, d->n_rows)) return operator_fail(what, "pre_stride out of range");
  const bool rows = d->n_rows > 0;
  if (rows && ((!d->a && a_rows > 0) || (!d->b && b_rows > 0))) return operator_fail(what, "NULL a or b");
  if ((rows || tn) && !d->out) return operator_fail(what, "NULL out");
  if (epi == Epilogue::kGatedBack && rows && !pre) return operator_fail(what, "NULL pre");
  if (((uintptr_t)d->a | (uintptr_t)d->b | (uintptr_t)pre) % 2) return operator_fail(what, "a, b or pre misaligned", WT_E_ALIGN);
  const int64_t out_size = d->out_dtype == WT_DT_F32 ? 4 : 2;
  if ((uintptr_t)d->out % out_size) return operator_fail(what, "out misaligned", WT_E_ALIGN);

  *a = ProductArgs{};
  a->offsets = d->offsets;
  a->counts = d->counts;
  a->row_index = d->row_index;
  a->a = (uint64_t)(uintptr_t)d->a;
  a->b = (uint64_t)(uintptr_t)d->b;
  a->out = (uint64_t)(uintptr_t)d->out;
  a->pre = (uint64_t)(uintptr_t)pre;
  a->a_stride = 2 * d->a_stride;
  a->b_stride = 2 * d->b_stride;
  a->b_expert = !tn && d->n_experts > 1 ? 2 * d->b_expert_stride : 0;
  a->out_stride = d->out_stride;
  a->out_expert = tn && d->n_experts > 1 ? d->out_expert_stride : 0;
  a->pre_stride = pre ? pre_stride : 0;
  a->n_rows = d->n_rows;
  a->n_index_rows = d->row_index ? d->n_index_rows : d->n_rows;
  a->n_experts = d->n_experts;
  a->m = tn ? (int32_t)d->m : 0;
  a->n = (int32_t)d->n;
  a->k = tn ? 0 : (int32_t)d->k;
  a->act = d->act;
  a->out_f32 = d->out_dtype == WT_DT_F32;
  return WT_OK;
}

wt_status mxfp4_product_args(const char *what, const wt_mxfp4_product_desc *d, ProductArgs *a) {
  if (!d) return operator_fail(what, "NULL description");
  const wt_status st = check_rows(what, d->n_rows, d->n_experts, d->offsets, d->counts);
  if (st != WT_OK) return st;
  if (d->gated != 0 && d->gated != 1) return operator_fail(what, "gated must be 0 or 1");
  if (!size_ok(d->n) || !size_ok(d->k)) return operator_fail(what, "n or k out of range");
  if (d->out_dtype != WT_DT_F32 && d->out_dtype != WT_DT_BF16) return operator_fail(what, "unknown out type");
  if (d->gated && d->out_dtype != WT_DT_BF16) return operator_fail(what, "out must be BF16");
  if (d->gated && d->act != WT_ACT_SILU && d->act != WT_ACT_GELU) return operator_fail(what, "unknown activation");
  const int64_t nb = (d->k + 31) / 32, b_rows = d->n * (1 + d->gated);
  if (!stride_ok(d->a_stride, 16 * nb, d->n_rows)) return operator_fail(what, "a_stride out of range");
  if (!stride_ok(d->a_scale_stride, nb, d->n_rows)) return operator_fail(what, "a_scale_stride out of range");
  if (!stride_ok(d->b_stride, 16 * nb, b_rows)) return operator_fail(what, "b_stride out of range");
  if (!stride_ok(d->b_scale_stride, nb, b_rows)) return operator_fail(what, "b_scale_stride out of range");
  if (!stride_ok(d->out_stride, d->n, d->n_rows)) return operator_fail(what, "out_stride out of range");
  const int64_t most = max_stride(d->n_experts) / 2;
  if (d->n_experts > 1 && (d->b_expert_stride < 0 || d->b_expert_stride > most)) return operator_fail(what, "b_expert_stride out of range");
  if (d->n_experts > 1 && (d->b_scale_expert_stride < 0 || d->b_scale_expert_stride > most))
    return operator_fail(what, "b_scale_expert_stride out of range");
  if (d->n_rows > 0 && (!d->a || !d->b || !d->a_scales || !d->b_scales || !d->out)) return operator_fail(what, "NULL pointer");
  const int64_t codes = (int64_t)((uintptr_t)d->a | (uintptr_t)d->b) | d->a_stride | d->b_stride |
                        (d->n_experts > 1 ? d->b_expert_stride : 0);
  if (codes % 16) return operator_fail(what, "codes not 16-byte aligned", WT_E_ALIGN);
  const int64_t scales = (int64_t)((uintptr_t)d->a_scales | (uintptr_t)d->b_scales) | d->a_scale_stride |
                         d->b_scale_stride | (d->n_experts > 1 ? d->b_scale_expert_stride : 0);
  if (scales % 4) return operator_fail(what, "scales not 4-byte aligned", WT_E_ALIGN);
  const int64_t out_size = d->out_dtype == WT_DT_F32 ? 4 : 2;
  if ((uintptr_t)d->out % out_size) return operator_fail(what, "out misaligned", WT_E_ALIGN);

  *a = ProductArgs{};
  a->offsets = d->offsets;
  a->counts = d->counts;
  a->a = (uint64_t)(uintptr_t)d->a;
  a->b = (uint64_t)(uintptr_t)d->b;
  a->a_scales = (uint64_t)(uintptr_t)d->a_scales;
  a->b_scales = (uint64_t)(uintptr_t)d->b_scales;
  a->out = (uint64_t)(uintptr_t)d->out;
  a->a_stride = d->a_stride;
  a->b_stride = d->b_stride;
  a->b_expert = d->n_experts > 1 ? d->b_expert_stride : 0;
  a->a_scale_stride = d->a_scale_stride;
  a->b_scale_stride = d->b_scale_stride;
  a->b_scale_expert = d->n_experts > 1 ? d->b_scale_expert_stride : 0;
  a->out_stride = d->out_stride;
  a->n_rows = d->n_rows;
  a->n_index_rows = d->n_rows;
  a->n_experts = d->n_experts;
  a->n = (int32_t)d->n;
  a->k = (int32_t)d->k;
  a->act = d->act;
  a->out_f32 = d->out_dtype == WT_DT_F32;
  return WT_OK;
}

bool product_aligned(const ProductArgs &a, int form, Epilogue epi) {
  const int64_t far = (int64_t)1 << 31;
  const int64_t bits = (int64_t)(a.a | a.b) | a.a_stride | a.b_stride | a.b_expert;
  if (bits % 4) return false;
  const bool tn = form == WT_PRODUCT_TN;
  // 256 rows of a tile, and a step along the sum behind the last
  if (a.a_stride > far / 512 || a.b_stride > far / 512) return false;
  if (a.row_index && a.n_index_rows * (tn ? a.b_stride : a.a_stride) >= far) return false;
  if (epi == Epilogue::kGated && (int64_t)(a.n + 512) * a.b_stride >= far) return false;
  if (tn) return a.m % 2 == 0 && a.n % 2 == 0;
  return a.k % 2 == 0 && (form == WT_PRODUCT_NT || a.n % 2 == 0);
}

}  // namespace wt

using namespace wt;

extern "C" {

void wt_product_desc_init(wt_product_desc *desc) {
  if (!desc) return;
  std::memset(desc, 0, sizeof *desc);
  desc->n_experts = 1;
  desc->out_dtype = WT_DT_BF16;
}

void wt_mxfp4_product_desc_init(wt_mxfp4_product_desc *desc) {
  if (!desc) return;
  std::memset(desc, 0, sizeof *desc);
  desc->n_experts = 1;
  desc->out_dtype = WT_DT_BF16;
}

}  // extern "C"
