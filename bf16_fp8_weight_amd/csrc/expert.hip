// expert.hip -- the experts' BF16 products and the gated feed-forward block.
#include <hip/hip_runtime.h>

#include <string>

#include "expert_tile.h"
#include "hip_util.h"
#include "plan.h"
#include "wt.h"

namespace wt {
namespace {

constexpr int kCus = 256;
constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;

template <int Form, Epilogue Epi, int BM, int BN, int WM, int WN, bool Aligned>
wt_status launch(const char *what, ProductArgs a, hipStream_t stream) {
  constexpr int columns = Epi == Epilogue::kGated ? BN / 2 : BN;
  const int64_t n_tiles = (a.n + columns - 1) / columns;
  const int64_t grid = grid_of(a, Form, BM, n_tiles);
  // Measured (us): gradient of 8192 rows of 12 experts x 2048 columns, 304 tiles, 353 with the rests last and 398 without;
  // x 7168 columns, 1064 tiles, 499 and 473; 16384 rows of 24 experts x 2048 gated, 1216 tiles, 1017 and 937: the rests'
  // weights are read twice.
  a.rests_last = grid <= 2 * kCus;
  if (grid > kMaxGrid) return operator_fail(what, "too many tiles");
  if (grid == 0) return WT_OK;
  auto kernel = product_any_kernel<Form, Epi, false, 128, 128, 2, 2>;
  if constexpr (Aligned) kernel = product_kernel<Form, Epi, false, BM, BN, WM, WN, false>;
  if constexpr (Aligned && Form == kTN)
    if (a.row_index) kernel = product_kernel<Form, Epi, false, BM, BN, WM, WN, true>;
  hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(64 * WM * WN), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return operator_fail(what, hip_msg("launch", e), WT_E_HIP);
  return WT_OK;
}

template <int Form, Epilogue Epi>
wt_status run(const char *what, const ProductArgs &a, hipStream_t stream) {
  if (!product_aligned(a, Form, Epi)) return launch<Form, Epi, 128, 128, 2, 2, false>(what, a, stream);
  const int columns = Epi == Epilogue::kGated ? 128 : 256;
  const int64_t tiles = grid_of(a, Form, 256, (a.n + columns - 1) / columns);
  return tiles < kCus ? launch<Form, Epi, 128, 128, 2, 2, true>(what, a, stream)
                      : launch<Form, Epi, 256, 256, 2, 4, true>(what, a, stream);
}

}  // namespace
}  // namespace wt

using namespace wt;

extern "C" {

wt_status wt_expert_product(const wt_product_desc *desc, void *stream) {
  const char *what = "wt_expert_product";
  try {
    ProductArgs a;
    const wt_status st = product_args(what, desc, Epilogue::kPlain, nullptr, 0, &a);
    if (st != WT_OK) return st;
    const StreamDevice on((hipStream_t)stream);
    if (desc->form == WT_PRODUCT_NT) return run<kNT, Epilogue::kPlain>(what, a, (hipStream_t)stream);
    if (desc->form == WT_PRODUCT_NN) return run<kNN, Epilogue::kPlain>(what, a, (hipStream_t)stream);
    return run<kTN, Epilogue::kPlain>(what, a, (hipStream_t)stream);
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
    return run<kNT, Epilogue::kGated>(what, a, (hipStream_t)stream);
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
    return run<kNN, Epilogue::kGatedBack>(what, a, (hipStream_t)stream);
  } catch (...) {
    return caught_status();
  }
}

}  // extern "C"
