// expert_run.h -- the kernels of a form and their launch; which of them a product of given sizes takes is expert.cpp's.
// Included by one source for each form, which compiles that form's kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <string>

#include "expert_tile.h"
#include "hip_util.h"
#include "launch_parts.h"

namespace wt {

constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;

template <int Form, Epilogue Epi, int BM, int BN, int WM, int WN, int Split, int Sub, int Stages, bool Aligned>
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
  auto kernel = [] {
    if constexpr (Aligned) return product_kernel<Form, Epi, false, BM, BN, WM, WN, Split, Sub, Stages, false>;
    else return product_any_kernel<Form, Epi, false, BM, BN, WM, WN, Sub>;
  }();
  if constexpr (Aligned && Form == kTN)
    if (a.row_index) kernel = product_kernel<Form, Epi, false, BM, BN, WM, WN, Split, Sub, Stages, true>;
  constexpr uint32_t threads = 64 * WM * WN * Split;
  const hipError_t e = launch_parts(grid, threads, hipSuccess, [&](uint32_t first, uint32_t count) {
    a.first_group = first;
    hipLaunchKernelGGL(kernel, dim3(count), dim3(threads), 0, stream, a);
    return hipGetLastError();
  });
  if (e != hipSuccess) return operator_fail(what, hip_msg("launch", e), WT_E_HIP);
  return WT_OK;
}

// The kernel that product_kernel_of() names; a form has those that it can name.
template <int Form, Epilogue Epi>
wt_status run_product(const char *what, const ProductArgs &a, hipStream_t stream) {
  switch (product_kernel_of(a, Form, Epi)) {
    case Kernel::kAny128: return launch<Form, Epi, 128, 128, 2, 2, 1, 2, 2, false>(what, a, stream);
    case Kernel::kAny64: return launch<Form, Epi, 64, 64, Form == kNT ? 4 : 2, Form == kNT ? 1 : 2, 1, 2, 2, false>(what, a, stream);
    case Kernel::k16Split:
      if constexpr (Form != kTN) return launch<Form, Epi, 16, 64, 1, 1, 8, 2, 2, true>(what, a, stream);
      break;
    case Kernel::k64Split: return launch<Form, Epi, 64, 64, 1, 1, 4, 1, 2, true>(what, a, stream);
    case Kernel::k64x128: return launch<Form, Epi, 64, 128, 2, 2, 1, 1, 4, true>(what, a, stream);
    case Kernel::k128: return launch<Form, Epi, 128, 128, 2, 2, 1, 2, 2, true>(what, a, stream);
    case Kernel::k128Wide: return launch<Form, Epi, 128, 128, 4, 2, 1, 1, 4, true>(what, a, stream);
    case Kernel::k256: return launch<Form, Epi, 256, 256, 2, 4, 1, 1, 4, true>(what, a, stream);
    default: break;
  }
  return operator_fail(what, "no kernel");
}

}  // namespace wt
