// expert_run.h -- which kernel a product of given sizes takes, and its launch.
// Included by one source for each form, which compiles that form's kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <string>

#include "expert_tile.h"
#include "hip_util.h"

namespace wt {

constexpr int kCus = 256;
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
  hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(64 * WM * WN * Split), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return operator_fail(what, hip_msg("launch", e), WT_E_HIP);
  return WT_OK;
}

// Which kernel. All rules go by the number of tiles (an upper bound, since the rows of each expert are on the device)
// against 256 CUs. Measured on MI355X, us (k x n; kernel 16 | 64 | 64w = 64 x 128 | 128x = eight waves | 128 | 256 = rows of a tile):
//   64 rows, 2048 x 2048, NT: 6.7 | 9.0 | 13.0 | 12.6 | 16.1          64 rows, 1024 x 2816 gated: 9.8 | 7.4 | - | 9.2 | 11.3 | 13.2
//   200 rows, 512 x 512, NN: 6.3 | 5.9 | 6.9 | 8.8 | 8.3              256 rows, 2816 x 1024 gated: 26.5 | 11.6 | 16.5 | 23.0 | 22.5
//   512 rows, 2048 x 2048, NT: - | 12.2 | 13.3 | 18.0 | 17.6          256 rows, 1024 x 2816 gated: - | 11.0 | 9.6 | 12.3 | 12.1
//   1024 rows, 2048 x 2048, NT: 49.7 | 21.1 | 15.5 | 20.3 | 24.5      1024 rows, 2816 x 1024 gated: - | 28.4 | 21.3 | 27.2 | 32.3
//   1003 rows of 5 experts, NN, 2736 x 1000: 41.4 | 29.8 | 21.8 | 30.9 | 36.6 | 54.8; 2048 rows, NT, 2048 x 1536: - | 30.6 | 25.2 | 20.8 | 24.9
//   4096 rows, 4096 x 4096, NT: - | - | - | 152 | 114 | 106           TN: - | - | - | 132 | 117 | 102
//   2000 rows of 24 experts, 7168 x 2048 gated: - | - | - | 372 | 300 | 336; 8192 cubed, NT: - | - | - | 1196 | 1010 | 804
//   256 rows of 96 experts, 7168 x 2048 gated: 945 | 986 | - | 868 | 859 | 981; 2048 x 7168: 492 | 532 | - | 418 | 445 | 462
// A tile's way through shared memory is what bounds the small ones (a step of 64 x 128 takes 0.13 us, of 128 x 128 0.2 to
// 0.25), so they pay as long as each has a CU of its own. Waves that split the sum shorten the chain of steps (two stages,
// which leave room for two workgroups, are up to 7 % faster than four); 256 x 256 pays from two thirds of a round of
// tiles on (128 | 256: 121 tiles, 2800 rows, 4096 x 2800 NT 62 | 78; 180, 2944 rows, 2048 x 3840 NT 53.5 | 46.5, NN 55 | 46.6; 203, 7312
// rows, 2560 x 864 gated 74 | 62), if experts fill them (rows an expert, 128 | 256): 24 x 7168 x 2048 gated: 83: 300 | 336, 250: 530 | 553, 400: 720 | 716, 500: 839 |
// 750; 16 x 4096 x 4096 NT: 200: 166 | 197, 256: 205 | 226, 400: 273 | 234. (256 x 128 and 128 x 256: 683 rows of 12 experts, 7168 x 2048
// through the gate 365 and 342 against 346; 24 experts' gated batch 1139 and 1109 against 925.)
// Any alignment (64 | 64 x 128 | 128): 2001 rows, 4001 x 777, NT 49 | 61 | 76, NN 68 | 76 | 106, its TN 56 | 57 | 61; 777 x 4001
// NT 43 | 39 | 29; 333 rows, 501 x 1001 gated 9.4 | 12.1 | 16.9; 8001 rows, 4097 x 4097 655 | 538 | 437.
template <int Form, Epilogue Epi>
wt_status run_product(const char *what, const ProductArgs &a, hipStream_t stream) {
  const int64_t halves = Epi == Epilogue::kGated ? 2 : 1;  // of a tile's columns are out's
  auto tiles = [&](int rows, int columns) { return grid_of(a, Form, rows, (a.n * halves + columns - 1) / columns); };
  if (!product_aligned(a, Form, Epi)) {
    if (tiles(128, 128) >= kCus) return launch<Form, Epi, 128, 128, 2, 2, 1, 2, 2, false>(what, a, stream);
    return launch<Form, Epi, 64, 64, Form == kNT ? 4 : 2, Form == kNT ? 1 : 2, 1, 2, 2, false>(what, a, stream);
  }
  if constexpr (Form != kTN)
    if (tiles(16, 64) <= kCus) return launch<Form, Epi, 16, 64, 1, 1, 8, 2, 2, true>(what, a, stream);
  if (tiles(64, 64) <= kCus) return launch<Form, Epi, 64, 64, 1, 1, 4, 1, 2, true>(what, a, stream);
  if (tiles(64, 128) <= kCus) return launch<Form, Epi, 64, 128, 2, 2, 1, 1, 4, true>(what, a, stream);
  if (3 * tiles(256, 256) >= 2 * kCus && (Form == kTN || a.n_rows > 256 * (int64_t)a.n_experts))
    return launch<Form, Epi, 256, 256, 2, 4, 1, 1, 4, true>(what, a, stream);
  return tiles(128, 128) >= kCus ? launch<Form, Epi, 128, 128, 2, 2, 1, 2, 2, true>(what, a, stream)
                                 : launch<Form, Epi, 128, 128, 4, 2, 1, 1, 4, true>(what, a, stream);
}

}  // namespace wt
