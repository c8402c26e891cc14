// expert.cpp -- the checks of the experts' products: a description is refused
// here or becomes the arguments of a kernel -- and which kernel that is. No GPU call.
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

int64_t grid_of(const ProductArgs &a, int form, int bm, int64_t n_tiles) {
  if (form == WT_PRODUCT_TN) return (((int64_t)(a.m + bm - 1) / bm * n_tiles + kXcds - 1) / kXcds) * kXcds * a.n_experts;
  // experts' last tiles; how many there are is known here for a dense layer
  const int64_t rests = !a.offsets ? a.n_rows % bm != 0 : a.n_rows < a.n_experts ? a.n_rows : a.n_experts;
  return ((a.n_rows / bm * n_tiles + kXcds - 1) / kXcds + (rests * n_tiles + kXcds - 1) / kXcds) * kXcds;
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
// A tile's way through shared memory is what bounds the small ones (32 terms of a sum take 0.19 us in a tile of 64 x 128, 0.23 in 128 x 128 with
// eight waves, 0.33 with four, 0.72 in 256 x 256), so they pay as long as each has a CU of its own. Waves that split the sum shorten the chain of steps (two stages,
// which leave room for two workgroups, are up to 7 % faster than four); 256 x 256 pays from two thirds of a round of
// tiles on (128 | 256: 121 tiles, 2800 rows, 4096 x 2800 NT 62 | 78; 180, 2944 rows, 2048 x 3840 NT 53.5 | 46.5, NN 55 | 46.6; 203, 7312
// rows, 2560 x 864 gated 74 | 62), if experts fill them (rows an expert, 128 | 256): 24 x 7168 x 2048 gated: 83: 300 | 336, 250: 530 | 553, 400: 720 | 716, 500: 839 |
// 750; 16 x 4096 x 4096 NT: 200: 166 | 197, 256: 205 | 226, 400: 273 | 234. (256 x 128 and 128 x 256: 683 rows of 12 experts, 7168 x 2048
// through the gate 365 and 342 against 346; 24 experts' gated batch 1139 and 1109 against 925.)
// Any alignment (64 | 64 x 128 | 128): 2001 rows, 4001 x 777, NT 49 | 61 | 76, NN 68 | 76 | 106, its TN 56 | 57 | 61; 777 x 4001
// NT 43 | 39 | 29; 333 rows, 501 x 1001 gated 9.4 | 12.1 | 16.9; 8001 rows, 4097 x 4097 655 | 538 | 437.
// Weights' gradients: tiles are the matrices' own (the grid rounds each expert's up to 8, which count for nothing), and a tile whose grid
// has room for twice the results or more is too large: workgroups without a tile still wait for a CU's shared memory. Measured (out,
// rows an expert; 64 | 64w | 128 | 128x | 256): 63 x (48 x 40): 10: 7.1 | 6.5 | 7.3 | 8.5 | 8.6, 100: 7.5 | 7.5 | 8.6 | 9.7 | 12.1; 32 x (256 x 256): 100: 7.2 |
// 7.1 | 8.1 | 8.2 | 13.9, 700: 18.9 | 19.4 | 25.7 | 21.9 | 43.0; 300 x (64 x 64): 10: 10.6 | 7.6 | 12.1 | 10.9 | 21.4; 300 x (512 x 256): 100: 70 | 34.1 | 35.1 |
// 34.8 | 51.3; 24 x (640 x 640): 83: 24.8 | 12.7 | 13.9 | 14.2 | 17.5, 333: 32.3 | 20.5 | 20.8 | 20.5 | 26.4; 50 x (128 x 512): 13.0 | 8.3 | 9.7 | 10.7 | 14.0.
// From two thirds of a round of tiles on that are filled, 256 x 256 (128 | 128x | 256): 12 x (7168 x 4096): 50: 264 | 267 | 202, 100: 300 | 332 | 241,
// 200: 385 | 393 | 303, 400: 527 | 479 | 404, 683: 708 | 654 | 538; 12 x (1024 x 2048): 100: 20.9 | 21.3 | 21.5, 400: 35.7 | 35.2 | 33.7, 683: 45.7 | 47.2 | 43.8;
// 24 x (1368 x 1000): 83: 32.5 | 30.8 | 30.9, 333: 55.0 | 47.5 | 45.4; dense, 4096 rows: 3328 x 3328 97.5 | 95.1 | 81.8, 2816 x 2816 (121 tiles) 59.8 | 66.0 | 80.2; 8192 x
// 8192: 100 rows 37.6 | 42.4 | 42.9, 2000 rows 249 | 267 | 211. Any alignment (64 | 128): 63 x (41 x 49): 7.7 | 10.5; 300 x (65 x 65): 10.0 | 20.2; 32 x (255 x
// 255): 12.5 | 18.8; 5 x (1001 x 2735): 30.5 | 28.3.
Kernel product_kernel_of(const ProductArgs &a, int form, Epilogue epi) {
  const bool tn = form == WT_PRODUCT_TN;
  const int64_t halves = epi == Epilogue::kGated ? 2 : 1;  // of a tile's columns are out's
  auto across = [&](int columns) { return (a.n * halves + columns - 1) / columns; };
  auto tiles = [&](int rows, int columns) {
    return tn ? ((int64_t)a.m + rows - 1) / rows * across(columns) * a.n_experts : grid_of(a, form, rows, across(columns));
  };
  auto too_large = [&](int edge) {
    return tn && grid_of(a, form, edge, across(edge)) * edge * edge >= 2 * (int64_t)a.m * a.n * a.n_experts;
  };
  if (!product_aligned(a, form, epi)) return tiles(128, 128) >= kCus && !too_large(128) ? Kernel::kAny128 : Kernel::kAny64;
  if (!tn && tiles(16, 64) <= kCus) return Kernel::k16Split;
  if (tiles(64, 64) <= kCus) return Kernel::k64Split;
  if (tiles(64, 128) <= kCus || too_large(128)) return Kernel::k64x128;
  if (3 * tiles(256, 256) >= 2 * kCus && (tn ? !too_large(256) : a.n_rows > 256 * (int64_t)a.n_experts)) return Kernel::k256;
  return tiles(128, 128) >= kCus ? Kernel::k128 : Kernel::k128Wide;
}

// Which kernel, as for product_kernel_of(). Measured on MI355X, us (k x n; kernel 32 | 64 | 128 | 256 = rows of a tile): one row, 2816 x 1024 6.6 |
// 7.1 | 8.3 | 12.1; 64 rows, 1024 x 2816 gated 6.3 | 6.5 | 7.9 | 9.9; 100 rows, 7168 x 4096 9.4 | 12.4 | 17.1 | 27.4; 256 rows, 2816 x 1024
// gated 7.3 | 7.8 | 10.9 | 23.8; 512 rows, 2048 x 2048 10.4 | 7.1 | 9.2 | 19.1; 1024 rows 19.3 | 9.5 | 9.6 | 19.4; 2048 rows, 4096 x 4096
// 94.5 | 47.2 | 26.2 | 33.0; 4096 rows - | - | 49.1 | 46.7; 256 rows of 96 experts, 7168 x 2048 gated 300 | - | 258 | 304; 2000 rows of 24
// experts - | - | 100 | 108; 6000 rows 181 | 193; 9600 rows 241 | 246; 12000 rows 286 | 252; 8192 cubed - | - | 327 | 296.
// Tiles of 256 want sums of 3584 terms or more besides (28 steps). By the sum's length, 1024 | 2048 | 2816 | 3584 | 4096 | 7168 | 14336, tiles of 128 and of
// 256 rows: 2944 rows x 3840, 180 tiles: 16.4 18.3 | 22.9 24.1 | 28.1 28.4 | 33.4 32.6 | 37.1 35.4 | 59.4 52.4 | 110 92.6; 3328 x 4096: - | 27.3 26.1 | 33.1
// 31.2 | 39.9 36.1 | 43.4 39.5 | 67.5 58.1; 8192 x 8192: 67.6 80.3 | 105 112 | 133 136 | 163 157 | 182 172; 4096 x 4096 gated: - | 55.2 57.4 | 69.0 69.4 |
// 82.8 80.9 | 93.0 87.5; 8192 rows of 12 experts x 2048: - | 35.3 42.3 | - | 53.2 57.7 | 59.0 63.3 | 91.8 98.5; 16384 rows of 24 experts x 2048 gated, 4096: 214
// 198; 12288 rows of 12 experts x 7168, 2048: 159 156.
Kernel mxfp4_kernel_of(const ProductArgs &a, Epilogue epi) {
  const int64_t far = (int64_t)1 << 31;
  // 31-bit offsets within a tile's rows, as in product_aligned(): 256 of them, and gated from the gate rows to the up rows
  const int64_t most = far / 512, b_most = epi == Epilogue::kGated ? far / ((int64_t)a.n + 512) : most;
  const bool near = a.a_stride <= most && a.b_stride <= b_most && a.a_scale_stride <= most && a.b_scale_stride <= b_most;
  if (!near) return Kernel::kAny128;
  const int64_t halves = epi == Epilogue::kGated ? 2 : 1;
  auto tiles = [&](int rows, int columns) { return grid_of(a, WT_PRODUCT_NT, rows, (a.n * halves + columns - 1) / columns); };
  if (tiles(32, 64) <= kCus) return Kernel::k32Split;
  if (tiles(64, 64) <= kCus) return Kernel::k64Split;
  if (a.k >= 3584 && 3 * tiles(256, 256) >= 2 * kCus && a.n_rows > 256 * (int64_t)a.n_experts) return Kernel::k256;
  return Kernel::k128;
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
