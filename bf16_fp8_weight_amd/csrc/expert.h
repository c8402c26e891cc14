// expert.h -- what the experts' products share between their host checks
// (expert.cpp, no GPU call: checks, choice of a kernel) and their kernels (expert_tile.h, expert.hip,
// mxfp4.hip).
#pragma once

#include <cstdint>
#include <string>

#include "wt.h"

struct ihipStream_t;  // hipStream_t is a pointer to it

namespace wt {

// What a product's kernel takes. Addresses and strides of a, b and their scales
// in bytes, those of out and pre in elements.
struct ProductArgs {
  const int32_t *offsets, *counts;  // offsets NULL: one expert that owns every row
  const int32_t *row_index;         // of the gathered operand, or NULL
  uint64_t a, b, a_scales, b_scales, out, pre;
  int64_t a_stride, b_stride, b_expert;
  int64_t a_scale_stride, b_scale_stride, b_scale_expert;
  int64_t out_stride, out_expert, pre_stride;
  int64_t n_rows, n_index_rows;
  int32_t n_experts;
  int32_t m, n, k;      // n: columns of out (of h in the gated forms)
  int32_t act, out_f32;
  int32_t rests_last;   // order of the tiles, see find_rows()
  uint32_t first_group;  // of this launch among the call's workgroups
};

enum class Epilogue { kPlain, kGated, kGatedBack };

// Whether a product's operands can be copied to shared memory in 16-byte pieces
// under 31-bit offsets (the kernels' windows): addresses, strides and the ends of rows are
// multiples of 4 bytes; a tile's rows, a gathered array and an expert's gate rows
// span less than 2^31 bytes.
bool product_aligned(const ProductArgs &a, int form, Epilogue epi);

constexpr int kCus = 256;
constexpr int kXcds = 8;

// Workgroups that deal out all tiles of bm rows and n_tiles columns of tiles. The rows of each expert are on the device: the
// grid holds the tiles of any experts whose rows add up to n_rows at most, and of more than that (they overlap) not all.
int64_t grid_of(const ProductArgs &a, int form, int bm, int64_t n_tiles);

// Which kernel a product takes: rows x columns of its tiles; kAny: operands of any alignment, kSplit: waves that split the sum,
// kWide: eight waves to a tile of 128 x 128.
enum class Kernel { kAny64, kAny128, k16Split, k32Split, k64Split, k64x128, k128, k128Wide, k256 };
Kernel product_kernel_of(const ProductArgs &a, int form, Epilogue epi);
Kernel mxfp4_kernel_of(const ProductArgs &a, Epilogue epi);

// Fills *a from a description that it has checked; `what` names the call in the
// thread's error text.
wt_status product_args(const char *what, const wt_product_desc *d, Epilogue epi, const void *pre, int64_t pre_stride,
                       ProductArgs *a);
wt_status mxfp4_product_args(const char *what, const wt_mxfp4_product_desc *d, ProductArgs *a);

// The caller's error text, set; returns st.
wt_status operator_fail(const char *what, const std::string &m, wt_status st = WT_E_INVAL);

// Enqueues a product of form Form (WT_PRODUCT_*): expert_nt.hip, expert_nn.hip, expert_tn.hip.
template <int Form, Epilogue Epi>
wt_status run_product(const char *what, const ProductArgs &a, ihipStream_t *stream);

constexpr int64_t kProductMaxRows = (int64_t)1 << 27;
constexpr int64_t kProductMaxSize = (int64_t)1 << 24;
constexpr int kProductMaxExperts = 1024;

}  // namespace wt
