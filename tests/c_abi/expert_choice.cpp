// Prints, for each description on stdin, the kernel that a product of it takes. No GPU code.
// A line: p FORM EPILOGUE N_ROWS N_EXPERTS OFFSETS N_INDEX_ROWS(-1: none) M N K A_STRIDE B_STRIDE
//     or: m GATED N_ROWS N_EXPERTS OFFSETS N K A_STRIDE A_SCALE_STRIDE B_STRIDE B_SCALE_STRIDE
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>

#include "expert.h"
#include "plan.h"

using namespace wt;

int main() {
  static const char *const names[] = {"any64", "any128", "16split", "32split", "64split", "64x128", "128", "128wide", "256"};
  const auto at = (void *)(uintptr_t)0x10000;
  for (std::string line; std::getline(std::cin, line);) {
    std::istringstream in(line);
    std::string kind;
    ProductArgs a;
    in >> kind;
    Kernel kernel;
    if (kind == "p") {
      wt_product_desc d;
      wt_product_desc_init(&d);
      int epi = 0, offsets = 0;
      in >> d.form >> epi >> d.n_rows >> d.n_experts >> offsets >> d.n_index_rows >> d.m >> d.n >> d.k >> d.a_stride >> d.b_stride;
      if (!in) return std::printf("malformed: %s\n", line.c_str()), 1;
      if (offsets) d.offsets = (const int32_t *)at;
      if (d.n_index_rows >= 0) d.row_index = (const int32_t *)at;
      d.a = d.b = d.out = at;
      d.out_stride = 2 * d.n;
      d.out_expert_stride = d.m * d.out_stride;
      if (d.form != WT_PRODUCT_TN) d.b_expert_stride = d.b_stride * (d.form == WT_PRODUCT_NT ? 2 * d.n : d.k);
      if (product_args("choice", &d, (Epilogue)epi, epi ? at : nullptr, 2 * d.n, &a) != WT_OK)
        return std::printf("refused: %s: %s\n", line.c_str(), wt_plan_last_error(nullptr)), 1;
      kernel = product_kernel_of(a, d.form, (Epilogue)epi);
    } else {
      wt_mxfp4_product_desc d;
      wt_mxfp4_product_desc_init(&d);
      int offsets = 0;
      in >> d.gated >> d.n_rows >> d.n_experts >> offsets >> d.n >> d.k >> d.a_stride >> d.a_scale_stride >> d.b_stride >> d.b_scale_stride;
      if (!in) return std::printf("malformed: %s\n", line.c_str()), 1;
      if (offsets) d.offsets = (const int32_t *)at;
      d.a = d.b = d.a_scales = d.b_scales = d.out = at;
      d.b_expert_stride = d.b_stride * d.n * 2, d.b_scale_expert_stride = d.b_scale_stride * d.n * 2;
      d.out_stride = d.n;
      if (mxfp4_product_args("choice", &d, &a) != WT_OK)
        return std::printf("refused: %s: %s\n", line.c_str(), wt_plan_last_error(nullptr)), 1;
      kernel = mxfp4_kernel_of(a, d.gated ? Epilogue::kGated : Epilogue::kPlain);
    }
    std::printf("%s\n", names[(int)kernel]);
  }
  return 0;
}
