// expert_tn.hip -- kernels of WT_PRODUCT_TN: gradients of weights.
#include "expert_run.h"

namespace wt {

template wt_status run_product<kTN, Epilogue::kPlain>(const char *, const ProductArgs &, hipStream_t);

}  // namespace wt
