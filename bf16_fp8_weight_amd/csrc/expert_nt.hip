// expert_nt.hip -- kernels of WT_PRODUCT_NT: projections, plain and gated.
#include "expert_run.h"

namespace wt {

template wt_status run_product<kNT, Epilogue::kPlain>(const char *, const ProductArgs &, hipStream_t);
template wt_status run_product<kNT, Epilogue::kGated>(const char *, const ProductArgs &, hipStream_t);

}  // namespace wt
