// expert_nn.hip -- kernels of WT_PRODUCT_NN: gradients of rows, plain and through the gate.
#include "expert_run.h"

namespace wt {

template wt_status run_product<kNN, Epilogue::kPlain>(const char *, const ProductArgs &, hipStream_t);
template wt_status run_product<kNN, Epilogue::kGatedBack>(const char *, const ProductArgs &, hipStream_t);

}  // namespace wt
