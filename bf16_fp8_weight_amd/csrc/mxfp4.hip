// mxfp4.hip -- MXFP4: rows to codes and scales, back to values, and products of
// such rows. The format and the rounding are defined in wt.h.
//
// Quantisation: four lanes to a block of 32 elements. The scale is a power of two,
// taken from the exponent bits of the largest magnitude; v_cvt_scalef32_pk_fp4
// divides by it (exactly), rounds to the nearest even code and saturates, in one
// instruction for two elements. Both directions are bound by memory: 22016 x 4096 BF16
// take 36.6 us to codes and 33.9 back (6.2 and 6.7 TB/s of the arrays' bytes, part of them from
// the last-level cache; 48.7 and 38 when they are not there). Eight, 16 or 32 elements to a lane and two or four blocks in
// flight made no difference (34.8 to 37.0); 32 elements in one lane's registers spilled.
#include <hip/hip_runtime.h>

#include <string>

#include "expert_tile.h"
#include "fp8_math.h"
#include "hip_util.h"
#include "launch_parts.h"
#include "plan.h"
#include "wave.h"
#include "wt.h"

namespace wt {
namespace {

constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;
constexpr int kThreads = 256;
constexpr int kLanes = 4;  // of a block, 8 elements each

struct RoundArgs {
  uint64_t x, codes, scales;  // x: the values that are read or written
  const int32_t *index;
  int64_t n_rows, n_out, cols, x_stride, code_stride, scale_stride;
  uint32_t nb, n_blocks;
  uint32_t first_group;  // of this launch among the call's workgroups
};

// The first `valid` (at most 8) values from element `at` on, as fp32.
template <bool F32>
__device__ __forceinline__ void load8(uint64_t x, uint64_t at, int valid, float (&v)[8]) {
  if (F32) {
    const uint64_t p = x + 4 * at;
    if (valid >= 8) {
      const f32x4 lo = load_at<f32x4>(p), hi = load_at<f32x4>(p + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < valid ? load_at<float>(p + 4 * i) : 0.0f;
    }
  } else {
    const u32x4 w = load_chunk(x + 2 * at, valid);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// 2^(c - 127), c < 255; 2^-127 is subnormal.
__device__ __forceinline__ float scale_of(int c) { return __uint_as_float(c > 0 ? (uint32_t)c << 23 : 1u << 22); }

template <bool F32>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_kernel(RoundArgs a) {
  const uint32_t block = (a.first_group + blockIdx.x) * (uint32_t)(kThreads / kLanes) + threadIdx.x / kLanes;
  const int l = threadIdx.x % kLanes;
  uint32_t i = 0, b = 0;
  int64_t src = -1;
  if (block < a.n_blocks) {
    i = block / a.nb, b = block - i * a.nb;
    src = a.index ? (int64_t)a.index[i] : (int64_t)i;
  }
  const bool mine = src >= 0 && src < a.n_rows;
  const int64_t c0 = 32 * (int64_t)b + 8 * l;
  float v[8] = {};
  if (mine) load8<F32>(a.x, (uint64_t)(src * a.x_stride + c0), (int)min((int64_t)8, a.cols - c0), v);
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  top = lanes_max<kLanes>(top);  // every lane of the block takes part
  if (!mine) return;
  const int exponent = (int)(top >> 23);  // biased; subnormals count as the lowest
  const bool bad = exponent == 255;
  const int c = bad ? 255 : top == 0 ? 127 : max(exponent - 2, 0);
  const float scale = scale_of(bad ? 127 : c);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
  st_global<uint32_t>(a.codes + (uint64_t)((int64_t)i * a.code_stride + c0 / 2), bad ? 0u : q);
  if (l == 0) st_global<uint8_t>(a.scales + (uint64_t)((int64_t)i * a.scale_stride + b), (uint8_t)c);
}

// A code's value times a power of two is exact: values have at most two digits.
template <bool F32>
__global__ void __launch_bounds__(kThreads) mxfp4_dequantize_kernel(RoundArgs a) {
  const uint32_t block = (a.first_group + blockIdx.x) * (uint32_t)(kThreads / kLanes) + threadIdx.x / kLanes;
  if (block >= a.n_blocks) return;
  const int l = threadIdx.x % kLanes;
  const uint32_t i = block / a.nb, b = block - i * a.nb;
  const int64_t c0 = 32 * (int64_t)b + 8 * l;
  if (c0 >= a.cols) return;
  const int n = (int)min((int64_t)8, a.cols - c0);
  const uint32_t q = ld_global<uint32_t>(a.codes + (uint64_t)((int64_t)i * a.code_stride + c0 / 2));
  const int c = ld_global<uint8_t>(a.scales + (uint64_t)((int64_t)i * a.scale_stride + b));
  const float scale = scale_of(c);
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3)};
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = c == 255 ? __uint_as_float(0x7FC00000u) : p[e >> 1][e & 1] * scale;
  const int64_t at = (int64_t)i * a.x_stride + c0;
  if (F32) store8<float>(a.x, at, v, n);
  else store8<__bf16>(a.x, at, v, n);
}

wt_status check_round(const char *what, int32_t dtype, int64_t n_rows, int64_t n_out, int64_t cols, int64_t x_stride,
                      int64_t code_stride, int64_t scale_stride) {
  if (dtype != WT_DT_F32 && dtype != WT_DT_BF16) return operator_fail(what, "unknown type");
  if (n_rows < 0 || n_out < 0) return operator_fail(what, "negative row count");
  if (cols < 1 || cols >= (int64_t)1 << 31) return operator_fail(what, "cols out of range");
  const int64_t nb = (cols + 31) / 32;
  if (x_stride < cols || code_stride < 16 * nb || scale_stride < nb) return operator_fail(what, "row stride too small");
  const int64_t rows = n_rows > n_out ? n_rows : n_out, most = ((int64_t)1 << 59) / (rows > 1 ? rows : 1);
  if (x_stride > most || code_stride > most || scale_stride > most) return operator_fail(what, "row stride too large");
  if (n_out > (((int64_t)1 << 31) - 1) / nb) return operator_fail(what, "rows * ceil(cols / 32) >= 2^31");
  return WT_OK;
}

hipError_t launch_round(void (*kernel)(RoundArgs), RoundArgs a, hipStream_t stream) {
  const uint32_t groups = (a.n_blocks + kThreads / kLanes - 1) / (kThreads / kLanes);
  return launch_parts(groups, kThreads, hipSuccess, [&](uint32_t first, uint32_t count) {
    a.first_group = first;
    hipLaunchKernelGGL(kernel, dim3(count), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
  });
}

template <Epilogue Epi, int BM, int BN, int WM, int WN, int Split, int Sub, int Stages, bool Near>
wt_status launch(const char *what, ProductArgs a, hipStream_t stream) {
  constexpr int columns = Epi == Epilogue::kGated ? BN / 2 : BN;
  const int64_t n_tiles = (a.n + columns - 1) / columns;
  const int64_t grid = grid_of(a, kNT, BM, n_tiles);
  a.rests_last = grid <= 2 * kCus;  // as in expert_run.h
  if (grid > kMaxGrid) return operator_fail(what, "too many tiles");
  if (grid == 0) return WT_OK;
  auto kernel = [] {
    if constexpr (Near) return product_kernel<kNT, Epi, true, BM, BN, WM, WN, Split, Sub, Stages, false>;
    else return product_any_kernel<kNT, Epi, true, BM, BN, WM, WN, Sub>;
  }();
  constexpr uint32_t threads = 64 * WM * WN * Split;
  const hipError_t e = launch_parts(grid, threads, hipSuccess, [&](uint32_t first, uint32_t count) {
    a.first_group = first;
    hipLaunchKernelGGL(kernel, dim3(count), dim3(threads), 0, stream, a);
    return hipGetLastError();
  });
  if (e != hipSuccess) return operator_fail(what, hip_msg("launch", e), WT_E_HIP);
  return WT_OK;
}

// The kernel that mxfp4_kernel_of() names.
template <Epilogue Epi>
wt_status run(const char *what, const ProductArgs &a, hipStream_t stream) {
  switch (mxfp4_kernel_of(a, Epi)) {
    case Kernel::kAny128: return launch<Epi, 128, 128, 2, 2, 1, 2, 2, false>(what, a, stream);
    case Kernel::k32Split: return launch<Epi, 32, 64, 1, 1, 4, 2, 2, true>(what, a, stream);
    case Kernel::k64Split: return launch<Epi, 64, 64, 1, 1, 4, 1, 2, true>(what, a, stream);
    case Kernel::k256: return launch<Epi, 256, 256, 2, 4, 1, 1, 4, true>(what, a, stream);
    case Kernel::k128: return launch<Epi, 128, 128, 2, 2, 1, 2, 2, true>(what, a, stream);
    default: break;
  }
  return operator_fail(what, "no kernel");
}

}  // namespace
}  // namespace wt

using namespace wt;

extern "C" {

wt_status wt_mxfp4_quantize(const void *x, int32_t dtype, int64_t n_rows, int64_t cols, int64_t x_row_stride,
                            const int32_t *row_index, int64_t n_out, void *codes, int64_t code_row_stride,
                            void *scales, int64_t scale_row_stride, void *stream) {
  const char *what = "wt_mxfp4_quantize";
  try {
    const wt_status st = check_round(what, dtype, n_rows, n_out, cols, x_row_stride, code_row_stride, scale_row_stride);
    if (st != WT_OK) return st;
    if (n_out == 0) return WT_OK;
    if (!codes || !scales || (n_rows > 0 && !x)) return operator_fail(what, "NULL pointer");
    if ((uintptr_t)x % (dtype == WT_DT_F32 ? 4 : 2)) return operator_fail(what, "x misaligned", WT_E_ALIGN);
    if ((uintptr_t)row_index % 4) return operator_fail(what, "row_index misaligned", WT_E_ALIGN);
    if ((uintptr_t)codes % 4 || code_row_stride % 4) return operator_fail(what, "codes not 4-byte aligned", WT_E_ALIGN);
    RoundArgs a{(uint64_t)(uintptr_t)x, (uint64_t)(uintptr_t)codes, (uint64_t)(uintptr_t)scales, row_index, n_rows,
                n_out, cols, x_row_stride, code_row_stride, scale_row_stride, (uint32_t)((cols + 31) / 32), 0, 0};
    a.n_blocks = (uint32_t)(n_out * a.nb);
    const StreamDevice on((hipStream_t)stream);
    const auto kernel = dtype == WT_DT_F32 ? mxfp4_quantize_kernel<true> : mxfp4_quantize_kernel<false>;
    const hipError_t e = launch_round(kernel, a, (hipStream_t)stream);
    if (e != hipSuccess) return operator_fail(what, hip_msg("launch", e), WT_E_HIP);
    return WT_OK;
  } catch (...) {
    return caught_status();
  }
}

wt_status wt_mxfp4_dequantize(const void *codes, int64_t code_row_stride, const void *scales,
                              int64_t scale_row_stride, int64_t n_rows, int64_t cols, void *out, int32_t dtype,
                              int64_t out_row_stride, void *stream) {
  const char *what = "wt_mxfp4_dequantize";
  try {
    const wt_status st = check_round(what, dtype, n_rows, n_rows, cols, out_row_stride, code_row_stride, scale_row_stride);
    if (st != WT_OK) return st;
    if (n_rows == 0) return WT_OK;
    if (!codes || !scales || !out) return operator_fail(what, "NULL pointer");
    if ((uintptr_t)out % (dtype == WT_DT_F32 ? 4 : 2)) return operator_fail(what, "out misaligned", WT_E_ALIGN);
    if ((uintptr_t)codes % 4 || code_row_stride % 4) return operator_fail(what, "codes not 4-byte aligned", WT_E_ALIGN);
    RoundArgs a{(uint64_t)(uintptr_t)out, (uint64_t)(uintptr_t)codes, (uint64_t)(uintptr_t)scales, nullptr, n_rows,
                n_rows, cols, out_row_stride, code_row_stride, scale_row_stride, (uint32_t)((cols + 31) / 32), 0, 0};
    a.n_blocks = (uint32_t)(n_rows * a.nb);
    const StreamDevice on((hipStream_t)stream);
    const auto kernel = dtype == WT_DT_F32 ? mxfp4_dequantize_kernel<true> : mxfp4_dequantize_kernel<false>;
    const hipError_t e = launch_round(kernel, a, (hipStream_t)stream);
    if (e != hipSuccess) return operator_fail(what, hip_msg("launch", e), WT_E_HIP);
    return WT_OK;
  } catch (...) {
    return caught_status();
  }
}

wt_status wt_mxfp4_product(const wt_mxfp4_product_desc *desc, void *stream) {
  const char *what = "wt_mxfp4_product";
  try {
    ProductArgs a;
    const wt_status st = mxfp4_product_args(what, desc, &a);
    if (st != WT_OK) return st;
    const StreamDevice on((hipStream_t)stream);
    return desc->gated ? run<Epilogue::kGated>(what, a, (hipStream_t)stream)
                       : run<Epilogue::kPlain>(what, a, (hipStream_t)stream);
  } catch (...) {
    return caught_status();
  }
}

}  // extern "C"
