// dispatch.hip -- the row map of a dispatch: token copies grouped by expert
// in a stable order. The definition is in wt.h.
//
// Three launches: each workgroup counts its tile of copies per expert; one
// workgroup turns the tiles' counts into each tile's first row per expert;
// each workgroup ranks its copies and writes both maps. Every rank comes from
// counts and lane masks, never from the order of atomics.
#include <hip/hip_runtime.h>

#include <string>

#include "hip_util.h"
#include "plan.h"
#include "wt.h"

namespace wt {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxExperts = 1024;
constexpr int kTile = 2048;  // copies of one workgroup
constexpr int kScanThreads = 1024;

struct RowsArgs {
  const int32_t *index;
  int64_t n_pairs;
  int32_t top_k, n_experts, align;
  int64_t n_rows;
  int32_t *row_token, *pair_row, *offsets, *counts;
  int32_t *tile_rows;  // [tile][expert]: counts, then first rows
  int32_t *used;       // [expert]: copies (also where counts is NULL)
  int32_t n_tiles;
};

__device__ __forceinline__ int expert_at(const RowsArgs &a, int64_t i, int64_t end) {
  const int e = i < end ? a.index[i] : -1;
  return e >= 0 && e < a.n_experts ? e : -1;
}

// Copies per expert of pairs [lo, hi), one histogram per wave: wave w takes
// the w-th quarter of the tile, so that ranks follow the pairs' order.
__device__ __forceinline__ void count_tile(const RowsArgs &a, int64_t lo, int64_t hi, int (*hist)[kMaxExperts]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int e = threadIdx.x; e < kWaves * kMaxExperts; e += kThreads) (&hist[0][0])[e] = 0;
  __syncthreads();
  const int64_t from = lo + wave * (kTile / kWaves), to = from + kTile / kWaves < hi ? from + kTile / kWaves : hi;
  for (int64_t i = from + lane; i < to; i += 64) {
    const int e = expert_at(a, i, to);
    if (e >= 0) atomicAdd(&hist[wave][e], 1);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) rows_count_kernel(RowsArgs a) {
  __shared__ int hist[kWaves][kMaxExperts];
  const int64_t lo = (int64_t)blockIdx.x * kTile, hi = lo + kTile < a.n_pairs ? lo + kTile : a.n_pairs;
  count_tile(a, lo, hi, hist);
  for (int e = threadIdx.x; e < a.n_experts; e += kThreads)
    a.tile_rows[(int64_t)blockIdx.x * a.n_experts + e] = (hist[0][e] + hist[1][e]) + (hist[2][e] + hist[3][e]);
}

// One workgroup, thread e for expert e: the copies of every tile before it,
// then the experts' first rows (a scan over the padded counts).
__global__ void __launch_bounds__(kScanThreads) rows_scan_kernel(RowsArgs a) {
  __shared__ int scan[kScanThreads];
  const int e = threadIdx.x;
  int total = 0;
  if (e < a.n_experts)
    for (int32_t t = 0; t < a.n_tiles; ++t) {
      int32_t *p = a.tile_rows + (int64_t)t * a.n_experts + e;
      const int c = *p;
      *p = total;
      total += c;
    }
  const int padded = (total + a.align - 1) / a.align * a.align;
  scan[e] = padded;
  __syncthreads();
  for (int d = 1; d < kScanThreads; d *= 2) {
    const int before = e >= d ? scan[e - d] : 0;
    __syncthreads();
    scan[e] += before;
    __syncthreads();
  }
  if (e < a.n_experts) {
    const int start = scan[e] - padded;
    a.offsets[e] = start;
    a.used[e] = total;
    if (a.counts) a.counts[e] = total;
    if (e == a.n_experts - 1) a.offsets[e + 1] = scan[e];
  }
}

// Lanes of the wave with the same expert as this one.
__device__ __forceinline__ uint64_t same_expert(int e) {
  uint64_t m = __ballot(e >= 0);
#pragma unroll
  for (int bit = 0; bit < 10; ++bit) {
    const uint64_t on = __ballot((e >> bit) & 1);
    m &= (e >> bit) & 1 ? on : ~on;
  }
  return m;
}

__global__ void __launch_bounds__(kThreads) rows_place_kernel(RowsArgs a) {
  __shared__ int next[kWaves][kMaxExperts];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t lo = (int64_t)blockIdx.x * kTile, hi = lo + kTile < a.n_pairs ? lo + kTile : a.n_pairs;
  if (lo < hi) {
    count_tile(a, lo, hi, next);
    // each wave's first row per expert
    for (int e = threadIdx.x; e < a.n_experts; e += kThreads) {
      int at = a.offsets[e] + a.tile_rows[(int64_t)blockIdx.x * a.n_experts + e];
      for (int w = 0; w < kWaves; ++w) {
        const int c = next[w][e];
        next[w][e] = at;
        at += c;
      }
    }
    __syncthreads();
    const int64_t from = lo + wave * (kTile / kWaves), to = from + kTile / kWaves < hi ? from + kTile / kWaves : hi;
    for (int64_t base = from; base < to; base += 64) {
      const int64_t i = base + lane;
      const int e = expert_at(a, i, to);
      const uint64_t same = same_expert(e);
      int row = -1;
      if (e >= 0) {
        const int before = __popcll(same & (((uint64_t)1 << lane) - 1));
        row = next[wave][e] + before;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (before == 0) next[wave][e] = row + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (row >= a.n_rows) row = -1;
        else if (a.row_token) a.row_token[row] = (int32_t)(i / a.top_k);
      }
      if (i < to && a.pair_row) a.pair_row[i] = row;
    }
  }
  if (!a.row_token) return;
  // rows that hold no copy: behind each expert's copies, and behind the last expert
  for (int e = blockIdx.x; e < a.n_experts; e += gridDim.x) {
    const int64_t end = a.offsets[e + 1] < a.n_rows ? a.offsets[e + 1] : a.n_rows;
    for (int64_t r = (int64_t)a.offsets[e] + a.used[e] + threadIdx.x; r < end; r += kThreads) a.row_token[r] = -1;
  }
  for (int64_t r = (int64_t)a.offsets[a.n_experts] + (int64_t)blockIdx.x * kThreads + threadIdx.x; r < a.n_rows;
       r += (int64_t)gridDim.x * kThreads)
    a.row_token[r] = -1;
}

wt_status fail(const char *what, const std::string &m, wt_status st = WT_E_INVAL) {
  set_thread_error(std::string(what) + ": " + m);
  return st;
}

wt_status check_sizes(const char *what, int64_t n_tokens, int32_t top_k, int32_t n_experts) {
  if (n_experts < 1 || n_experts > kMaxExperts) return fail(what, "n_experts out of range");
  if (top_k < 1) return fail(what, "top_k out of range");
  if (n_tokens < 0 || n_tokens > (((int64_t)1 << 31) - 1) / top_k) return fail(what, "n_tokens out of range");
  return WT_OK;
}

int64_t tiles_of(int64_t pairs) { return (pairs + kTile - 1) / kTile; }

}  // namespace
}  // namespace wt

using namespace wt;

extern "C" {

wt_status wt_dispatch_workspace_bytes(int64_t n_tokens, int32_t top_k, int32_t n_experts, size_t *bytes) {
  const char *what = "wt_dispatch_workspace_bytes";
  const wt_status st = check_sizes(what, n_tokens, top_k, n_experts);
  if (st != WT_OK) return st;
  if (!bytes) return fail(what, "NULL result");
  *bytes = (size_t)(4 * (tiles_of(n_tokens * top_k) + 1) * n_experts);
  return WT_OK;
}

wt_status wt_dispatch_rows(const int32_t *index, int64_t n_tokens, int32_t top_k, int32_t n_experts,
                           int32_t row_align, int64_t n_rows, int32_t *row_token, int32_t *pair_row,
                           int32_t *offsets, int32_t *counts, void *workspace, size_t workspace_bytes, void *stream) {
  const char *what = "wt_dispatch_rows";
  try {
    size_t need = 0;
    wt_status st = check_sizes(what, n_tokens, top_k, n_experts);
    if (st == WT_OK) st = wt_dispatch_workspace_bytes(n_tokens, top_k, n_experts, &need);
    if (st != WT_OK) return st;
    if (row_align < 1 || row_align > 4096) return fail(what, "row_align out of range");
    const int64_t pairs = n_tokens * top_k;
    if (pairs + (int64_t)n_experts * (row_align - 1) >= ((int64_t)1 << 31)) return fail(what, "too many rows");
    if (n_rows < 0 || n_rows >= ((int64_t)1 << 31)) return fail(what, "n_rows out of range");
    if ((pairs > 0 && !index) || !offsets || !workspace) return fail(what, "NULL index, offsets or workspace");
    if (((uintptr_t)index | (uintptr_t)row_token | (uintptr_t)pair_row | (uintptr_t)offsets | (uintptr_t)counts |
         (uintptr_t)workspace) % 4)
      return fail(what, "misaligned pointer", WT_E_ALIGN);
    if (workspace_bytes < need) return fail(what, "workspace too small", WT_E_RANGE);
    RowsArgs a{};
    a.index = index;
    a.n_pairs = pairs;
    a.top_k = top_k;
    a.n_experts = n_experts;
    a.align = row_align;
    a.n_rows = n_rows;
    a.row_token = row_token;
    a.pair_row = pair_row;
    a.offsets = offsets;
    a.counts = counts;
    a.n_tiles = (int32_t)tiles_of(pairs);
    a.used = (int32_t *)workspace;
    a.tile_rows = a.used + n_experts;
    const hipStream_t s = (hipStream_t)stream;
    if (a.n_tiles > 0) hipLaunchKernelGGL(rows_count_kernel, dim3((uint32_t)a.n_tiles), dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(rows_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, a);
    hipLaunchKernelGGL(rows_place_kernel, dim3(a.n_tiles > 0 ? (uint32_t)a.n_tiles : 1u), dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(what, hip_msg("launch", e), WT_E_HIP);
    return WT_OK;
  } catch (...) {
    set_thread_error("internal error");
    return WT_E_INVAL;
  }
}

}  // extern "C"
