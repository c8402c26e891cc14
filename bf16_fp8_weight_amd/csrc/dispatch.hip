// dispatch.hip -- the row map of a dispatch: token copies grouped by expert
// in a stable order. The definition is in wt.h.
//
// A copy's row = its expert's first row + the copies of that expert in the
// tiles before its own, in the waves before its own, and in the lanes before
// its own. Counts come from integer histograms and lane masks, never from the
// order of atomics. Up to kRowsSingle copies one workgroup places them all (one
// launch); beyond, a first launch counts each tile and the second one's
// workgroups each add up what they need of all tiles' counts (side by side, where
// a scan kernel between the two took 12 us alone; four experts to a load, where
// one to a load took 2.7 us more with 64 tiles). Workgroups behind the last tile
// take part in filling the rows that hold no copy; with one tile each of them
// counts the copies for itself. Nothing here is bound by bytes: 16384 tokens
// move 1.8 MB in 10.6 us (replayed from a graph; 10.8 to 11.2 for a call from
// Python), which go to two launches (3 + 8 us), five barriers, and reads and
// scattered writes that wait for L2.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "hip_util.h"
#include "plan.h"
#include "wave.h"
#include "wt.h"

namespace wt {
namespace {

constexpr int kMaxExperts = 1024;
// Copies of a workgroup's tile: kRowsTile, half of it up to kRowsFew, more beyond
// kMaxTiles tiles. Measured on MI355X, 8 copies of each token over 384 experts,
// replayed from a graph (with the rule as it is, row_align 1: 1024 tokens 8.2 us,
// 4096 9.1, 8192 9.7, 16384 10.3, 65536 14.0), tiles of 1024 / 2048 / 4096 copies: 1024 tokens 8.3 / 8.9 / 11.1 us, 4096
// tokens 9.2 / 9.3 / 11.5, 8192 tokens 10.3 / 9.9 / 11.7, 16384 tokens 11.7 /
// 11.1 / 12.2; at most 64 / 128 / 256 tiles: 65536 tokens 17.9 / 14.1 / 15.1 us.
constexpr int64_t kRowsTile = 2048;
constexpr int64_t kRowsFew = 32768;
constexpr int kMaxTiles = 128;
// Copies up to which one workgroup takes them all; one workgroup / two launches:
// 512 tokens 7.6 / 8.0 us, 1024 tokens 11.6 / 8.3.
constexpr int64_t kRowsSingle = 4096;
// Rows for which there is one workgroup to fill them. 128 tokens over 384 experts
// in tiles of 128 rows, with one workgroup per 1024 / 4096 / 16384 rows 5.2 / 5.3
// / 6.5 us (in tiles of 16 rows 5.6 / 8.5 / 8.5), 9.6 us when one fills them all.
constexpr int64_t kRowsFill = 1024;
constexpr int64_t kMaxFill = 256;

struct RowsArgs {
  const int32_t *index;
  int64_t n_pairs;
  int32_t top_k, n_experts, align;
  int64_t n_rows;
  int32_t *row_token, *pair_row, *offsets, *counts;
  int32_t *tile_counts;  // [tile][expert], 16-byte aligned rows
  int64_t tile;          // copies of a tile, a multiple of 64 times the workgroup's waves
  int32_t n_tiles;
};

// Waves of a workgroup: 16, or 8 beyond 512 experts (each wave has a histogram
// of 4 bytes per expert); a thread then looks after one or two experts.
constexpr int kManyExperts = 512;

// Copies that a lane loads at once. 1 / 2 / 4 of them: 512 tokens 8.3 / 7.6 / 7.5
// us, 128 tokens 4.8 / 4.8 / 5.0.
constexpr int kAhead = 2;

__host__ __device__ constexpr int counts_row(int n_experts) { return (n_experts + 3) / 4 * 4; }

__device__ __forceinline__ int expert_at(const RowsArgs &a, int64_t i, int64_t end) {
  const int e = i < end ? a.index[i] : -1;
  return e >= 0 && e < a.n_experts ? e : -1;
}

__global__ void __launch_bounds__(1024) rows_count_kernel(RowsArgs a) {
  extern __shared__ int lds[];
  const int64_t lo = blockIdx.x * a.tile, hi = lo + a.tile < a.n_pairs ? lo + a.tile : a.n_pairs;
  for (int e = threadIdx.x; e < a.n_experts; e += blockDim.x) lds[e] = 0;
  __syncthreads();
  for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) {
    const int e = expert_at(a, i, hi);
    if (e >= 0) atomicAdd(&lds[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.n_experts; e += blockDim.x) a.tile_counts[blockIdx.x * counts_row(a.n_experts) + e] = lds[e];
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

template <bool Single, int Waves>
__global__ void __launch_bounds__(64 * Waves) rows_place_kernel(RowsArgs a) {
  extern __shared__ int lds[];
  constexpr int Threads = 64 * Waves, Per = Waves == 16 ? 1 : 2;  // experts of a thread
  __shared__ int scan[Waves];
  const int E = a.n_experts, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int *next = lds;                 // [wave][expert]: counts, then next rows
  int *before = next + Waves * E;  // [expert]: copies in the tiles before
  int *total = before + E;         // [expert]: copies in all tiles
  int *start = total + E;          // [expert + 1]: first rows
  const int64_t lo = Single ? 0 : blockIdx.x * a.tile, hi = lo + a.tile < a.n_pairs ? lo + a.tile : a.n_pairs;
  const int64_t part = a.tile / Waves, from = lo + wave * part, to = from + part < hi ? from + part : hi;
  for (int e = threadIdx.x; e < (Waves + 2) * E; e += Threads) lds[e] = 0;
  __syncthreads();
#pragma unroll 1
  for (int64_t base = from; base < to; base += 64 * kAhead) {
    int e[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) e[j] = expert_at(a, base + 64 * j + lane, to);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (e[j] >= 0) atomicAdd(&next[wave * E + e[j]], 1);
  }
  if (!Single) {
    // thread = (four experts, every parts-th tile)
    const int quads = counts_row(E) / 4, parts = Threads / quads, quad = threadIdx.x % quads;
    if ((int)threadIdx.x < parts * quads) {
      int b[4] = {0, 0, 0, 0}, t[4] = {0, 0, 0, 0};
#pragma unroll 4
      for (int k = threadIdx.x / quads; k < a.n_tiles; k += parts) {
        const int4 c = *(const int4 *)(a.tile_counts + (int64_t)k * counts_row(E) + 4 * quad);
        const int v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b[i] += k < (int)blockIdx.x ? v[i] : 0;
          t[i] += v[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * quad + i < E) {
          atomicAdd(&before[4 * quad + i], b[i]);
          atomicAdd(&total[4 * quad + i], t[i]);
        }
    }
  }
  __syncthreads();
  // first rows: a scan of the padded counts over the experts, a run of Per of them to each thread
  int used[Per][Waves], all[Per], size[Per], sum = 0;
#pragma unroll
  for (int p = 0; p < Per; ++p) {
    const int e = threadIdx.x * Per + p;
    int own = 0;
#pragma unroll
    for (int w = 0; w < Waves; ++w) used[p][w] = e < E ? next[w * E + e] : 0;
#pragma unroll
    for (int w = 0; w < Waves; ++w) own += used[p][w];
    all[p] = Single ? own : e < E ? total[e] : 0;
    size[p] = (int)(((uint32_t)all[p] + a.align - 1) / (uint32_t)a.align) * a.align;
    sum += size[p];
  }
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(upto, d);
    if (lane >= d) upto += up;
  }
  if (lane == 63) scan[wave] = upto;
  __syncthreads();
  int at = upto - sum;
#pragma unroll
  for (int w = 0; w < Waves; ++w) at += w < wave ? scan[w] : 0;
#pragma unroll
  for (int p = 0; p < Per; ++p) {
    const int e = threadIdx.x * Per + p;
    if (e < E) {
      int row = at + before[e];
#pragma unroll
      for (int w = 0; w < Waves; ++w) {
        next[w * E + e] = row;
        row += used[p][w];
      }
      start[e] = at;
      total[e] = all[p];
      if (blockIdx.x == 0) {
        a.offsets[e] = at;
        if (a.counts) a.counts[e] = all[p];
      }
      at += size[p];
      if (e == E - 1) {
        start[E] = at;
        if (blockIdx.x == 0) a.offsets[E] = at;
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int64_t base = !Single || blockIdx.x == 0 ? from : to; base < to; base += 64 * kAhead) {
    int expert[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) expert[j] = expert_at(a, base + 64 * j + lane, to);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (base + 64 * j >= to) break;
      const int64_t i = base + 64 * j + lane;
      const int e = expert[j];
      const uint64_t same = same_expert(e);
      int row = -1;
      if (e >= 0) {
        const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
        row = next[wave * E + e] + rank;
        wave_lds_fence();
        if (rank == 0) next[wave * E + e] = row + __popcll(same);
        wave_lds_fence();
        if (row >= a.n_rows) row = -1;
        else if (a.row_token) a.row_token[row] = (int32_t)((uint32_t)i / (uint32_t)a.top_k);
      }
      if (i < to && a.pair_row) a.pair_row[i] = row;
    }
  }
  if (!a.row_token) return;
  // rows that hold no copy: behind each expert's copies (a wave per expert), and behind the last expert
  for (int e = a.align > 1 ? blockIdx.x * Waves + wave : E; e < E; e += gridDim.x * Waves) {
    const int64_t end = start[e + 1] < a.n_rows ? start[e + 1] : a.n_rows;
    for (int64_t r = (int64_t)start[e] + total[e] + lane; r < end; r += 64) a.row_token[r] = -1;
  }
  for (int64_t r = (int64_t)start[E] + blockIdx.x * Threads + threadIdx.x; r < a.n_rows;
       r += (int64_t)gridDim.x * Threads)
    a.row_token[r] = -1;
}

// Copies of a tile.
int64_t tile_of(int64_t pairs) {
  if (pairs <= kRowsFew) return kRowsTile / 2;
  return std::max(kRowsTile, (pairs + kMaxTiles - 1) / kMaxTiles);
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

}  // namespace
}  // namespace wt

using namespace wt;

extern "C" {

wt_status wt_dispatch_workspace_bytes(int64_t n_tokens, int32_t top_k, int32_t n_experts, size_t *bytes) {
  const char *what = "wt_dispatch_workspace_bytes";
  try {
    const wt_status st = check_sizes(what, n_tokens, top_k, n_experts);
    if (st != WT_OK) return st;
    if (!bytes) return fail(what, "NULL result");
    const int64_t pairs = n_tokens * top_k, tile = tile_of(pairs);
    *bytes = (size_t)(4 * counts_row(n_experts) * ((pairs + tile - 1) / tile) + 16);
    return WT_OK;
  } catch (...) {
    return caught_status();
  }
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
    const bool single = pairs <= kRowsSingle;
    const int waves = n_experts <= kManyExperts ? 16 : 8, unit = 64 * waves;
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
    a.tile_counts = (int32_t *)(((uintptr_t)workspace + 15) / 16 * 16);
    a.tile = single ? pairs : tile_of(pairs);
    a.tile = (a.tile + unit - 1) / unit * unit;
    if (a.tile == 0) a.tile = unit;
    a.n_tiles = (int32_t)((pairs + a.tile - 1) / a.tile);
    const hipStream_t s = (hipStream_t)stream;
    // workgroups behind the last tile only fill rows
    const int64_t fill = row_token ? std::min<int64_t>(n_rows / kRowsFill, kMaxFill) : 0;
    const uint32_t grid = (uint32_t)std::max<int64_t>({1, a.n_tiles, fill}), threads = 64u * waves;
    const uint32_t lds = 4u * ((waves + 3) * n_experts + 1);
    if (!single && a.n_tiles > 0)
      hipLaunchKernelGGL(rows_count_kernel, dim3((uint32_t)a.n_tiles), dim3(threads), 4u * n_experts, s, a);
    const auto kernel = single ? (waves == 16 ? rows_place_kernel<true, 16> : rows_place_kernel<true, 8>)
                               : (waves == 16 ? rows_place_kernel<false, 16> : rows_place_kernel<false, 8>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), lds, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(what, hip_msg("launch", e), WT_E_HIP);
    return WT_OK;
  } catch (...) {
    return caught_status();
  }
}

}  // extern "C"
