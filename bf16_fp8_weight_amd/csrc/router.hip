// router.hip -- expert selection, per-expert counts and the balance loss of
// a routed layer, forward and backward, for gfx950. The definition is in wt.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "fp8_math.h"
#include "hip_util.h"
#include "plan.h"
#include "wave.h"
#include "wt.h"

namespace wt {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;

struct RouterArgs {
  uint64_t logits;
  const float *bias;
  const int32_t *offsets;
  int32_t n_tokens, n_experts, top_k, n_seqs;
  int64_t stride;
  int32_t tile;  // tokens of one workgroup
  bool bf16, softmax, normalize;
  float scale, coef;
};

// First token of sequence q (q = n_seqs: one behind the last), kept inside
// [0, n_tokens] whatever the array holds.
__device__ __forceinline__ int32_t seq_start(const RouterArgs &a, int32_t q) {
  if (!a.offsets) return q == 0 ? 0 : a.n_tokens;
  const int32_t x = a.offsets[q];
  return x < 0 ? 0 : x > a.n_tokens ? a.n_tokens : x;
}

// Lowest q with seq_start(q + 1) > t, or n_seqs.
__device__ __forceinline__ int32_t seq_of(const RouterArgs &a, int32_t t) {
  int32_t lo = 0, hi = a.n_seqs;
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (seq_start(a, mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The runs of a workgroup's tokens [t, end) that belong to one sequence, or
// to none (seq < 0).
struct Runs {
  int32_t t, end, q;
  __device__ Runs(const RouterArgs &a, int32_t first, int32_t last) : t(first), end(last), q(seq_of(a, first)) {}
  __device__ bool next(const RouterArgs &a, int32_t *lo, int32_t *hi, int32_t *seq) {
    if (t >= end) return false;
    while (q < a.n_seqs && seq_start(a, q + 1) <= t) ++q;
    *lo = t;
    const int32_t start = q < a.n_seqs ? seq_start(a, q) : end;
    if (q >= a.n_seqs || start > t) {
      *seq = -1;
      *hi = start < end ? start : end;
    } else {
      *seq = q;
      const int32_t stop = seq_start(a, q + 1);
      *hi = stop < end ? stop : end;
    }
    t = *hi;
    return true;
  }
};

// A token's logits: lane l holds experts l, l + 64, ... (-infinity beyond the last).
template <int NJ>
__device__ __forceinline__ void load_row(const RouterArgs &a, int64_t t, int lane, float x[NJ]) {
  const uint64_t row = a.logits + (a.bf16 ? 2ull : 4ull) * (uint64_t)(t * a.stride);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 64 * j;
    x[j] = -INFINITY;
    if (e < a.n_experts)
      x[j] = a.bf16 ? bf16_lo(ld_global<uint16_t>(row + 2ull * e)) : ld_global<float>(row + 4ull * e);
  }
}

// What turns a logit into its score (softmax: exp(x - top) inv) and a score
// into its probability (sigmoid: s inv).
struct Norm {
  float top, inv;
};

__device__ __forceinline__ float score_of(const RouterArgs &a, const Norm &n, float x) {
  return a.softmax ? expf(x - n.top) * n.inv : 1.0f / (1.0f + expf(-x));
}

template <int NJ>
__device__ __forceinline__ Norm scores(const RouterArgs &a, const float x[NJ], float s[NJ]) {
  Norm n{0.0f, 1.0f};
  if (a.softmax) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) m = fmaxf(m, x[j]);
    m = wave_max(m);
    n.top = m == -INFINITY ? 0.0f : m;
  }
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    s[j] = score_of(a, n, x[j]);
    z += s[j];
  }
  z = wave_sum(z);
  if (a.softmax) {
    n.inv = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] *= n.inv;
  } else {
    n.inv = 1.0f / (z + 1e-20f);
  }
  return n;
}

__device__ __forceinline__ bool selectable(float x) { return x > -INFINITY; }  // false for NaN

// Two keys closer than this may stand in the wrong order: a score carries at
// most 4 fp32 roundings (exponential, sum, quotient, product: below 5e-7 of
// it) and the sum with the bias one of the key.
__device__ __forceinline__ float near_tie(float key) { return 2e-6f * (1.0f + fabsf(key)); }

// Selection in 64 bits for a token with two keys too close to order in 32
// (out of line, from the logits again: it is rare and must cost no registers).
template <int NJ>
__device__ __attribute__((noinline)) int select_exact(const RouterArgs &a, int64_t t, int lane) {
  float x[NJ];
  double k[NJ];
  load_row<NJ>(a, t, lane, x);
  double top = -INFINITY, z = 0.0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) top = fmax(top, selectable(x[j]) ? (double)x[j] : -INFINITY);
  for (int d = 32; d; d >>= 1) top = fmax(top, __shfl_xor(top, d));
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    k[j] = a.softmax ? exp((double)x[j] - top) : 1.0 / (1.0 + exp(-(double)x[j]));
    z += selectable(x[j]) ? k[j] : 0.0;
  }
  for (int d = 32; d; d >>= 1) z += __shfl_xor(z, d);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 64 * j;
    k[j] = selectable(x[j]) && e < a.n_experts ? (a.softmax ? k[j] / z : k[j]) + (double)a.bias[e] : -INFINITY;
  }
  int index = -1;
  for (int r = 0; r < a.top_k; ++r) {
    double best = -INFINITY;
    int at = kMaxExperts;
#pragma unroll
    for (int j = NJ - 1; j >= 0; --j)
      if (k[j] >= best && k[j] > -INFINITY) best = k[j], at = lane + 64 * j;
    for (int d = 32; d; d >>= 1) {
      const double ob = __shfl_xor(best, d);
      const int oa = __shfl_xor(at, d);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if (at >= kMaxExperts) break;
    if (lane == r) index = at;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (lane + 64 * j == at) k[j] = -INFINITY;
  }
  return index;
}

// Selection: lane r < top_k receives the r-th expert (-1: none left).
// A round takes the greatest key over the wave and, by ballots in the order
// of the expert's number, the lowest expert that has it. With a bias the keys
// carry roundings: rounds go on behind the last place until a different key
// shows that its border is safe, and a near tie decides in 64 bits.
template <int NJ>
__device__ __forceinline__ int select_topk(const RouterArgs &a, int64_t t, const float x[NJ], const float s[NJ],
                                           const float b[NJ], int lane) {
  float k[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const float key = a.bias ? s[j] + b[j] : x[j];
    k[j] = selectable(x[j]) && selectable(key) ? key : -INFINITY;  // never NaN from here on
  }
  int index = -1;
  bool close = false;
  float key0 = 0.0f, x0 = 0.0f, b0 = 0.0f;
  for (int r = 0;; ++r) {
    if (!a.bias && r == a.top_k) break;
    float m = k[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) m = fmaxf(m, k[j]);
    m = wave_max(m);
    if (m == -INFINITY) break;
    int at = 0;
    float xr = 0.0f, br = 0.0f;
    bool found = false;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (!found) {
        const uint64_t who = __ballot(k[j] == m);
        if (who) {
          const int l = __builtin_ctzll(who);
          found = true;
          at = l + 64 * j;
          if (a.bias) {
            xr = __shfl(x[j], l);
            br = __shfl(b[j], l);
          }
          if (lane == l) k[j] = -INFINITY;
        }
      }
    if (a.bias) {
      const bool same = r > 0 && xr == x0 && br == b0;
      if (r > 0 && !same && key0 - m <= near_tie(key0)) close = true;
      if (r >= a.top_k && !same) break;
      key0 = m, x0 = xr, b0 = br;
    }
    if (r < a.top_k && lane == r) index = at;
  }
  return close ? select_exact<NJ>(a, t, lane) : index;
}

struct ForwardOut {
  int32_t *index;
  float *weight;
  float *part_p;    // [tile + sequence][expert]: sums of probabilities
  int32_t *part_c;  // and selections of the tokens that the two share
};

// Forward pass over tokens. One wave per token; a workgroup's tile of tokens
// is cut at the sequences' borders, and the tokens that tile i shares with
// sequence q leave their sums at row i + q: along the tokens each step to the
// next pair raises i or q, so no two pairs share a row, no sum needs an
// atomic, and the order of every sum is fixed.
template <int NJ>
__global__ void __launch_bounds__(kThreads) router_forward_kernel(RouterArgs a, ForwardOut o) {
  __shared__ float sum[kWaves][64 * NJ];
  __shared__ int cnt[64 * NJ];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t first = blockIdx.x * a.tile;
  const int32_t last = a.n_tokens - first < a.tile ? a.n_tokens : first + a.tile;
  float b[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) b[j] = a.bias && lane + 64 * j < a.n_experts ? a.bias[lane + 64 * j] : 0.0f;
  Runs runs(a, first, last);
  int32_t lo, hi, q;
  while (runs.next(a, &lo, &hi, &q)) {
    if (q < 0) {
      for (int64_t i = (int64_t)lo * a.top_k + threadIdx.x; i < (int64_t)hi * a.top_k; i += kThreads) {
        o.index[i] = -1;
        o.weight[i] = 0.0f;
      }
      continue;
    }
    for (int e = threadIdx.x; e < a.n_experts; e += kThreads) cnt[e] = 0;
    __syncthreads();
    float acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = 0.0f;
    for (int32_t t = lo + wave; t < hi; t += kWaves) {
      float x[NJ], s[NJ];
      load_row<NJ>(a, t, lane, x);
      const Norm n = scores<NJ>(a, x, s);
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[j] += a.softmax ? s[j] : s[j] * n.inv;
      const int index = select_topk<NJ>(a, t, x, s, b, lane);
      float w = 0.0f;
      if (index >= 0) {
        const uint64_t row = a.logits + (a.bf16 ? 2ull : 4ull) * (uint64_t)((int64_t)t * a.stride);
        w = score_of(a, n, a.bf16 ? bf16_lo(ld_global<uint16_t>(row + 2ull * index)) : ld_global<float>(row + 4ull * index));
        atomicAdd(&cnt[index], 1);
      }
      if (a.normalize) w /= wave_sum(w) + 1e-20f;
      if (lane < a.top_k) {
        o.index[(int64_t)t * a.top_k + lane] = index;
        o.weight[(int64_t)t * a.top_k + lane] = w * a.scale;
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) sum[wave][lane + 64 * j] = acc[j];
    __syncthreads();
    const int64_t row = ((int64_t)blockIdx.x + q) * a.n_experts;
    for (int e = threadIdx.x; e < a.n_experts; e += kThreads) {
      o.part_p[row + e] = (sum[0][e] + sum[1][e]) + (sum[2][e] + sum[3][e]);
      o.part_c[row + e] = cnt[e];
    }
    __syncthreads();
  }
}

constexpr int kChunk = 16;  // experts of one workgroup in the reductions

__device__ __forceinline__ double sum_of_16(double x, double *lds) {
  // rows of 16 experts: thread = 16 row + expert; sums over the 16 rows
  lds[threadIdx.x] = x;
  __syncthreads();
  for (int d = 8; d; d >>= 1) {
    if ((int)(threadIdx.x >> 4) < d) lds[threadIdx.x] += lds[threadIdx.x + 16 * d];
    __syncthreads();
  }
  const double r = lds[threadIdx.x & 15];
  __syncthreads();
  return r;
}

// Per sequence and 16 experts: the tiles' partial sums, the counts, and these
// experts' part of the loss.
__global__ void __launch_bounds__(kThreads)
    router_reduce_kernel(RouterArgs a, const float *part_p, const int32_t *part_c, int32_t *seq_counts,
                         double *part_loss) {
  __shared__ double lds[kThreads];
  const int32_t q = blockIdx.x, e = blockIdx.y * kChunk + (threadIdx.x & 15), row = threadIdx.x >> 4;
  const int32_t lo = seq_start(a, q), hi = seq_start(a, q + 1);
  double p = 0.0, c = 0.0;
  if (hi > lo && e < a.n_experts) {
    const int32_t last = (hi - 1) / a.tile;
    for (int32_t i = lo / a.tile + row; i <= last; i += 16) {
      const int64_t at = ((int64_t)i + q) * a.n_experts + e;
      p += (double)part_p[at];
      c += (double)part_c[at];
    }
  }
  p = sum_of_16(p, lds);
  c = sum_of_16(c, lds);
  double part = 0.0;
  if (row == 0 && e < a.n_experts) {
    seq_counts[(int64_t)q * a.n_experts + e] = (int32_t)c;
    const double n = hi > lo ? (double)(hi - lo) : 1.0;
    part = c * p / (n * n);
  }
  // over the 16 experts: lanes 0..15 of the first wave
  if (threadIdx.x < 64) {
    for (int d = 8; d; d >>= 1) part += __shfl_xor(part, d);
    if (threadIdx.x == 0) part_loss[(int64_t)q * gridDim.y + blockIdx.y] = part;
  }
}

// Block 0: the loss from its parts. The others: counts over all sequences of
// 16 experts each.
__global__ void __launch_bounds__(kThreads)
    router_finish_kernel(RouterArgs a, const int32_t *seq_counts, const double *part_loss, int64_t n_parts,
                         int32_t *counts, float *loss) {
  __shared__ double lds[kThreads];
  if (blockIdx.x == 0) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n_parts; i += kThreads) s += part_loss[i];
    s = sum_of_16(s, lds);
    if (threadIdx.x < 64) {
      if (threadIdx.x >= 16) s = 0.0;
      for (int d = 8; d; d >>= 1) s += __shfl_xor(s, d);
      if (threadIdx.x == 0)
        *loss = (float)(s * (double)a.coef * (double)a.n_experts / ((double)a.top_k * (double)a.n_seqs));
    }
    return;
  }
  const int32_t e = (blockIdx.x - 1) * kChunk + (threadIdx.x & 15);
  double c = 0.0;
  if (e < a.n_experts)
    for (int32_t q = threadIdx.x >> 4; q < a.n_seqs; q += 16) c += (double)seq_counts[(int64_t)q * a.n_experts + e];
  c = sum_of_16(c, lds);
  if (threadIdx.x < 16 && e < a.n_experts) counts[e] = (int32_t)c;
}

struct BackwardIo {
  const int32_t *index;
  const int32_t *seq_counts;
  const float *dweight;
  const float *dloss;
  uint64_t dlogits;
  int64_t dstride;
};

__device__ __forceinline__ void store_logit(const RouterArgs &a, uint64_t row, int e, float x) {
  if (a.bf16)
    st_global<uint16_t>(row + 2ull * e, __builtin_bit_cast(uint16_t, (__bf16)x));
  else
    st_global<float>(row + 4ull * e, x);
}

// Backward pass: one wave per token, scores recomputed from the logits (which
// have to be read anyway). Of the loss, d/dp_e is the same for all tokens of a
// sequence and stays in registers; of the weights, the top_k values go to
// their experts' lanes through the wave's row of shared memory.
template <int NJ>
__global__ void __launch_bounds__(kThreads) router_backward_kernel(RouterArgs a, BackwardIo o) {
  __shared__ float direct[kWaves][64 * NJ];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float *mine = direct[wave];
#pragma unroll
  for (int j = 0; j < NJ; ++j) mine[lane + 64 * j] = 0.0f;
  const int32_t first = blockIdx.x * a.tile;
  const int32_t last = a.n_tokens - first < a.tile ? a.n_tokens : first + a.tile;
  const uint64_t size = a.bf16 ? 2 : 4;
  Runs runs(a, first, last);
  int32_t lo, hi, q;
  while (runs.next(a, &lo, &hi, &q)) {
    float b[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) b[j] = 0.0f;
    if (q >= 0 && o.dloss) {
      const double n = (double)(seq_start(a, q + 1) - seq_start(a, q));
      const float f =
          (float)((double)*o.dloss * (double)a.coef * a.n_experts / ((double)a.n_seqs * (double)a.top_k * n * n));
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (lane + 64 * j < a.n_experts) b[j] = f * (float)o.seq_counts[(int64_t)q * a.n_experts + lane + 64 * j];
    }
    for (int32_t t = lo + wave; t < hi; t += kWaves) {
      const uint64_t drow = o.dlogits + size * (uint64_t)((int64_t)t * o.dstride);
      if (q < 0) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (lane + 64 * j < a.n_experts) store_logit(a, drow, lane + 64 * j, 0.0f);
        continue;
      }
      const uint64_t row = a.logits + size * (uint64_t)((int64_t)t * a.stride);
      int at = -1;
      float d = 0.0f, sel = 0.0f;
      if (o.dweight && lane < a.top_k) {
        at = o.index[(int64_t)t * a.top_k + lane];
        if (at < 0 || at >= a.n_experts) at = -1;
        else d = o.dweight[(int64_t)t * a.top_k + lane] * a.scale;
      }
      float x[NJ], s[NJ];
      load_row<NJ>(a, t, lane, x);
      const Norm n = scores<NJ>(a, x, s);
      if (o.dweight) {
        if (at >= 0)
          sel = score_of(a, n, a.bf16 ? bf16_lo(ld_global<uint16_t>(row + 2ull * at)) : ld_global<float>(row + 4ull * at));
        if (a.normalize) {
          const float z = wave_sum(sel) + 1e-20f;
          d = (d - wave_sum(d * sel) / z) / z;
        }
        if (at >= 0) atomicAdd(&mine[at], d);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      float g[NJ], dot = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        g[j] = o.dweight ? mine[lane + 64 * j] : 0.0f;
        dot += (a.softmax ? b[j] + g[j] : b[j]) * s[j];
      }
      if (o.dweight) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (at >= 0) mine[at] = 0.0f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      dot = wave_sum(dot);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = lane + 64 * j;
        if (e >= a.n_experts) continue;
        const float dx = a.softmax ? s[j] * (b[j] + g[j] - dot)
                                   : ((b[j] - dot * n.inv) * n.inv + g[j]) * s[j] * (1.0f - s[j]);
        store_logit(a, drow, e, dx);
      }
    }
  }
}

// Tokens of one workgroup.
int32_t tile_of(int64_t n_tokens) {
  int32_t tile = 4;
  while (tile < 64 && n_tokens > (int64_t)tile * 1024) tile *= 2;
  return tile;
}

int chunks_of(int n_experts) { return (n_experts + kChunk - 1) / kChunk; }

struct Workspace {
  int64_t part_p, part_c, part_loss, bytes;
};

Workspace workspace_of(const wt_router_desc &d) {
  const int64_t tile = tile_of(d.n_tokens);
  const int64_t rows = (d.n_tokens + tile - 1) / tile + d.n_seqs;
  Workspace w;
  w.part_p = 0;
  w.part_c = 4 * rows * d.n_experts;
  w.part_loss = (w.part_c + 4 * rows * d.n_experts + 15) / 16 * 16;
  w.bytes = w.part_loss + 8 * (int64_t)d.n_seqs * chunks_of(d.n_experts);
  return w;
}

wt_status fail(const char *what, const std::string &m, wt_status st = WT_E_INVAL) {
  set_thread_error(std::string(what) + ": " + m);
  return st;
}

wt_status check_desc(const char *what, const wt_router_desc *d) {
  if (!d) return fail(what, "NULL description");
  if (d->n_experts < 1 || d->n_experts > kMaxExperts) return fail(what, "n_experts out of range");
  if (d->top_k < 1 || d->top_k > kMaxTopK || d->top_k > d->n_experts) return fail(what, "top_k out of range");
  if (d->n_tokens < 0 || d->n_tokens > (((int64_t)1 << 31) - 1) / d->top_k) return fail(what, "n_tokens out of range");
  if (d->logits_dtype != WT_DT_F32 && d->logits_dtype != WT_DT_BF16) return fail(what, "unknown logits type");
  if (d->score != WT_SCORE_SIGMOID && d->score != WT_SCORE_SOFTMAX) return fail(what, "unknown score");
  if (d->normalize != 0 && d->normalize != 1) return fail(what, "normalize must be 0 or 1");
  if (!std::isfinite(d->scale) || !std::isfinite(d->balance_coef)) return fail(what, "scale or balance_coef not finite");
  if (d->n_seqs < 1 || d->n_seqs > (1 << 20)) return fail(what, "n_seqs out of range");
  if (!d->seq_offsets && d->n_seqs != 1) return fail(what, "several sequences without seq_offsets");
  return WT_OK;
}

wt_status check_memory_args(const char *what, const wt_router_desc *d) {
  const int64_t size = d->logits_dtype == WT_DT_BF16 ? 2 : 4;
  if (d->logits_stride < d->n_experts || d->logits_stride > ((int64_t)1 << 40)) return fail(what, "logits_stride out of range");
  if (d->n_tokens > 0 && !d->logits) return fail(what, "NULL logits");
  if ((uintptr_t)d->logits % size) return fail(what, "logits misaligned", WT_E_ALIGN);
  if ((uintptr_t)d->bias % 4 || (uintptr_t)d->seq_offsets % 4) return fail(what, "bias or seq_offsets misaligned", WT_E_ALIGN);
  return WT_OK;
}

RouterArgs args_of(const wt_router_desc &d) {
  RouterArgs a{};
  a.logits = (uint64_t)(uintptr_t)d.logits;
  a.bias = d.bias;
  a.offsets = d.seq_offsets;
  a.n_tokens = (int32_t)d.n_tokens;
  a.n_experts = d.n_experts;
  a.top_k = d.top_k;
  a.n_seqs = d.n_seqs;
  a.stride = d.logits_stride;
  a.tile = tile_of(d.n_tokens);
  a.bf16 = d.logits_dtype == WT_DT_BF16;
  a.softmax = d.score == WT_SCORE_SOFTMAX;
  a.normalize = d.normalize;
  a.scale = d.scale;
  a.coef = d.balance_coef;
  return a;
}

// Calls f with the number of 64-expert columns as a constant.
template <class F>
void with_columns(int n_experts, F f) {
  const int nj = (n_experts + 63) / 64;
  if (nj <= 1) f(std::integral_constant<int, 1>());
  else if (nj <= 2) f(std::integral_constant<int, 2>());
  else if (nj <= 3) f(std::integral_constant<int, 3>());
  else if (nj <= 4) f(std::integral_constant<int, 4>());
  else if (nj <= 6) f(std::integral_constant<int, 6>());
  else if (nj <= 8) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
}

}  // namespace
}  // namespace wt

using namespace wt;

extern "C" {

void wt_router_desc_init(wt_router_desc *desc) {
  if (!desc) return;
  std::memset(desc, 0, sizeof *desc);
  desc->top_k = 1;
  desc->n_seqs = 1;
  desc->scale = 1.0f;
}

wt_status wt_router_workspace_bytes(const wt_router_desc *desc, size_t *bytes) {
  const char *what = "wt_router_workspace_bytes";
  const wt_status st = check_desc(what, desc);
  if (st != WT_OK) return st;
  if (!bytes) return fail(what, "NULL result");
  *bytes = (size_t)workspace_of(*desc).bytes;
  return WT_OK;
}

wt_status wt_router_forward(const wt_router_desc *desc, int32_t *index, float *weight, int32_t *counts,
                            int32_t *seq_counts, float *loss, void *workspace, size_t workspace_bytes, void *stream) {
  const char *what = "wt_router_forward";
  try {
    wt_status st = check_desc(what, desc);
    if (st == WT_OK) st = check_memory_args(what, desc);
    if (st != WT_OK) return st;
    if (desc->n_tokens > 0 && (!index || !weight)) return fail(what, "NULL index or weight");
    if (!seq_counts || !loss || !workspace) return fail(what, "NULL seq_counts, loss or workspace");
    if (((uintptr_t)index | (uintptr_t)weight | (uintptr_t)counts | (uintptr_t)seq_counts | (uintptr_t)loss) % 4)
      return fail(what, "output misaligned", WT_E_ALIGN);
    if ((uintptr_t)workspace % 16) return fail(what, "workspace not 16-byte aligned", WT_E_ALIGN);
    const Workspace w = workspace_of(*desc);
    if (workspace_bytes < (size_t)w.bytes) return fail(what, "workspace too small", WT_E_RANGE);
    const RouterArgs a = args_of(*desc);
    const hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)workspace;
    float *part_p = (float *)(base + w.part_p);
    int32_t *part_c = (int32_t *)(base + w.part_c);
    double *part_loss = (double *)(base + w.part_loss);
    const uint32_t tiles = (uint32_t)((a.n_tokens + a.tile - 1) / a.tile), chunks = (uint32_t)chunks_of(a.n_experts);
    if (tiles > 0)
      with_columns(a.n_experts, [&](auto nj) {
        hipLaunchKernelGGL((router_forward_kernel<decltype(nj)::value>), dim3(tiles), dim3(kThreads), 0, s, a,
                           ForwardOut{index, weight, part_p, part_c});
      });
    hipLaunchKernelGGL(router_reduce_kernel, dim3((uint32_t)a.n_seqs, chunks), dim3(kThreads), 0, s, a, part_p, part_c,
                       seq_counts, part_loss);
    hipLaunchKernelGGL(router_finish_kernel, dim3(counts ? 1 + chunks : 1), dim3(kThreads), 0, s, a, seq_counts,
                       part_loss, (int64_t)a.n_seqs * chunks, counts, loss);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(what, hip_msg("launch", e), WT_E_HIP);
    return WT_OK;
  } catch (...) {
    set_thread_error("internal error");
    return WT_E_INVAL;
  }
}

wt_status wt_router_backward(const wt_router_desc *desc, const int32_t *index, const int32_t *seq_counts,
                             const float *dweight, const float *dloss, void *dlogits, int64_t dlogits_stride,
                             void *stream) {
  const char *what = "wt_router_backward";
  try {
    wt_status st = check_desc(what, desc);
    if (st == WT_OK) st = check_memory_args(what, desc);
    if (st != WT_OK) return st;
    if (dlogits_stride < desc->n_experts || dlogits_stride > ((int64_t)1 << 40))
      return fail(what, "dlogits_stride out of range");
    if (desc->n_tokens == 0) return WT_OK;
    if (!dlogits) return fail(what, "NULL dlogits");
    if (dweight && !index) return fail(what, "dweight without index");
    if (dloss && !seq_counts) return fail(what, "dloss without seq_counts");
    if (((uintptr_t)index | (uintptr_t)seq_counts | (uintptr_t)dweight | (uintptr_t)dloss) % 4)
      return fail(what, "input misaligned", WT_E_ALIGN);
    if ((uintptr_t)dlogits % (desc->logits_dtype == WT_DT_BF16 ? 2 : 4))
      return fail(what, "dlogits misaligned", WT_E_ALIGN);
    if (dlogits == desc->logits && dlogits_stride != desc->logits_stride)
      return fail(what, "dlogits on the logits with another stride", WT_E_OVERLAP);
    const RouterArgs a = args_of(*desc);
    const uint32_t tiles = (uint32_t)((a.n_tokens + a.tile - 1) / a.tile);
    const BackwardIo io{index, seq_counts, dweight, dloss, (uint64_t)(uintptr_t)dlogits, dlogits_stride};
    with_columns(a.n_experts, [&](auto nj) {
      hipLaunchKernelGGL((router_backward_kernel<decltype(nj)::value>), dim3(tiles), dim3(kThreads), 0,
                         (hipStream_t)stream, a, io);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(what, hip_msg("launch", e), WT_E_HIP);
    return WT_OK;
  } catch (...) {
    set_thread_error("internal error");
    return WT_E_INVAL;
  }
}

}  // extern "C"
