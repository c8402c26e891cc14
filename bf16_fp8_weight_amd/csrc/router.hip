// router.hip -- expert selection, per-expert counts and the balance loss of
// a routed layer, forward and backward, for gfx950. The definition is in wt.h.
//
// Forward: one pass over the logits leaves selections, weights and, per tile
// of tokens and sequence, sums of probabilities and counts; one or two small
// launches reduce those. 16384 tokens x 384 experts are 26 MB, 5.6 us at the
// card's copy rate, and take 17.8 us, 22.8 us with the reductions. The pass is
// bound by latency: its 273 vector and 202 scalar instructions a token need some
// 7 us to issue, but each token's selection is one chain of dependent steps, and
// the waves wait for 48 % of their cycles. Backward: one pass that reads the
// logits again and writes their gradient, 51 MB in 11.5 us (4.5 TB/s).
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

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int64_t kMaxTokens = (int64_t)1 << 27;  // sixteen threads each (backward) stay below a launch's 2^32

constexpr int kWaves = 8;  // of a workgroup of the forward pass

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

// Lowest q with seq_start(q + 1) > t, or n_seqs: a search that probes 64
// places at once, so that up to 64 sequences cost one load.
__device__ __forceinline__ int32_t seq_of(const RouterArgs &a, int32_t t) {
  const int lane = threadIdx.x & 63;
  int32_t lo = 0, hi = a.n_seqs;
  while (hi - lo > 64) {
    const int32_t step = (hi - lo + 63) >> 6, at = min(lo + (lane + 1) * step, hi);
    const int n = __popcll(__ballot(seq_start(a, at) <= t));
    lo = min(lo + n * step, hi);
    hi = min(lo + step, hi);
  }
  const bool behind = lo + lane < hi && seq_start(a, lo + lane + 1) <= t;
  return lo + __popcll(__ballot(behind));
}

// The runs of a workgroup's tokens [t, end) that belong to one sequence, or
// to none (seq < 0).
struct Runs {
  int32_t t, end, q;
  __device__ Runs(const RouterArgs &a, int32_t first, int32_t last) : t(first), end(last), q(seq_of(a, first)) {}
  __device__ bool next(const RouterArgs &a, int32_t *lo, int32_t *hi, int32_t *seq) {
    if (t >= end) return false;
    int32_t start = end, stop = end;
    for (; q < a.n_seqs; ++q) {
      start = seq_start(a, q);
      stop = seq_start(a, q + 1);
      if (stop > t) break;
    }
    *lo = t;
    if (q >= a.n_seqs || start > t) {
      *seq = -1;
      *hi = q < a.n_seqs && start < end ? start : end;
    } else {
      *seq = q;
      *hi = stop < end ? stop : end;
    }
    t = *hi;
    return true;
  }
};

// The wave's number in its workgroup, known to be uniform: what depends on it
// (the token, its rows' addresses) then lives in scalar registers.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

__device__ __forceinline__ uint64_t row_of(uint64_t base, int64_t t, int64_t stride, bool bf16) {
  return base + (uint64_t)(t * stride) * (bf16 ? 2u : 4u);
}

__device__ __forceinline__ float load_at(uint64_t row, uint32_t e, bool bf16) {
  return bf16 ? bf16_lo(ld_global<uint16_t>(row + 2u * e)) : ld_global<float>(row + 4u * e);
}

__device__ __forceinline__ float load_logit(const RouterArgs &a, int64_t t, uint32_t e) {
  return load_at(row_of(a.logits, t, a.stride, a.bf16), e, a.bf16);
}

// A row as a buffer: accesses beyond its last expert read 0 and write nothing,
// so that no lane needs a branch or an address of its own.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(uint64_t row, int n, bool bf16) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)row, 0, n * (bf16 ? 2 : 4), 0x00020000);
}

// A token's logits as they lie in memory: lane l holds experts l, l + 64, ...
// Nothing touches the values before logits_of, so that a row can be on its way
// while the one before it is worked on.
template <int NJ>
__device__ __forceinline__ void load_row(const RouterArgs &a, int64_t t, uint32_t lane, uint32_t raw[NJ]) {
  const auto row = row_buffer(row_of(a.logits, t, a.stride, a.bf16), a.n_experts, a.bf16);
  if (a.bf16) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) raw[j] = __builtin_amdgcn_raw_buffer_load_b16(row, 2 * lane + 128 * j, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) raw[j] = __builtin_amdgcn_raw_buffer_load_b32(row, 4 * lane + 256 * j, 0, 0);
  }
}

// The logits of a loaded row, -infinity beyond the last expert.
template <int NJ>
__device__ __forceinline__ void logits_of(const RouterArgs &a, uint32_t lane, const uint32_t raw[NJ], float x[NJ]) {
  const uint32_t shift = a.bf16 ? 16 : 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    x[j] = lane + 64 * j < (uint32_t)a.n_experts ? __uint_as_float(raw[j] << shift) : -INFINITY;
}

// What turns a logit into its score (softmax: exp(x - top) inv) and a score
// into its probability (sigmoid: s inv).
struct Norm {
  float top, inv;
};

// exp(x) as 2^(x log2 e): the rounding of the product makes it off by |x|
// 2^-24 of the result, so by less than 2^-24 of 1 / e at the most where the
// result is below 1 (all there is here: 1 / (1 + exp) and exp(x - top)).
// Relative to a small score the error grows with |x|, to 4e-6 at x = -60; a
// longer argument would cost further instructions for every logit.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

template <bool Softmax>
__device__ __forceinline__ float score_of(const Norm &n, float x) {
  return Softmax ? fast_exp(x - n.top) * n.inv : __builtin_amdgcn_rcpf(1.0f + fast_exp(-x));
}

template <int NJ, bool Softmax>
__device__ __forceinline__ Norm scores(const float x[NJ], float s[NJ]) {
  Norm n{0.0f, 1.0f};
  if (Softmax) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) m = fmaxf(m, x[j]);
    m = wave_max(m);
    n.top = m == -INFINITY ? 0.0f : m;
  }
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    s[j] = score_of<Softmax>(n, x[j]);
    z += s[j];
  }
  z = wave_sum(z);
  if (Softmax) {
    n.inv = z == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(z);
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] *= n.inv;
  } else {
    n.inv = __builtin_amdgcn_rcpf(z + 1e-20f);
  }
  return n;
}

__device__ __forceinline__ bool selectable(float x) { return x > -INFINITY; }  // false for NaN

constexpr float kLowest = -0x1.fffffep+127f;  // no selectable key is below it

// exp in 64 bits with few registers: x = n ln 2 + r, the series of r by
// Horner's rule from a table of 1 / k in scalar memory (|r| < 0.35: fourteen
// terms leave 1e-19), in a loop because it runs for few tokens and must not
// cost the others' registers.
__constant__ const double kInverse[15] = {0.0,       1.0,       1.0 / 2,  1.0 / 3,  1.0 / 4,  1.0 / 5,  1.0 / 6, 1.0 / 7,
                                          1.0 / 8,   1.0 / 9,   1.0 / 10, 1.0 / 11, 1.0 / 12, 1.0 / 13, 1.0 / 14};
__device__ __forceinline__ double exp64(double x) {
  if (!(x > -745.0)) return x <= -745.0 ? 0.0 : x;  // NaN stays
  if (x > 709.0) return INFINITY;
  const double n = rint(x * 0x1.71547652b82fep+0);
  const double r = fma(n, -0x1.abc9e3b39803fp-56, fma(n, -0x1.62e42fefa39efp-1, x));
  double p = 1.0;
#pragma unroll 1
  for (int k = 14; k > 0; --k) p = fma(p, r * kInverse[k], 1.0);
  return ldexp(p, (int)n);
}

// Top and sum of a softmax in 64 bits.
__device__ __forceinline__ void softmax64(const RouterArgs &a, int64_t t, int lane, double *top, double *z) {
  double m = -INFINITY, sum = 0.0;
#pragma unroll 1
  for (int e = lane; e < a.n_experts; e += 64) {
    const float x = load_logit(a, t, e);
    m = fmax(m, selectable(x) ? (double)x : -INFINITY);
  }
#pragma unroll 1
  for (int d = 32; d; d >>= 1) m = fmax(m, __shfl_xor(m, d));
#pragma unroll 1
  for (int e = lane; e < a.n_experts; e += 64) sum += exp64((double)load_logit(a, t, e) - m);
#pragma unroll 1
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  *top = m;
  *z = sum;
}

// An expert's key in 64 bits (-infinity: not selectable).
template <bool Softmax, bool Bias>
__device__ __forceinline__ double exact_key(const RouterArgs &a, int64_t t, int e, double top, double z) {
  const double x = (double)load_logit(a, t, e);
  double key = x;
  if (Bias) {
    const double y = exp64(Softmax ? x - top : -x);
    key = (Softmax ? y : 1.0) / (Softmax ? z : 1.0 + y) + (double)a.bias[e];
  }
  return x > -INFINITY && key > -INFINITY ? key : -INFINITY;
}

// Two keys closer than this may stand in the wrong order, in units of 2^-24
// of which a key carries: for the sigmoid 0.8 from the exponential (see
// fast_exp; its own last bit counts s (1 - s) <= 1/4), 1 from the sum and 2
// from v_rcp_f32; for softmax, of the score, 2 from the exponential, 1 / e from
// its argument, 24 from the sum over the experts, 2 from quotient and product;
// and 1 of the key from the sum with the bias. Twice that for a pair.
template <bool Softmax>
__device__ __forceinline__ float near_tie(float key, float score) {
  return 0x1p-23f * ((Softmax ? 0.5f + 28.0f * score : 3.8f) + fabsf(key));
}

// A wave's candidates of a selection.
struct Candidates {
  float key[64];
  float score[64];
  uint32_t expert[64];
};

// fp32 to an unsigned number of the same order, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// A place for each lane of the mask: how many lower lanes there are, plus base.
__device__ __forceinline__ int place(uint64_t who, int base) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, (uint32_t)base));
}

// Packs the experts of the lane masks to one per lane, in the order of their
// numbers.
template <int NJ>
__device__ __forceinline__ void collect(const uint64_t who[NJ], const float k[NJ], const float s[NJ], int lane,
                                        Candidates &c) {
  int base = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    if (who[j]) {
      const int at = place(who[j], base);
      if (who[j] >> lane & 1) {
        c.key[at] = k[j];
        c.score[at] = s[j];
        c.expert[at] = lane + 64 * j;
      }
      base += __popcll(who[j]);
    }
  wave_lds_fence();
}

// Ranks the wave's `count` <= 64 candidates by keys in 64 bits and leaves them
// in that order.
template <bool Softmax, bool Bias>
__device__ __forceinline__ void rank_exact(const RouterArgs &a, int64_t t, int lane, int count, Candidates &c) {
  double top = 0.0, z = 1.0;
  if (Softmax && Bias) softmax64(a, t, lane, &top, &z);
  const float s = c.score[lane];
  const uint32_t e = c.expert[lane];
  const double key = lane < count ? exact_key<Softmax, Bias>(a, t, e, top, z) : 0.0;
  int rank = lane < count ? 0 : lane;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const double other = __shfl(key, i);
    rank += lane < count && (other > key || (other == key && i < lane)) ? 1 : 0;
  }
  wave_lds_fence();
  c.score[rank] = s;
  c.expert[rank] = e;
  wave_lds_fence();
}

// Selection one expert after the other by keys in 64 bits, for a token with
// more candidates than lanes (many equal keys). Returns how many were found.
template <bool Softmax, bool Bias>
__device__ __forceinline__ int select_rounds(const RouterArgs &a, int64_t t, const Norm &n, int lane, Candidates &c) {
  double top = 0.0, z = 1.0, last = INFINITY;
  if (Softmax && Bias) softmax64(a, t, lane, &top, &z);
  int count = 0, last_e = -1;
  for (; count < a.top_k; ++count) {
    // the greatest key behind the last one taken, and of equals the lowest expert
    double best = -INFINITY;
    int at = kMaxExperts;
#pragma unroll 1
    for (int e = lane; e < a.n_experts; e += 64) {
      const double k = exact_key<Softmax, Bias>(a, t, e, top, z);
      if ((k < last || (k == last && e > last_e)) && k > best) best = k, at = e;
    }
#pragma unroll 1
    for (int d = 32; d; d >>= 1) {
      const double ob = __shfl_xor(best, d);
      const int oa = __shfl_xor(at, d);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if (at >= kMaxExperts) break;
    if (lane == 0) {
      c.expert[count] = at;
      c.score[count] = score_of<Softmax>(n, load_logit(a, t, at));
    }
    last = best;
    last_e = at;
  }
  wave_lds_fence();
  return count;
}

// Selection: lane r < top_k receives the r-th expert (-1: none left) and its
// score.
//
// A threshold is sought that at least top_k + 1 of the 64 lanes' greatest keys
// reach, and few more: nine halvings of the two octaves below the greatest
// (a compare and a count of a lane mask each). The experts whose keys reach
// it, at most 64, are packed to one per lane in the order of their numbers,
// and each counts the greater keys: its rank (equal keys, seen when two lanes
// claim a rank, are counted apart by lane). With the scores that is most of a
// token's 273 vector instructions (384 experts); taking the greatest key top_k
// times needs 35 each time.
//
// With a bias the keys carry roundings. Where two neighbours of the first
// top_k + 1 (or of a run of equals across that border and the next behind it)
// are too close and not of the same logit and bias, all experts within reach
// of the last place are ranked by keys in 64 bits. More than 64 candidates
// (many equal keys) are selected one after the other.
template <int NJ, bool Softmax, bool Bias>
__device__ __forceinline__ void select_topk(const RouterArgs &a, int64_t t, const Norm &norm, const float x[NJ],
                                            const float s[NJ], const float b[NJ], int lane, Candidates &c, int *index,
                                            float *score) {
  float k[NJ], h = -INFINITY;  // a key that is NaN reaches no threshold
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    k[j] = Bias ? (x[j] == -INFINITY ? -INFINITY : s[j] + b[j]) : x[j];
    h = fmaxf(h, k[j]);
  }
  const uint32_t u = h > -INFINITY ? ordered(h) : 0u, top = wave_max_u32(u);
  *index = -1;
  *score = 0.0f;
  if (top == 0) return;
  const int need = a.top_k + 1;
  // keys down to a quarter of the greatest, or all there are
  constexpr uint32_t kSpan = 0x01000000u;
  uint32_t lo = top > kSpan ? top - kSpan : 1u, step;  // lo + step stays below 2^32
  if (__popcll(__ballot(u >= lo)) >= need) {
#pragma unroll
    for (step = kSpan / 2; step > kSpan >> 10; step >>= 1) lo += __popcll(__ballot(u >= lo + step)) >= need ? step : 0u;
  } else {
    lo = 1u;
    for (step = 0x80000000u; step > kSpan >> 10; step >>= 1) lo += __popcll(__ballot(u >= lo + step)) >= need ? step : 0u;
  }
  // keys that lie close together take more steps
  while (__popcll(__ballot(u >= lo)) > need + 8 && step) {
    lo += __popcll(__ballot(u >= lo + step)) >= need ? step : 0u;
    step >>= 1;
  }
  // 0x00800000 is the number of the lowest fp32 value, which every key reaches; the numbers below it are those of
  // -infinity and of NaNs, which no key would
  const bool all = lo <= 0x00800000u;
  const float least = all ? kLowest : from_ordered(lo);
  uint64_t who[NJ];
  int count = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    who[j] = __ballot(k[j] >= least);
    count += __popcll(who[j]);
  }
  float reach = least;
  bool decided = count <= 64;
  if (decided) {
    collect<NJ>(who, k, s, lane, c);
    const bool mine = lane < count;  // this lane holds a candidate
    const float key = mine ? c.key[lane] : -INFINITY;
    float sc = c.score[lane];
    uint32_t ex = c.expert[lane];
    int rank = 0;
    for (int i = 0; i < count; i += 4) {  // lanes from count on hold -infinity
      rank += lane_value(key, i) > key ? 1 : 0;
      rank += lane_value(key, i + 1) > key ? 1 : 0;
      rank += lane_value(key, i + 2) > key ? 1 : 0;
      rank += lane_value(key, i + 3) > key ? 1 : 0;
    }
    rank = mine ? rank : lane;  // lanes without a candidate stay behind them
    wave_lds_fence();
    c.expert[rank] = lane;
    wave_lds_fence();
    if (__ballot(c.expert[rank] != (uint32_t)lane)) {  // equal keys: by lane
      for (int i = 0; i < count; i += 4) {
        rank += lane_value(key, i) == key && lane > i && mine ? 1 : 0;
        rank += lane_value(key, i + 1) == key && lane > i + 1 && mine ? 1 : 0;
        rank += lane_value(key, i + 2) == key && lane > i + 2 && mine ? 1 : 0;
        rank += lane_value(key, i + 3) == key && lane > i + 3 && mine ? 1 : 0;
      }
    }
    wave_lds_fence();
    c.key[rank] = key;
    c.score[rank] = sc;
    c.expert[rank] = ex;
    wave_lds_fence();
    if (Bias) {
      // lane r against r + 1; the greatest score of a candidate bounds the pair's
      const bool pair = lane + 1 < count;
      const float k0 = c.key[lane], k1 = c.key[(lane + 1) & 63];
      const float most = Softmax ? wave_max(mine ? sc : 0.0f) : 0.0f;
      const uint64_t close = __ballot(pair && k0 - k1 <= near_tie<Softmax>(k0, most));
      if (close & ((2ull << (a.top_k - 1)) - 1)) {
        const uint32_t er = c.expert[lane];
        const float xe = mine ? load_logit(a, t, er) : 0.0f, be = mine ? a.bias[er] : 0.0f;
        const uint64_t same = __ballot(pair && xe == __shfl_down(xe, 1) && be == __shfl_down(be, 1));
        const int border = a.top_k - 1 + __builtin_ctzll(~(same >> (a.top_k - 1)));  // first unlike pair from there on
        const bool open = border + 1 < count ? (close >> border) & 1 : count > a.top_k && !all;
        decided = !open && !(close & ~same & ((1ull << (a.top_k - 1)) - 1));
        // everything within reach of the last place. The difference may pass the lowest fp32 value: experts that are
        // switched off, and columns behind the last expert, have the key -infinity and must not come within reach.
        if (count > a.top_k) {
          const float last = lane_value(k0, a.top_k - 1);
          reach = fmaxf(fminf(least, last - near_tie<Softmax>(last, Softmax ? 1.0f : 0.0f)), kLowest);
        }
      }
    }
  }
  if (!decided) {
    count = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      who[j] = __ballot(k[j] >= reach);
      count += __popcll(who[j]);
    }
    wave_lds_fence();
    if (count <= 64) {
      collect<NJ>(who, k, s, lane, c);
      rank_exact<Softmax, Bias>(a, t, lane, count, c);
    } else {
      count = select_rounds<Softmax, Bias>(a, t, norm, lane, c);
    }
  }
  if (lane < a.top_k && lane < count) {
    *index = (int)c.expert[lane];
    *score = c.score[lane];
  }
  wave_lds_fence();
}

struct ForwardOut {
  int32_t *index;
  float *weight;
  float *part_p;    // [tile + sequence][expert]: sums of probabilities
  int32_t *part_c;  // and selections of the tokens that the two share
};

// What a token's selection leaves: its row of both outputs and its counts.
__device__ __forceinline__ void put_token(const RouterArgs &a, const ForwardOut &o, int32_t t, int lane, int index,
                                          float score, int *cnt) {
  float w = score;
  if (a.normalize) w *= __builtin_amdgcn_rcpf(wave_sum(w) + 1e-20f);
  if (index >= 0) atomicAdd(&cnt[index], 1);
  if (lane < a.top_k) {
    o.index[(int64_t)t * a.top_k + lane] = index;
    o.weight[(int64_t)t * a.top_k + lane] = index >= 0 ? w * a.scale : 0.0f;  // a NaN sum reaches experts alone
  }
}

// Forward pass over tokens, a wave to a token, its next row's loads ahead of
// it. A workgroup's tile of tokens is cut at the sequences' borders, and the
// tokens that tile i shares with sequence q leave their sums at row i + q:
// along the tokens each step to the next pair raises i or q, so no two pairs
// share a row, no sum needs an atomic, and the order of every sum is fixed.
// Probabilities are added in fp32 over the at most 8 tokens of a wave and the
// eight waves, which keeps a sum within 15 roundings; sums of tiles are in fp64.
//
// The runs of a tile are worked on one after the other, with three barriers
// each, so a batch of very short sequences takes longer: 256 tokens x 200 in 1 /
// 8 / 64 / 256 sequences 8.5 / 11.7 / 16.8 / 29.2 us (replayed from a graph),
// 2048 x 384 in 1 / 13 / 64 / 1024 of them 11.8 / 14.0 / 16.2 / 62 us, 16384 x
// 384 in 13 / 64 / 1024 / 4096 of them 22.9 / 25.3 / 70.8 / 202 us.
//
// Up to 384 experts six waves fit a SIMD (80 registers) instead of four, which
// 16384 tokens do not need (one time with both) and longer batches do, compared
// in one run: 24000 x 384 26.7 against 30.7 us, 65536 x 384 48.5 against 52.2.
// Softmax scores with a bias would spill registers for it; beyond 384 experts it
// has not been tried (16384 x 512 24.6 us, without it).
template <int NJ, bool Softmax, bool Bias>
__global__ void __launch_bounds__(64 * kWaves, NJ > 6 || (Softmax && Bias) ? 1 : 6) router_forward_kernel(RouterArgs a, ForwardOut o) {
  constexpr int W = kWaves, Threads = 64 * W;
  __shared__ float sum[W][64 * NJ];
  __shared__ int cnt[64 * NJ];
  __shared__ Candidates cand[W];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int32_t first = blockIdx.x * a.tile;
  const int32_t last = a.n_tokens - first < a.tile ? a.n_tokens : first + a.tile;
  int32_t t = first + wave;  // this wave's next token
  uint32_t ahead[NJ];
  float b[NJ];
  if (t < last) load_row<NJ>(a, t, lane, ahead);
#pragma unroll
  for (int j = 0; j < NJ; ++j) b[j] = Bias ? a.bias[min(lane + 64 * j, a.n_experts - 1)] : 0.0f;
  Runs runs(a, first, last);
  int32_t lo, hi, q;
  while (runs.next(a, &lo, &hi, &q)) {
    if (q < 0) {
      for (int64_t i = (int64_t)lo * a.top_k + threadIdx.x; i < (int64_t)hi * a.top_k; i += Threads) {
        o.index[i] = -1;
        o.weight[i] = 0.0f;
      }
      while (t < hi) t += W;
      if (t < last) load_row<NJ>(a, t, lane, ahead);
      continue;
    }
    for (int e = threadIdx.x; e < a.n_experts; e += Threads) cnt[e] = 0;
    __syncthreads();
    float acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = 0.0f;
    for (; t < hi; t += W) {
      float x[NJ], s[NJ], w;
      int index;
      logits_of<NJ>(a, lane, ahead, x);
      if (t + W < last) load_row<NJ>(a, t + W, lane, ahead);
      const Norm n = scores<NJ, Softmax>(x, s);
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[j] += Softmax ? s[j] : s[j] * n.inv;
      select_topk<NJ, Softmax, Bias>(a, t, n, x, s, b, lane, cand[wave], &index, &w);
      put_token(a, o, t, lane, index, w, cnt);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) sum[wave][lane + 64 * j] = acc[j];
    __syncthreads();
    const int64_t row = ((int64_t)blockIdx.x + q) * a.n_experts;
    for (int e = threadIdx.x; e < a.n_experts; e += Threads) {
      float p = sum[0][e];
#pragma unroll
      for (int i = 1; i < W; ++i) p += sum[i][e];
      o.part_p[row + e] = p;
      o.part_c[row + e] = cnt[e];
    }
    __syncthreads();
  }
}

constexpr int kThreads = 256;  // of the reductions
constexpr int kChunk = 16;     // experts of one of their workgroups

// Per sequence and 16 experts: the tiles' partial sums, the counts, and these
// experts' part of the loss.
__global__ void __launch_bounds__(kThreads)
    router_reduce_kernel(RouterArgs a, const float *part_p, const int32_t *part_c, int32_t *seq_counts,
                         double *part_loss) {
  __shared__ double sp[kThreads];
  __shared__ int sc[kThreads];
  const int32_t q = blockIdx.x, e = blockIdx.y * kChunk + (threadIdx.x & 15), row = threadIdx.x >> 4;
  const int32_t lo = seq_start(a, q), hi = seq_start(a, q + 1);
  double p = 0.0;
  int c = 0;
  if (hi > lo && e < a.n_experts) {
    const int32_t last = (hi - 1) / a.tile;
#pragma unroll 4
    for (int32_t i = lo / a.tile + row; i <= last; i += kThreads / kChunk) {
      const int64_t at = ((int64_t)i + q) * a.n_experts + e;
      p += (double)part_p[at];
      c += part_c[at];
    }
  }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = c;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  double part = 0.0;
  if (threadIdx.x < kChunk && e < a.n_experts) {
    p = 0.0;
    c = 0;
#pragma unroll
    for (int i = 0; i < kThreads / kChunk; ++i) {
      p += sp[kChunk * i + threadIdx.x];
      c += sc[kChunk * i + threadIdx.x];
    }
    seq_counts[(int64_t)q * a.n_experts + e] = c;
    const double n = hi > lo ? (double)(hi - lo) : 1.0;
    part = (double)c * p / (n * n);
  }
  for (int d = 8; d; d >>= 1) part += __shfl_xor(part, d);
  if (threadIdx.x == 0) part_loss[(int64_t)q * gridDim.y + blockIdx.y] = part;
}

__device__ __forceinline__ float loss_of(const RouterArgs &a, double s) {
  return (float)(s * (double)a.coef * (double)a.n_experts / ((double)a.top_k * (double)a.n_seqs));
}

// Block 0: the loss from its parts. The others: counts over all sequences of
// 16 experts each.
__global__ void __launch_bounds__(kThreads)
    router_finish_kernel(RouterArgs a, const int32_t *seq_counts, const double *part_loss, int64_t n_parts,
                         int32_t *counts, float *loss) {
  __shared__ double sp[kThreads / 64];
  __shared__ int sc[kThreads];
  if (blockIdx.x == 0) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n_parts; i += kThreads) s += part_loss[i];
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) sp[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) *loss = loss_of(a, (sp[0] + sp[1]) + (sp[2] + sp[3]));
    return;
  }
  const int32_t e = (blockIdx.x - 1) * kChunk + (threadIdx.x & 15);
  int c = 0;
  if (e < a.n_experts)
    for (int32_t q = threadIdx.x >> 4; q < a.n_seqs; q += kThreads / kChunk) c += seq_counts[(int64_t)q * a.n_experts + e];
  sc[threadIdx.x] = c;
  __syncthreads();
  if (threadIdx.x < kChunk && e < a.n_experts) {
    c = 0;
    for (int i = 0; i < kThreads / kChunk; ++i) c += sc[kChunk * i + threadIdx.x];
    counts[e] = c;
  }
}

// Both reductions of one sequence in one workgroup, for few partial sums (a
// second launch would cost more than the reads one after the other).
constexpr int kSmallThreads = 1024;
__global__ void __launch_bounds__(kSmallThreads)
    router_small_kernel(RouterArgs a, const float *part_p, const int32_t *part_c, int32_t *seq_counts,
                        int32_t *counts, float *loss) {
  __shared__ double sp[kSmallThreads];
  __shared__ int sc[kSmallThreads];
  const int E = a.n_experts, rows = kSmallThreads / E, e = threadIdx.x % E, row = threadIdx.x / E;
  const int32_t lo = seq_start(a, 0), hi = seq_start(a, 1);
  double p = 0.0, total = 0.0;
  int c = 0;
  if (hi > lo && row < rows) {
    const int32_t last = (hi - 1) / a.tile;
#pragma unroll 4
    for (int32_t i = lo / a.tile + row; i <= last; i += rows) {
      const int64_t at = (int64_t)i * E + e;
      p += (double)part_p[at];
      c += part_c[at];
    }
  }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = c;
  __syncthreads();
  if (row == 0) {
    for (int i = 1; i < rows; ++i) {
      p += sp[i * E + e];
      c += sc[i * E + e];
    }
    seq_counts[e] = c;
    if (counts) counts[e] = c;
    const double n = hi > lo ? (double)(hi - lo) : 1.0;
    total = (double)c * p / (n * n);
  }
  __syncthreads();
  for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
  if ((threadIdx.x & 63) == 0) sp[threadIdx.x >> 6] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kSmallThreads / 64; ++i) total += sp[i];
    *loss = loss_of(a, total);
  }
}

struct BackwardIo {
  const int32_t *index;
  const int32_t *seq_counts;
  const float *dweight;
  const float *dloss;
  uint64_t dlogits;
  int64_t dstride;
};

template <int NJ>
__device__ __forceinline__ void store_row(const RouterArgs &a, const BackwardIo &o, int64_t t, uint32_t lane,
                                          const float x[NJ]) {
  const auto row = row_buffer(row_of(o.dlogits, t, o.dstride, a.bf16), a.n_experts, a.bf16);
  if (a.bf16) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)x[j]), row, 2 * lane + 128 * j, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[j]), row, 4 * lane + 256 * j, 0, 0);
  }
}

// Backward pass, a wave to a token, scores recomputed from the logits (which
// have to be read anyway). Of the loss, d/dp_e is the same for all tokens of a
// sequence and stays in registers; of the weights, the top_k values meet their
// experts' lanes in the wave's row of shared memory: first the scores lie
// there for the selected to be picked up, then the selected's gradients. An
// expert in several places adds up by one atomic instruction of one wave, whose
// lanes shared memory takes in their order (a test holds it to that).
constexpr int kBackWaves = 4;
template <int NJ, bool Softmax>
__global__ void __launch_bounds__(64 * kBackWaves) router_backward_kernel(RouterArgs a, BackwardIo o) {
  constexpr int W = kBackWaves;
  __shared__ float rows[W][64 * NJ];
  const int lane = threadIdx.x & 63, wave = wave_id();
  float *row = rows[wave];
  const int32_t first = blockIdx.x * a.tile;
  const int32_t last = a.n_tokens - first < a.tile ? a.n_tokens : first + a.tile;
  int32_t t = first + wave;
  if (t >= last) return;
  const bool chosen = o.dweight && lane < a.top_k;  // this lane carries a selected expert
  uint32_t ahead[NJ];
  float dw = 0.0f;
  int at = -1;
  load_row<NJ>(a, t, lane, ahead);
  if (chosen) {
    at = o.index[(int64_t)t * a.top_k + lane];
    dw = o.dweight[(int64_t)t * a.top_k + lane];
  }
  const float dloss = o.dloss ? *o.dloss : 0.0f;
  int32_t q = seq_of(a, t), start = 0, stop = -1;  // [start, stop): of sequence q, or the padding before or behind
  bool padding = false;
  float b[NJ];
  for (; t < last; t += W) {
    if (t >= stop) {
      start = stop = a.n_tokens;
      for (; q < a.n_seqs; ++q) {
        start = seq_start(a, q);
        stop = seq_start(a, q + 1);
        if (stop > t) break;
      }
      padding = q >= a.n_seqs || start > t;
      if (padding) stop = q < a.n_seqs ? start : a.n_tokens;
#pragma unroll
      for (int j = 0; j < NJ; ++j) b[j] = 0.0f;
      if (!padding && o.dloss) {
        const float n = (float)(stop - start);
        const float f = dloss * a.coef * (float)a.n_experts / ((float)a.n_seqs * (float)a.top_k) / n / n;
        const int32_t *c = o.seq_counts + (int64_t)q * a.n_experts;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          b[j] = f * (float)c[min(lane + 64 * j, a.n_experts - 1)];
      }
    }
    float x[NJ], s[NJ], g[NJ];
    logits_of<NJ>(a, lane, ahead, x);
    const int sel = at >= 0 && at < a.n_experts ? at : -1;
    float d = sel >= 0 ? dw * a.scale : 0.0f;
    if (t + W < last) {
      load_row<NJ>(a, t + W, lane, ahead);
      if (chosen) {
        at = o.index[(int64_t)(t + W) * a.top_k + lane];
        dw = o.dweight[(int64_t)(t + W) * a.top_k + lane];
      }
    }
    if (padding) {
      store_row<NJ>(a, o, t, lane, b);  // zeros
      continue;
    }
    const Norm n = scores<NJ, Softmax>(x, s);
    if (!Softmax) {
      // x becomes the sigmoid's slope s (1 - s). 1 - s is exp(-x) s: a difference would have no digits left for a
      // confident expert, whose 1 - s is small. An exponential that is infinite meets a score of 0.
#pragma unroll
      for (int j = 0; j < NJ; ++j) x[j] = s[j] * (s[j] * fminf(fast_exp(-x[j]), 0x1.fffffep+127f));
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) g[j] = 0.0f;
    if (o.dweight) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) row[lane + 64 * j] = s[j];
      wave_lds_fence();
      const float ss = sel >= 0 ? row[sel] : 0.0f;
      wave_lds_fence();
#pragma unroll
      for (int j = 0; j < NJ; ++j) row[lane + 64 * j] = 0.0f;
      if (a.normalize) {
        // with z = sum + 1e-20, d_j - sum(d s) / z = c_j - sum(c s) / z + d_0 1e-20 / z for c = d - d_0: what all
        // of a token's gradients share cancels before it is rounded (entirely, if one expert is selected)
        const float r = __builtin_amdgcn_rcpf(wave_sum(ss) + 1e-20f), d0 = lane_value(d, 0), c = d - d0;
        const float cs = wave_sum(c * ss);
        if (sel >= 0) d = (c - cs * r + d0 * (1e-20f * r)) * r;
      }
      wave_lds_fence();
      if (sel >= 0) atomicAdd(&row[sel], d);
      wave_lds_fence();
#pragma unroll
      for (int j = 0; j < NJ; ++j) g[j] = row[lane + 64 * j];
      wave_lds_fence();
    }
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) dot += (Softmax ? b[j] + g[j] : b[j]) * s[j];
    dot = wave_sum(dot);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      g[j] = Softmax ? s[j] * (b[j] + g[j] - dot)
                       : ((b[j] - dot * n.inv) * n.inv + g[j]) * x[j];
    store_row<NJ>(a, o, t, lane, g);
  }
}

// Tokens of one workgroup. More of them leave fewer partial sums, fewer fill
// the card with fewer tokens. Measured on MI355X, forward with 4, 8 and 16
// waves to a workgroup and 1, 2, 4 tokens to a wave: 16384 x 384 31.3 / 26.6 /
// 24.4, 30.7 / 25.9 / 23.3 and - / 26.6 / 24.2 us, 5003 x 160 17.5 / 15.5 /
// 16.5, 14.8 / 14.3 / 20.5 and 15.6 / - / 21.2 us; few tokens with 1 and 2 to
// each of 8 waves: 64 x 384 8.8 / 10.4 us, 128 x 384 9.3 / 10.6, 512 x 384 9.5 /
// 11.5, 2048 x 160 11.6 / 12.9, 4096 x 384 15.4 / 14.8, 8192 x 384 21.8 / 17.8; backward (4 waves) of the
// first 14.6 / 12.5 / 11.8 us, of the second 7.6 / 7.6 / 7.6 us.
int32_t tile_of(int64_t n_tokens) {
  return n_tokens <= 2048 ? 8 : n_tokens <= 8192 ? 16 : n_tokens <= 32768 ? 32 : 64;
}
int32_t back_tile_of(int64_t n_tokens) { return n_tokens <= 8192 ? 4 : 16; }

// Partial sums of one sequence up to which one workgroup reduces them. Measured
// on MI355X, the whole forward pass of 384 experts with one workgroup / with two
// launches: 1 token 7.5 / 8.9 us, 64 tokens (3,456 sums) 8.7 / 9.4, 192 tokens
// (9,600) 9.7 / 9.8, 256 tokens (12,672) 10.1 / 9.7. With several sequences, one
// after the other in that workgroup: 128 tokens in 2 of them 10.1 / 9.4 us, in 8
// (160 experts) 15.1 / 8.5.
constexpr int64_t kSmallSums = 8192;

int chunks_of(int n_experts) { return (n_experts + kChunk - 1) / kChunk; }

struct Workspace {
  int64_t rows, part_p, part_c, part_loss, bytes;
};

Workspace workspace_of(const wt_router_desc &d) {
  const int64_t tile = tile_of(d.n_tokens);
  const int64_t rows = (d.n_tokens + tile - 1) / tile + d.n_seqs;
  Workspace w;
  w.rows = rows;
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
  if (d->n_tokens < 0 || d->n_tokens > kMaxTokens || d->n_tokens * d->top_k >= (int64_t)1 << 31)
    return fail(what, "n_tokens out of range");
  if (d->logits_dtype != WT_DT_F32 && d->logits_dtype != WT_DT_BF16) return fail(what, "unknown logits type");
  if (d->score != WT_SCORE_SIGMOID && d->score != WT_SCORE_SOFTMAX) return fail(what, "unknown score");
  if (d->normalize != 0 && d->normalize != 1) return fail(what, "normalize must be 0 or 1");
  if (!std::isfinite(d->scale) || !std::isfinite(d->balance_coef)) return fail(what, "scale or balance_coef not finite");
  if (d->n_seqs < 1 || d->n_seqs > (1 << 20)) return fail(what, "n_seqs out of range");
  if (!d->seq_offsets && d->n_seqs != 1) return fail(what, "several sequences without seq_offsets");
  return WT_OK;
}

// Row strides whose last row still has a 64-bit byte offset.
int64_t max_stride(int64_t n_tokens) { return ((int64_t)1 << 60) / (n_tokens > 1 ? n_tokens : 1); }

wt_status check_memory_args(const char *what, const wt_router_desc *d) {
  const int64_t size = d->logits_dtype == WT_DT_BF16 ? 2 : 4;
  if (d->logits_stride < d->n_experts || d->logits_stride > max_stride(d->n_tokens))
    return fail(what, "logits_stride out of range");
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

// Calls f with the number of 64-expert columns as a constant, the next one that
// there is: 257 to 384 experts cost the same, and 513 to 1024. 16384 tokens over
// 256 / 320 / 384 / 512 / 640 / 1024 experts, forward 21 / 22.8 / 23.0 / 24.6 /
// 40.4 / 42.4 us, backward 10.6 / 12.0 / 12.3 / 14.6 / 21 / 27.7 us.
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
  try {
    const wt_status st = check_desc(what, desc);
    if (st != WT_OK) return st;
    if (!bytes) return fail(what, "NULL result");
    *bytes = (size_t)workspace_of(*desc).bytes;
    return WT_OK;
  } catch (...) {
    return caught_status();
  }
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
        constexpr int N = decltype(nj)::value;
        const auto kernel = a.softmax ? (a.bias ? router_forward_kernel<N, true, true> : router_forward_kernel<N, true, false>)
                                      : (a.bias ? router_forward_kernel<N, false, true> : router_forward_kernel<N, false, false>);
        hipLaunchKernelGGL(kernel, dim3(tiles), dim3(64 * kWaves), 0, s, a,
                           ForwardOut{index, weight, part_p, part_c});
      });
    if (a.n_seqs == 1 && w.rows * a.n_experts <= kSmallSums) {
      hipLaunchKernelGGL(router_small_kernel, dim3(1), dim3(kSmallThreads), 0, s, a, part_p, part_c, seq_counts, counts,
                         loss);
    } else {
      hipLaunchKernelGGL(router_reduce_kernel, dim3((uint32_t)a.n_seqs, chunks), dim3(kThreads), 0, s, a, part_p,
                         part_c, seq_counts, part_loss);
      hipLaunchKernelGGL(router_finish_kernel, dim3(counts ? 1 + chunks : 1), dim3(kThreads), 0, s, a, seq_counts,
                         part_loss, (int64_t)a.n_seqs * chunks, counts, loss);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(what, hip_msg("launch", e), WT_E_HIP);
    return WT_OK;
  } catch (...) {
    return caught_status();
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
    if (dlogits_stride < desc->n_experts || dlogits_stride > max_stride(desc->n_tokens))
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
    RouterArgs a = args_of(*desc);
    a.tile = back_tile_of(a.n_tokens);
    const uint32_t tiles = (uint32_t)((a.n_tokens + a.tile - 1) / a.tile);
    const BackwardIo io{index, seq_counts, dweight, dloss, (uint64_t)(uintptr_t)dlogits, dlogits_stride};
    with_columns(a.n_experts, [&](auto nj) {
      constexpr int N = decltype(nj)::value;
      const auto kernel = a.softmax ? router_backward_kernel<N, true> : router_backward_kernel<N, false>;
      hipLaunchKernelGGL(kernel, dim3(tiles), dim3(64 * kBackWaves), 0, (hipStream_t)stream, a, io);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(what, hip_msg("launch", e), WT_E_HIP);
    return WT_OK;
  } catch (...) {
    return caught_status();
  }
}

}  // extern "C"
