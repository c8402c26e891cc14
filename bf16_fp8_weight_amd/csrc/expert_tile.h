// expert_tile.h -- device code of the experts' products: the tile of a workgroup,
// its operands' way through shared memory, the matrix instructions and what is
// done with the sums. The definitions are in wt.h.
//
// A workgroup of WM x WN waves computes BM x BN results. Both operands pass
// through shared memory in steps of 64 Sub bytes along the sum (32 BF16 elements or
// 128 MXFP4 codes each), in 16-byte chunks:
//   - an operand whose rows run along the sum (a and b of NT, a of NN) as its rows
//     of 4 Sub chunks, chunk c of row r at slot c ^ swizzle_along(r), so that what is read
//     in one cycle lies in different banks;
//   - one whose rows run across it (b of NN, a and b of TN) as it comes, 32 Sub rows of
//     BM or BN elements, read back transposed (ds_read_b64_tr_b16: a 16-lane group
//     fetches 4 rows x 16 columns, each lane receiving a column); there chunk c
//     of row k lies at slot c ^ swizzle(k), because those 4 rows would share banks.
// The matrix instructions take b's tile as their first operand: a lane then holds four
// neighbouring columns of one row of out. BF16 takes 16 x 16 x 32; 32 x 32 x 16 were
// slower in the whole kernel (8192 x 8192 x 8192: 1240 to 1270 TFLOP/s against 1330 to
// 1350). MXFP4 takes 32 x 32 x 64, which reach 8.8 PFLOP/s over registers alone (7.0 on
// random values, under the power limit) where 16 x 16 x 128 reach 6.3 (5.7).
//
// product_kernel (aligned operands) is bound by the matrix units where there are tiles for
// every CU, and there by power: matrix instructions alone, from registers, reach 1.61 PFLOP/s on
// random BF16 values. 8192 x 8192 x 8192, from card to card: NT 1312 to 1375 TFLOP/s, NN 1354 to 1426, TN 1355 to 1433 (matrix units busy
// 75 % of the time), MXFP4 3600 to 3740 (50 %; its 256 x 256 tiles spill 4 and 5 registers, reloaded in the first copies and the last steps).
// With few rows it is bound by the weights' bytes (those of the experts that have rows at 5.1 to 6.2 TB/s), with few of both
// by the chain of steps. product_any_kernel (any stride) is bound by loads that
// straddle cache lines: 2001 rows, 4001 x 777, NT 49 us, NN 68; 8001 rows, 4097 x 4097, 433 us (620 TFLOP/s).
#pragma once

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "expert.h"

namespace wt {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Calls f with the integral constants 0 .. N - 1.
template <class F, int... I>
__device__ __forceinline__ void static_calls(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F f) {
  static_calls(f, std::make_integer_sequence<int, N>());
}

enum Form { kNT = WT_PRODUCT_NT, kNN = WT_PRODUCT_NN, kTN = WT_PRODUCT_TN };

// MXFP4: a row's scales are copied for 512 codes at a time. Those of 128, a word to
// a row, made as many requests as the operands (8192 x 8192 x 8192 360 us).
constexpr int kScaleRow = 16;

// ------------------------------------------------------------- activations
// Both are x s(y) with s(y) = 1 / (1 + exp(-y)): SiLU y = x; GELU's
// (1 + tanh(z)) / 2 = s(2 z). With t = exp(-|y|) both s and 1 - s are t / (1 + t) or
// 1 / (1 + t), without a difference that cancels or an exponential that overflows. t is taken as the square of h =
// exp(-|y| / 2), and x and the slope's factor meet one h before the other: below y = -87.3 t leaves the normal numbers
// (exp2 gives 0 for those), while x s still is one of BF16's, down to 2^-133.
// exp2 and the reciprocal are good to a last place of fp32 and exp2's argument to
// 2^-22 |y|, far below the BF16 result's 2^-8.
struct Act {
  float value, slope, scale;  // the activation is value scale, its slope is slope scale
};

__device__ __forceinline__ Act activation(int act, float x) {
  constexpr float kLog2e = 1.44269504f, kC = 1.59576912f;  // 2 sqrt(2 / pi)
  float y = x, dy = 1.0f;
  if (act == WT_ACT_GELU) {
    const float x2 = x * x;
    y = kC * x * (1.0f + 0.044715f * x2);
    dy = kC * (1.0f + 3.0f * 0.044715f * x2);
  }
  const float h = __builtin_amdgcn_exp2f(-0.5f * kLog2e * fabsf(y)), t = h * h, r = __builtin_amdgcn_rcpf(1.0f + t);
  // s = p (p r) and 1 - s; a NaN is in all of them
  const float p = y >= 0.0f ? 1.0f : h, rest = y >= 0.0f ? t * r : r;
  Act f;
  f.scale = p * r;
  // -FLT_MAX times a logistic of 0 is the limit 0, where -infinity would make a NaN
  f.value = fmaxf(x, -FLT_MAX) * p;
  // s (1 + (1 - s) x dy); where x dy passes these limits, t is 0, and with it 1 - s or p
  f.slope = (1.0f + rest * __builtin_amdgcn_fmed3f(x * dy, -1e13f, 1e13f)) * p;
  return f;
}

// ------------------------------------------------------- which tile is whose
struct Rows {
  int expert;
  int64_t first;  // of the row space
  int count;
};

// An expert's rows, cut to the row space.
__device__ __forceinline__ void expert_rows(const ProductArgs &a, int e, int &first, int &count) {
  const int n_rows = (int)a.n_rows;
  if (!a.offsets) {
    first = 0;
    count = n_rows;
    return;
  }
  const int lo = a.offsets[e];
  // offsets may be any two numbers: their difference has 33 bits
  const int64_t n = a.counts ? a.counts[e] : (int64_t)a.offsets[e + 1] - lo;
  first = min(max(lo, 0), n_rows);
  // a first row below 0 takes its part of the count along
  const int64_t end = lo + max(n, (int64_t)0);
  count = (int)max((int64_t)0, min(end, (int64_t)n_rows) - first);
}

template <int Ctrl, int RowMask>
__device__ __forceinline__ uint32_t dpp_add(uint32_t x) {
  return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, Ctrl, RowMask, 0xF, false);
}
// Sums of a lane's value and those of the lanes before it, over the wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x = dpp_add<0x111, 0xF>(x);  // row_shr:1, 2, 4, 8: within 16 lanes
  x = dpp_add<0x112, 0xF>(x);
  x = dpp_add<0x114, 0xF>(x);
  x = dpp_add<0x118, 0xF>(x);
  x = dpp_add<0x142, 0xA>(x);  // rows 1 and 3 take in the last lane of rows 0 and 2
  return dpp_add<0x143, 0xC>(x);  // rows 2 and 3 that of row 1
}
__device__ __forceinline__ uint32_t last_lane(uint32_t x) { return (uint32_t)__builtin_amdgcn_readlane((int)x, 63); }

// Workgroups go round the 8 XCDs, each with an L2 of its own: tiles are dealt so that
// an XCD's are neighbours. Up to kRowGroup row tiles take turns under one
// column tile, so that what the XCD's 32 CUs read at a time are few rows of both operands.
constexpr int kRowGroup = 8;

// Place u among m_tiles x n_tiles tiles.
__device__ __forceinline__ void place_tile(uint32_t u, uint32_t m_tiles, uint32_t n_tiles, int &mt, int &nt) {
  const uint32_t group = u / (kRowGroup * n_tiles), in = u - group * kRowGroup * n_tiles;
  const uint32_t height = min(m_tiles - group * kRowGroup, (uint32_t)kRowGroup);
  nt = (int)(in / height);
  mt = (int)(group * kRowGroup + in - (uint32_t)nt * height);
}

// The lane (of the first n, at most 64) whose value comes at place `order` when they are sorted from the largest down.
__device__ __forceinline__ int lane_in_order(int value, int n, int order) {
  const int lane = threadIdx.x & 63;
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const int v = __builtin_amdgcn_readlane(value, i);
    rank += v > value || (v == value && i < lane);
  }
  return __builtin_ctzll(__ballot(lane < n && rank == order));
}

// The tile of a workgroup, or false if there are not that many. Each XCD gets an eighth of all experts' tiles. With
// a.rests_last the tiles that hold the rest of an expert's rows come behind all others, the largest first (up to 64 experts):
// they take less time (products of rows that are not there are left out), so they fill up the last round.
template <int BM>
__device__ __forceinline__ bool find_rows(const ProductArgs &a, uint32_t block, uint32_t n_tiles, Rows &r, int &mt, int &nt) {
  const int lane = threadIdx.x & 63, E = a.n_experts;
  int first = 0, count = 0;
  uint32_t mine = 0, scan = 0, all = 0, all_rests = 0;
  auto look = [&](int base) {
    first = count = 0;
    if (base + lane < E) expert_rows(a, base + lane, first, count);
    mine = (uint32_t)(count + (a.rests_last ? 0 : BM - 1)) / BM;
  };
  for (int base = 0; base < E; base += 64) {
    look(base);
    scan = wave_scan(mine);
    all += last_lane(scan);
    if (a.rests_last) all_rests += (uint32_t)__popcll(__ballot((uint32_t)count % BM != 0));
  }
  const uint64_t tiles = (uint64_t)all * n_tiles, per = (tiles + kXcds - 1) / kXcds;
  uint64_t t = (uint64_t)(block % kXcds) * per + block / kXcds;
  const bool rest = block / kXcds >= per;
  if (rest) {
    t = block - per * kXcds;  // dealt one by one
    if (t >= (uint64_t)all_rests * n_tiles) return false;
  } else if (t >= tiles) {
    return false;
  }
  uint32_t at = (uint32_t)(t / n_tiles), before = 0;  // row tile
  if (rest) nt = (int)(t - (uint64_t)at * n_tiles);
  for (int base = 0; base < E; base += 64) {
    if (E > 64) look(base);
    int l = -1;
    if (rest) {
      const uint32_t rows = (uint32_t)count % BM;
      if (E <= 64) {
        l = lane_in_order((int)rows, E, (int)at);
      } else {
        scan = wave_scan(rows != 0);
        const uint64_t hit = __ballot(at - before < scan && rows != 0);
        if (hit) l = __builtin_ctzll(hit);
      }
    } else {
      if (E > 64) scan = wave_scan(mine);
      const uint64_t hit = __ballot(at - before < scan && mine > 0);
      if (hit) l = __builtin_ctzll(hit);
    }
    if (l >= 0) {
      r.expert = base + l;
      r.first = __builtin_amdgcn_readlane(first, l);
      r.count = __builtin_amdgcn_readlane(count, l);
      if (rest) {
        mt = r.count / BM;
      } else {
        const uint32_t m_tiles = (uint32_t)__builtin_amdgcn_readlane((int)mine, l);
        const uint32_t begin = before + (uint32_t)__builtin_amdgcn_readlane((int)scan, l) - m_tiles;
        place_tile((uint32_t)(t - (uint64_t)begin * n_tiles), m_tiles, n_tiles, mt, nt);
      }
      return true;
    }
    before += last_lane(scan);
  }
  return false;
}

// TN: every expert has m x n tiles, whether it has rows or not, and the time of a tile goes by the rows. Each XCD gets an eighth
// of every expert's tiles, those of the experts with the most rows first (up to 64 experts; more are taken as they come).
__device__ __forceinline__ bool find_matrix(const ProductArgs &a, uint32_t block, uint32_t m_tiles, uint32_t n_tiles, Rows &r,
                                            int &mt, int &nt) {
  const int lane = threadIdx.x & 63, E = a.n_experts;
  const uint32_t each = m_tiles * n_tiles, per = (each + kXcds - 1) / kXcds;
  const uint32_t slot = block / kXcds, order = slot / per;
  // the XCDs take turns in getting an expert's last part, which may be smaller
  const uint32_t u = (block + order) % kXcds * per + slot % per;
  if (order >= (uint32_t)E || u >= each) return false;
  int first = 0, count = -1;
  r.expert = (int)order;
  if (E > 1 && E <= 64) {
    if (lane < E) expert_rows(a, lane, first, count);
    r.expert = lane_in_order(count, E, (int)order);
    r.first = __builtin_amdgcn_readlane(first, r.expert);
    r.count = __builtin_amdgcn_readlane(count, r.expert);
  } else {
    expert_rows(a, r.expert, first, count);
    r.first = __builtin_amdgcn_readfirstlane(first);
    r.count = __builtin_amdgcn_readfirstlane(count);
  }
  place_tile(u, m_tiles, n_tiles, mt, nt);
  return true;
}

// ------------------------------------------------------------ shared memory
// Rows across the sum: the 4 rows of a 16-lane group, and those of the group
// that reads beside it (8 rows on), in different 32-byte slots; rows of 64 elements have four.
template <int N>
__device__ __forceinline__ uint32_t swizzle(uint32_t k) { return ((k & 3) | (N >= 128 ? k >> 3 & 1 : 0) << 2) << 1; }

// Rows along the sum, 64 or 128 bytes each: ds_read_b128 serves the lanes 0-3, 12-15, 20-23 and 24-27 together (then 4-11, 16-19 and
// 28-31, and so on), which are rows 0-15 in two chunks for BF16 and the rows of these numbers for MXFP4. Without this split
// MXFP4's reads took twice as long. BF16 has no conflicts left in any form, MXFP4 in 38 % of shared memory's cycles (8192 x 8192 x 8192).
template <bool F4, int Sub>
__device__ __forceinline__ uint32_t swizzle_along(uint32_t row) { return Sub == 2 ? row >> 1 & 7 : F4 ? row >> 2 & 3 : row >> 1 & 3; }

// One operand's tile of a step: N rows of the operand (along the sum) or 32 Sub rows of N elements (across it).
template <int N, bool Across, bool F4, int Sub, int Threads>
struct Place {
  static constexpr int kChunks = N * 4 * Sub;  // 16-byte chunks
  static constexpr int kEach = kChunks / Threads;
  static constexpr int kRow = Across ? N / 8 : 4 * Sub;  // chunks of a row in shared memory
  static_assert(kChunks % Threads == 0, "chunks per thread");
  static_assert(!Across || N >= 64, "the swizzle spans 8 or 16 chunks");
  // Chunk q of the tile holds (row, chunk) of the operand.
  static __device__ __forceinline__ void source(int q, int &row, int &chunk) {
    row = q / kRow;
    chunk = (q % kRow) ^ (int)(Across ? swizzle<N>(row) : swizzle_along<F4, Sub>(row));
  }
};

// Global memory at a byte address, at any alignment of 2 bytes. (Through generic pointers the accesses would count as
// shared memory's too, and every read of a step would wait for the next step's loads.)
template <class V, int Align = 2>
__device__ __forceinline__ V load_at(uint64_t p) {
  typedef V Any __attribute__((aligned(Align)));
  return *(const __attribute__((address_space(1))) Any *)(uintptr_t)p;
}
template <class V>
__device__ __forceinline__ void store_at(uint64_t p, V v) {
  typedef V Any __attribute__((aligned(2)));
  *(__attribute__((address_space(1))) Any *)(uintptr_t)p = v;
}

// Eight BF16 elements of which the first `valid` exist.
__device__ __forceinline__ u32x4 load_chunk(uint64_t p, int64_t valid) {
  u32x4 v = {0, 0, 0, 0};
  if (valid >= 8) {
    v = load_at<u32x4>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) v[i >> 1] |= (uint32_t)load_at<uint16_t>(p + 2 * i) << (16 * (i & 1));
  }
  return v;
}

// The last `n` (uniform, 1 to 7) of eight elements as the first ones; what lies behind them is not looked at.
__device__ __forceinline__ u32x4 last_first(u32x4 v, int n) {
  const int drop = 8 - n;
  if (drop & 4) v = u32x4{v.z, v.w, 0, 0};
  if (drop & 2) v = u32x4{v.y, v.z, v.w, 0};
  if (drop & 1) v = u32x4{v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16};
  return v;
}

// ----------------------------------------------------------------- the tile
// Sub: steps are 64 Sub bytes along the sum.
template <int Form, Epilogue Epi, bool F4, int BM, int BN, int WM, int WN, int Sub>
struct Tile {
  static constexpr int kForm = Form;
  static constexpr Epilogue kEpi = Epi;
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr bool kAcrossA = Form == kTN, kAcrossB = Form != kNT;
  static constexpr int kStepBytes = 64 * Sub, kStep = (F4 ? 128 : 32) * Sub;  // of a row along the sum; elements
  static constexpr int kSub = Sub, kScaleSteps = 4 / Sub;  // steps of a row of scales
  static constexpr int kS = F4 ? 32 : 16;  // of a matrix instruction
  static constexpr int kPer = F4 ? 2 : 1, kKK = kPer * Sub;  // matrix instructions along 64 bytes of the sum, and along a step
  typedef typename std::conditional<F4, f32x16, f32x4>::type Acc;
  static constexpr int kTM = BM / WM / kS, kTN_ = BN / WN / kS;
  static constexpr int kColumns = Epi == Epilogue::kGated ? BN / 2 : BN;  // of out (h)
  static constexpr int kLdsA = BM * kStepBytes, kLdsB = BN * kStepBytes;
  static constexpr int kLds = kLdsA + kLdsB;
  // Scales of kScaleSteps steps, copied 64 rows at a time
  static constexpr int kScaleRowsA = (BM + 63) / 64 * 64, kScaleRowsB = (BN + 63) / 64 * 64;
  static constexpr int kLdsScales = F4 ? (kScaleRowsA + kScaleRowsB) * kScaleRow : 0;
  using PlaceA = Place<BM, kAcrossA, F4, Sub, kThreads>;
  using PlaceB = Place<BN, kAcrossB, F4, Sub, kThreads>;

  // Row of b's matrix that row r of the tile holds (its last one for those behind it); the gated forms have gate rows in the
  // lower half and the same columns' up rows in the upper.
  static __device__ __forceinline__ int64_t b_row(const ProductArgs &a, int n0, int r) {
    const int c = min(n0 + r % kColumns, a.n - 1);
    return r < kColumns ? c : (int64_t)a.n + c;
  }

  static constexpr int kWaveColumns = kColumns / WN;  // columns of out of a wave
  // Row (column) of b's tile where fragment j begins, without the wave's first; gated: up fragments behind the gate's.
  static constexpr int b_frag(int j) {
    return Epi == Epilogue::kGated && j >= kTN_ / 2 ? kColumns + kS * (j - kTN_ / 2) : kS * j;
  }

  // Where a lane reads its part of the wave's first fragments (bytes into a step's operands). Of each 64 bytes of the sum the
  // lanes' part p = lane / kS takes chunk p (MXFP4: chunks 2 p and 2 p + 1, one for each matrix instruction). Fragment i of rows
  // that run along the sum lies kS i rows on: row r0 + lane % kS; its other chunks are found by an exclusive or. Across: columns
  // c0 .. c0 + 15; the swizzle moves chunks within 16, so that fragment i is found by an exclusive or.
  struct Lane {
    uint32_t a, b, sa, sb;
  };
  static __device__ __forceinline__ uint32_t lane_along(int r0) {
    const uint32_t lane = threadIdx.x & 63;
    return (r0 + lane % kS) * kStepBytes + ((lane / kS * kPer) ^ swizzle_along<F4, Sub>(lane % kS)) * 16;
  }
  template <int N, int Each>
  static __device__ __forceinline__ uint32_t lane_across(int c0) {
    static_assert(kS == 16 && (Each == 32 || Each == 64 || Each == 128), "a wave's columns do not carry into the swizzle");
    const uint32_t lane = threadIdx.x & 63, i = lane & 15, k = (lane >> 4) * 8 + (i >> 2);
    return k * (2 * N) + ((c0 / 8 + (i >> 1 & 1)) ^ swizzle<N>(k)) * 16 + (i & 1) * 8;  // swizzle(k + 4) is the same
  }
  static __device__ __forceinline__ Lane lane_of(int wm, int wn) {
    const uint32_t lane = threadIdx.x & 63, scale = lane % kS * kScaleRow + lane / kS * kPer;
    const int r0 = wm * (BM / WM), c0 = wn * kWaveColumns;
    Lane l;
    if constexpr (kAcrossA) l.a = lane_across<BM, BM / WM>(r0);
    else l.a = lane_along(r0);
    if constexpr (kAcrossB) l.b = lane_across<BN, BN / WN>(c0) + kLdsA;
    else l.b = lane_along(c0) + kLdsA;
    l.sa = r0 * kScaleRow + scale;
    l.sb = (kScaleRowsA + c0) * kScaleRow + scale;
    return l;
  }

  typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
  typedef __attribute__((address_space(3))) const uint16_t lds_u16;
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  template <int N>
  static __device__ __forceinline__ u32x4 read_across(uint32_t at) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)(at + 4 * 2 * N));
    u32x4 v;
    __builtin_memcpy(&v, &lo, 8);
    __builtin_memcpy((char *)&v + 8, &hi, 8);
    return v;
  }

  // A wave's share of a step's operands, in registers.
  struct Fragments {
    u32x4 a[kTM][kKK], b[kTN_][kKK];
    uint32_t sa[F4 ? kTM : 1][Sub], sb[F4 ? kTN_ : 1][Sub];  // scales, two to a register
  };

  // Where a step's operands and scales lie in shared memory. keep: mask of the lane's scales that are the row's (what is
  // behind them may be anything, NaN among it).
  struct From {
    uint32_t operands, scales, keep[Sub];
  };
  // The exclusive or that finds matrix instruction kk's chunk.
  static constexpr uint32_t chunk_bits(int kk) { return 64u * (kk / kPer) + 16u * (kk % kPer); }
  static __device__ __forceinline__ void read_a(const From &from, const Lane &l, int i, int kk, Fragments &f) {
    if constexpr (kAcrossA) f.a[i][kk] = read_across<BM>(from.operands + (l.a ^ (uint32_t)(2 * kS * i)) + 64 * BM * kk);
    else f.a[i][kk] = *(lds_u32x4 *)(uintptr_t)(from.operands + (l.a ^ chunk_bits(kk)) + kS * i * kStepBytes);
    if constexpr (F4)
      if (kk % kPer == kPer - 1)
        f.sa[i][kk / kPer] = *(lds_u16 *)(uintptr_t)(from.scales + l.sa + kS * kScaleRow * i + 4 * (kk / kPer)) & from.keep[kk / kPer];
  }
  static __device__ __forceinline__ void read_b(const From &from, const Lane &l, int j, int kk, Fragments &f) {
    if constexpr (kAcrossB) f.b[j][kk] = read_across<BN>(from.operands + (l.b ^ (uint32_t)(2 * kS * j)) + 64 * BN * kk);
    else f.b[j][kk] = *(lds_u32x4 *)(uintptr_t)(from.operands + (l.b ^ chunk_bits(kk)) + b_frag(j) * kStepBytes);
    if constexpr (F4)
      if (kk % kPer == kPer - 1)
        f.sb[j][kk / kPer] = *(lds_u16 *)(uintptr_t)(from.scales + l.sb + kScaleRow * b_frag(j) + 4 * (kk / kPer)) & from.keep[kk / kPer];
  }
  static __device__ __forceinline__ void read(const From &from, const Lane &l, Fragments &f) {
#pragma unroll
    for (int kk = 0; kk < kKK; ++kk) {
#pragma unroll
      for (int j = 0; j < kTN_; ++j) read_b(from, l, j, kk, f);
#pragma unroll
      for (int i = 0; i < kTM; ++i) read_a(from, l, i, kk, f);
    }
  }
  // `left`: scale blocks of the row from this step's first on.
  static __device__ __forceinline__ From from_of(uint32_t operands, uint32_t scales, int64_t left) {
    From f;
    f.operands = operands;
    f.scales = scales;
#pragma unroll
    for (int u = 0; u < Sub; ++u) {
      const int first = 4 * u + (threadIdx.x & 63) / kS * kPer;
      f.keep[u] = first + 1 < left ? 0xFFFFu : first < left ? 0xFFu : 0u;
    }
    return f;
  }

  // Row i of the products with chunk kk, a's fragment from fa and b's from fb.
  template <int kk>
  static __device__ __forceinline__ void multiply(const Fragments &fa, const Fragments &fb, int i, Acc (&acc)[kTM][kTN_]) {
#pragma unroll
    for (int j = 0; j < kTN_; ++j) {
      const u32x4 x = fb.b[j][kk], y = fa.a[i][kk];
      if constexpr (F4) {
        // the codes are the lower half of the operand, the upper is not looked at
        const i32x8 b = (i32x8)__builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
        const i32x8 a = (i32x8)__builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1);
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[i][j], 4, 4, kk % kPer, (int)fb.sb[j][kk / kPer],
                                                                    kk % kPer, (int)fa.sa[i][kk / kPer]);
      } else {
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), acc[i][j], 0, 0, 0);
      }
    }
  }
};

// ------------------------------------------------------------------ results
// Of eight neighbouring columns `n` exist.
template <class V>
__device__ __forceinline__ void store8(uint64_t out, int64_t at, const float (&v)[8], int n) {
  const uint64_t p = out + (uint64_t)at * sizeof(V);
  typedef V V8 __attribute__((ext_vector_type(8)));
  if (n >= 8) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (V)v[i];
    store_at<V8>(p, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store_at<V>(p + sizeof(V) * i, (V)v[i]);
  }
}

__device__ __forceinline__ void load_pre(uint64_t pre, int64_t at, int n, float (&v)[8]) {
  const u32x4 w = load_chunk(pre + 2 * (uint64_t)at, n);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// What becomes of eight neighbouring sums of one row: `row` of out, `column` of out (h), n of them exist.
template <Epilogue Epi>
__device__ __forceinline__ void finish8(const ProductArgs &a, uint64_t out, int64_t row, int column, int n, const float (&s)[8],
                                        const float (&up)[8]) {
  if (Epi == Epilogue::kPlain) {
    if (a.out_f32) store8<float>(out, row * a.out_stride + column, s, n);
    else store8<__bf16>(out, row * a.out_stride + column, s, n);
  } else if (Epi == Epilogue::kGated) {
    if (a.pre) {
      store8<__bf16>(a.pre, row * a.pre_stride + column, s, n);
      store8<__bf16>(a.pre, row * a.pre_stride + a.n + column, up, n);
    }
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Act t = activation(a.act, s[i]);
      h[i] = t.value * t.scale * up[i];
    }
    store8<__bf16>(out, row * a.out_stride + column, h, n);
  } else {
    // d(pre) leaves in BF16, as the operand of two products: in fp32 they would take it as two BF16 terms, twice the matrix
    // instructions (1.1 of 1.66 ms of 8192 rows of 12 experts, 7168, 2048). What it costs: 0.00235 of the gradients' norm against
    // 0.00166 with d(pre) in fp32; the results themselves are BF16, of which 0.00166 is the rounding.
    float g[8], u[8], dg[8], du[8];
    load_pre(a.pre, row * a.pre_stride + column, n, g);
    load_pre(a.pre, row * a.pre_stride + a.n + column, n, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Act t = activation(a.act, g[i]);
      const float dh = s[i] * t.scale;
      dg[i] = dh * u[i] * t.slope;
      du[i] = dh * t.value;
    }
    store8<__bf16>(out, row * a.out_stride + column, dg, n);
    store8<__bf16>(out, row * a.out_stride + a.n + column, du, n);
  }
}

// Eight neighbouring columns of a lane's row out of two fours of neighbouring columns, by exchange with another lane.
// 16 x 16: lane group g = lane / 16 has columns 4 g .. of fragments x and y; the even groups get 4 g .. + 7 of x, the odd ones
// 4 (g - 1) .. + 7 of y. 32 x 32: half h has columns 4 h .. of x and 8 + 4 h .. of the same fragment as y, and gets 8 h .. + 7.
template <int S, class V>
__device__ __forceinline__ void eight(const V &x, int x0, const V &y, int y0, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = __float_as_uint(x[x0 + i]), q = __float_as_uint(y[y0 + i]);
    const auto r = S == 16 ? __builtin_amdgcn_permlane16_swap(p, q, false, false) : __builtin_amdgcn_permlane32_swap(p, q, false, false);
    v[i] = __uint_as_float(r[0]);
    v[4 + i] = __uint_as_float(r[1]);
  }
}

// T: the tile; acc: sums of TM x TN fragments from row row0 of the tile and column column0 of out on.
template <class T, class Acc, int TM, int TN>
__device__ __forceinline__ void finish_tile(const ProductArgs &a, const Rows &r, int m0, int m_left, int row0, int column0,
                                            const Acc (&acc)[TM][TN]) {
  constexpr int S = T::kS, Form = T::kForm;
  constexpr Epilogue Epi = T::kEpi;
  const int lane = threadIdx.x & 63, g = lane / S;
  const uint64_t out = a.out + (Form == kTN ? (uint64_t)(a.out_expert * r.expert) * (a.out_f32 ? 4 : 2) : 0);
  constexpr int kCols = Epi == Epilogue::kGated ? TN / 2 : TN;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = row0 + S * i + lane % S;
#pragma unroll
    for (int p = 0; p < kCols * S / 16; p += 2) {  // 32 columns
      constexpr int kUp = Epi == Epilogue::kGated ? kCols : 0;
      const int x = p * 16 / S, y = (p + 1) * 16 / S;
#pragma unroll
      for (int half = 0; half < S / 16; ++half) {
        const int column = column0 + 16 * p + (S == 16 ? 16 * (g & 1) + 8 * (g >> 1) : 16 * half + 8 * g);
        float s[8], up[8];
        if constexpr (S == 16) {
          eight<S>(acc[i][x], 0, acc[i][y], 0, s);
          if (kUp) eight<S>(acc[i][x + kUp], 0, acc[i][y + kUp], 0, up);
        } else {
          eight<S>(acc[i][x], 8 * half, acc[i][x], 8 * half + 4, s);
          if (kUp) eight<S>(acc[i][x + kUp], 8 * half, acc[i][x + kUp], 8 * half + 4, up);
        }
        if (row < m_left && column < a.n)
          finish8<Epi>(a, out, (Form == kTN ? 0 : r.first) + m0 + row, column, a.n - column, s, up);
      }
    }
  }
}

// ------------------------------------------------- operands of any alignment
// The next step's chunks are loaded to registers before the present one is
// computed and stored to the other half of shared memory behind it.
template <int Form, Epilogue Epi, bool F4, int BM, int BN, int WM, int WN, int Sub>
__global__ void __launch_bounds__(64 * WM * WN) product_any_kernel(ProductArgs a) {
  using T = Tile<Form, Epi, F4, BM, BN, WM, WN, Sub>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][T::kLds + T::kLdsScales];
  Rows r;
  int mt, nt;
  const uint32_t n_tiles = (uint32_t)(a.n + T::kColumns - 1) / T::kColumns;
  const bool mine = Form == kTN ? find_matrix(a, a.first_group + blockIdx.x, (uint32_t)(a.m + BM - 1) / BM, n_tiles, r, mt, nt)
                                : find_rows<BM>(a, a.first_group + blockIdx.x, n_tiles, r, mt, nt);
  if (!mine) return;
  const int tid = threadIdx.x, wave = tid >> 6, wm = wave / WN, wn = wave % WN;
  const int m0 = mt * BM, n0 = nt * T::kColumns;
  const int64_t K = Form == kTN ? r.count : a.k;
  const int m_left = (Form == kTN ? a.m : r.count) - m0;
  const uint64_t b_base = a.b + (Form == kTN ? 0 : (uint64_t)(a.b_expert * r.expert));

  // Of each chunk: where it lies in the first step, how many of its elements exist (along the sum: of its row; across it: of
  // the columns), and its row in the step. The chunks that a step has in full are loaded without a question.
  constexpr int kA = T::PlaceA::kEach, kB = T::PlaceB::kEach;
  u32x4 ra[kA], rb[kB];
  uint32_t rs[Sub] = {};
  uint64_t pa[kA], pb[kB];
  int64_t va[kA], vb[kB];
  bool cut_a[kA] = {}, cut_b[kB] = {};
  const int64_t f4_row = (int64_t)(a.k + 31) / 32 * 16;  // bytes of codes
  const int64_t along = F4 ? f4_row / 16 * 8 : a.k;      // elements, codes in chunks that count as 8
  const bool gather_b = Form == kTN && a.row_index;
  bool full = true;
#pragma unroll
  for (int i = 0; i < kA; ++i) {
    int row, chunk;
    T::PlaceA::source(tid + i * T::kThreads, row, chunk);
    if (T::kAcrossA) {
      pa[i] = a.a + (uint64_t)((r.first + row) * a.a_stride + 2 * (int64_t)(m0 + 8 * chunk));
      va[i] = m_left - 8 * chunk;
      // columns that do not exist may hold anything: the tile's first ones; a chunk that ends behind the last column is loaded
      // as the eight before it and moved
      if (va[i] <= 0 && m_left >= 8) pa[i] -= 16 * chunk, va[i] = 8;
      cut_a[i] = va[i] > 0 && va[i] < 8;
      if (cut_a[i] && a.m >= 8) pa[i] -= 2 * (8 - va[i]);
      full = full && (va[i] >= 8 || (cut_a[i] && a.m >= 8));
    } else {
      // so may rows that do not exist
      int64_t from = r.first + m0 + min(row, m_left - 1);
      bool there = true;
      if (!F4 && a.row_index) {
        from = a.row_index[from];
        there = from >= 0 && from < a.n_index_rows;
      }
      pa[i] = a.a + (uint64_t)(there ? from * a.a_stride + 16 * chunk : 0);
      va[i] = there ? along - 8 * chunk : 0;
      full = full && there;
    }
  }
#pragma unroll
  for (int i = 0; i < kB; ++i) {
    int row, chunk;
    T::PlaceB::source(tid + i * T::kThreads, row, chunk);
    if (T::kAcrossB) {
      pb[i] = b_base + (uint64_t)((gather_b ? 0 : (Form == kTN ? r.first + row : row) * a.b_stride) + 2 * (int64_t)(n0 + 8 * chunk));
      vb[i] = a.n - n0 - 8 * chunk;
      if (vb[i] <= 0 && a.n - n0 >= 8) pb[i] -= 16 * chunk, vb[i] = 8;
      cut_b[i] = vb[i] > 0 && vb[i] < 8;
      if (cut_b[i] && a.n >= 8) pb[i] -= 2 * (8 - vb[i]);
      full = full && (vb[i] >= 8 || (cut_b[i] && a.n >= 8));
    } else {
      pb[i] = b_base + (uint64_t)(T::b_row(a, n0, row) * a.b_stride + 16 * chunk);
      vb[i] = along - 8 * chunk;
    }
  }
  full = __all(full);
  // the tiles with the last columns, if those do not fill a chunk
  const bool cuts_a = T::kAcrossA && m_left < BM && a.m % 8, cuts_b = T::kAcrossB && a.n - n0 < BN && a.n % 8;
  auto load = [&](int64_t k0) __attribute__((always_inline)) {  // k0 in elements
    const int64_t k1 = F4 ? k0 / 4 : k0;  // as `along` counts
    const bool whole = full && (F4 ? k1 + T::kStep / 4 <= along : k0 + T::kStep <= K);
    const uint64_t move_a = (uint64_t)(T::kAcrossA ? k0 * a.a_stride : 2 * k1), move_b = (uint64_t)(T::kAcrossB ? k0 * a.b_stride : 2 * k1);
    uint64_t at_b[kB];
    bool there_b[kB];
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      int row, chunk;
      T::PlaceB::source(tid + i * T::kThreads, row, chunk);
      at_b[i] = pb[i] + move_b;
      there_b[i] = !T::kAcrossB || k0 + row < K;
      if (gather_b && there_b[i]) {
        const int64_t from = a.row_index[r.first + k0 + row];
        there_b[i] = from >= 0 && from < a.n_index_rows;
        at_b[i] = pb[i] + (uint64_t)(there_b[i] ? from * a.b_stride : 0);
      }
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < kA; ++i) ra[i] = load_at<u32x4>(pa[i] + move_a);
      if (gather_b) {
#pragma unroll
        for (int i = 0; i < kB; ++i) rb[i] = there_b[i] ? load_at<u32x4>(at_b[i]) : u32x4{0, 0, 0, 0};
      } else {
#pragma unroll
        for (int i = 0; i < kB; ++i) rb[i] = load_at<u32x4>(at_b[i]);
      }
      if (cuts_a) {
#pragma unroll
        for (int i = 0; i < kA; ++i) ra[i] = cut_a[i] ? last_first(ra[i], a.m % 8) : ra[i];
      }
      if (cuts_b) {
#pragma unroll
        for (int i = 0; i < kB; ++i) rb[i] = cut_b[i] ? last_first(rb[i], a.n % 8) : rb[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kA; ++i) {
        int row, chunk;
        T::PlaceA::source(tid + i * T::kThreads, row, chunk);
        ra[i] = load_chunk(pa[i] + move_a + (cut_a[i] && a.m >= 8 ? 2 * (8 - va[i]) : 0),
                           T::kAcrossA ? (k0 + row < K ? va[i] : 0) : va[i] - k1);
      }
#pragma unroll
      for (int i = 0; i < kB; ++i)
        rb[i] = load_chunk(at_b[i] + (cut_b[i] && a.n >= 8 ? 2 * (8 - vb[i]) : 0), T::kAcrossB ? (there_b[i] ? vb[i] : 0) : vb[i] - k1);
    }
    if constexpr (F4) {  // the scales of a row's blocks
      static_assert(!F4 || BM + BN == T::kThreads, "a row of scales to a thread");
#pragma unroll
      for (int u = 0; u < Sub; ++u) {
        const int64_t at = k0 / 32 + 4 * u;
        rs[u] = 0;
        if (at >= (a.k + 31) / 32) continue;
        if (tid < BM) {
          rs[u] = load_at<uint32_t>(a.a_scales + (uint64_t)((r.first + m0 + min(tid, m_left - 1)) * a.a_scale_stride + at));
        } else {
          const int64_t s = T::b_row(a, n0, tid - BM);
          rs[u] = load_at<uint32_t>(a.b_scales + (uint64_t)(a.b_scale_expert * r.expert + s * a.b_scale_stride + at));
        }
      }
    }
  };
  auto store = [&](uint8_t *to) {
#pragma unroll
    for (int i = 0; i < T::PlaceA::kEach; ++i) *(u32x4 *)(to + 16 * (tid + i * T::kThreads)) = ra[i];
#pragma unroll
    for (int i = 0; i < T::PlaceB::kEach; ++i) *(u32x4 *)(to + T::kLdsA + 16 * (tid + i * T::kThreads)) = rb[i];
    if constexpr (F4) {
#pragma unroll
      for (int u = 0; u < Sub; ++u) *(uint32_t *)(to + T::kLds + kScaleRow * tid + 4 * u) = rs[u];
    }
  };

  typename T::Acc acc[T::kTM][T::kTN_];
#pragma unroll
  for (int i = 0; i < T::kTM; ++i)
#pragma unroll
    for (int j = 0; j < T::kTN_; ++j) acc[i][j] = typename T::Acc{};
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&lds[0][0];
  const typename T::Lane lane = T::lane_of(wm, wn);
  if (K > 0) {
    load(0);
    store(lds[0]);
    __syncthreads();
    int at = 0;
    for (int64_t k0 = 0; k0 < K; k0 += T::kStep, at ^= 1) {
      const bool more = k0 + T::kStep < K;
      if (more) load(k0 + T::kStep);
      typename T::Fragments f;
      const uint32_t from = lds0 + at * (T::kLds + T::kLdsScales);
      T::read(T::from_of(from, from + T::kLds, (a.k - k0 + 31) / 32), lane, f);
      static_for<T::kKK>([&](auto half) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::kTM; ++i) T::template multiply<decltype(half)::value>(f, f, i, acc);
      });
      if (more) store(lds[at ^ 1]);
      __syncthreads();
    }
  }

  finish_tile<T>(a, r, m0, m_left, wm * (BM / WM), n0 + wn * T::kWaveColumns, acc);
}

// ------------------------------------------------------ aligned operands
// buffer_load ... lds copies 16 bytes a lane straight into shared memory, at
// consecutive places of a wave (from M0 on), so the swizzle is in the addresses that are
// read. What lies outside of [base, base + bytes) reads as 0 and touches no
// memory: rows behind the last, and offsets set to kNowhere.
constexpr uint32_t kNowhere = 0x80000000u;

// The compiler does not count these loads: wait_for_copies() waits for them. It is told of M0, which it uses for operations of
// its own (messages, indexed registers), none of them in these kernels now. (It warns
// that it does not save M0 itself, which nothing here expects.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int Add>
__device__ __forceinline__ void copy16(u32x4 buffer, uint32_t lds, uint32_t offset) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buffer), "n"(Add) : "memory", "scc", "m0");
}
template <int Add>
__device__ __forceinline__ void copy4(u32x4 buffer, uint32_t lds, uint32_t offset) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buffer), "n"(Add) : "memory", "scc", "m0");
}
#pragma clang diagnostic pop

// All but the last `Pending` of this wave's copies have arrived and what it read has been read; then the workgroup meets.
template <int Pending, bool Meet>
__device__ __forceinline__ void wait_for_copies() {
  if (Meet) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(Pending) : "memory");
  else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(Pending) : "memory");
}

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
__device__ __forceinline__ uint64_t uniform(uint64_t x) { return (uint64_t)uniform((uint32_t)(x >> 32)) << 32 | uniform((uint32_t)x); }

// What a step copies of an operand: `bytes` from `base` on, `last_bytes` in the last step.
struct Window {
  uint64_t base;
  uint32_t move;  // bytes from step to step
  uint32_t bytes, last_bytes;
  __device__ __forceinline__ u32x4 buffer(bool last) const {
    return u32x4{uniform((uint32_t)base), uniform((uint32_t)(base >> 32)), uniform(last ? last_bytes : bytes), 0x00020000u};
  }
};

__device__ __forceinline__ Window window(uint64_t base, int64_t move, int64_t bytes, int64_t last_bytes) {
  // (an operand without rows has less than no bytes)
  return {uniform(base), uniform((uint32_t)move), uniform((uint32_t)max(bytes, (int64_t)0)), uniform((uint32_t)max(last_bytes, (int64_t)0))};
}

// WM x WN waves share a tile (Split = 1), or Split waves take a part of the sum each, of the same tile and with operands of
// their own, and add up their sums in the end (WM = WN = 1).
// Indexed: rows along the sum (b of TN) are taken through row_index.
template <int Form, Epilogue Epi, bool F4, int BM, int BN, int WM, int WN, int Split, int Sub, int kStages, bool Indexed>
__global__ void __launch_bounds__(64 * WM * WN * Split, WM * WN * Split == 4 && Sub * Split * kStages * (BM + BN) > 1280 ? 1 : 2) product_kernel(ProductArgs a) {
  using T = Tile<Form, Epi, F4, BM, BN, WM, WN, Sub>;
  constexpr int kStepBytes = T::kStepBytes, kScaleSteps = T::kScaleSteps;
  using PA = typename T::PlaceA;
  using PB = typename T::PlaceB;
  static_assert(Split == 1 || (WM == 1 && WN == 1), "a wave has the whole tile or the whole sum");
  constexpr int kIndexSteps = 2 / Sub, kIndexPairs = kStages / kIndexSteps + 2,
                kIndexRows = Indexed ? 256 * kIndexPairs : 0;  // of a wave: 64 row numbers, that is steps; how often; bytes
  // rows of scales: those of the steps that are copied ahead, and of the present step's
  constexpr int kScaleRing = (kStages + kScaleSteps - 1) / kScaleSteps + 1;
  constexpr int kRing = kStages * T::kLds + kScaleRing * T::kLdsScales;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Split * kRing + WM * WN * Split * kIndexRows];
  Rows r;
  int mt, nt;
  const uint32_t n_tiles = (uint32_t)(a.n + T::kColumns - 1) / T::kColumns;
  const bool mine = Form == kTN ? find_matrix(a, a.first_group + blockIdx.x, (uint32_t)(a.m + BM - 1) / BM, n_tiles, r, mt, nt)
                                : find_rows<BM>(a, a.first_group + blockIdx.x, n_tiles, r, mt, nt);
  if (!mine) return;
  const int waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = Split > 1 ? waves : 0, wave = Split > 1 ? 0 : waves, wm = wave / WN, wn = wave % WN;
  const int tid = Split > 1 ? threadIdx.x & 63 : threadIdx.x;  // among those that share the tile
  const int m0 = mt * BM, n0 = nt * T::kColumns;
  const int m_left = (Form == kTN ? a.m : r.count) - m0;
  const int64_t K = Form == kTN ? r.count : a.k;
  constexpr int kCopies = PA::kEach + PB::kEach;  // of a thread and step (scales and row numbers come on top now and then)
  const int all_steps = (int)((K + T::kStep - 1) / T::kStep);
  // This wave's steps of the sum: whole kScaleSteps of them for MXFP4.
  constexpr int kUnit = F4 ? kScaleSteps : 1;
  const int units = (all_steps + kUnit - 1) / kUnit;
  const int step0 = units * part / Split * kUnit, steps = min(units * (part + 1) / Split * kUnit, all_steps) - step0;
  const int last_step = all_steps - 1 - step0;  // of the sum, counted from step0

  // Along the sum: bytes of a row that the last step has. Across it: rows.
  const int64_t row_bytes = F4 ? (int64_t)(a.k + 31) / 32 * 16 : 2 * (int64_t)a.k;
  const int last_bytes = (int)(row_bytes - (int64_t)(all_steps - 1) * kStepBytes);
  const int last_rows = (int)(K - (int64_t)(all_steps - 1) * T::kStep);

  Window wa, wb;
  uint32_t oa[PA::kEach], ob[PB::kEach];
  if (T::kAcrossA) {
    const int64_t width = 2 * (int64_t)min(a.m - m0, BM);
    wa = window(a.a + (uint64_t)(r.first * a.a_stride + 2 * (int64_t)m0), T::kStep * a.a_stride, (T::kStep - 1) * a.a_stride + width,
                (last_rows - 1) * a.a_stride + width);
  } else {
    const bool gather = !F4 && a.row_index;
    const int64_t before = (gather ? a.n_index_rows - 1 : min(m_left, BM) - 1) * a.a_stride;
    wa = window(a.a + (uint64_t)(gather ? 0 : (r.first + m0) * a.a_stride), kStepBytes, before + kStepBytes, before + last_bytes);
  }
#pragma unroll
  for (int i = 0; i < PA::kEach; ++i) {
    int row, chunk;
    PA::source(tid + i * T::kThreads, row, chunk);
    uint32_t at = (uint32_t)row;
    if (!T::kAcrossA && !F4 && a.row_index) {
      const int64_t from = row < m_left ? a.row_index[r.first + m0 + row] : -1;
      at = from >= 0 && from < a.n_index_rows ? (uint32_t)from : kNowhere;
    }
    oa[i] = at == kNowhere ? kNowhere : at * (uint32_t)a.a_stride + 16u * chunk;
  }
  const uint64_t b_base = a.b + (Form == kTN ? 0 : (uint64_t)(a.b_expert * r.expert));
  if (T::kAcrossB) {
    const int64_t width = 2 * (int64_t)min(a.n - n0, BN);
    const uint64_t base = b_base + (uint64_t)((Form == kTN && !Indexed ? r.first * a.b_stride : 0) + 2 * (int64_t)n0);
    const int64_t all = (a.n_index_rows - 1) * a.b_stride + width;
    wb = Indexed ? window(base, 0, all, all)
                 : window(base, T::kStep * a.b_stride, (T::kStep - 1) * a.b_stride + width, (last_rows - 1) * a.b_stride + width);
  } else {
    // gated: the up rows lie a.n rows behind the gate rows
    const int64_t before = (Epi == Epilogue::kGated ? a.n + min(a.n - n0, T::kColumns) - 1 : min(a.n - n0, BN) - 1) * a.b_stride;
    wb = window(b_base + (uint64_t)(n0 * a.b_stride), kStepBytes, before + kStepBytes, before + last_bytes);
  }
#pragma unroll
  for (int i = 0; i < PB::kEach; ++i) {
    int row, chunk;
    PB::source(tid + i * T::kThreads, row, chunk);
    if (Epi == Epilogue::kGated && row >= T::kColumns) row += a.n - T::kColumns;  // up rows
    ob[i] = (uint32_t)row * (uint32_t)a.b_stride + 16u * chunk;
  }
  wa.base += (uint64_t)step0 * wa.move;
  wb.base += (uint64_t)step0 * wb.move;

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&lds[0] + part * kRing;

  // Indexed: each wave copies the numbers of 64 rows at a time, kIndexPairs of them ahead.
  typedef __attribute__((address_space(3))) const int32_t lds_i32;
  const uint32_t lds_index = lds0 + (uint32_t)(Split - part) * kRing + (uint32_t)waves * kIndexRows;
  const Window wi = Indexed ? window((uint64_t)(uintptr_t)(a.row_index + r.first), 0, 4 * K, 4 * K) : Window{};
  auto copy_index = [&](int step) __attribute__((always_inline)) {  // a multiple of kIndexSteps
    const uint32_t at = 4u * (uint32_t)((step0 + step) * T::kStep + (threadIdx.x & 63));
    copy4<0>(wi.buffer(false), uniform(lds_index + (uint32_t)(step / kIndexSteps % kIndexPairs) * 256), at);
  };
  auto load_rows = [&](int step) __attribute__((always_inline)) {  // where b's rows of a step lie
#pragma unroll
    for (int i = 0; i < PB::kEach; ++i) {
      int row, chunk;
      PB::source(tid + i * T::kThreads, row, chunk);
      const int from = *(lds_i32 *)(uintptr_t)(lds_index + (uint32_t)(step % (kIndexSteps * kIndexPairs)) * (128 * Sub) + 4 * row);
      const bool there = (int64_t)(step0 + step) * T::kStep + row < K && from >= 0 && from < a.n_index_rows;
      ob[i] = there ? (uint32_t)from * (uint32_t)a.b_stride + 16u * chunk : kNowhere;
    }
  };

  // Scales: 64 rows of a or b, kScaleSteps steps of each, to a copy; the waves that share the tile take turns.
  constexpr int kScaleJobs = F4 ? (T::kScaleRowsA + T::kScaleRowsB) / 64 : 0, kScaleCopies = kScaleJobs / (WM * WN);
  static_assert(kScaleJobs % (WM * WN) == 0, "as many copies for every wave");
  Window ws[kScaleCopies > 0 ? kScaleCopies : 1];
  uint32_t os[kScaleCopies > 0 ? kScaleCopies : 1];
  const int blocks = (a.k + 31) / 32, last_scales = (all_steps - 1) / kScaleSteps * kScaleSteps;
  if constexpr (F4) {
#pragma unroll
    for (int i = 0; i < kScaleCopies; ++i) {
      const int job = wave + i * WM * WN;
      const bool of_a = job < T::kScaleRowsA / 64;
      const int64_t stride = of_a ? a.a_scale_stride : a.b_scale_stride;
      int row = (of_a ? job : job - T::kScaleRowsA / 64) * 64 + (threadIdx.x & 63);
      const bool there = row < (of_a ? BM : BN);
      const int64_t rows = of_a ? min(m_left, BM) : Epi == Epilogue::kGated ? a.n + min(a.n - n0, T::kColumns) : min(a.n - n0, BN);
      if (!of_a && Epi == Epilogue::kGated && row >= T::kColumns) row += a.n - T::kColumns;
      ws[i] = window((of_a ? a.a_scales + (uint64_t)((r.first + m0) * stride)
                           : a.b_scales + (uint64_t)(a.b_scale_expert * r.expert + n0 * stride)) + (uint64_t)step0 * (4 * Sub),
                     kScaleRow, (rows - 1) * stride + kScaleRow, (rows - 1) * stride + (blocks + 3) / 4 * 4 - 4 * Sub * last_scales);
      os[i] = there ? (uint32_t)row * (uint32_t)stride : kNowhere;
    }
  }
  auto copy_scales = [&](int step) __attribute__((always_inline)) {  // a multiple of kScaleSteps
#pragma unroll
    for (int i = 0; i < kScaleCopies; ++i) {
      const uint32_t to = uniform(lds0 + kStages * T::kLds + (uint32_t)(step / kScaleSteps % kScaleRing) * T::kLdsScales + 1024u * (wave + i * WM * WN));
      copy16<0>(ws[i].buffer(step0 + step == last_scales), to, os[i]);
      ws[i].base += ws[i].move;
    }
  };

  // One of a step's copies; the last step's rows along the sum may end before its 64 bytes.
  auto copy = [&](auto piece, int step, bool last) __attribute__((always_inline)) {
    constexpr int p = decltype(piece)::value;
    const uint32_t to = uniform(lds0 + (uint32_t)(step % kStages) * T::kLds + 1024u * wave);
    if constexpr (p < PA::kEach) {
      uint32_t at = oa[p];
      if (!T::kAcrossA && last) {
        int row, chunk;
        PA::source(tid + p * T::kThreads, row, chunk);
        at = 16 * chunk < last_bytes ? at : kNowhere;
      }
      copy16<p * T::kThreads * 16>(wa.buffer(last), to, at);
    } else {
      constexpr int i = p - PA::kEach;
      uint32_t at = ob[i];
      if (!T::kAcrossB && last) {
        int row, chunk;
        PB::source(tid + i * T::kThreads, row, chunk);
        at = 16 * chunk < last_bytes ? at : kNowhere;
      }
      copy16<T::kLdsA + i * T::kThreads * 16>(wb.buffer(last), to, at);
    }
  };
  auto advance = [&](int step) __attribute__((always_inline)) {  // behind the copies of `step`
    wa.base += wa.move;
    wb.base += wb.move;
    if (Indexed && step + 1 < steps) load_rows(step + 1);
  };

  typename T::Acc acc[T::kTM][T::kTN_];
#pragma unroll
  for (int i = 0; i < T::kTM; ++i)
#pragma unroll
    for (int j = 0; j < T::kTN_; ++j) acc[i][j] = typename T::Acc{};

  // A step's products use fragments that were read during the step before; the copies run kStages - 1 steps ahead. a's first
  // fragments are read again as soon as their row of products is through; b's, which every row needs, and a's last, which
  // would be late, have registers for two steps.
  const typename T::Lane lane = T::lane_of(wm, wn);
  typename T::Fragments f[2];
  constexpr int kLate = F4 || T::kTM < 2 ? 1 : 2, kOnce = T::kTM - kLate;
  auto from_step = [&](int step, bool tail) __attribute__((always_inline)) -> typename T::From {
    return T::from_of(lds0 + (uint32_t)(step % kStages) * T::kLds,
                      lds0 + kStages * T::kLds + (uint32_t)(step / kScaleSteps % kScaleRing) * T::kLdsScales + step % kScaleSteps * (4 * Sub),
                      tail ? blocks - 4 * Sub * (step0 + step) : 4 * Sub);
  };
  // Rows along the sum that end within a 16-byte chunk: what was copied behind their end becomes 0.
  auto cut_last = [&](int step) __attribute__((always_inline)) {
    if (F4 || last_bytes % 16 == 0) return;
    constexpr int kRowsAlong = BM + (T::kAcrossB ? 0 : BN);
    typedef __attribute__((address_space(3))) uint16_t lds_u16;
    for (int row = tid; row < kRowsAlong; row += T::kThreads) {
      const int in = row < BM ? row : row - BM;
      const uint32_t at = lds0 + (uint32_t)(step % kStages) * T::kLds + (row < BM ? 0 : T::kLdsA) + in * kStepBytes +
                          ((uint32_t)(last_bytes / 16) ^ swizzle_along<F4, Sub>(in)) * 16;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (2 * e >= last_bytes % 16) *(lds_u16 *)(uintptr_t)(at + 2 * e) = 0;
    }
    wait_for_copies<63, Split == 1>();
  };
  auto turn = [&](auto rows, auto tail, int step, typename T::Fragments &now, typename T::Fragments &next) __attribute__((always_inline)) {
    constexpr int Live = decltype(rows)::value;
    constexpr bool Tail = decltype(tail)::value;
    // the next step's operands are there, and nobody reads this step's any more
    if (!Tail || step + kStages <= steps) wait_for_copies<(kStages - 2) * kCopies, Split == 1>();
    else wait_for_copies<0, Split == 1>();
    if (Tail && Form != kTN && step + 1 == last_step) cut_last(step + 1);
    const typename T::From from = from_step(step + 1, Tail);
    const int ahead = step + kStages;
    if (F4 && ahead % kScaleSteps == 0 && (!Tail || ahead < steps)) copy_scales(ahead);
    if (Indexed && step % kIndexSteps == 0 && step + kIndexSteps * kIndexPairs < steps) copy_index(step + kIndexSteps * kIndexPairs);
    constexpr int kRows = T::kKK * T::kTM;  // of products
    static_for<kRows>([&](auto row) __attribute__((always_inline)) {
      constexpr int u = decltype(row)::value, i = u % T::kTM, kk = u / T::kTM;
      if constexpr (u < kLate * T::kKK && kOnce + u / T::kKK < Live) T::read_a(from, lane, kOnce + u / T::kKK, u % T::kKK, next);
      static_for<T::kKK * T::kTN_>([&](auto col) __attribute__((always_inline)) {
        constexpr int v = decltype(col)::value;
        if constexpr (v * kRows / (T::kKK * T::kTN_) / 2 == u && Live > 0) T::read_b(from, lane, v % T::kTN_, v / T::kTN_, next);
      });
      if (!Tail || ahead < steps) static_for<kCopies>([&](auto piece) __attribute__((always_inline)) {
          if constexpr (decltype(piece)::value * kRows / kCopies == u) copy(piece, ahead, Tail && ahead == last_step);
        });
      if constexpr (i < Live) T::template multiply<kk>(i < kOnce ? f[0] : now, now, i, acc);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (i < kOnce && i < Live) T::read_a(from, lane, i, kk, f[0]);
    });
    if (!Tail || ahead < steps) advance(ahead);
  };
  if (steps > 0) {
    if (Indexed) {
#pragma unroll 1
      for (int i = 0; i < kIndexSteps * kIndexPairs && i < steps; i += kIndexSteps) copy_index(i);
      wait_for_copies<0, false>();
      load_rows(0);
    }
#pragma unroll 1
    for (int i = 0; i < kStages && i < steps; ++i) {
      if (F4 && i % kScaleSteps == 0) copy_scales(i);
      static_for<kCopies>([&](auto piece) __attribute__((always_inline)) { copy(piece, i, i == last_step); });
      advance(i);
    }
    if (steps >= kStages) wait_for_copies<(kStages - 1) * kCopies, Split == 1>();
    else wait_for_copies<0, Split == 1>();
    if (Form != kTN && last_step == 0) cut_last(0);
    T::read(from_step(0, true), lane, f[0]);
    // rows: fragments of a that the wave multiplies
    auto loop = [&](auto rows) __attribute__((always_inline)) {
      int step = 0;
#pragma unroll 1
      for (; step + 1 + kStages < steps - 1; step += 2) {
        turn(rows, std::false_type(), step, f[0], f[1]);
        turn(rows, std::false_type(), step + 1, f[1], f[0]);
      }
#pragma unroll 1
      for (; step < steps; step += 2) {
        turn(rows, std::true_type(), step, f[0], f[1]);
        if (step + 1 < steps) turn(rows, std::true_type(), step + 1, f[1], f[0]);
      }
    };
    // an expert's last tile: waves leave out all or half of their rows if there are none
    const int live = m_left - wm * (BM / WM);
    constexpr bool kWhole = Form == kTN || Split > 1;
    if (kWhole || live > BM / WM / 2) loop(std::integral_constant<int, T::kTM>());
    else if (live > 0) loop(std::integral_constant<int, kWhole ? T::kTM : T::kTM / 2>());
    else loop(std::integral_constant<int, kWhole ? T::kTM : 0>());
  }
  if constexpr (Split == 1) {
    finish_tile<T>(a, r, m0, m_left, wm * (BM / WM), n0 + wn * T::kWaveColumns, acc);
  } else {
    // Row i of the fragments is added up, in the order of the parts, and finished by wave i.
    constexpr int kWords = sizeof(typename T::Acc) / 16, kPart = T::kTM * T::kTN_ * kWords;  // of 16 bytes and 64 lanes
    static_assert(Split * kPart * 1024 <= Split * kRing && T::kTM <= Split, "sums take the place of the operands");
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    const uint32_t sums = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&lds[0] + 16 * tid;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T::kTM; ++i)
#pragma unroll
      for (int j = 0; j < T::kTN_; ++j)
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * w + e];
          *(lds_f32x4 *)(uintptr_t)(sums + 1024 * (part * kPart + (i * T::kTN_ + j) * kWords + w)) = v;
        }
    __syncthreads();
    if (part >= T::kTM) return;
    typename T::Acc sum[1][T::kTN_];
#pragma unroll
    for (int j = 0; j < T::kTN_; ++j)
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        f32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < Split; ++p) v += *(lds_f32x4 *)(uintptr_t)(sums + 1024 * (p * kPart + (part * T::kTN_ + j) * kWords + w));
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[0][j][4 * w + e] = v[e];
      }
    finish_tile<T>(a, r, m0, m_left, part * T::kS, n0, sum);
  }
}

}  // namespace wt
