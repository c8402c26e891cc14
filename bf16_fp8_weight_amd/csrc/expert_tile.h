// expert_tile.h -- device code of the experts' products: the tile of a workgroup,
// its operands' way through shared memory, the matrix instructions and what is
// done with the sums. The definitions are in wt.h.
//
// A workgroup of WM x WN waves computes BM x BN results. Both operands pass
// through shared memory in steps of 128 bytes along the sum (64 BF16 elements or
// 256 MXFP4 codes), in 16-byte chunks:
//   - an operand whose rows run along the sum (a and b of NT, a of NN) as its rows
//     of 8 chunks, chunk c of row r at slot c ^ (r & 7), so that the 16 rows that
//     the lanes of a matrix instruction read at once lie in different banks;
//   - one whose rows run across it (b of NN, a and b of TN) as it comes, 64 rows of
//     BM or BN elements, read back transposed (ds_read_b64_tr_b16: a 16-lane group
//     fetches 4 rows x 16 columns, each lane receiving a column); there chunk c
//     of row k lies at slot c ^ swizzle(k), because those 4 rows would share banks.
// The matrix instructions take b's tile as their first operand: a lane then holds
// four neighbouring columns of one row of out.
#pragma once

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "expert.h"

namespace wt {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

enum Form { kNT = WT_PRODUCT_NT, kNN = WT_PRODUCT_NN, kTN = WT_PRODUCT_TN };

constexpr int kStepBytes = 128;  // of a row along the sum

// ------------------------------------------------------------- activations
// Both are x s(y) with s(y) = 1 / (1 + exp(-y)): SiLU y = x; GELU's
// (1 + tanh(z)) / 2 = s(2 z). With t = exp(-|y|) both s and 1 - s are t / (1 + t) or
// 1 / (1 + t), without a difference that cancels or an exponential that overflows.
// exp2 and the reciprocal are good to a last place of fp32 and exp2's argument to
// 2^-22 |y|, far below the BF16 result's 2^-8.
struct Act {
  float value, slope;
};

__device__ __forceinline__ Act activation(int act, float x) {
  constexpr float kLog2e = 1.44269504f, kC = 1.59576912f;  // 2 sqrt(2 / pi)
  float y = x, dy = 1.0f;
  if (act == WT_ACT_GELU) {
    const float x2 = x * x;
    y = kC * x * (1.0f + 0.044715f * x2);
    dy = kC * (1.0f + 3.0f * 0.044715f * x2);
  }
  const float t = __builtin_amdgcn_exp2f(-kLog2e * fabsf(y)), r = __builtin_amdgcn_rcpf(1.0f + t), q = t * r;
  const float s = y >= 0.0f ? r : q, rest = y >= 0.0f ? q : r;  // a NaN is in both
  Act f;
  // -FLT_MAX times a logistic of 0 is the limit 0, where -infinity would make a NaN
  f.value = fmaxf(x, -FLT_MAX) * s;
  // s (1 - s) is 0 in fp32 long before x dy could overflow
  f.slope = s + s * rest * (fminf(fmaxf(x, -1e4f), 1e4f) * fminf(dy, 1e9f));
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
  const int n = a.counts ? a.counts[e] : a.offsets[e + 1] - lo;
  first = min(max(lo, 0), n_rows);
  // a first row below 0 takes its part of the count along
  const int64_t end = (int64_t)lo + max(n, 0);
  count = (int)max((int64_t)0, min(end, (int64_t)n_rows) - first);
}

__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {  // inclusive, over 64 lanes
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Tile t of the row tiles x column tiles of all experts, or false if there are
// not that many. Workgroups go round the 8 XCDs, each with an L2 of its own: tiles are
// dealt so that an XCD's are neighbours. Within an expert up to kRowGroup row tiles
// take turns under one column tile, so that what the XCD's 32 CUs read at a time are few
// rows of both operands.
constexpr int kXcds = 8, kRowGroup = 8;

template <int BM>
__device__ __forceinline__ bool find_rows(const ProductArgs &a, uint32_t block, uint32_t n_tiles, Rows &r, int &mt, int &nt) {
  const int lane = threadIdx.x & 63, E = a.n_experts;
  uint32_t total = 0;
  int first = 0, count = 0;
  uint32_t mine = 0, scan = 0;
  for (int base = 0; base < E; base += 64) {
    mine = 0;
    if (base + lane < E) {
      expert_rows(a, base + lane, first, count);
      mine = (uint32_t)(count + BM - 1) / BM;
    }
    scan = wave_scan(mine);
    total += __builtin_amdgcn_readlane(scan, 63);
  }
  const uint64_t tiles = (uint64_t)total * n_tiles;
  const uint64_t per = (tiles + kXcds - 1) / kXcds;
  if (block / kXcds >= per) return false;
  const uint64_t t64 = (uint64_t)(block % kXcds) * per + block / kXcds;
  if (t64 >= tiles) return false;
  // the expert that holds row tile t / n_tiles
  const uint32_t at = (uint32_t)(t64 / n_tiles);
  uint32_t before = 0;
  for (int base = 0; base < E; base += 64) {
    if (E > 64) {
      mine = 0;
      if (base + lane < E) {
        expert_rows(a, base + lane, first, count);
        mine = (uint32_t)(count + BM - 1) / BM;
      }
      scan = wave_scan(mine);
    }
    const uint64_t hit = __ballot(at - before < scan && mine > 0);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      r.expert = base + l;
      r.first = __builtin_amdgcn_readlane(first, l);
      r.count = __builtin_amdgcn_readlane(count, l);
      const uint32_t m_tiles = __builtin_amdgcn_readlane(mine, l);
      const uint32_t begin = before + __builtin_amdgcn_readlane(scan, l) - m_tiles;
      const uint32_t u = (uint32_t)(t64 - (uint64_t)begin * n_tiles);  // within the expert
      const uint32_t group = u / (kRowGroup * n_tiles), in = u - group * kRowGroup * n_tiles;
      const uint32_t height = min(m_tiles - group * kRowGroup, (uint32_t)kRowGroup);
      nt = (int)(in / height);
      mt = (int)(group * kRowGroup + in - (uint32_t)nt * height);
      return true;
    }
    before += __builtin_amdgcn_readlane(scan, 63);
  }
  return false;
}

// TN: every expert has m x n tiles, whether it has rows or not.
__device__ __forceinline__ bool find_matrix(const ProductArgs &a, uint32_t block, uint32_t m_tiles, uint32_t n_tiles, Rows &r,
                                            int &mt, int &nt) {
  const uint32_t each = m_tiles * n_tiles, tiles = each * a.n_experts, per = (tiles + kXcds - 1) / kXcds;
  const uint32_t t = block % kXcds * per + block / kXcds;
  if (block / kXcds >= per || t >= tiles) return false;
  r.expert = t / each;
  int first;
  expert_rows(a, r.expert, first, r.count);
  r.first = first;
  const uint32_t u = t - r.expert * each, group = u / (kRowGroup * n_tiles), in = u - group * kRowGroup * n_tiles;
  const uint32_t height = min(m_tiles - group * kRowGroup, (uint32_t)kRowGroup);
  nt = (int)(in / height);
  mt = (int)(group * kRowGroup + in - (uint32_t)nt * height);
  return true;
}

// ------------------------------------------------------------ shared memory
// Rows across the sum: the 4 rows of a 16-lane group, and those of the group
// that reads beside it (8 rows on), in different 32-byte slots.
__device__ __forceinline__ uint32_t swizzle(uint32_t k) { return ((k & 3) | (k >> 3 & 1) << 2) << 1; }

// One operand's tile of a step: N rows of the operand (along the sum) or 64 rows of N elements (across it).
template <int N, bool Across, int Threads>
struct Place {
  static constexpr int kChunks = N * 8;  // 16-byte chunks
  static constexpr int kEach = kChunks / Threads;
  static constexpr int kRow = Across ? N / 8 : 8;  // chunks of a row in shared memory
  static_assert(kChunks % Threads == 0, "chunks per thread");
  static_assert(!Across || N >= 128, "the swizzle spans 16 chunks");
  // Chunk q of the tile holds (row, chunk) of the operand.
  static __device__ __forceinline__ void source(int q, int &row, int &chunk) {
    row = q / kRow;
    chunk = (q % kRow) ^ (int)(Across ? swizzle(row) : row & 7);
  }
};

// Eight BF16 elements of which the first `valid` exist, at any 2-byte address.
__device__ __forceinline__ u32x4 load_chunk(uint64_t p, int64_t valid) {
  u32x4 v = {0, 0, 0, 0};
  const uint16_t *s = (const uint16_t *)(uintptr_t)p;
  if (valid >= 8) {
    __builtin_memcpy(&v, s, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) v[i >> 1] |= (uint32_t)s[i] << (16 * (i & 1));
  }
  return v;
}

// ----------------------------------------------------------------- the tile
template <int Form, Epilogue Epi, bool F4, int BM, int BN, int WM, int WN>
struct Tile {
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr bool kAcrossA = Form == kTN, kAcrossB = Form != kNT;
  static constexpr int kStep = F4 ? 256 : 64;  // elements of the sum
  static constexpr int kTM = BM / WM / 16, kTN_ = BN / WN / 16;
  static constexpr int kColumns = Epi == Epilogue::kGated ? BN / 2 : BN;  // of out (h)
  static constexpr int kLdsA = BM * kStepBytes, kLdsB = BN * kStepBytes;
  static constexpr int kLdsScales = F4 ? (BM + BN) * 8 : 0;
  static constexpr int kLds = kLdsA + kLdsB + kLdsScales;
  using PlaceA = Place<BM, kAcrossA, kThreads>;
  using PlaceB = Place<BN, kAcrossB, kThreads>;

  // Row of b's matrix that row r of the tile holds; the gated forms have gate rows
  // in the lower half and the same columns' up rows in the upper.
  static __device__ __forceinline__ int64_t b_row(const ProductArgs &a, int n0, int r, bool &ok) {
    if (Epi != Epilogue::kGated) {
      ok = n0 + r < a.n;
      return n0 + r;
    }
    const int c = n0 + r % kColumns;
    ok = c < a.n;
    return r < kColumns ? c : (int64_t)a.n + c;
  }

  // First row of b's tile that matrix fragment j of wave column wn covers.
  static __device__ __forceinline__ int b_frag(int wn, int j) {
    if (Epi != Epilogue::kGated) return wn * (BN / WN) + 16 * j;
    constexpr int half = kTN_ / 2;
    return (j < half ? 0 : kColumns) + wn * (kColumns / WN) + 16 * (j % half);
  }
  static __device__ __forceinline__ int out_column(int wn, int j) {  // j < kTN_ / 2 when gated
    return Epi == Epilogue::kGated ? wn * (kColumns / WN) + 16 * j : wn * (BN / WN) + 16 * j;
  }

  // Fragment of an operand whose rows run along the sum: row r0 + lane % 16, chunk
  // kk * 4 + lane / 16 (MXFP4: lane / 16 * 2 + kk, so that a lane's two scales are neighbours).
  static __device__ __forceinline__ u32x4 read_along(const uint8_t *lds, int r0, int kk) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int chunk = (F4 ? g * 2 + kk : kk * 4 + g) ^ (lane & 7);
    return *(const u32x4 *)(lds + (r0 + (lane & 15)) * kStepBytes + chunk * 16);
  }
  // Fragment of one whose rows run across: columns c0 .. c0 + 15, the same places of the sum.
  template <int N>
  static __device__ __forceinline__ u32x4 read_across(const uint8_t *lds, int c0, int kk) {
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    const uint32_t k = kk * 32 + g * 8 + (i >> 2);
    const uint32_t slot = (uint32_t)(c0 / 8 + ((i & 3) >> 1)) ^ swizzle(k);  // swizzle(k + 4) is the same
    const uint8_t *p = lds + k * (2 * N) + slot * 16 + (i & 1) * 8;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * 2 * N));
    u32x4 v;
    __builtin_memcpy(&v, &lo, 8);
    __builtin_memcpy((char *)&v + 8, &hi, 8);
    return v;
  }

  static __device__ __forceinline__ f32x4 multiply(u32x4 b, u32x4 a, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  }
  template <int Kk>
  static __device__ __forceinline__ f32x4 multiply_f4(u32x4 b, u32x4 a, f32x4 c, uint32_t sb, uint32_t sa) {
    const i32x8 vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    const i32x8 va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, c, 4, 4, Kk, (int)sb, Kk, (int)sa);
  }

  // Adds one step to the sums. `blocks`: scale blocks of the row that this step still has (MXFP4).
  static __device__ __forceinline__ void step(const uint8_t *lds, int wm, int wn, int blocks, f32x4 (&acc)[kTM][kTN_]) {
    const uint8_t *la = lds, *lb = lds + kLdsA;
    if constexpr (F4) {
      const int lane = threadIdx.x & 63, g = lane >> 4;
      const uint8_t *sa = lds + kLdsA + kLdsB + (lane & 15) * 8 + g * 2, *sb = sa + BM * 8;
      // scales behind the row's last block may be anything, NaN among it
      const uint32_t keep = 2 * g + 1 < blocks ? 0xFFFFu : 2 * g < blocks ? 0xFFu : 0u;
      uint32_t xa[kTM], xb[kTN_];
#pragma unroll
      for (int i = 0; i < kTM; ++i) xa[i] = *(const uint16_t *)(sa + (wm * (BM / WM) + 16 * i) * 8) & keep;
#pragma unroll
      for (int j = 0; j < kTN_; ++j) xb[j] = *(const uint16_t *)(sb + b_frag(wn, j) * 8) & keep;
      half_f4<0>(la, lb, wm, wn, xa, xb, acc);
      half_f4<1>(la, lb, wm, wn, xa, xb, acc);
    } else {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        u32x4 fa[kTM], fb[kTN_];
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
          const int r0 = wm * (BM / WM) + 16 * i;
          fa[i] = kAcrossA ? read_across<BM>(la, r0, kk) : read_along(la, r0, kk);
        }
#pragma unroll
        for (int j = 0; j < kTN_; ++j) fb[j] = kAcrossB ? read_across<BN>(lb, b_frag(wn, j), kk) : read_along(lb, b_frag(wn, j), kk);
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
          for (int j = 0; j < kTN_; ++j) acc[i][j] = multiply(fb[j], fa[i], acc[i][j]);
      }
    }
  }
  template <int Kk>
  static __device__ __forceinline__ void half_f4(const uint8_t *la, const uint8_t *lb, int wm, int wn, const uint32_t (&xa)[kTM],
                                                 const uint32_t (&xb)[kTN_], f32x4 (&acc)[kTM][kTN_]) {
    u32x4 fa[kTM], fb[kTN_];
#pragma unroll
    for (int i = 0; i < kTM; ++i) fa[i] = read_along(la, wm * (BM / WM) + 16 * i, Kk);
#pragma unroll
    for (int j = 0; j < kTN_; ++j) fb[j] = read_along(lb, b_frag(wn, j), Kk);
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN_; ++j) acc[i][j] = multiply_f4<Kk>(fb[j], fa[i], acc[i][j], xb[j], xa[i]);
  }
};

// ------------------------------------------------------------------ results
__device__ __forceinline__ void store4(uint64_t out, int64_t at, f32x4 v, int n, bool f32, bool wide) {
  if (f32) {
    float *p = (float *)(uintptr_t)out + at;
    if (wide && n >= 4) {
      *(f32x4 *)p = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = v[i];
    }
    return;
  }
  __bf16 *p = (__bf16 *)(uintptr_t)out + at;
  const bf16x4 r = {(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w};
  if (wide && n >= 4) {
    *(bf16x4 *)p = r;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = r[i];
  }
}

__device__ __forceinline__ f32x4 load_pre(uint64_t pre, int64_t at, int n, bool wide) {
  const __bf16 *p = (const __bf16 *)(uintptr_t)pre + at;
  f32x4 v = {0, 0, 0, 0};
  if (wide && n >= 4) {
    const bf16x4 r = *(const bf16x4 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)r[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] = (float)p[i];
  }
  return v;
}

// What becomes of four neighbouring sums of one row: `row` of out, `column` of out (h), n of them exist.
template <Epilogue Epi>
__device__ __forceinline__ void finish4(const ProductArgs &a, uint64_t out, int64_t row, int column, int n, f32x4 s, f32x4 up) {
  const bool wide = a.out_wide;
  if (Epi == Epilogue::kPlain) {
    store4(out, row * a.out_stride + column, s, n, a.out_f32, wide);
  } else if (Epi == Epilogue::kGated) {
    if (a.pre) {
      store4(a.pre, row * a.pre_stride + column, s, n, false, wide);
      store4(a.pre, row * a.pre_stride + a.n + column, up, n, false, wide);
    }
    f32x4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = activation(a.act, s[i]).value * up[i];
    store4(out, row * a.out_stride + column, h, n, false, wide);
  } else {
    const f32x4 g = load_pre(a.pre, row * a.pre_stride + column, n, wide);
    const f32x4 u = load_pre(a.pre, row * a.pre_stride + a.n + column, n, wide);
    f32x4 dg, du;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Act t = activation(a.act, g[i]);
      dg[i] = s[i] * u[i] * t.slope;
      du[i] = s[i] * t.value;
    }
    store4(out, row * a.out_stride + column, dg, n, false, wide);
    store4(out, row * a.out_stride + a.n + column, du, n, false, wide);
  }
}

template <int Form, Epilogue Epi, bool F4, int BM, int BN, int WM, int WN, int TM, int TN>
__device__ __forceinline__ void finish_tile(const ProductArgs &a, const Rows &r, int m0, int n0, int m_left, int wm, int wn,
                                            const f32x4 (&acc)[TM][TN]) {
  using T = Tile<Form, Epi, F4, BM, BN, WM, WN>;
  const int lane = threadIdx.x & 63;
  const uint64_t out = a.out + (Form == kTN ? (uint64_t)(a.out_expert * r.expert) * (a.out_f32 ? 4 : 2) : 0);
  constexpr int kCols = Epi == Epilogue::kGated ? TN / 2 : TN;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = wm * (BM / WM) + 16 * i + (lane & 15);
    if (row >= m_left) continue;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const int column = n0 + T::out_column(wn, j) + 4 * (lane >> 4);
      if (column < a.n)
        finish4<Epi>(a, out, (Form == kTN ? 0 : r.first) + m0 + row, column, a.n - column, acc[i][j],
                     Epi == Epilogue::kGated ? acc[i][j + kCols] : acc[i][j]);
    }
  }
}

// ------------------------------------------------- operands of any alignment
// The next step's chunks are loaded to registers before the present one is
// computed and stored to the other half of shared memory behind it.
template <int Form, Epilogue Epi, bool F4, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN) product_any_kernel(ProductArgs a) {
  using T = Tile<Form, Epi, F4, BM, BN, WM, WN>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][T::kLds];
  Rows r;
  int mt, nt;
  const uint32_t n_tiles = (uint32_t)(a.n + T::kColumns - 1) / T::kColumns;
  const bool mine = Form == kTN ? find_matrix(a, blockIdx.x, (uint32_t)(a.m + BM - 1) / BM, n_tiles, r, mt, nt)
                                : find_rows<BM>(a, blockIdx.x, n_tiles, r, mt, nt);
  if (!mine) return;
  const int tid = threadIdx.x, wave = tid >> 6, wm = wave / WN, wn = wave % WN;
  const int m0 = mt * BM, n0 = nt * T::kColumns;
  const int64_t K = Form == kTN ? r.count : a.k;
  const int m_left = (Form == kTN ? a.m : r.count) - m0;
  const uint64_t b_base = a.b + (Form == kTN ? 0 : (uint64_t)(a.b_expert * r.expert));

  u32x4 ra[T::PlaceA::kEach], rb[T::PlaceB::kEach];
  uint32_t rs[F4 ? 2 : 1] = {};
  auto gathered = [&](int64_t row) -> int64_t {  // a row of the row space to one of the operand, -1: zeros
    if (!a.row_index) return row;
    const int64_t i = a.row_index[row];
    return i >= 0 && i < a.n_index_rows ? i : -1;
  };
  const int64_t f4_row = (int64_t)(a.k + 31) / 32 * 16;  // bytes of codes
  auto load = [&](int64_t k0) {  // k0 in elements
#pragma unroll
    for (int i = 0; i < T::PlaceA::kEach; ++i) {
      int row, chunk;
      T::PlaceA::source(tid + i * T::kThreads, row, chunk);
      ra[i] = u32x4{0, 0, 0, 0};
      if (F4) {
        const int64_t at = k0 / 2 + 16 * chunk;
        if (row < m_left && at < f4_row) ra[i] = *(const u32x4 *)(uintptr_t)(a.a + (uint64_t)((r.first + m0 + row) * a.a_stride + at));
      } else if (T::kAcrossA) {
        if (k0 + row < K)
          ra[i] = load_chunk(a.a + (uint64_t)((r.first + k0 + row) * a.a_stride + 2 * (int64_t)(m0 + 8 * chunk)), m_left - 8 * chunk);
      } else if (row < m_left) {
        const int64_t s = gathered(r.first + m0 + row);
        if (s >= 0) ra[i] = load_chunk(a.a + (uint64_t)(s * a.a_stride + 2 * (k0 + 8 * chunk)), K - k0 - 8 * chunk);
      }
    }
#pragma unroll
    for (int i = 0; i < T::PlaceB::kEach; ++i) {
      int row, chunk;
      T::PlaceB::source(tid + i * T::kThreads, row, chunk);
      rb[i] = u32x4{0, 0, 0, 0};
      if (T::kAcrossB) {
        if (k0 + row < K) {
          const int64_t s = Form == kTN ? gathered(r.first + k0 + row) : k0 + row;
          if (s >= 0) rb[i] = load_chunk(b_base + (uint64_t)(s * a.b_stride + 2 * (int64_t)(n0 + 8 * chunk)), a.n - n0 - 8 * chunk);
        }
      } else {
        bool ok;
        const int64_t s = T::b_row(a, n0, row, ok);
        if (F4) {
          const int64_t at = k0 / 2 + 16 * chunk;
          if (ok && at < f4_row) rb[i] = *(const u32x4 *)(uintptr_t)(b_base + (uint64_t)(s * a.b_stride + at));
        } else if (ok) {
          rb[i] = load_chunk(b_base + (uint64_t)(s * a.b_stride + 2 * (k0 + 8 * chunk)), K - k0 - 8 * chunk);
        }
      }
    }
    if constexpr (F4) {  // the scales of two rows' four blocks
      static_assert(!F4 || (BM + BN) * 2 == 2 * T::kThreads, "two words of scales to a thread");
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int word = tid + i * T::kThreads, row = word >> 1;
        const int64_t at = k0 / 32 + 4 * (word & 1);
        rs[i] = 0;
        if (at >= (a.k + 31) / 32) continue;
        if (row < BM) {
          if (row < m_left) rs[i] = *(const uint32_t *)(uintptr_t)(a.a_scales + (uint64_t)((r.first + m0 + row) * a.a_scale_stride + at));
        } else {
          bool ok;
          const int64_t s = T::b_row(a, n0, row - BM, ok);
          if (ok) rs[i] = *(const uint32_t *)(uintptr_t)(a.b_scales + (uint64_t)(a.b_scale_expert * r.expert + s * a.b_scale_stride + at));
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
      for (int i = 0; i < 2; ++i) *(uint32_t *)(to + T::kLdsA + T::kLdsB + 4 * (tid + i * T::kThreads)) = rs[i];
    }
  };

  f32x4 acc[T::kTM][T::kTN_];
#pragma unroll
  for (int i = 0; i < T::kTM; ++i)
#pragma unroll
    for (int j = 0; j < T::kTN_; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  if (K > 0) {
    load(0);
    store(lds[0]);
    __syncthreads();
    int at = 0;
    for (int64_t k0 = 0; k0 < K; k0 += T::kStep, at ^= 1) {
      const bool more = k0 + T::kStep < K;
      if (more) load(k0 + T::kStep);
      T::step(lds[at], wm, wn, F4 ? (int)((a.k - k0 + 31) / 32) : 0, acc);
      if (more) store(lds[at ^ 1]);
      __syncthreads();
    }
  }

  finish_tile<Form, Epi, F4, BM, BN, WM, WN>(a, r, m0, n0, m_left, wm, wn, acc);
}

// ------------------------------------------------------ aligned operands
// buffer_load ... lds copies 16 bytes a lane straight into shared memory, at
// consecutive places of a wave (from M0 on), so the swizzle is in the addresses that are
// read. What lies outside of [base, base + bytes) reads as 0 and touches no
// memory: rows behind the last, and offsets set to kNowhere.
constexpr uint32_t kNowhere = 0x80000000u;

// The compiler does not count these loads: wait_and_meet() waits for all of them.
__device__ __forceinline__ void copy16(u32x4 buffer, uint32_t lds, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buffer) : "memory");
}
__device__ __forceinline__ void copy4(u32x4 buffer, uint32_t lds, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buffer) : "memory");
}

// What this wave copied has arrived and what it read has been read; then the workgroup meets.
__device__ __forceinline__ void wait_and_meet() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A window over an operand that moves along the sum; everything in it is uniform.
struct Window {
  uint64_t base;
  int64_t bytes;  // from base to the operand's end
  __device__ __forceinline__ u32x4 buffer() const {
    const int64_t n = bytes < 0 ? 0 : bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0;
    u32x4 r;
    r.x = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)base);
    r.y = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32)) & 0xFFFFu;
    r.z = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)n);
    r.w = 0x00020000u;
    return r;
  }
  __device__ __forceinline__ void move(int64_t by) {
    base += (uint64_t)by;
    bytes -= by;
  }
};

template <int Form, Epilogue Epi, bool F4, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, 2) product_kernel(ProductArgs a) {
  using T = Tile<Form, Epi, F4, BM, BN, WM, WN>;
  using PA = typename T::PlaceA;
  using PB = typename T::PlaceB;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][T::kLds];
  Rows r;
  int mt, nt;
  const uint32_t n_tiles = (uint32_t)(a.n + T::kColumns - 1) / T::kColumns;
  const bool mine = Form == kTN ? find_matrix(a, blockIdx.x, (uint32_t)(a.m + BM - 1) / BM, n_tiles, r, mt, nt)
                                : find_rows<BM>(a, blockIdx.x, n_tiles, r, mt, nt);
  if (!mine) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
  const int m0 = mt * BM, n0 = nt * T::kColumns;
  const int m_left = (Form == kTN ? a.m : r.count) - m0;
  // bytes of a row along the sum, or rows across it
  const int64_t row_bytes = F4 ? (int64_t)(a.k + 31) / 32 * 16 : 2 * (int64_t)a.k;
  const int64_t K = Form == kTN ? r.count : a.k;
  const int steps = (int)((K + T::kStep - 1) / T::kStep);

  Window wa, wb;
  uint32_t oa[PA::kEach], ob[PB::kEach];
  auto index_of = [&](int64_t row) -> uint32_t {  // of the gathered operand, kNowhere if there is none
    const int64_t i = a.row_index[row];
    return i >= 0 && i < a.n_index_rows ? (uint32_t)i : kNowhere;
  };
  const bool gather_a = Form != kTN && !F4 && a.row_index, gather_b = Form == kTN && a.row_index;
  if (T::kAcrossA) {
    wa = {a.a + (uint64_t)(r.first * a.a_stride + 2 * (int64_t)m0), (K - 1) * a.a_stride + 2 * (int64_t)(a.m - m0)};
  } else if (gather_a) {
    wa = {a.a, (a.n_index_rows - 1) * a.a_stride + row_bytes};
  } else {
    wa = {a.a + (uint64_t)((r.first + m0) * a.a_stride), (int64_t)(m_left - 1) * a.a_stride + row_bytes};
  }
#pragma unroll
  for (int i = 0; i < PA::kEach; ++i) {
    int row, chunk;
    PA::source(tid + i * T::kThreads, row, chunk);
    uint32_t at = (uint32_t)row;
    if (gather_a) at = row < m_left ? index_of(r.first + m0 + row) : kNowhere;
    oa[i] = at == kNowhere ? kNowhere : at * (uint32_t)a.a_stride + 16u * chunk;
  }
  const uint64_t b_base = a.b + (Form == kTN ? 0 : (uint64_t)(a.b_expert * r.expert));
  if (T::kAcrossB) {
    const int64_t rows = gather_b ? a.n_index_rows : K;
    wb = {b_base + (uint64_t)((Form == kTN && !gather_b ? r.first * a.b_stride : 0) + 2 * (int64_t)n0),
          (rows - 1) * a.b_stride + 2 * (int64_t)(a.n - n0)};
  } else {
    const int64_t rows = Epi == Epilogue::kGated ? 2 * (int64_t)a.n : a.n;
    wb = {b_base + (uint64_t)(n0 * a.b_stride), (rows - n0 - 1) * a.b_stride + row_bytes};
  }
#pragma unroll
  for (int i = 0; i < PB::kEach; ++i) {
    int row, chunk;
    PB::source(tid + i * T::kThreads, row, chunk);
    if (Epi == Epilogue::kGated && row >= T::kColumns) row += a.n - T::kColumns;  // up rows
    ob[i] = (uint32_t)row * (uint32_t)a.b_stride + 16u * chunk;
  }
  uint32_t next_row[PB::kEach];  // of b, gathered: one step ahead
  auto load_rows = [&](int step) {
#pragma unroll
    for (int i = 0; i < PB::kEach; ++i) {
      int row, chunk;
      PB::source(tid + i * T::kThreads, row, chunk);
      const int64_t k = (int64_t)step * T::kStep + row;
      next_row[i] = k < K ? index_of(r.first + k) : kNowhere;
    }
  };
  if (gather_b && steps > 0) load_rows(0);

  Window sa{}, sb{};
  uint32_t osa = 0, osb = 0;
  static_assert(!F4 || (BM * 2 == T::kThreads && BN * 2 == T::kThreads), "one word of scales to a thread");
  if (F4) {
    const int64_t nb = (a.k + 31) / 32, words = (nb + 3) / 4 * 4;
    sa = {a.a_scales + (uint64_t)((r.first + m0) * a.a_scale_stride), (int64_t)(m_left - 1) * a.a_scale_stride + words};
    const int64_t rows = Epi == Epilogue::kGated ? 2 * (int64_t)a.n : a.n;
    sb = {a.b_scales + (uint64_t)(a.b_scale_expert * r.expert + n0 * a.b_scale_stride), (rows - n0 - 1) * a.b_scale_stride + words};
    int row = tid >> 1;
    osa = (uint32_t)row * (uint32_t)a.a_scale_stride + 4u * (tid & 1);
    if (Epi == Epilogue::kGated && row >= T::kColumns) row += a.n - T::kColumns;
    osb = (uint32_t)row * (uint32_t)a.b_scale_stride + 4u * (tid & 1);
  }

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&lds[0][0] + 1024u * wave;
  auto fetch = [&](int step) {
    const uint32_t to = lds0 + (step & 1) * T::kLds;
    const u32x4 ba = wa.buffer(), bb = wb.buffer();
    // the row's end lies within the last step: chunks behind it are not the next row's
    const int64_t left = row_bytes - (int64_t)step * kStepBytes;
    const bool cut = left < kStepBytes;
#pragma unroll
    for (int i = 0; i < PA::kEach; ++i) {
      uint32_t at = oa[i];
      if (!T::kAcrossA && cut) {
        int row, chunk;
        PA::source(tid + i * T::kThreads, row, chunk);
        at = 16 * chunk < left ? at : kNowhere;
      }
      copy16(ba, to + i * T::kThreads * 16, at);
    }
#pragma unroll
    for (int i = 0; i < PB::kEach; ++i) {
      uint32_t at = ob[i];
      int row, chunk;
      PB::source(tid + i * T::kThreads, row, chunk);
      if (!T::kAcrossB && cut) at = 16 * chunk < left ? at : kNowhere;
      if (gather_b) at = next_row[i] == kNowhere ? kNowhere : next_row[i] * (uint32_t)a.b_stride + 16u * chunk;
      copy16(bb, to + T::kLdsA + i * T::kThreads * 16, at);
    }
    wa.move(T::kAcrossA ? 64 * a.a_stride : kStepBytes);
    if (!gather_b) wb.move(T::kAcrossB ? 64 * a.b_stride : kStepBytes);
    if (F4) {
      const uint32_t scales = to - 1024u * wave + T::kLdsA + T::kLdsB + 256u * wave;
      copy4(sa.buffer(), scales, osa);
      copy4(sb.buffer(), scales + BM * 8, osb);
      sa.move(8);
      sb.move(8);
    }
    if (gather_b && step + 1 < steps) load_rows(step + 1);
  };

  f32x4 acc[T::kTM][T::kTN_];
#pragma unroll
  for (int i = 0; i < T::kTM; ++i)
#pragma unroll
    for (int j = 0; j < T::kTN_; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  if (steps > 0) fetch(0);
  for (int step = 0; step < steps; ++step) {
    // this step's operands are there, and nobody reads the other half any more
    wait_and_meet();
    if (step + 1 < steps) fetch(step + 1);
    T::step(lds[step & 1], wm, wn, F4 ? (a.k + 31) / 32 - 8 * step : 0, acc);
  }
  finish_tile<Form, Epi, F4, BM, BN, WM, WN>(a, r, m0, n0, m_left, wm, wn, acc);
}

// Row tiles that n_rows rows of n_experts experts can make.
inline int64_t most_row_tiles(const ProductArgs &a, int bm) {
  const int64_t experts = a.offsets ? a.n_experts : 1;
  const int64_t some = a.n_rows < experts ? a.n_rows : experts;  // with rows
  return (a.n_rows - some) / bm + some;
}

}  // namespace wt
