// adamw.hip -- the AdamW step over many parameter shards: gradient norm and
// update kernels for gfx950, and the entry points that run them. The
// definition (formulas, rounding of 8-bit states, random bits) is in wt.h.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <new>
#include <string>

#include "adamw.h"
#include "fp8_math.h"
#include "hip_util.h"
#include "plan.h"
#include "wave.h"
#include "wt.h"

namespace wt {
namespace {

constexpr int kThreads = 256;  // of the norm kernel

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A step reads and writes each byte once: streaming (non-temporal) accesses.
// Measured on MI355X over 176 M elements, plain / loads / stores / both: 32-bit
// states 930 / 916 / 929 / 888 us, 8-bit 510 / 522 / 501 / 492 us.
template <class T>
__device__ __forceinline__ T ld_stream(uint64_t a) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_nontemporal_load((gcptr<T>)(uintptr_t)a);
#else
  return ld_global<T>(a);
#endif
}
template <class T>
__device__ __forceinline__ void st_stream(uint64_t a, T v) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_nontemporal_store(v, (gptr<T>)(uintptr_t)a);
#else
  st_global<T>(a, v);
#endif
}

// ------------------------------------------------------------ scalars
__host__ __device__ inline double int_pow(double b, int64_t t) {
  double r = 1.0;
  for (uint64_t k = (uint64_t)t; k; k >>= 1) {
    if (k & 1) r *= b;
    b *= b;
  }
  return r;
}

__host__ __device__ inline AdamScalars step_scalars(double lr, double beta1, double beta2, double eps, int64_t step,
                                                    uint64_t seed) {
  AdamScalars s;
  const int64_t t = step < 1 ? 1 : step;
  s.lr = (float)lr;
  s.lr_bias1 = (float)(lr / (1.0 - int_pow(beta1, t)));
  s.b1 = (float)beta1;
  s.ib1 = (float)(1.0 - beta1);
  s.b2 = (float)beta2;
  s.ib2 = (float)(1.0 - beta2);
  s.inv_bias2 = (float)(1.0 / sqrt(1.0 - int_pow(beta2, t)));
  s.eps = (float)eps;
  uint64_t z = seed + (uint64_t)t * 0x9E3779B97F4A7C15ull;
  z ^= z >> 32;
  z *= 0x6A09E667F3BCC909ull;
  z ^= z >> 29;
  z *= 0xBB67AE8584CAA73Bull;
  z ^= z >> 32;
  s.k0 = (uint32_t)z;
  s.k1 = (uint32_t)(z >> 32);
  return s;
}

struct AdamArgs {
  const AdamTensor *tensors;
  const AdamItem *items;
  const AdamNorm *norm;     // null: no norm was computed
  const int64_t *step_dev;  // null: `s` holds the step's scalars
  const float *lr_dev;
  double lr, beta1, beta2, eps;
  int64_t step;
  uint64_t seed;
  AdamScalars s;
  float grad_scale;
};

// ------------------------------------------------------------ random bits
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// Random word of element j of a block whose key is mix32(block ^ k0) + k1.
__device__ __forceinline__ uint32_t random_word(uint32_t key, uint32_t j) { return mix32(key + j * 0x9E3779B9u); }

// ------------------------------------------------------------ element access
// Four elements at index i of an array, of which those below `left` exist
// (left >= 4 when Full). Vector: the array's chunks start at the alignment of
// one access.
template <bool Full>
__device__ __forceinline__ void load_f32(uint64_t a, int64_t i, int64_t left, bool vec, float x[4]) {
  a += 4ull * (uint64_t)i;
  if (Full || (vec && left >= 4)) {
    const u32x4 v = ld_stream<u32x4>(a);
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = e < left ? ld_global<float>(a + 4 * e) : 0.0f;
}

template <bool Full>
__device__ __forceinline__ void store_f32(uint64_t a, int64_t i, int64_t left, bool vec, const float x[4]) {
  a += 4ull * (uint64_t)i;
  if (Full || (vec && left >= 4)) {
    const u32x4 v = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    st_stream<u32x4>(a, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) st_global<float>(a + 4 * e, x[e]);
}

template <bool Full>
__device__ __forceinline__ void load_bf16(uint64_t a, int64_t i, int64_t left, bool vec, float x[4]) {
  a += 2ull * (uint64_t)i;
  if (Full || (vec && left >= 4)) {
    const u32x2 v = ld_stream<u32x2>(a);
    x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = e < left ? bf16_lo(ld_global<uint16_t>(a + 2 * e)) : 0.0f;
}

template <bool Full>
__device__ __forceinline__ void store_bf16(uint64_t a, int64_t i, int64_t left, bool vec, const uint32_t h[4]) {
  a += 2ull * (uint64_t)i;
  if (Full || (vec && left >= 4)) {
    const u32x2 v = {h[0] | h[1] << 16, h[2] | h[3] << 16};
    st_stream<u32x2>(a, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) st_global<uint16_t>(a + 2 * e, (uint16_t)h[e]);
}

template <bool Full>
__device__ __forceinline__ uint32_t load_codes(uint64_t a, int64_t i, int64_t left, bool vec) {
  a += (uint64_t)i;
  if (Full || (vec && left >= 4)) return ld_stream<uint32_t>(a);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) w |= (uint32_t)ld_global<uint8_t>(a + e) << (8 * e);
  return w;
}

template <bool Full>
__device__ __forceinline__ void store_codes(uint64_t a, int64_t i, int64_t left, bool vec, uint32_t w) {
  a += (uint64_t)i;
  if (Full || (vec && left >= 4)) {
    st_stream<uint32_t>(a, w);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) st_global<uint8_t>(a + e, (uint8_t)(w >> (8 * e)));
}

__device__ __forceinline__ void decode4(uint32_t w, float scale, float x[4]) {
  x[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0) * scale;
  x[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * scale;
  x[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * scale;
  x[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * scale;
}

__device__ __forceinline__ uint32_t bf16_nearest(float x) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}

// fp32 -> BF16, the magnitude rounded up where the 16 dropped bits plus the
// random ones reach a whole step. An infinity has no bits to carry; a NaN gives
// up its payload, which could.
__device__ __forceinline__ uint32_t bf16_random(float x, uint32_t r16) {
  return ((x == x ? __float_as_uint(x) : 0x7FC00000u) + r16) >> 16;
}

constexpr uint32_t kFiniteEnd = 0x7F800000u;  // magnitude bits from here up: infinity, NaN
constexpr float kTinyAmax = 0x1p-100f;        // below: the block is held as zeros

// Square root, correctly rounded for x in [2^-100, 2^127) (equal to sqrtf on
// every mantissa of two binades, tests compare the states it makes bit for
// bit), one bit off at most below; NaN for 0 and for subnormal x, which the
// caller's slow path takes. Five instructions against sqrtf's seventeen.
__device__ __forceinline__ float fast_sqrt(float x) {
  const float y = __builtin_amdgcn_rsqf(x);
  const float g = x * y;
  return fmaf(fmaf(-g, g, x), 0.5f * y, g);
}

// Magnitude bits from which a block takes the slow path: 2^125 and more
// (448 / amax is near the end of the normal range), infinity, NaN.
constexpr uint32_t kPlainEnd = 0x7E000000u;

// Scale of a block, amax / 448, and the factor x -> code units, 448 / amax,
// both correctly rounded: an approximate reciprocal (exact for the constant)
// and its residual, after Markstein. Equal to IEEE division on every mantissa
// for amax in [2^-100, 2^125).
__device__ __forceinline__ void state_scale(uint32_t amax_bits, float *scale, float *inv) {
  const float a = __uint_as_float(amax_bits);
  const bool live = a >= kTinyAmax;
  constexpr float r448 = 1.0f / 448.0f;
  const float s0 = a * r448;
  const float s = fmaf(fmaf(-s0, 448.0f, a), r448, s0);
  float r = __builtin_amdgcn_rcpf(a);
  r = fmaf(fmaf(-a, r, 1.0f), r, r);
  const float i0 = 448.0f * r;
  const float i = fmaf(fmaf(-i0, a, 448.0f), r, i0);
  *scale = live ? s : 1.0f;
  *inv = live ? i : 0.0f;
}

__device__ __forceinline__ void state_scale_slow(uint32_t amax_bits, float *scale, float *inv) {
  const float a = __uint_as_float(amax_bits);
  const bool live = a >= kTinyAmax;
  *scale = live ? a / 448.0f : 1.0f;
  *inv = live ? 448.0f / a : 0.0f;
}

// Four values as E4M3 codes: |x| inv + rho rounded down in units of the
// format. v_cvt_sr_fp8_f32 adds the top 20 bits of its random operand below
// the kept mantissa bits and cuts, subnormal codes included (equal to the
// definition on 4.2 M random values over the whole range). It does not
// saturate, and need not: |x| inv exceeds 448 by two roundings at most, two
// units of those 20 bits, and with 16 random bits the sum stays below the
// next code. Root: a positive root never rounds to zero.
template <bool Root, bool Slow>
__device__ __forceinline__ uint32_t encode4(const float x[4], float inv, const uint32_t w[4]) {
  int q = 0;
  float y[4];
  uint32_t bad = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = x[e] * inv;
    if (Root && (!Slow || (x[e] > 0.0f && inv > 0.0f))) y[e] = fmaxf(y[e], 0x1p-9f);
    if (Slow && (__float_as_uint(x[e]) & 0x7FFFFFFFu) >= kFiniteEnd) bad |= 0xFFu << (8 * e);
  }
#define WT_RND(e) (int)(Root ? w[e] & 0xFFFF0000u : w[e] << 16)
  q = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], WT_RND(0), q, 0);
  q = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], WT_RND(1), q, 1);
  q = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], WT_RND(2), q, 2);
  q = __builtin_amdgcn_cvt_sr_fp8_f32(y[3], WT_RND(3), q, 3);
#undef WT_RND
  return ((uint32_t)q & ~bad) | (bad & 0x7F7F7F7Fu);
}

__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  return b < kFiniteEnd ? b : 0u;
}

// b x + ib y, each product and the sum rounded by itself (no fused multiply
// and add): what the stored states are made of is the same, bit for bit, as
// separate fp32 operations in any program give. A moment that came out one
// bit off would now and then round to the other code, and a code that heads
// its block moves the block's next scale by a whole step.
__device__ __forceinline__ float blend(float b, float x, float ib, float y) {
#pragma clang fp contract(off)
  const float p = b * x, q = ib * y;
  return p + q;
}

// ------------------------------------------------------------ update
// One item, eight elements to a thread. Sixteen lanes share a 128-element
// block, lane l owning its 4-element chunks l and l + 16, so each access of a
// wave covers consecutive bytes (fp32 256, BF16 128, codes 64 per block) and
// the block's amax is a DPP max over a row of 16 lanes.
//
// Bound by HBM: 28 bytes an element with 32-bit states, a master and BF16
// gradients, 16.1 with 8-bit ones. Measured on MI355X over 176 M elements:
// 0.84 ms (5.86 TB/s) and 0.47-0.48 ms (6.0 TB/s), where a prepare kernel that
// reads and writes as much reaches 6.2 TB/s. With 8 bits some 55 vector
// instructions an element run beside it (the roots and quotients of the first
// version, 80 of them, held it at 5.2 TB/s), which is why rare values (zeros,
// infinities, NaN) take a path of their own.
template <int Bits, bool Full>
__device__ __forceinline__ void update_item(const AdamTensor &t, uint32_t chunk, const AdamScalars &s, float gs) {
  const uint32_t tid = threadIdx.x, l = tid & 15;
  const bool vec = t.flags & kAdamVector;
  const bool gbf = t.flags & kAdamGradBf16, has_master = t.flags & kAdamMaster, has_param = t.flags & kAdamParam;
  const float decay = fmaf(-(s.lr * t.lr_mul), t.weight_decay, 1.0f);
  const float rate = s.lr_bias1 * t.lr_mul;
  const uint32_t b = chunk * (adam_item(Bits) / kAdamBlock) + (tid >> 4);
  const int64_t i0 = (int64_t)b * kAdamBlock + 4 * l;
  float g[8], p[8], m[8], v[8], sm = 1.0f, sv = 1.0f;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int64_t i = i0 + 64 * c, left = t.n - i;
    if (gbf) load_bf16<Full>(t.grad, i, left, vec, g + 4 * c);
    else load_f32<Full>(t.grad, i, left, vec, g + 4 * c);
    if (has_master) load_f32<Full>(t.master, i, left, vec, p + 4 * c);
    else load_bf16<Full>(t.param, i, left, vec, p + 4 * c);
    if (Bits == 32) {
      load_f32<Full>(t.m, i, left, vec, m + 4 * c);
      load_f32<Full>(t.v, i, left, vec, v + 4 * c);
    }
  }
  if (Bits == 8) {
    if (Full || (int64_t)b * kAdamBlock < t.n) {
      sm = ld_global<float>(t.m_scale + 4ull * b);
      sv = ld_global<float>(t.v_scale + 4ull * b);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t i = i0 + 64 * c, left = t.n - i;
      decode4(load_codes<Full>(t.m, i, left, vec), sm, m + 4 * c);
      decode4(load_codes<Full>(t.v, i, left, vec), sv, v + 4 * c);
    }
  }
  // moments and the root of the second
  float root[8];
  uint32_t am = 0, av = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = g[e] * gs;
    m[e] = blend(s.b1, m[e], s.ib1, x);
    if (Bits == 8) v[e] *= v[e];
    v[e] = blend(s.b2, v[e], s.ib2, x * x);
    root[e] = Bits == 8 ? fast_sqrt(v[e]) : sqrtf(v[e]);
    if (Bits == 8) {
      am = max(am, __float_as_uint(m[e]) & 0x7FFFFFFFu);
      av = max(av, __float_as_uint(root[e]));  // no sign, unless it is a NaN's
    }
  }
  // some lane of the wave has a zero or subnormal v, a huge value, an infinity or NaN
  const bool slow = Bits == 8 && __any(max(am, av) >= kPlainEnd);
  if (slow) {
    am = av = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      root[e] = sqrtf(v[e]);
      am = max(am, finite_bits(m[e]));
      av = max(av, finite_bits(root[e]));
    }
  }
  if (Bits == 32) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      store_f32<Full>(t.m, i0 + 64 * c, t.n - i0 - 64 * c, vec, m + 4 * c);
      store_f32<Full>(t.v, i0 + 64 * c, t.n - i0 - 64 * c, vec, v + 4 * c);
    }
  }
  const uint32_t key = Bits == 8 || !has_master ? mix32((t.block0 + b) ^ s.k0) + s.k1 : 0u;
  // parameters; 1 / d by v_rcp_f32 (one bit): d lies in the normal range, and what the update is off by is far
  // below a rounding of p
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float u = m[e] * __builtin_amdgcn_rcpf(fmaf(root[e], s.inv_bias2, s.eps));
    p[e] = fmaf(-rate, u, p[e] * decay);
  }
  uint32_t h[8];
  if (has_master) {
#pragma unroll
    for (int c = 0; c < 2; ++c) store_f32<Full>(t.master, i0 + 64 * c, t.n - i0 - 64 * c, vec, p + 4 * c);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = bf16_nearest(p[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      h[e] = bf16_random(p[e], (random_word(key, 4 * l + 64 * (e >> 2) + (e & 3)) * 0x9E3779B9u) >> 16);
  }
  if (has_param) {
#pragma unroll
    for (int c = 0; c < 2; ++c) store_bf16<Full>(t.param, i0 + 64 * c, t.n - i0 - 64 * c, vec, h + 4 * c);
  }
  if (Bits == 8) {
    float im, iv;
    am = lanes_max<16>(am);  // every lane of the row takes part
    av = lanes_max<16>(av);
    if (!slow) {
      state_scale(am, &sm, &im);
      state_scale(av, &sv, &iv);
    } else {
      state_scale_slow(am, &sm, &im);
      state_scale_slow(av, &sv, &iv);
    }
    if (l == 0 && (Full || (int64_t)b * kAdamBlock < t.n)) {
      st_global<float>(t.m_scale + 4ull * b, sm);
      st_global<float>(t.v_scale + 4ull * b, sv);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t i = i0 + 64 * c, left = t.n - i;
      uint32_t w[4], cm, cv;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = random_word(key, 4 * l + 64 * c + e);
      if (!slow) {
        cm = encode4<false, false>(m + 4 * c, im, w);
        cv = encode4<true, false>(root + 4 * c, iv, w);
      } else {
        cm = encode4<false, true>(m + 4 * c, im, w);
        cv = encode4<true, true>(root + 4 * c, iv, w);
      }
      store_codes<Full>(t.m, i, left, vec, cm);
      store_codes<Full>(t.v, i, left, vec, cv);
    }
  }
}

template <int Bits>
__global__ void __launch_bounds__(adam_item(Bits) / 8) adamw_update_kernel(AdamArgs a) {
  const AdamItem item = ld_table(a.items, blockIdx.x);
  const AdamTensor t = ld_table(a.tensors, item.tensor);
  float gs = a.grad_scale;
  if (a.norm) {
    if (a.norm->skip) return;
    gs *= a.norm->clip;
  }
  AdamScalars s = a.s;
  // two powers, a root and two quotients in fp64 in every thread, replayed from a graph: 96 vectors of 896 elements 4.6
  // -> 5.6 us (32-bit states) and 5.5 -> 6.4 us (8-bit), 17 M elements 56.8 -> 57.9 and 34.9 -> 36.1 us; nothing that
  // shows over 176 M
  if (a.step_dev || a.lr_dev)
    s = step_scalars(a.lr_dev ? (double)*a.lr_dev : a.lr, a.beta1, a.beta2, a.eps, a.step_dev ? *a.step_dev : a.step,
                     a.seed);
  if ((t.flags & kAdamVector) && ((int64_t)item.chunk + 1) * adam_item(Bits) <= t.n)
    update_item<Bits, true>(t, item.chunk, s, gs);
  else
    update_item<Bits, false>(t, item.chunk, s, gs);
}

// ------------------------------------------------------------ norm
template <int Item, bool Full>
__device__ __forceinline__ double item_squares(const AdamGradItem &t) {
  const bool vec = t.flags & kAdamVector, gbf = t.flags & kAdamGradBf16;
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < Item / (4 * kThreads); ++c) {
    const int64_t i = 4 * (c * kThreads + (int)threadIdx.x), left = (int64_t)t.count - i;
    float g[4];
    if (gbf) load_bf16<Full>(t.grad, i, left, vec, g);
    else load_f32<Full>(t.grad, i, left, vec, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += (double)(g[e] * g[e]);
  }
  return sum;
}

__device__ __forceinline__ double block_sum(double x, double *lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Sum of the squares of every gradient, per workgroup: each square in fp32, all
// sums in fp64 (fp32 sums of a thread's 8 or 16 squares would be infinite from
// gradients of 4.6e18 on, where a square is up to 1.8e19).
template <int Item>
__global__ void __launch_bounds__(kThreads)
    adamw_norm_kernel(const AdamGradItem *items, uint32_t n_items, double *partials) {
  __shared__ double lds[4];
  double sum = 0.0;
  AdamGradItem next = blockIdx.x < n_items ? ld_table(items, blockIdx.x) : AdamGradItem{0, 0, 0};
  for (uint32_t k = blockIdx.x; k < n_items; k += gridDim.x) {
    const AdamGradItem t = next;
    if (k + gridDim.x < n_items) next = ld_table(items, k + gridDim.x);
    const bool full = (t.flags & kAdamVector) && t.count == Item;
    sum += full ? item_squares<Item, true>(t) : item_squares<Item, false>(t);
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) partials[blockIdx.x] = sum;
}

// The norm and what follows from it, from the workgroups' sums in a fixed
// order. A launch of its own costs 4 us; having the norm kernel's last
// workgroup do it cost 27 us (1024 workgroups) to 45 us (2048), whether they
// counted on one counter or on one per 64: each one's release writes back
// its XCD's L2.
__global__ void __launch_bounds__(kThreads)
    adamw_clip_kernel(const double *partials, uint32_t n, AdamNorm *norm, float grad_scale, double max_norm,
                      float *norm_out) {
  __shared__ double lds[4];
  double x[kAdamNormGrid / kThreads], sum = 0.0;
#pragma unroll
  for (uint32_t k = 0; k < kAdamNormGrid / kThreads; ++k)
    x[k] = k * kThreads + threadIdx.x < n ? partials[k * kThreads + threadIdx.x] : 0.0;
#pragma unroll
  for (uint32_t k = 0; k < kAdamNormGrid / kThreads; ++k) sum += x[k];
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) {
    const double r = sqrt(sum) * fabs((double)grad_scale);
    double clip = 1.0;
    if (max_norm > 0.0 && max_norm < r + 1e-6) clip = max_norm / (r + 1e-6);
    norm->clip = (float)clip;
    norm->skip = r <= 3.4028234663852886e38 ? 0u : 1u;  // false for NaN
    if (norm_out) *norm_out = (float)r;
  }
}

}  // namespace
}  // namespace wt

using namespace wt;

struct wt_adamw {
  AdamLayout L;
  AdamOffsets at{};
  int device = 0;
  uint8_t *mem = nullptr;
  std::atomic<bool> busy{false};
};

namespace {

wt_status fail(const std::string &m, wt_status st) {
  set_thread_error("wt_adamw: " + m);
  return st;
}

wt_status check_tensors(const wt_adamw_tensor *t, size_t n, bool s8, int device, std::string *err) {
  for (size_t i = 0; i < n; ++i) {
    if (t[i].n == 0) continue;
    const uint64_t e = (uint64_t)t[i].n, nb = (e + kAdamBlock - 1) / kAdamBlock;
    const struct {
      const void *p;
      uint64_t bytes;
      const char *what;
    } parts[] = {{t[i].param, 2 * e, "param"},
                 {t[i].master, 4 * e, "master"},
                 {t[i].grad, (t[i].grad_dtype == WT_DT_BF16 ? 2 : 4) * e, "grad"},
                 {t[i].m, (s8 ? 1 : 4) * e, "m"},
                 {t[i].v, (s8 ? 1 : 4) * e, "v"},
                 {s8 ? t[i].m_scale : nullptr, 4 * nb, "m_scale"},
                 {s8 ? t[i].v_scale : nullptr, 4 * nb, "v_scale"}};
    for (const auto &q : parts) {
      if (!q.p) continue;
      const wt_status st = check_memory(q.p, q.bytes, WT_MEM_DEVICE, device,
                                        "tensor " + std::to_string(i) + ": " + q.what, err);
      if (st != WT_OK) return st;
    }
  }
  return WT_OK;
}

wt_status create_impl(const wt_adamw_tensor *tensors, size_t n, const wt_adamw_options &o, wt_adamw *a) {
  std::string err;
  wt_status st = build_adamw(tensors, n, o, &a->L, &err);
  if (st != WT_OK) return fail(err, st);
  int count = 0, dev = o.device;
  hipError_t e = hipGetDeviceCount(&count);
  if (e == hipSuccess && dev < 0) e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(hip_msg("device query", e), WT_E_HIP);
  if (dev >= count) return fail("no such device", WT_E_INVAL);
  a->device = dev;
  DeviceGuard guard(dev);
  st = check_tensors(tensors, n, o.state_bits == 8, dev, &err);
  if (st != WT_OK) return fail(err, st);
  a->at = adamw_offsets(a->L);
  e = hipMalloc((void **)&a->mem, a->at.bytes);
  if (e == hipErrorOutOfMemory) {
    (void)hipGetLastError();
    return fail("device allocation failed", WT_E_NOMEM);
  }
  if (e == hipSuccess) e = hipMemset(a->mem, 0, a->at.bytes);
  if (e == hipSuccess && !a->L.tensors.empty())
    e = hipMemcpy(a->mem + a->at.tensors, a->L.tensors.data(), a->L.tensors.size() * sizeof(AdamTensor),
                  hipMemcpyHostToDevice);
  if (e == hipSuccess && !a->L.items.empty())
    e = hipMemcpy(a->mem + a->at.items, a->L.items.data(), a->L.items.size() * sizeof(AdamItem),
                  hipMemcpyHostToDevice);
  if (e == hipSuccess && !a->L.grads.empty())
    e = hipMemcpy(a->mem + a->at.grads, a->L.grads.data(), a->L.grads.size() * sizeof(AdamGradItem),
                  hipMemcpyHostToDevice);
  if (e == hipSuccess) e = hipDeviceSynchronize();  // the tables are there before a step on any stream
  if (e != hipSuccess) return fail(hip_msg("device tables", e), WT_E_HIP);
  // the launch needs only their numbers from here on
  std::vector<AdamItem>().swap(a->L.items);
  std::vector<AdamGradItem>().swap(a->L.grads);
  return WT_OK;
}

wt_status step_impl(wt_adamw *a, const wt_adamw_hyper *h, hipStream_t stream) {
  std::string err;
  wt_status st = check_adamw_hyper(h, &err);
  if (st != WT_OK) return fail(err, st);
  DeviceGuard guard(a->device);
  const uint32_t n_items = (uint32_t)a->L.info.n_items;
  AdamArgs k{};
  k.tensors = (const AdamTensor *)(a->mem + a->at.tensors);
  k.items = (const AdamItem *)(a->mem + a->at.items);
  k.step_dev = h->step_dev;
  k.lr_dev = h->lr_dev;
  k.lr = h->lr;
  k.beta1 = h->beta1;
  k.beta2 = h->beta2;
  k.eps = h->eps;
  k.step = h->step;
  k.seed = h->seed;
  k.s = step_scalars(h->lr, h->beta1, h->beta2, h->eps, h->step, h->seed);
  k.grad_scale = (float)h->grad_scale;
  if (h->max_norm > 0 || h->norm_out) {
    AdamNorm *norm = (AdamNorm *)(a->mem + a->at.norm);
    const uint32_t grid = n_items < 1 ? 1 : n_items < kAdamNormGrid ? n_items : kAdamNormGrid;
    const auto kernel = a->L.state_bits == 8 ? adamw_norm_kernel<adam_item(8)> : adamw_norm_kernel<adam_item(32)>;
    double *partials = (double *)(a->mem + a->at.partials);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, stream, (const AdamGradItem *)(a->mem + a->at.grads),
                       n_items, partials);
    hipLaunchKernelGGL(adamw_clip_kernel, dim3(1), dim3(kThreads), 0, stream, partials, grid, norm, k.grad_scale,
                       h->max_norm, h->norm_out);
    k.norm = norm;
  }
  if (n_items > 0) {
    if (a->L.state_bits == 8)
      hipLaunchKernelGGL((adamw_update_kernel<8>), dim3(n_items), dim3(adam_item(8) / 8), 0, stream, k);
    else
      hipLaunchKernelGGL((adamw_update_kernel<32>), dim3(n_items), dim3(adam_item(32) / 8), 0, stream, k);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(hip_msg("launch", e), WT_E_HIP);
  return WT_OK;
}

void free_adamw(wt_adamw *a) {
  if (a->mem) {
    DeviceGuard guard(a->device);
    (void)hipDeviceSynchronize();
    (void)hipFree(a->mem);
  }
  delete a;
}

}  // namespace

extern "C" {

wt_status wt_adamw_create(const wt_adamw_tensor *tensors, size_t n_tensors, const wt_adamw_options *opts,
                          wt_adamw **out) {
  if (!out) return WT_E_INVAL;
  *out = nullptr;
  wt_adamw *a = nullptr;
  wt_status st;
  try {
    a = new wt_adamw();
    st = create_impl(tensors, n_tensors, resolve_adamw_opts(opts), a);
  } catch (...) {
    st = caught_status();
  }
  if (st == WT_OK)
    *out = a;
  else if (a)
    free_adamw(a);
  return st;
}

wt_status wt_adamw_step(wt_adamw *adamw, const wt_adamw_hyper *hyper, void *stream) {
  if (!adamw) return WT_E_INVAL;
  bool expected = false;
  if (!adamw->busy.compare_exchange_strong(expected, true)) {
    set_thread_error("wt_adamw: a step of this handle is being enqueued by another thread");
    return WT_E_STATE;
  }
  wt_status st;
  try {
    st = step_impl(adamw, hyper, (hipStream_t)stream);
  } catch (...) {
    st = caught_status();
  }
  adamw->busy.store(false);
  return st;
}

wt_status wt_adamw_get_info(const wt_adamw *adamw, wt_adamw_info *info) {
  if (!adamw || !info) return WT_E_INVAL;
  *info = adamw->L.info;
  return WT_OK;
}

void wt_adamw_destroy(wt_adamw *adamw) {
  if (adamw) free_adamw(adamw);
}

}  // extern "C"
