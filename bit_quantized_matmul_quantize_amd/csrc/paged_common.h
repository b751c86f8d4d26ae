// What the kernels of the paged key-value cache share: where a token's values
// lie, and which sequence and tile a workgroup takes.
#pragma once

#include <algorithm>

#include "bqmm_internal.h"

namespace bqmm {

// Positions and lengths stay below this, so that their sums stay below 2^31.
constexpr int32_t kMaxPlaces = 1 << 30;

// A block holds a page's values of one key head: page * d values in units of 16
// bytes, and behind int8 codes a binary32 scale per token.  In bytes:
__host__ __device__ inline uint32_t paged_block_bytes(uint32_t page, uint32_t d, uint32_t bits) {
  return bits == 16u ? page * d * 2u : page * (d + 4u);
}

// Sequence i's part of a call.
struct PagedSpan {
  uint32_t first;  // its first new token's row
  uint32_t n;      // its new tokens
  int32_t at;      // the place of its first new token in the sequence (below 0: before its beginning)
  int32_t keys;    // the tokens that the cache holds of it
};

// Whatever starts and lens hold, rows stay inside [0, tokens) and places inside
// the table.
__device__ __forceinline__ PagedSpan paged_span(const PagedArgs &a, uint32_t i) {
  const int64_t s0 = a.starts[i], s1 = a.starts[i + 1u], len = a.lens[i];
  const int64_t lo = min(max(s0, (int64_t)0), (int64_t)a.tokens), hi = min(max(s1, (int64_t)0), (int64_t)a.tokens);
  const int64_t at = len - s1 + lo, room = (int64_t)a.width << a.page_shift;
  PagedSpan p;
  p.first = (uint32_t)lo;
  p.n = hi > lo ? (uint32_t)(hi - lo) : 0u;
  p.at = (int32_t)min(max(at, (int64_t)-kMaxPlaces), (int64_t)kMaxPlaces);
  p.keys = (int32_t)min(max(len, (int64_t)0), room);
  return p;
}

// The sum over a wave's lanes up to and with this one's.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const uint32_t lane = __lane_id();
#pragma unroll
  for (uint32_t d = 1; d < 64u; d *= 2u) {
    const uint32_t u = __shfl_up(v, d, 64);
    if (lane >= d) v += u;
  }
  return v;
}

// The sequence that item `item` belongs to, where sequence i has items(i) of
// them, one sequence's after the other's, and the item's number there.  False
// past the last.  Taken by whole waves: 64 sequences at a time.
template <class Items>
__device__ __forceinline__ bool paged_find(uint32_t item, uint32_t count, Items items, uint32_t *seq, uint32_t *inside) {
  const uint32_t lane = __lane_id();
  for (uint32_t base = 0; base < count; base += 64u) {
    const uint32_t mine = base + lane < count ? items(base + lane) : 0u;
    const uint32_t upto = count == 1u ? mine : wave_scan(mine);
    const uint64_t past = __ballot(upto > item);
    if (past) {
      const uint32_t who = (uint32_t)__builtin_ctzll(past);
      *seq = __builtin_amdgcn_readfirstlane(base + who);
      const uint32_t before = (uint32_t)__builtin_amdgcn_readlane((int)(upto - mine), (int)who);
      *inside = __builtin_amdgcn_readfirstlane(item - before);
      return true;
    }
    item -= (uint32_t)__builtin_amdgcn_readlane((int)upto, count == 1u ? 0 : 63);
  }
  return false;
}

// ---- attention ------------------------------------------------------------------

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
// The running maximum of the scores (base 2) is set this far above the largest one, so that
// it is raised, and sums are rescaled, rarely: weights are at most 1, and of the largest score
// at least 2^-8, which costs no bits.
constexpr float kSlack = 8.0f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Caps up to here take the short form of the cap below: off by at most 2^-22 of the cap,
// 2^-16, less than the weights' own rounding.
constexpr float kShortCap = 64.0f;

// The arguments with what the kernels take of scale and cap.
inline PagedArgs score_args(PagedArgs a) {
  // Scores base 2 are the products times this, or made of them by the cap at once.  Not 0 where
  // the scale is, so that the score of a key that is not seen stays -infinity; 2^-149 of any
  // product is below 2^-20.
  a.scale2 = a.cap != 0.0f ? 1.0f : std::max(a.scale * kLog2e, 0x1p-149f);
  a.cap2 = a.cap * kLog2e;
  // (beyond binary32 it would make a NaN of a product of 0)
  a.cap_inv2 = a.cap != 0.0f ? std::min(2.0f * kLog2e * a.scale / a.cap, 3.0e38f) : 0.0f;
  a.cap_inv = a.cap != 0.0f ? 1.0f / a.cap : 0.0f;
  return a;
}

// Of a product x, s = scale x:  c tanh(s / c) = c (1 - 2 / (1 + exp(2 s / c))), base 2
__device__ __forceinline__ float capped(float x, float cap2, float inv2) {
  return cap2 - 2.0f * cap2 * __builtin_amdgcn_rcpf(1.0f + exp2_hw(x * inv2));
}
// The same, off by at most 2^-21 of the score, for large caps: where t = s / c is small, the
// difference above leaves nothing of it; tanh(t) = t + t^3 p(t^2), with p fitted to [0, 0.625^2]
// (to 2^-27 of tanh(t)).
__device__ __forceinline__ float capped_large(float x, const PagedArgs &a) {
  const float s = x * a.scale, t = s * a.cap_inv, u = t * t;
  float p = fmaf(u, -0x1.76abe4p-8f, 0x1.5256cap-6f);
  p = fmaf(u, p, -0x1.b84446p-5f);
  p = fmaf(u, p, 0x1.110768p-3f);
  p = fmaf(u, p, -0x1.555534p-2f);
  const float low = s * kLog2e, far = a.cap2 - 2.0f * a.cap2 * __builtin_amdgcn_rcpf(1.0f + exp2_hw(t * (2.0f * kLog2e)));
  return fabsf(t) < 0.625f ? fmaf(low * u, p, low) : far;
}

__device__ __forceinline__ v8bf as_bf(const v4u &u) { return __builtin_bit_cast(v8bf, u); }

__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  v2bf v;
  v[0] = (__bf16)lo;
  v[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}
// sum + the two values, in binary32.
__device__ __forceinline__ float add_two_bf16(uint32_t two, float sum) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, two), __builtin_bit_cast(v2bf, 0x3F803F80u), sum, false);
}
// Eight codes as bf16 (exact).
__device__ __forceinline__ v4u bf16_of_codes(uint32_t a, uint32_t b) {
  v4u r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? b : a;
    const float x0 = (float)(int8_t)w, x1 = (float)(int8_t)(w >> 8), x2 = (float)(int8_t)(w >> 16), x3 = (float)(int8_t)(w >> 24);
    r[2 * i] = __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302u);
    r[2 * i + 1] = __builtin_amdgcn_perm(__float_as_uint(x3), __float_as_uint(x2), 0x07060302u);
  }
  return r;
}

// Of eight bf16: the finite ones, zero for the others.
__device__ __forceinline__ v4u finite_only(v4u u) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((u[i] & 0x7F80u) == 0x7F80u) u[i] &= 0xFFFF0000u;
    if ((u[i] & 0x7F800000u) == 0x7F800000u) u[i] &= 0xFFFFu;
  }
  return u;
}
// The others: 1 for an infinity, 256 for a negative one, 65536 for a NaN, and what a
// sum of up to 255 of each adds to a sum of finite values.
__device__ __forceinline__ v4u not_finite_marks(const v4u &u) {
  v4u r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto mark = [](uint32_t h) { return (h & 0x7FFFu) > 0x7F80u ? 0x4780u : h == 0x7F80u ? 0x3F80u : h == 0xFF80u ? 0x4380u : 0u; };
    r[i] = mark(u[i] & 0xFFFFu) | mark(u[i] >> 16) << 16;
  }
  return r;
}
__device__ __forceinline__ float of_marks(float sum) {
  const uint32_t n = (uint32_t)sum, plus = n & 0xFFu, minus = n & 0xFF00u;
  return n == 0u ? 0.0f : __uint_as_float(n >> 16 || (plus && minus) ? 0x7FC00000u : plus ? 0x7F800000u : 0xFF800000u);
}

__device__ __forceinline__ bool any_not_finite(const v4u &u) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (u[i] & 0x7F800000u) == 0x7F800000u || (u[i] & 0x7F80u) == 0x7F80u;
  return bad;
}

}  // namespace bqmm
