// RMS norm with the residual's addition and an int8, q8_1 or bf16 output, and
// the int8 row quantizer alone.
//
//   h = bf16_rne(x + residual)       (written back to residual; h = x without one)
//   r = 1 / sqrt(mean(h^2) + eps)    (the mean and r in binary64)
//   t = h * weight                   (binary32: the product of two bf16 is exact)
//   bf16:  y = bf16_rne(t * r)
//   q8_1:  quantize_act_q8_1's rule on that y
//   int8:  code = rint(127 t / top), scale = top * r / 127,  top = max |t| of the row
//
// r is common to a row, so the int8 codes do not depend on it and are exact:
// 127 t has at most 23 significant bits, and its correctly rounded quotient by
// the 16-bit top decides every tie (a quotient that is no half differs from
// one by more than half a step of binary32).  The row quantizer is the same
// with t = x and r = 1.
//
// Bound by memory: the row is read once, held in registers as t between the
// reduction (sum of squares, largest |t|) and the output, and written once.
// 4096 rows of 5120 with the residual to int8 (147 MB): 24.0 us, 6.1 TB/s (part
// of it in the 256 MB cache; a 2 x 2.1 GB copy reaches 4.8); 36.5 us while the roundings to bf16 and the codes took twice the instructions
// (the vector ALU then bound it as much as memory).  One row of 2048: 2.7 us.
// One workgroup per row; a lane owns kNV vectors of eight consecutive values
// (16-byte loads), so a row of k values takes k / (8 kNV) lanes.  Rows beyond
// kMaxHeld values are read a second time instead of being held.
#include "bqmm_internal.h"

namespace bqmm {
namespace {

enum { kOutBf16 = 0, kOutInt8 = 1, kOutQ81 = 2 };

constexpr int kMaxThreads = kNormMaxThreads;
constexpr uint32_t kMaxHeld = kNormMaxThreads * kNormMaxVectors * 8u;  // 32768 values of a row in registers

// Eight bf16 values, two to a word.  Rows of odd length start at any even
// address: 16-byte accesses with the alignment of a bf16 value (gfx950 takes
// them as they are).
struct __attribute__((packed, aligned(2))) Pack8 {
  uint32_t w[4];
};

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two values rounded to bf16 side by side (one instruction; a NaN stays one).
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2f f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, v2bf));
}

__device__ __forceinline__ void load8(const uint16_t *p, uint32_t c, uint32_t k, uint32_t (&v)[4]) {
  if (c + 8u <= k) {
    const Pack8 a = *reinterpret_cast<const Pack8 *>(p + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (c + 2u * i < k ? p[c + 2u * i] : 0u) | (c + 2u * i + 1u < k ? (uint32_t)p[c + 2u * i + 1u] << 16 : 0u);
  }
}

__device__ __forceinline__ void store8(uint16_t *p, uint32_t c, uint32_t k, const uint32_t (&v)[4]) {
  if (c + 8u <= k) {
    *reinterpret_cast<Pack8 *>(p + c) = Pack8{{v[0], v[1], v[2], v[3]}};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < k) p[c + i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
  }
}

struct RowStats {
  double sum;    // of h^2
  uint32_t top;  // bits of the largest |t|; a NaN is above every number
};

// Over the workgroup; every lane gets the result.
__device__ __forceinline__ RowStats reduce_row(RowStats s) {
  __shared__ double sums[16];
  __shared__ uint32_t tops[16];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    s.sum += __shfl_xor(s.sum, d);
    s.top = max(s.top, (uint32_t)__shfl_xor((int)s.top, d));
  }
  const uint32_t waves = blockDim.x >> 6;
  if (waves == 1u) return s;
  if ((threadIdx.x & 63u) == 0u) {
    sums[threadIdx.x >> 6] = s.sum;
    tops[threadIdx.x >> 6] = s.top;
  }
  __syncthreads();
  s.sum = sums[0];
  s.top = tops[0];
  for (uint32_t w = 1; w < waves; ++w) {
    s.sum += sums[w];
    s.top = max(s.top, tops[w]);
  }
  return s;
}

// What the output stage needs of a row.
struct RowScale {
  double r;
  float top, mul, inv;  // int8: top and 127 t scaled by a power of two, 1 / top
  bool live;            // else every code is zero
};

template <int kOut, bool kNorm>
__device__ __forceinline__ RowScale row_scale(const RowStats &s, uint32_t k, double eps) {
  RowScale c{};
  c.r = kNorm ? rsqrt(s.sum / (double)k + eps) : 1.0;
  if constexpr (kOut == kOutInt8) {
    const float top = __uint_as_float(s.top);
    // a power of two that brings top to [2^-29, 2): neither 127 t nor 1 / top nor 127 p overflows
    const float p = ldexpf(1.0f, min(127 - (int)(s.top >> 23), 120));
    c.live = s.top > 0u && s.top < 0x7F800000u;
    c.top = c.live ? top * p : 1.0f;
    c.mul = 127.0f * p;
    c.inv = 1.0f / c.top;
  }
  return c;
}

// Eight values at column c: codes or bf16, and for q8_1 the block's (d, s).
template <int kOut, bool kNorm>
__device__ __forceinline__ void put8(const float (&t)[8], const RowScale &rs, uint8_t *out, uint64_t row,
                                     uint32_t c, uint32_t k, uint32_t kpad, uint64_t scale_off) {
  if constexpr (kOut == kOutInt8) {
    uint32_t packed[2] = {0u, 0u};
    if (rs.live) {
      uint32_t code[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // the correctly rounded quotient: one residual step from a reciprocal that is itself correctly rounded
        const float num = t[i] * rs.mul;
        const float q0 = num * rs.inv;
        const float q = fmaf(fmaf(-q0, rs.top, num), rs.inv, q0);
        // beside 1.5 * 2^23 only whole numbers are left, the nearest (ties to even), in the low bits
        code[i] = __float_as_uint(q + 12582912.0f);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the low bytes of four
        const uint32_t ab = __builtin_amdgcn_perm(code[4 * h + 1], code[4 * h], 0x0C0C0400u);
        const uint32_t cd = __builtin_amdgcn_perm(code[4 * h + 3], code[4 * h + 2], 0x04000C0Cu);
        packed[h] = ab | cd;
      }
    }
    *reinterpret_cast<uint2 *>(out + row * kpad + c) = make_uint2(packed[0], packed[1]);
  } else {
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = round2((float)((double)t[2 * i] * rs.r), (float)((double)t[2 * i + 1] * rs.r));
    if constexpr (kOut == kOutBf16) {
      store8(reinterpret_cast<uint16_t *>(out) + row * k, c, k, y);
    } else {
      float v[8], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = low(y[i]);
        v[2 * i + 1] = high(y[i]);
        amax = fmaxf(amax, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
      }
      amax = fmaxf(amax, __shfl_xor(amax, 1));
      amax = fmaxf(amax, __shfl_xor(amax, 2));
      const uint32_t dh = f32_to_f16_bits(amax / 127.0f);
      const float d = f16_bits_to_f32(dh);
      int sum = 0;
      uint32_t packed[2] = {0u, 0u};
      if (d != 0.0f && dh != 0x7C00u) {  // (an infinite scale gives zero codes)
        const float inv = 1.0f / d;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // the correctly rounded quotient again, then halves away from zero: a quotient of 8 by 11
          // significant bits that is no half is further from one than the sum's rounding
          const float q0 = v[i] * inv;
          const float q = fminf(truncf(fabsf(fmaf(fmaf(-q0, d, v[i]), inv, q0)) + 0.5f), 127.0f) * (v[i] < 0.0f ? -1.0f : 1.0f);
          sum += (int)q;
          packed[i / 4] |= ((uint32_t)(int)q & 0xFFu) << (8 * (i % 4));
        }
      }
      sum += __shfl_xor(sum, 1);
      sum += __shfl_xor(sum, 2);
      *reinterpret_cast<uint2 *>(out + row * kpad + c) = make_uint2(packed[0], packed[1]);
      if ((threadIdx.x & 3u) == 0u)
        *reinterpret_cast<uint32_t *>(out + scale_off + 4ull * (row * (kpad / 32u) + c / 32u)) =
            dh | (f32_to_f16_bits(d * (float)sum) << 16);
    }
  }
}

// h and t of eight values; adds them to the row's statistics.  Values past k are zero.
template <int kOut, bool kRes, bool kNorm>
__device__ __forceinline__ void take8(const uint32_t (&x)[4], const uint32_t (&res)[4], const uint32_t (&w)[4],
                                      uint32_t (&h)[4], float (&t)[8], RowStats &s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = kRes ? round2(low(x[i]) + low(res[i]), high(x[i]) + high(res[i])) : x[i];
    const float a = low(h[i]), b = high(h[i]);
    t[2 * i] = kNorm ? a * low(w[i]) : a;
    t[2 * i + 1] = kNorm ? b * high(w[i]) : b;
    if constexpr (kNorm) s.sum = fma((double)a, (double)a, fma((double)b, (double)b, s.sum));
    if constexpr (kOut == kOutInt8)
      s.top = max(s.top, max(__float_as_uint(t[2 * i]) & 0x7FFFFFFFu, __float_as_uint(t[2 * i + 1]) & 0x7FFFFFFFu));
  }
}

template <int kOut>
__device__ __forceinline__ uint32_t padded(uint32_t k, uint32_t kpad) {
  return kOut == kOutBf16 ? (k + 7u) / 8u * 8u : kpad;
}

template <int kOut, bool kNorm>
__device__ __forceinline__ void put_row_scale(const RowStats &s, const RowScale &rs, uint8_t *out, uint64_t row,
                                              uint64_t scale_off) {
  if constexpr (kOut == kOutInt8)
    if (threadIdx.x == 0)
      *reinterpret_cast<float *>(out + scale_off + 4ull * row) =
          (float)((double)__uint_as_float(s.top) * rs.r / 127.0);
}

// A row held in registers: kNV vectors of eight per lane.
template <int kNV, int kOut, bool kRes, bool kNorm>
__global__ __launch_bounds__(kMaxThreads) void norm_rows_kernel(const uint16_t *__restrict__ x,
                                                                uint16_t *__restrict__ residual,
                                                                const uint16_t *__restrict__ weight,
                                                                uint8_t *__restrict__ out, uint32_t k, uint32_t kpad,
                                                                double eps, uint64_t scale_off) {
  const uint64_t row = blockIdx.x;
  const uint32_t kend = padded<kOut>(k, kpad);
  float t[kNV][8];
  RowStats s{0.0, 0u};
  {
    uint32_t xv[kNV][4], rv[kNV][4], wv[kNV][4];
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const uint32_t c = (j * blockDim.x + threadIdx.x) * 8u;
      load8(x + row * k, c, k, xv[j]);
      if constexpr (kRes) load8(residual + row * k, c, k, rv[j]);
      if constexpr (kNorm) load8(weight, c, k, wv[j]);
    }
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const uint32_t c = (j * blockDim.x + threadIdx.x) * 8u;
      uint32_t h[4];
      take8<kOut, kRes, kNorm>(xv[j], rv[j], wv[j], h, t[j], s);
      if constexpr (kRes)
        if (c < k) store8(residual + row * k, c, k, h);
    }
  }
  if constexpr (kNorm || kOut == kOutInt8) s = reduce_row(s);
  const RowScale rs = row_scale<kOut, kNorm>(s, k, eps);
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    const uint32_t c = (j * blockDim.x + threadIdx.x) * 8u;
    // kpad is a multiple of 32: the four lanes of a q8_1 block go together
    if (c < kend) put8<kOut, kNorm>(t[j], rs, out, row, c, k, kpad, scale_off);
  }
  put_row_scale<kOut, kNorm>(s, rs, out, row, scale_off);
}

// A row too long for that: h is read again (from the residual, where this
// same lane has written it, or from x) for the output.
template <int kOut, bool kRes, bool kNorm>
__global__ __launch_bounds__(kMaxThreads) void norm_long_rows_kernel(const uint16_t *x, uint16_t *residual,
                                                                     const uint16_t *__restrict__ weight,
                                                                     uint8_t *__restrict__ out, uint32_t k,
                                                                     uint32_t kpad, double eps, uint64_t scale_off) {
  const uint64_t row = blockIdx.x;
  const uint32_t kend = padded<kOut>(k, kpad);
  RowStats s{0.0, 0u};
  uint32_t xv[4], rv[4], wv[4], h[4];
  float t[8];
  if constexpr (kNorm || kOut == kOutInt8) {
    for (uint32_t c = threadIdx.x * 8u; c < k; c += blockDim.x * 8u) {
      load8(x + row * k, c, k, xv);
      if constexpr (kRes) load8(residual + row * k, c, k, rv);
      if constexpr (kNorm) load8(weight, c, k, wv);
      take8<kOut, kRes, kNorm>(xv, rv, wv, h, t, s);
      if constexpr (kRes) store8(residual + row * k, c, k, h);
    }
    s = reduce_row(s);
  }
  const RowScale rs = row_scale<kOut, kNorm>(s, k, eps);
  for (uint32_t c = threadIdx.x * 8u; c < kend; c += blockDim.x * 8u) {
    RowStats unused{0.0, 0u};
    load8((kRes ? residual : x) + row * k, c, k, xv);
    if constexpr (kNorm) load8(weight, c, k, wv);
    take8<kOut, false, kNorm>(xv, rv, wv, h, t, unused);
    put8<kOut, kNorm>(t, rs, out, row, c, k, kpad, scale_off);
  }
  put_row_scale<kOut, kNorm>(s, rs, out, row, scale_off);
}

template <int kNV, int kOut, bool kRes, bool kNorm>
void launch_held(const uint16_t *x, uint16_t *res, const uint16_t *w, uint8_t *out, uint32_t m, uint32_t k,
                 uint32_t kpad, double eps, uint64_t scale_off, uint32_t threads, hipStream_t s) {
  hipLaunchKernelGGL((norm_rows_kernel<kNV, kOut, kRes, kNorm>), dim3(m), dim3(threads), 0, s, x, res, w, out, k,
                     kpad, eps, scale_off);
}

template <int kOut, bool kRes, bool kNorm>
hipError_t launch_norm(const void *x, void *residual, const void *weight, void *out, uint32_t m, uint32_t k,
                       double eps, hipStream_t s) {
  const uint32_t to = kOut == kOutInt8 ? 128u : kOut == kOutQ81 ? 256u : 8u;
  const uint32_t kpad = norm_padded(k, to);
  const uint64_t scale_off = (uint64_t)m * kpad;
  const uint16_t *xp = static_cast<const uint16_t *>(x);
  uint16_t *rp = static_cast<uint16_t *>(residual);
  const uint16_t *wp = static_cast<const uint16_t *>(weight);
  uint8_t *op = static_cast<uint8_t *>(out);
  if (kpad > kMaxHeld) {
    hipLaunchKernelGGL((norm_long_rows_kernel<kOut, kRes, kNorm>), dim3(m), dim3(kMaxThreads), 0, s, xp, rp, wp, op,
                       k, kpad, eps, scale_off);
    return hipGetLastError();
  }
  // As few vectors per lane as 512 lanes allow, and the lanes those take: k =
  // 5120 runs 320 lanes of two vectors, where 256 would leave half of every
  // third vector idle.
  const uint32_t threads = norm_threads(kpad);
  switch (norm_vectors(kpad)) {
    case 1: launch_held<1, kOut, kRes, kNorm>(xp, rp, wp, op, m, k, kpad, eps, scale_off, threads, s); break;
    case 2: launch_held<2, kOut, kRes, kNorm>(xp, rp, wp, op, m, k, kpad, eps, scale_off, threads, s); break;
    case 4: launch_held<4, kOut, kRes, kNorm>(xp, rp, wp, op, m, k, kpad, eps, scale_off, threads, s); break;
    default: launch_held<8, kOut, kRes, kNorm>(xp, rp, wp, op, m, k, kpad, eps, scale_off, threads, s); break;
  }
  return hipGetLastError();
}

template <int kOut>
hipError_t launch_add_rms_norm(const void *x, void *residual, const void *weight, void *out, uint32_t m, uint32_t k,
                               double eps, hipStream_t s) {
  return residual ? launch_norm<kOut, true, true>(x, residual, weight, out, m, k, eps, s)
                  : launch_norm<kOut, false, true>(x, residual, weight, out, m, k, eps, s);
}

}  // namespace

hipError_t launch_add_rms_norm_bf16(const void *x, void *residual, const void *weight, void *out, uint32_t m,
                                    uint32_t k, double eps, hipStream_t s) {
  return launch_add_rms_norm<kOutBf16>(x, residual, weight, out, m, k, eps, s);
}

hipError_t launch_add_rms_norm_quantize_int8(const void *x, void *residual, const void *weight, void *out, uint32_t m,
                                             uint32_t k, double eps, hipStream_t s) {
  return launch_add_rms_norm<kOutInt8>(x, residual, weight, out, m, k, eps, s);
}

hipError_t launch_add_rms_norm_quantize_q8_1(const void *x, void *residual, const void *weight, void *out, uint32_t m,
                                             uint32_t k, double eps, hipStream_t s) {
  return launch_add_rms_norm<kOutQ81>(x, residual, weight, out, m, k, eps, s);
}

hipError_t launch_quantize_rows_int8(const void *x, void *out, uint32_t rows, uint32_t k, hipStream_t s) {
  return launch_norm<kOutInt8, false, false>(x, nullptr, nullptr, out, rows, k, 0.0, s);
}

}  // namespace bqmm
