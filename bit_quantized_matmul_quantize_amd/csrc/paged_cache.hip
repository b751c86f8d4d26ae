// Writing a paged key-value cache and reading it back.
//
// Writing: per token, each head of q and k is normed (optional), and its first
// rot values are rotated in pairs (i, i + rot / 2),
//   t[i] c - t[i + rot/2] s,   t[i + rot/2] c + t[i] s,
// with the cosine and sine of frequency i at the position of the frequency's
// axis; q goes out in bf16, k and v into the cache, in bf16 or as int8 codes
// rint(127 t / top) with a scale top / 127 per token and head.
//
// Bound by bytes: 2 read and 2 or 1 + 4/d written a value, a few operations each: a
// prompt of 8192, 32 heads over 8 of 128, in bf16 205 MB in 50 us, 4.1 TB/s (39 us where the
// last call's lie in the 256 MB cache).
// A workgroup takes 16 consecutive places of a sequence, aligned to 16, so that
// they lie in one page and fill whole 16-byte units of it: a unit of k is 8 or 16
// values of one token, and a unit of v one value of 8 or 16 tokens, for which the
// tile of v is turned in LDS.  A thread keeps its token and its pair of 8-value
// runs from head to head, and with them the cosines and sines.
#include "paged_common.h"

#include <algorithm>

namespace bqmm {
namespace {

constexpr uint32_t kTile = 16;     // places
constexpr uint32_t kThreads = 256;
// Workgroups that the heads of a tile are shared out to: enough of them in all, and
// four turns each where that leaves more (looking up the angles costs about two).
// 2130 tokens of 6 sequences, 16 heads over 2 of 256, written and read: with 512 as
// enough 24.3 us, with 1024 25.7; a prompt of 8192, 32 heads over 8: with up to 2048
// 51 us, with 1024 55.
constexpr uint32_t kEnough = 512, kMore = 2048;

struct Tile {
  PagedSpan span;
  uint32_t seq;
  int32_t place0;      // the tile's first place (a multiple of 16)
  uint32_t low, high;  // the new tokens' places in the tile, from place0 on
};

__device__ __forceinline__ uint32_t tiles_of(const PagedSpan &p) {
  return p.n == 0u ? 0u : (p.n + ((uint32_t)p.at & (kTile - 1u)) + kTile - 1u) / kTile;
}

__device__ __forceinline__ bool find_tile(const PagedArgs &a, uint32_t item, Tile *t) {
  uint32_t inside;
  if (!paged_find(item, a.count, [&](uint32_t i) { return tiles_of(paged_span(a, i)); }, &t->seq, &inside)) return false;
  t->span = paged_span(a, t->seq);
  const int32_t before = t->span.at & (int32_t)(kTile - 1u);
  t->place0 = t->span.at - before + (int32_t)(inside * kTile);
  t->low = inside == 0u ? (uint32_t)before : 0u;
  t->high = min((uint32_t)(t->span.at + (int32_t)t->span.n - t->place0), kTile);
  return true;
}

// The tile's page, -1 where there is none.
__device__ __forceinline__ int64_t tile_page(const PagedArgs &a, const Tile &t) {
  if (t.place0 < 0 || t.place0 >= (int64_t)a.width << a.page_shift) return -1;
  const uint32_t id = (uint32_t)a.table[(uint64_t)t.seq * a.width + ((uint32_t)t.place0 >> a.page_shift)];
  return id < a.pages ? (int64_t)id : -1;
}

struct __attribute__((aligned(4))) Float8 {
  float x[8];
};
__device__ __forceinline__ void unpack8(const uint4 &r, float *x) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf16_to_f32(w[e] & 0xFFFFu);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float *x) {
  return make_uint4(two_bf16(x[0], x[1]), two_bf16(x[2], x[3]), two_bf16(x[4], x[5]), two_bf16(x[6], x[7]));
}

// Codes of 16 values whose row's largest magnitude has the bits `top`.  A row with a NaN
// or an infinity gets zero codes.
__device__ __forceinline__ void quantize16(const float *x, uint32_t top, uint32_t *codes, float *scale) {
  const bool some = top != 0u && top < 0x7F800000u;
  // a power of two that brings top to [2^-29, 2): neither 127 t nor 1 / top nor 127 p overflows
  const float p = ldexpf(1.0f, min(127 - (int)(top >> 23), 120));
  const float t = some ? __uint_as_float(top) * p : 1.0f, mul = 127.0f * p, inv = 1.0f / t;
  *scale = __uint_as_float(top) / 127.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t c[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      // the correctly rounded quotient: one residual step from a reciprocal that is itself
      // correctly rounded (without it a half of the largest is off by a code for one row in nine)
      const float num = x[4 * w + b] * mul, q0 = num * inv;
      const float q = fmaf(fmaf(-q0, t, num), inv, q0);
      // beside 1.5 * 2^23 only whole numbers are left, the nearest (ties to even), in the low bits
      c[b] = some ? __float_as_uint(q + 12582912.0f) : 0u;
    }
    // the low bytes of four words
    const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(c[3], c[2], 0x0C0C0400u);
    codes[w] = lo | hi << 16;
  }
}

// Maximum and sum over the G lanes of a row (G a power of two).
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t G) {
  for (uint32_t d = 1; d < G; d *= 2u) v = max(v, (uint32_t)__shfl_xor((int)v, (int)d, 64));
  return v;
}
__device__ __forceinline__ float row_sum(float v, uint32_t G) {
  for (uint32_t d = 1; d < G; d *= 2u) v += __shfl_xor(v, (int)d, 64);
  return v;
}
__device__ __forceinline__ uint32_t top16(const float *x) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  return top;
}

// G: lanes of a row, each with two runs of 8 values.
// Workgroups (.., y) with y < parts share the heads of q and k, the others those of v.
template <uint32_t G>
__global__ __launch_bounds__(kThreads) void paged_write_kernel(PagedArgs a, uint32_t parts) {
  constexpr uint32_t kHeads = kThreads / (kTile * G);  // heads at once
  constexpr uint32_t kPitch = G * 16u;                 // of a token in the tile
  __shared__ __attribute__((aligned(16))) uint16_t turn[kHeads * kTile * kPitch];
  Tile t;
  if (!find_tile(a, blockIdx.x, &t)) return;
  const uint32_t lane = threadIdx.x % G, token = threadIdx.x / G % kTile, sub = threadIdx.x / (G * kTile);
  const uint32_t page = 1u << a.page_shift, block = paged_block_bytes(page, a.d, a.bits);
  const int64_t id = tile_page(a, t);
  const uint32_t off = (uint32_t)t.place0 & (page - 1u);  // of the tile in its page
  const bool mine = token >= t.low && token < t.high && lane < a.d / 16u;
  const uint64_t row = (uint64_t)t.span.first + (uint32_t)(t.place0 + (int32_t)token - t.span.at);

  if (blockIdx.y < parts) {
    // this lane's runs of a head: a pair that is rotated, or two that are not
    const uint32_t pairs = a.rot / 16u;
    const bool turned = lane < pairs;
    const uint32_t run0 = turned ? lane : 2u * lane, run1 = turned ? lane + pairs : run0 + 1u;
    // q and k: the first heads are on their way while the angles are looked up, the
    // next ones while these are computed
    const uint32_t heads = a.hq + a.hk, stride = parts * kHeads;
    auto load = [&](uint32_t h, uint4 (&raw)[2]) {
      if (mine && h < heads) {
        const uint16_t *p = h < a.hq ? a.q + row * a.q_token + h * a.q_head : a.k + row * a.k_token + (h - a.hq) * a.k_head;
        raw[0] = *reinterpret_cast<const uint4 *>(p + run0 * 8u);
        raw[1] = *reinterpret_cast<const uint4 *>(p + run1 * 8u);
      }
    };
    uint4 raw[2] = {};
    load(blockIdx.y * kHeads + sub, raw);
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.0f, s[e] = 0.0f;
    if (mine && turned) {
      const float nan = __uint_as_float(0x7FC00000u);
      if (!a.axis) {  // one row of the table a token, read as vectors
        const int32_t angle = a.positions ? a.positions[row] : t.place0 + (int32_t)token;
        const bool known = (uint32_t)angle < a.angles;
        const float *at = a.cos_sin + (uint64_t)(known ? angle : 0) * a.rot + lane * 8u;
        const Float8 cv = *reinterpret_cast<const Float8 *>(at), sv = *reinterpret_cast<const Float8 *>(at + a.rot / 2u);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = known ? cv.x[e] : nan, s[e] = known ? sv.x[e] : nan;
      } else {
        int32_t angle[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t axis = a.axis[lane * 8u + e];
          angle[e] = a.positions[(uint64_t)(axis < a.axes ? axis : 0u) * a.tokens + row];
          if (axis >= a.axes) angle[e] = -1;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool known = (uint32_t)angle[e] < a.angles;
          const float *at = a.cos_sin + (uint64_t)(known ? angle[e] : 0) * a.rot + lane * 8u + e;
          c[e] = known ? at[0] : nan;
          s[e] = known ? at[a.rot / 2u] : nan;
        }
      }
    }
    // the norms' weights of this lane's runs
    uint4 wq[2] = {}, wk[2] = {};
    if (lane < a.d / 16u) {
      if (a.q_norm) {
        wq[0] = *reinterpret_cast<const uint4 *>(a.q_norm + run0 * 8u);
        wq[1] = *reinterpret_cast<const uint4 *>(a.q_norm + run1 * 8u);
      }
      if (a.k_norm) {
        wk[0] = *reinterpret_cast<const uint4 *>(a.k_norm + run0 * 8u);
        wk[1] = *reinterpret_cast<const uint4 *>(a.k_norm + run1 * 8u);
      }
    }

    for (uint32_t h0 = blockIdx.y * kHeads; h0 < heads; h0 += stride) {
      const uint32_t h = h0 + sub;
      const bool is_q = h < a.hq, live = mine && h < heads;
      float x[16];
      unpack8(raw[0], x);
      unpack8(raw[1], x + 8);
      if (!live) {  // (of no row: zeros)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.0f;
      }
      load(h + stride, raw);
      if (a.q_norm || a.k_norm) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) sum = fmaf(x[e], x[e], sum);
        sum = row_sum(sum, G);
        if (live && (is_q ? a.q_norm : a.k_norm)) {
          const float r = 1.0f / sqrtf(sum / (float)a.d + a.eps);
          float w[16];
          unpack8(is_q ? wq[0] : wk[0], w);
          unpack8(is_q ? wq[1] : wk[1], w + 8);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
        }
      }
      if (turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = x[e], v = x[e + 8];
          x[e] = fmaf(u, c[e], -v * s[e]);
          x[e + 8] = fmaf(v, c[e], u * s[e]);
        }
      }
      if (is_q) {
        if (live) {
          uint16_t *p = a.out + (row * a.hq + h) * a.d;
          *reinterpret_cast<uint4 *>(p + run0 * 8u) = pack8(x);
          *reinterpret_cast<uint4 *>(p + run1 * 8u) = pack8(x + 8);
        }
      }
      if (a.bits == 16u) {
        if (!is_q && live && id >= 0) {
          uint8_t *p = a.k_cache + ((uint64_t)id * a.hk + (h - a.hq)) * block + (off + token) * 16u;
          *reinterpret_cast<uint4 *>(p + (uint64_t)run0 * page * 16u) = pack8(x);
          *reinterpret_cast<uint4 *>(p + (uint64_t)run1 * page * 16u) = pack8(x + 8);
        }
      } else if (__any(!is_q && live)) {
        const uint32_t top = row_max(top16(x), G);
        if (!is_q && live && id >= 0) {
          uint32_t codes[4];
          float scale;
          quantize16(x, top, codes, &scale);
          uint8_t *p = a.k_cache + ((uint64_t)id * a.hk + (h - a.hq)) * block;
          *reinterpret_cast<uint2 *>(p + ((run0 / 2u) * page + off + token) * 16u + (run0 & 1u) * 8u) = make_uint2(codes[0], codes[1]);
          *reinterpret_cast<uint2 *>(p + ((run1 / 2u) * page + off + token) * 16u + (run1 & 1u) * 8u) = make_uint2(codes[2], codes[3]);
          if (lane == 0u) *reinterpret_cast<float *>(p + page * a.d + (off + token) * 4u) = scale;
        }
      }
    }
    return;
  }
  if (id < 0) return;  // (the whole workgroup)

  // v: turned in LDS, so that whole units leave
  for (uint32_t h0 = (blockIdx.y - parts) * kHeads; h0 < a.hk; h0 += (gridDim.y - parts) * kHeads) {
    const uint32_t h = h0 + sub;
    const bool live = mine && h < a.hk;
    uint16_t *to = turn + (sub * kTile + token) * kPitch;
    __syncthreads();  // the last heads have left
    if (a.bits == 16u) {
      if (live) {
        const uint4 *p = reinterpret_cast<const uint4 *>(a.v + row * a.v_token + h * a.v_head) + 2u * lane;
        uint4 *w = reinterpret_cast<uint4 *>(to) + 2u * lane;
        w[0] = p[0];
        w[1] = p[1];
      }
    } else {
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.0f;
      if (live) {
        const uint4 *p = reinterpret_cast<const uint4 *>(a.v + row * a.v_token + h * a.v_head) + 2u * lane;
        unpack8(p[0], x);
        unpack8(p[1], x + 8);
      }
      const uint32_t top = row_max(top16(x), G);
      if (live) {
        uint32_t codes[4];
        float scale;
        quantize16(x, top, codes, &scale);
        *(reinterpret_cast<uint4 *>(to) + lane) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        if (lane == 0u)
          *reinterpret_cast<float *>(a.v_cache + ((uint64_t)id * a.hk + h) * block + page * a.d + (off + token) * 4u) = scale;
      }
    }
    __syncthreads();
    const uint32_t unit = a.bits == 16u ? 8u : 16u, groups = kTile / unit;
    for (uint32_t i = threadIdx.x; i < kHeads * groups * a.d; i += kThreads) {
      const uint32_t dim = i % a.d, group = i / a.d % groups, head = h0 + i / a.d / groups;
      if (head >= a.hk) break;
      const uint32_t t0 = group * unit, lo = max(t.low, t0), hi = min(t.high, t0 + unit);
      if (lo >= hi) continue;
      const uint16_t *from = turn + (i / a.d / groups) * kTile * kPitch;
      uint8_t *p = a.v_cache + ((uint64_t)id * a.hk + head) * block + ((uint64_t)(off / unit + group) * a.d + dim) * 16u;
      if (a.bits == 16u) {
        if (hi - lo == 8u) {
          uint32_t w[4];
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e)
            w[e] = from[(t0 + 2u * e) * kPitch + dim] | (uint32_t)from[(t0 + 2u * e + 1u) * kPitch + dim] << 16;
          *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          for (uint32_t e = lo; e < hi; ++e) reinterpret_cast<uint16_t *>(p)[e - t0] = from[e * kPitch + dim];
        }
      } else {
        const uint8_t *codes = reinterpret_cast<const uint8_t *>(from) + dim;
        if (hi - lo == 16u) {
          uint32_t w[4];
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            w[e] = 0;
#pragma unroll
            for (uint32_t b = 0; b < 4; ++b) w[e] |= (uint32_t)codes[(4u * e + b) * 2u * kPitch] << (8u * b);
          }
          *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          for (uint32_t e = lo; e < hi; ++e) p[e] = codes[e * 2u * kPitch];
        }
      }
    }
  }
}

// The same tiles back to rows: a workgroup's part of the heads of k, then of v.
// Units are read side by side and turned in LDS, rows leave whole.
__global__ __launch_bounds__(kThreads) void paged_read_kernel(PagedArgs a) {
  constexpr uint32_t kMost = 256 + 8;  // values of a token in the tile, and a pad against bank conflicts
  __shared__ __attribute__((aligned(16))) uint16_t turn[kTile * kMost];
  __shared__ float scales[kTile];
  Tile t;
  if (!find_tile(a, blockIdx.x, &t)) return;
  const uint32_t page = 1u << a.page_shift, block = paged_block_bytes(page, a.d, a.bits), pitch = a.d + 8u;
  const int64_t id = tile_page(a, t);
  const uint32_t off = (uint32_t)t.place0 & (page - 1u), unit = a.bits == 16u ? 8u : 16u;
  for (uint32_t h = blockIdx.y; h < 2u * a.hk; h += gridDim.y) {
    const bool is_k = h < a.hk;
    const uint32_t head = is_k ? h : h - a.hk;
    const uint8_t *from = (is_k ? a.k_cache : a.v_cache) + ((uint64_t)max(id, (int64_t)0) * a.hk + head) * block;
    __syncthreads();
    if (a.bits == 8u && threadIdx.x < kTile)
      scales[threadIdx.x] = reinterpret_cast<const float *>(from + page * a.d)[off + threadIdx.x];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kTile * a.d / unit; i += kThreads) {
      // (of k: token and unit; of v: value and group of tokens)
      const uint32_t inner = is_k ? i % kTile : i % a.d, outer = is_k ? i / kTile : i / a.d;
      const uint64_t at = is_k ? (uint64_t)outer * page + off + inner : (uint64_t)(off / unit + outer) * a.d + inner;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (id >= 0) u = *reinterpret_cast<const uint4 *>(from + at * 16u);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (uint32_t e = 0; e < 16u; ++e) {
        if (e >= unit) break;
        const uint32_t token = is_k ? inner : outer * unit + e, dim = is_k ? outer * unit + e : inner;
        uint32_t y;
        if (a.bits == 16u)
          y = w[(e / 2u) & 3u] >> (16u * (e & 1u)) & 0xFFFFu;
        else
          y = id < 0 ? 0u : f32_to_bf16_rne((float)(int8_t)(w[e / 4u] >> (8u * (e & 3u))) * scales[token]);
        turn[token * pitch + dim] = (uint16_t)y;
      }
    }
    __syncthreads();
    uint16_t *out = is_k ? a.k_out : a.v_out;
    for (uint32_t i = threadIdx.x; i < kTile * (a.d / 8u); i += kThreads) {
      const uint32_t token = i / (a.d / 8u), run = i % (a.d / 8u);
      if (token < t.low || token >= t.high) continue;
      const uint64_t row = (uint64_t)t.span.first + (uint32_t)(t.place0 + (int32_t)token - t.span.at);
      *reinterpret_cast<uint4 *>(out + (row * a.hk + head) * a.d + run * 8u) =
          *reinterpret_cast<const uint4 *>(turn + token * pitch + run * 8u);
    }
  }
}

// Tiles that a call can have, whatever starts and lens hold: one begins and one
// ends inside a sequence, and none is without a token.
uint32_t tiles_at_most(const PagedArgs &a) {
  return (uint32_t)std::min<uint64_t>(a.tokens, a.tokens / kTile + 2ull * a.count);
}

}  // namespace

hipError_t launch_paged_write(const PagedArgs &a, hipStream_t s) {
  const uint32_t G = a.d <= 16u ? 1u : a.d <= 32u ? 2u : a.d <= 64u ? 4u : a.d <= 128u ? 8u : 16u;
  const uint32_t at_once = kThreads / (kTile * G), tiles = tiles_at_most(a);
  const uint32_t all_qk = (a.hq + a.hk + at_once - 1u) / at_once, all_v = (a.hk + at_once - 1u) / at_once;
  // as many workgroups for v as its share is
  const uint32_t parts = std::min(all_qk, std::max({1u, kEnough / tiles, std::min(kMore / tiles, all_qk / 4u)}));
  const uint32_t parts_v = std::min(all_v, std::max(1u, (uint32_t)((uint64_t)parts * all_v / all_qk)));
  const dim3 grid(tiles, parts + parts_v);
  switch (G) {
    case 1: hipLaunchKernelGGL(paged_write_kernel<1>, grid, dim3(kThreads), 0, s, a, parts); break;
    case 2: hipLaunchKernelGGL(paged_write_kernel<2>, grid, dim3(kThreads), 0, s, a, parts); break;
    case 4: hipLaunchKernelGGL(paged_write_kernel<4>, grid, dim3(kThreads), 0, s, a, parts); break;
    case 8: hipLaunchKernelGGL(paged_write_kernel<8>, grid, dim3(kThreads), 0, s, a, parts); break;
    default: hipLaunchKernelGGL(paged_write_kernel<16>, grid, dim3(kThreads), 0, s, a, parts);
  }
  return hipGetLastError();
}

hipError_t launch_paged_read(const PagedArgs &a, hipStream_t s) {
  const uint32_t tiles = tiles_at_most(a);
  const dim3 grid(tiles, std::min(2u * a.hk, std::max(1u, kMore / tiles)));
  hipLaunchKernelGGL(paged_read_kernel, grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace bqmm
