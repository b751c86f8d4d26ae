// Attention of prompts over the paged key-value cache:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - max s),  s_j = scale q . k_j, capped,
// in one pass over the cache with the running maximum and sum of the softmax.
//
// Bound by the matrix cores (4 d operations for each head and pair of tokens),
// and by the exponentials beside them.  A workgroup takes 128 rows: the heads of
// consecutive tokens that share a key head, so that a tile of keys serves them
// all and few pairs are masked.  Tiles of keys and values come from the cache
// straight into LDS, in its units, while the last ones are computed; an int8
// cache goes through registers and lies in LDS as bf16 (codes are exact; scales
// are applied to scores and weights).
//
// S^T = K Q^T and O^T = V^T P^T: a lane's scores belong to one row, so that the
// softmax needs no exchange between lanes, and the weights of its keys are an
// operand of the second product as they are, given the order in which K's rows
// are read: row 8 b + 4 h + j of the first product is key 16 (b / 2) + 8 h + 4 (b % 2) + j.
#include <algorithm>

#include "paged_common.h"

namespace bqmm {
namespace {

constexpr uint32_t kWaves = 4;
constexpr uint32_t kThreads = 64 * kWaves;
constexpr uint32_t kRows = 32 * kWaves;

// 16 bytes a lane straight from memory into LDS: lane i's go to the wave's
// destination + 16 i.  The kernel waits itself; no register is written.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t offset, const uint8_t *base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(uint32_t lds, const uint8_t *from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}

// kDP: values of a head, rounded up (the ones beyond are zero).
template <uint32_t kDP, uint32_t kBits>
struct Shape {
  static constexpr uint32_t kKT = kDP <= 128 ? 64 : 32;      // keys of a tile
  static constexpr uint32_t kSubs = kKT / 16;                // parts of it that lie in one page
  static constexpr uint32_t kTile = kKT * kDP * 2;           // bytes of its keys, or values
  static constexpr uint32_t kStage = 2 * kTile + (kBits == 8 ? 2 * kKT * 4 : 0);
  static constexpr uint32_t kLoads = kTile / 16 / kThreads;  // bf16: of a thread, for keys, and for values
  static constexpr uint32_t kCodes = (kTile / 32 + kThreads - 1) / kThreads;  // int8
  static constexpr uint32_t kOutPitch = kDP * 2 + 16;        // bytes of a row of the output in LDS
  static constexpr uint32_t kLds = 2 * kStage > kRows * kOutPitch ? 2 * kStage : kRows * kOutPitch;
};

__device__ __forceinline__ uint32_t tiles_of(const PagedArgs &a, const PagedSpan &p) {
  return (uint32_t)(((uint64_t)p.n * (a.hq / a.hk) + kRows - 1u) / kRows);
}

template <uint32_t kDP, uint32_t kBits>
__global__ __launch_bounds__(kThreads, kDP <= 128 ? 2 : 1) void paged_prefill_kernel(PagedArgs a) {
  using S = Shape<kDP, kBits>;
  constexpr uint32_t kKT = S::kKT, kSubs = S::kSubs;
  constexpr uint32_t kHalves = kKT / 32;  // halves of a tile: 32 keys
  constexpr uint32_t kDS = kDP / 16;      // steps of the first product
  constexpr uint32_t kDB = kDP / 32;      // blocks of the second
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 31u, half = lane >> 5;
  const uint32_t head = blockIdx.x % a.hk, g = a.hq / a.hk;
  uint32_t seq, inside;
  if (!paged_find(blockIdx.x / a.hk, a.count, [&](uint32_t i) { return tiles_of(a, paged_span(a, i)); }, &seq, &inside)) return;
  const PagedSpan p = paged_span(a, seq);
  // the last tiles have the most keys: they begin first
  const uint32_t tile = tiles_of(a, p) - 1u - inside, rows = p.n * g;

  // what rows see: key <= place, and key > place - window
  auto place_of = [&](uint32_t row) { return p.at + (int32_t)(row / g); };
  auto low_of = [&](int32_t place) { return a.window ? (int32_t)max((int64_t)place + 1 - (int64_t)a.window, (int64_t)0) : 0; };
  const uint32_t row0 = tile * kRows, row1 = min(row0 + kRows, rows) - 1u;
  const int32_t end = min(p.keys, max(place_of(row1) + 1, 0));
  const int32_t begin = low_of(place_of(row0)) / (int32_t)kKT * (int32_t)kKT;
  const uint32_t wrow0 = row0 + wave * 32u, wrow1 = min(wrow0 + 32u, rows) - 1u;
  const bool idle = wrow0 >= rows;
  // keys that all rows of the wave see lie in [whole_low, whole_end), those that any sees in [any_low, any_end)
  const int32_t any_low = idle ? 0 : low_of(place_of(wrow0)), any_end = idle ? 0 : min(p.keys, place_of(wrow1) + 1);
  const int32_t whole_low = idle ? 0 : low_of(place_of(wrow1)), whole_end = idle ? 0 : min(p.keys, place_of(wrow0) + 1);

  const uint32_t row = wrow0 + r, token = row / g, hh = row % g;
  const bool live = row < rows;
  const int32_t pos = live ? p.at + (int32_t)token : -1, low = live ? low_of(pos) : 0;
  v4u q[kDS];
  {
    const uint16_t *from = a.q + (uint64_t)(p.first + (live ? token : 0u)) * a.q_token + (uint64_t)(head * g + hh) * a.q_head;
#pragma unroll
    for (uint32_t s = 0; s < kDS; ++s) {
      q[s] = v4u{0, 0, 0, 0};
      if (live && 16u * s < a.d) q[s] = *reinterpret_cast<const v4u *>(from + 16u * s + 8u * half);
    }
  }

  const uint32_t page = 1u << a.page_shift, block = paged_block_bytes(page, a.d, kBits);
  const uint64_t page_bytes = (uint64_t)block * a.hk;
  const int32_t *table = a.table + (uint64_t)seq * a.width;
  const uint8_t *kc = a.k_cache + (uint64_t)head * block, *vc = a.v_cache + (uint64_t)head * block;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

  if (a.d != kDP) {
    for (uint32_t i = threadIdx.x * 16u; i < 2u * S::kStage; i += kThreads * 16u) *reinterpret_cast<v4u *>(lds + i) = v4u{0, 0, 0, 0};
    __syncthreads();
  }

  auto ids_of = [&](int32_t key0, uint32_t (&ids)[kSubs]) {
#pragma unroll
    for (uint32_t t = 0; t < kSubs; ++t) {
      const uint32_t at = (uint32_t)(key0 + (int32_t)(16u * t)) >> a.page_shift;
      ids[t] = __builtin_amdgcn_readfirstlane(at < a.width ? (uint32_t)table[at] : ~0u);
    }
  };
  auto pick = [&](const uint32_t (&ids)[kSubs], uint32_t sub) {
    uint32_t id = ids[0];
#pragma unroll
    for (uint32_t t = 1; t < kSubs; ++t) id = sub == t ? ids[t] : id;
    return id < a.pages ? id : 0u;
  };

  // ---- bringing a tile: places in the tile that this thread brings
  constexpr uint32_t kParts = kBits == 16 ? S::kLoads : S::kCodes;
  constexpr uint32_t kUnit = 128 / kBits;
  v4u kr[kBits == 8 ? kParts : 1], vr[kBits == 8 ? kParts : 1];
  float scale_r = 0.0f;
  auto bring = [&](int32_t key0, const uint32_t (&ids)[kSubs], uint32_t stage) {
    const uint32_t off0 = (uint32_t)key0 & (page - 1u);
    const bool one_page = page >= kKT;
    const uint32_t id0 = ids[0] < a.pages ? ids[0] : 0u;
    const uint8_t *k0 = kc + id0 * page_bytes + off0 * 16u, *v0 = vc + id0 * page_bytes + (uint64_t)(off0 / kUnit) * a.d * 16u;
#pragma unroll
    for (uint32_t j = 0; j < kParts; ++j) {
      // (wave's 64 units follow each other, in LDS too)
      const uint32_t i = (wave + kWaves * j) * 64u + lane;
      const uint32_t ku = i / kKT, key = i % kKT, vg = i / kDP, dim = i % kDP;
      const bool has_k = ku * kUnit < a.d, has_v = dim < a.d && vg * kUnit < kKT;
      if constexpr (kBits == 16) {
        const uint32_t to = lds0 + stage * S::kStage + (wave + kWaves * j) * 1024u;
        if (one_page) {
          if (has_k) load_to_lds(to, (ku * page + key) * 16u, k0);
          if (has_v) load_to_lds(to + S::kTile, (vg * a.d + dim) * 16u, v0);
        } else {
          const uint32_t ks = key / 16u, vs = vg * kUnit / 16u;
          const uint32_t ko = (uint32_t)(key0 + (int32_t)key) & (page - 1u), vo = (uint32_t)(key0 + (int32_t)(vg * kUnit)) & (page - 1u);
          if (has_k) load_to_lds(to, kc + pick(ids, ks) * page_bytes + (ku * page + ko) * 16u);
          if (has_v) load_to_lds(to + S::kTile, vc + pick(ids, vs) * page_bytes + ((uint64_t)(vo / kUnit) * a.d + dim) * 16u);
        }
      } else {
        const uint32_t ko = (uint32_t)(key0 + (int32_t)key) & (page - 1u), vo = (uint32_t)(key0 + (int32_t)(vg * kUnit)) & (page - 1u);
        if (has_k) kr[j] = *reinterpret_cast<const v4u *>(kc + pick(ids, key / 16u) * page_bytes + (ku * page + ko) * 16u);
        if (has_v) vr[j] = *reinterpret_cast<const v4u *>(vc + pick(ids, vg) * page_bytes + ((uint64_t)(vo / kUnit) * a.d + dim) * 16u);
      }
    }
    if constexpr (kBits == 8) {
      if (threadIdx.x < 2u * kKT) {
        const uint32_t key = threadIdx.x % kKT, ko = (uint32_t)(key0 + (int32_t)key) & (page - 1u);
        const uint8_t *from = threadIdx.x < kKT ? kc : vc;
        scale_r = *reinterpret_cast<const float *>(from + pick(ids, key / 16u) * page_bytes + page * a.d + ko * 4u);
      }
    }
  };
  // an int8 tile from registers into LDS
  auto settle = [&](uint32_t stage) {
    if constexpr (kBits == 8) {
      uint8_t *to = lds + stage * S::kStage;
#pragma unroll
      for (uint32_t j = 0; j < kParts; ++j) {
        const uint32_t i = (wave + kWaves * j) * 64u + lane;
        const uint32_t ku = i / kKT, key = i % kKT, vg = i / kDP, dim = i % kDP;
        if (ku * kUnit < a.d) {
          *reinterpret_cast<v4u *>(to + (2u * ku * kKT + key) * 16u) = bf16_of_codes(kr[j][0], kr[j][1]);
          *reinterpret_cast<v4u *>(to + ((2u * ku + 1u) * kKT + key) * 16u) = bf16_of_codes(kr[j][2], kr[j][3]);
        }
        if (dim < a.d && vg * kUnit < kKT) {
          *reinterpret_cast<v4u *>(to + S::kTile + (2u * vg * kDP + dim) * 16u) = bf16_of_codes(vr[j][0], vr[j][1]);
          *reinterpret_cast<v4u *>(to + S::kTile + ((2u * vg + 1u) * kDP + dim) * 16u) = bf16_of_codes(vr[j][2], vr[j][3]);
        }
      }
      if (threadIdx.x < 2u * kKT) reinterpret_cast<float *>(to + 2u * S::kTile)[threadIdx.x] = scale_r;
    }
  };

  const float scale2 = a.scale * kLog2e, cap2 = a.cap * kLog2e, inv2 = a.cap != 0.0f ? 2.0f * kLog2e / a.cap : 0.0f;
  float m = -INFINITY, l = 0.0f;
  v16f o[kDB];
#pragma unroll
  for (uint32_t b = 0; b < kDB; ++b)
#pragma unroll
    for (uint32_t i = 0; i < 16; ++i) o[b][i] = 0.0f;
  // the key of this lane's row of K in a half tile
  const uint32_t k_row = 16u * (r >> 4) + 8u * ((r >> 2) & 1u) + 4u * ((r >> 3) & 1u) + (r & 3u);

  uint32_t ids[kSubs], next_ids[kSubs];
  ids_of(begin, ids);
  if (begin < end) bring(begin, ids, 0);
  settle(0);
  ids_of(begin + (int32_t)kKT, next_ids);
  uint32_t stage = 0;
  for (int32_t key0 = begin; key0 < end; key0 += (int32_t)kKT, stage ^= 1u) {
    // this tile has arrived, and nobody reads the other stage any more
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    const bool more = key0 + (int32_t)kKT < end;
    if (more) bring(key0 + (int32_t)kKT, next_ids, stage ^ 1u);
    uint32_t after_ids[kSubs];
    ids_of(key0 + 2 * (int32_t)kKT, after_ids);
    if (key0 < any_end && key0 + (int32_t)kKT > any_low) {
      const uint8_t *kt = lds + stage * S::kStage, *vt = kt + S::kTile;
      const float *scales = reinterpret_cast<const float *>(vt + S::kTile);
      uint32_t hole = 0;  // bit t: the tile's keys 16 t.. lie in no page
#pragma unroll
      for (uint32_t t = 0; t < kSubs; ++t) hole |= ids[t] >= a.pages ? 1u << t : 0u;
      const bool whole = !hole && key0 >= whole_low && key0 + (int32_t)kKT <= whole_end;
      v16f x[kHalves];
#pragma unroll
      for (uint32_t f = 0; f < kHalves; ++f) {
#pragma unroll
        for (uint32_t i = 0; i < 16; ++i) x[f][i] = 0.0f;
#pragma unroll
        for (uint32_t s = 0; s < kDS; ++s) {
          const v4u k = *reinterpret_cast<const v4u *>(kt + ((2u * s + half) * kKT + 32u * f + k_row) * 16u);
          x[f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf(k), as_bf(q[s]), x[f], 0, 0, 0);
        }
      }
      // x: scores base 2, of keys 32 f + 16 (i / 8) + 8 half + i % 8
#pragma unroll
      for (uint32_t f = 0; f < kHalves; ++f) {
        if constexpr (kBits == 8) {
#pragma unroll
          for (uint32_t i = 0; i < 16; i += 4) {
            const v4f s = *reinterpret_cast<const v4f *>(scales + 32u * f + 16u * (i / 8u) + 8u * half + i % 8u);
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) x[f][i + e] *= s[e];
          }
        }
        if (a.cap != 0.0f) {
#pragma unroll
          for (uint32_t i = 0; i < 16; ++i) x[f][i] = capped(x[f][i] * a.scale, cap2, inv2);
        } else {
#pragma unroll
          for (uint32_t i = 0; i < 16; ++i) x[f][i] *= scale2;
        }
        if (!whole) {
#pragma unroll
          for (uint32_t i = 0; i < 16; ++i) {
            const int32_t key = key0 + (int32_t)(32u * f + 16u * (i / 8u) + 8u * half + i % 8u);
            const bool seen = key <= pos && key >= low && key < p.keys && !(hole >> (2u * f + i / 8u) & 1u);
            x[f][i] = seen ? x[f][i] : -INFINITY;
          }
        }
      }
      float top = x[0][0];
#pragma unroll
      for (uint32_t f = 0; f < kHalves; ++f)
#pragma unroll
        for (uint32_t i = 0; i < 16; ++i) top = fmaxf(top, x[f][i]);
      if (__ballot(top > m + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m, top);
        const float keep = m == -INFINITY ? 0.0f : exp2_hw(m - next);
        m = next;
        l *= keep;
#pragma unroll
        for (uint32_t b = 0; b < kDB; ++b)
#pragma unroll
          for (uint32_t i = 0; i < 16; ++i) o[b][i] *= keep;
      }
      const float base = m == -INFINITY ? 0.0f : m;
      // weights, rounded to bf16 for the matrix cores: 2^-9 of each, as the output is rounded
      v4u w[kHalves][2];
#pragma unroll
      for (uint32_t f = 0; f < kHalves; ++f)
#pragma unroll
        for (uint32_t i = 0; i < 16; i += 2) {
          float y0 = exp2_hw(x[f][i] - base), y1 = exp2_hw(x[f][i + 1] - base);
          l += y0 + y1;
          if constexpr (kBits == 8) {
            const float2 s = *reinterpret_cast<const float2 *>(scales + kKT + 32u * f + 16u * (i / 8u) + 8u * half + i % 8u);
            y0 = x[f][i] == -INFINITY ? 0.0f : y0 * s.x;
            y1 = x[f][i + 1] == -INFINITY ? 0.0f : y1 * s.y;
          }
          w[f][i / 8u][i % 8u / 2u] = two_bf16(y0, y1);
        }
      bool bad = false;
      if constexpr (kBits == 16) {
        if (!whole) {
#pragma unroll 1
          for (uint32_t i = lane; i < S::kTile / 16u; i += 64u) bad |= any_not_finite(*reinterpret_cast<const v4u *>(vt + i * 16u));
          bad = __ballot(bad) != 0u;
        }
      }
      if (!bad) {
#pragma unroll
        for (uint32_t f = 0; f < kHalves; ++f)
#pragma unroll
          for (uint32_t kk = 0; kk < 2; ++kk)
#pragma unroll
            for (uint32_t b = 0; b < kDB; ++b) {
              const v4u v = *reinterpret_cast<const v4u *>(vt + ((4u * f + 2u * kk + half) * kDP + 32u * b + r) * 16u);
              o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf(v), as_bf(w[f][kk]), o[b], 0, 0, 0);
            }
      } else {
        // A NaN or an infinity among the values of a tile that not every row sees
        // whole: 0 * NaN must not reach the rows that do not see its key.  One
        // key at a time, added where it is seen.
#pragma unroll 1
        for (uint32_t key = 0; key < kKT; ++key) {
          const uint32_t group = key / 8u, e = key % 8u;
          const int32_t place = key0 + (int32_t)key;
          const bool seen = place <= pos && place >= low && place < p.keys && !(hole >> (key / 16u) & 1u);
          const bool here = half == (group & 1u);
          const uint32_t keep = here ? (e & 1u ? 0xFFFF0000u : 0xFFFFu) : 0u;
          v4u sel, mine = w[0][0];
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) sel[i] = e / 2u == i ? keep : 0u;
#pragma unroll
          for (uint32_t f = 0; f < kHalves; ++f)
#pragma unroll
            for (uint32_t kk = 0; kk < 2; ++kk) mine = group / 2u == 2u * f + kk ? w[f][kk] : mine;
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b) {
            const v4u v = *reinterpret_cast<const v4u *>(vt + ((group / 2u * 2u + half) * kDP + 32u * b + r) * 16u);
            v16f one;
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i) one[i] = 0.0f;
            one = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf(v & sel), as_bf(mine & sel), one, 0, 0, 0);
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i) o[b][i] += seen ? one[i] : 0.0f;
          }
        }
      }
    }
    if (more) settle(stage ^ 1u);
#pragma unroll
    for (uint32_t t = 0; t < kSubs; ++t) ids[t] = next_ids[t], next_ids[t] = after_ids[t];
  }

  // rows leave through LDS, where the stages were (each wave's own part)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  l += __shfl_xor(l, 32, 64);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint8_t *mine = lds + wave * 32u * S::kOutPitch;
#pragma unroll
  for (uint32_t b = 0; b < kDB; ++b)
#pragma unroll
    for (uint32_t i = 0; i < 16; i += 4)
      *reinterpret_cast<uint2 *>(mine + r * S::kOutPitch + (32u * b + 2u * i + 4u * half) * 2u) =
          make_uint2(two_bf16(o[b][i] * inv, o[b][i + 1] * inv), two_bf16(o[b][i + 2] * inv, o[b][i + 3] * inv));
  __syncthreads();
  const uint32_t pieces = a.d / 8u;
  for (uint32_t i = lane; i < 32u * pieces; i += 64u) {
    const uint32_t at = i / pieces, piece = i % pieces, to = wrow0 + at;
    if (to >= rows) break;
    *reinterpret_cast<uint4 *>(a.out + ((uint64_t)(p.first + to / g) * a.hq + head * g + to % g) * a.d + piece * 8u) =
        *reinterpret_cast<const uint4 *>(mine + at * S::kOutPitch + piece * 16u);
  }
}

template <uint32_t kDP, uint32_t kBits>
hipError_t launch(const PagedArgs &a, hipStream_t s) {
  constexpr uint32_t kLds = Shape<kDP, kBits>::kLds;
  auto *kernel = paged_prefill_kernel<kDP, kBits>;
  if (kLds > 65536u) {
    const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void *>(kernel), (int)kLds);
    if (e != hipSuccess) return e;
  }
  // (of a sequence with rows: at most one tile that is not full)
  const uint64_t rows = (uint64_t)a.tokens * (a.hq / a.hk), tiles = rows / kRows + std::min(a.count, a.tokens);
  hipLaunchKernelGGL(kernel, dim3((uint32_t)(tiles * a.hk)), dim3(kThreads), kLds, s, a);
  return hipGetLastError();
}

template <uint32_t kBits>
hipError_t launch_heads(const PagedArgs &a, hipStream_t s) {
  if (a.d <= 64u) return launch<64, kBits>(a, s);
  if (a.d <= 96u) return launch<96, kBits>(a, s);
  if (a.d <= 128u) return launch<128, kBits>(a, s);
  if (a.d <= 192u) return launch<192, kBits>(a, s);
  return launch<256, kBits>(a, s);
}

}  // namespace

hipError_t launch_paged_prefill(const PagedArgs &a, hipStream_t s) {
  return a.bits == 16u ? launch_heads<16>(a, s) : launch_heads<8>(a, s);
}

}  // namespace bqmm
