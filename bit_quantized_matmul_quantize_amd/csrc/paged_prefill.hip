// Attention of prompts over the paged key-value cache:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - max s),  s_j = scale q . k_j, capped,
// in one pass over the cache with the running maximum and sum of the softmax.
//
// Bound by the matrix cores (4 d operations for each head and pair of tokens),
// and by the exponentials beside them: 4096 tokens behind 12288, 32 heads over 8 of
// 128, 838 us, 1.1 PFLOP/s, the matrix cores 63% busy (834 to 882 on different cards).
// A workgroup takes 128 rows, 32 a wave, which each operand read from LDS then
// serves: the heads of consecutive tokens that share a key head, so that a tile of
// keys serves them all and few pairs are masked.  Tiles of keys and values come from the cache
// straight into LDS, in its units, while the last ones are computed; an int8
// cache goes through registers and lies in LDS as bf16 (codes are exact; scales
// are applied to scores and weights).
//
// S^T = K Q^T and O^T = V^T P^T: a lane's scores belong to one row, so that the
// softmax needs no exchange between lanes, and the weights of its keys are an
// operand of the second product as they are, given the order in which K's rows
// are read: row 8 b + 4 h + j of the first product is key 16 (b / 2) + 8 h + 4 (b % 2) + j.
#include "paged_common.h"

namespace bqmm {
namespace {

constexpr uint32_t kWaves = 4;
constexpr uint32_t kThreads = 64 * kWaves;
constexpr uint32_t kRows = 32 * kWaves;
// Up to so many workgroups (two to a compute unit) take two groups of waves each: a
// prompt of 1024 tokens 25 us (with one 27), of 2048 50 (53); one of 3000, with 752
// workgroups, 98 (84).
constexpr uint32_t kFew = 512;
constexpr uint32_t kCus = 256;

// 16 bytes a lane straight from memory into LDS: lane i's go to the wave's
// destination + 16 i.  The kernel waits itself; no register is written.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t offset, const uint8_t *base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(uint32_t lds, const uint8_t *from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}

// kRuns of them, 1024 bytes apart in memory and in LDS.
template <uint32_t kRuns>
__device__ __forceinline__ void load_run_to_lds(uint32_t lds, uint32_t offset, const uint8_t *base) {
  static_assert(kRuns >= 1 && kRuns <= 4, "");
  if constexpr (kRuns == 1)
    load_to_lds(lds, offset, base);
  else if constexpr (kRuns == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:1024" ::"s"(lds), "v"(offset), "s"(base) : "memory", "m0");
  else if constexpr (kRuns == 3)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:1024\n\tglobal_load_lds_dwordx4 %1, %2 offset:2048"
                 ::"s"(lds), "v"(offset), "s"(base) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:1024\n\tglobal_load_lds_dwordx4 %1, %2 offset:2048\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:%3" ::"s"(lds), "v"(offset), "s"(base), "n"(3 * 1024) : "memory", "m0");
}

// kDP: values of a head, rounded up (the ones beyond are zero).
template <uint32_t kDP, uint32_t kBits>
struct Shape {
  static constexpr uint32_t kKT = kDP <= 128 ? 64 : 32;      // keys of a tile
  static constexpr uint32_t kSubs = kKT / 16;                // parts of it that lie in one page
  static constexpr uint32_t kTile = kKT * kDP * 2;           // bytes of its keys, or values
  static constexpr uint32_t kStage = 2 * kTile + (kBits == 8 ? 3 * kKT * 4 : 0);  // (and its scales)
  static constexpr uint32_t kLoads = kTile / 16 / kThreads;  // bf16: of a thread, for keys, and for values
  static constexpr uint32_t kCodes = (kTile / 32 + kThreads - 1) / kThreads;  // int8
  static constexpr uint32_t kOutPitch = kDP * 2 + 16;        // bytes of a row of the output in LDS
  static constexpr uint32_t kLds = 2 * kStage > kRows * kOutPitch ? 2 * kStage : kRows * kOutPitch;
};

__device__ __forceinline__ uint32_t tiles_of(const PagedArgs &a, const PagedSpan &p) {
  return (uint32_t)(((uint64_t)p.n * (a.hq / a.hk) + kRows - 1u) / kRows);
}

// The tile of rows that workgroup `item` of a key head takes: those with the most
// keys first, since the last to end decide.  Sequences by their longest tile (up to
// 64 of them; more are taken as they come: prompts of 20 to 400 tokens behind up to 3000, 64
// sequences 209 us, with an empty one more 216, int8 244 and 279), their tiles from the last
// one back.
// kPairs: two workgroups share a compute unit, the second ones of all units come in
// reverse, so that the longest tiles have the shortest ones beside them: prompts of
// 1300, 700, 129 and fewer tokens behind up to 4000 143 us (in order 150).
template <bool kPairs>
__device__ __forceinline__ bool take_tile(const PagedArgs &a, uint32_t item, uint32_t *seq, uint32_t *tile) {
  const uint32_t lane = __lane_id();
  if (a.count > 64u) {
    uint32_t inside;
    if (!paged_find(item, a.count, [&](uint32_t i) { return tiles_of(a, paged_span(a, i)); }, seq, &inside)) return false;
    *tile = tiles_of(a, paged_span(a, *seq)) - 1u - inside;
    return true;
  }
  uint32_t mine = 0, keys = 0;
  if (lane < a.count) {
    const PagedSpan p = paged_span(a, lane);
    mine = tiles_of(a, p);
    keys = mine ? (uint32_t)min(p.keys, max(p.at + (int32_t)p.n, 0)) + 1u : 0u;
    if (a.window) keys = min(keys, a.window + p.n);
  }
  uint32_t before = 0, all = mine;
  if (a.count > 1u) {
    all = 0;
    for (uint32_t i = 0; i < a.count; ++i) {  // tiles of the sequences that come first
      const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)keys, (int)i), n = (uint32_t)__builtin_amdgcn_readlane((int)mine, (int)i);
      before += k > keys || (k == keys && i < lane) ? n : 0u;
      all += n;
    }
  }
  all = __builtin_amdgcn_readfirstlane(all);
  if (item >= all) return false;
  if constexpr (kPairs) {
    const uint32_t round = kCus / a.hk;  // tiles of the first workgroups of all compute units
    if (item >= round && item < 2u * round) item = min(all, 2u * round) - 1u - (item - round);
  }
  const uint64_t who = __ballot(item >= before && item - before < mine);
  const uint32_t w = (uint32_t)__builtin_ctzll(who);
  *seq = __builtin_amdgcn_readfirstlane(w);
  *tile = (uint32_t)__builtin_amdgcn_readlane((int)(mine - 1u - (item - before)), (int)w);
  return true;
}

// kExact: a head has kDP values, and a page has at least a tile's keys.
// kCap: 0: scores are as they are; 1: capped, by up to kShortCap; 2: by more.
// kGroups: groups of four waves; two of them share the tiles of keys of the same rows.
template <uint32_t kDP, uint32_t kBits, bool kExact, int kCap, uint32_t kGroups>
__global__ __launch_bounds__(kThreads * kGroups, 2) void paged_prefill_kernel(PagedArgs a) {
  using S = Shape<kDP, kBits>;
  constexpr uint32_t kKT = S::kKT, kSubs = S::kSubs;
  constexpr uint32_t kHalves = kKT / 32;  // halves of a tile: 32 keys
  constexpr uint32_t kDS = kDP / 16;      // steps of the first product
  constexpr uint32_t kDB = kDP / 32;      // blocks of the second, two steps each
  extern __shared__ __attribute__((aligned(16))) uint8_t all_lds[];

  // a group's threads and LDS
  const uint32_t group = kGroups == 1 ? 0u : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads), thread = threadIdx.x % kThreads;
  uint8_t *const lds = all_lds + group * (2u * S::kStage);
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(thread >> 6);
  const uint32_t r = lane & 31u, half = lane >> 5;
  const uint32_t head = blockIdx.x % a.hk, g = a.hq / a.hk;
  uint32_t seq, tile;
  if (!take_tile<kGroups == 1>(a, blockIdx.x / a.hk, &seq, &tile)) return;
  const PagedSpan p = paged_span(a, seq);
  const uint32_t rows = p.n * g;

  // what rows see: key <= place, and key > place - window
  auto place_of = [&](uint32_t row) { return p.at + (int32_t)(row / g); };
  auto low_of = [&](int32_t place) { return a.window ? (int32_t)max((int64_t)place + 1 - (int64_t)a.window, (int64_t)0) : 0; };
  const uint32_t row0 = tile * kRows, row1 = min(row0 + kRows, rows) - 1u;
  const int32_t end = min(p.keys, max(place_of(row1) + 1, 0));
  const int32_t first = low_of(place_of(row0)), begin = first / (int32_t)kKT * (int32_t)kKT;  // keys that any row sees: [first, end)
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

  const uint32_t d = kExact ? kDP : a.d;
  const uint32_t page = 1u << a.page_shift, block = paged_block_bytes(page, d, kBits);
  const uint64_t page_bytes = (uint64_t)block * a.hk;
  const int32_t *table = a.table + (uint64_t)seq * a.width;
  const uint8_t *kc = a.k_cache + (uint64_t)head * block, *vc = a.v_cache + (uint64_t)head * block;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

  if constexpr (!kExact) {
    for (uint32_t i = thread * 16u; i < 2u * S::kStage; i += kThreads * 16u) *reinterpret_cast<v4u *>(lds + i) = v4u{0, 0, 0, 0};
    __syncthreads();
  }

  // The page of the tile's keys 16 t..: in the lanes 16 t.. (and those a tile later).
  // A vector load: a scalar one would be waited for with the operands read from LDS.
  auto id_of = [&](int32_t key0) {
    const uint32_t at = (uint32_t)(key0 + (int32_t)(lane % kKT & ~15u)) >> a.page_shift;
    return at < a.width ? (uint32_t)table[at] : ~0u;
  };
  auto known = [&](uint32_t id) { return id < a.pages ? id : 0u; };

  // ---- bringing a tile: a wave's 64 units at a time follow each other, in LDS too
  constexpr uint32_t kParts = kBits == 16 ? S::kLoads : S::kCodes;
  constexpr uint32_t kUnit = 128 / kBits;
  constexpr bool kFull = kParts * kThreads * 16 == S::kTile * kBits / 16;  // every thread has a unit in every part
  v4u kr[kBits == 8 ? kParts : 1], vr[kBits == 8 ? kParts : 1];
  float k_scale = 0.0f, v_scale = 0.0f;
  auto bring_k = [&](int32_t key0, uint32_t id, uint32_t stage) {
    const uint32_t off0 = (uint32_t)key0 & (page - 1u), key = lane % kKT, ko = (uint32_t)(key0 + (int32_t)key) & (page - 1u);
    const bool one_page = kExact || page >= kKT;
    const uint32_t id0 = known(__builtin_amdgcn_readfirstlane(id));
    const uint8_t *k0 = kc + id0 * page_bytes + off0 * 16u;
    const uint8_t *mine = kc + known(id) * page_bytes;  // (its key is the same in all parts)
#pragma unroll
    for (uint32_t j = 0; j < kParts; ++j) {
      const uint32_t to = lds0 + stage * S::kStage + (wave * kParts + j) * 1024u;
      if constexpr (kBits == 16 && kExact) {
        load_to_lds(to, (lane / kKT * page + key) * 16u, k0 + (uint64_t)((wave * kParts + j) * (64u / kKT)) * page * 16u);
      } else {
        const uint32_t ku = ((wave * kParts + j) * 64u + lane) / kKT;
        const uint8_t *from = one_page ? k0 + (ku * page + key) * 16u : mine + (ku * page + ko) * 16u;
        if ((kExact && kFull) || ku * kUnit < d) {
          if constexpr (kBits == 16)
            load_to_lds(to, from);
          else
            kr[j] = *reinterpret_cast<const v4u *>(from);
        }
      }
    }
    if constexpr (kBits == 8) {
      if (thread < kKT) k_scale = *reinterpret_cast<const float *>(kc + known(id) * page_bytes + page * d + ko * 4u);
    }
  };
  auto bring_v = [&](int32_t key0, uint32_t id, uint32_t stage) {
    const uint32_t off0 = (uint32_t)key0 & (page - 1u);
    const bool one_page = kExact || page >= kKT;
    const uint32_t id0 = known(__builtin_amdgcn_readfirstlane(id));
    const uint8_t *v0 = vc + id0 * page_bytes + (uint64_t)(off0 / kUnit) * d * 16u;
    const uint32_t to = lds0 + stage * S::kStage + S::kTile + wave * kParts * 1024u;
    if constexpr (kBits == 16 && kExact) {
      load_run_to_lds<kParts>(to, lane * 16u, v0 + wave * kParts * 1024u);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < kParts; ++j) {
        const uint32_t i = (wave * kParts + j) * 64u + lane, vg = i / kDP, dim = i % kDP;
        const uint32_t vo = (uint32_t)(key0 + (int32_t)(vg * kUnit)) & (page - 1u);
        // (the lanes of a wave's 64 units may lie in two groups of keys where kDP is no multiple of 64)
        const uint32_t sub = vg * kUnit / 16u * 16u;
        const uint32_t vid = one_page ? id0 : known(kDP % 64u == 0u ? (uint32_t)__builtin_amdgcn_readlane((int)id, (int)__builtin_amdgcn_readfirstlane(sub % 64u)) : (uint32_t)__shfl((int)id, (int)(sub % 64u), 64));
        const uint8_t *from = one_page ? v0 + (vg * d + dim) * 16u : vc + vid * page_bytes + ((uint64_t)(vo / kUnit) * d + dim) * 16u;
        if ((kExact && kFull) || (dim < d && vg * kUnit < kKT)) {
          if constexpr (kBits == 16)
            load_to_lds(to + j * 1024u, from);
          else
            vr[j] = *reinterpret_cast<const v4u *>(from);
        }
      }
    }
    if constexpr (kBits == 8) {
      const uint32_t ko = (uint32_t)(key0 + (int32_t)(lane % kKT)) & (page - 1u);
      if (thread < kKT) v_scale = *reinterpret_cast<const float *>(vc + known(id) * page_bytes + page * d + ko * 4u);
    }
  };
  const int32_t all_low = low_of(place_of(row1)), all_end = min(p.keys, place_of(row0) + 1);  // seen by all rows
  auto whole_for_all = [&](int32_t key0, uint64_t hole) { return !hole && key0 >= all_low && key0 + (int32_t)kKT <= all_end; };
  // an int8 tile from registers into LDS
  auto settle = [&](uint32_t stage, bool whole) {
    if constexpr (kBits == 8) {
      uint8_t *to = lds + stage * S::kStage;
#pragma unroll
      for (uint32_t j = 0; j < kParts; ++j) {
        const uint32_t i = (wave * kParts + j) * 64u + lane;
        const uint32_t ku = i / kKT, key = i % kKT, vg = i / kDP, dim = i % kDP;
        asm volatile("" : "+v"(kr[j]), "+v"(vr[j]));  // (else every code is carried in a register of its own)
        if ((kExact && kFull) || ku * kUnit < d) {
          *reinterpret_cast<v4u *>(to + (2u * ku * kKT + key) * 16u) = bf16_of_codes(kr[j][0], kr[j][1]);
          *reinterpret_cast<v4u *>(to + ((2u * ku + 1u) * kKT + key) * 16u) = bf16_of_codes(kr[j][2], kr[j][3]);
        }
        if ((kExact && kFull) || (dim < d && vg * kUnit < kKT)) {
          *reinterpret_cast<v4u *>(to + S::kTile + (2u * vg * kDP + dim) * 16u) = bf16_of_codes(vr[j][0], vr[j][1]);
          *reinterpret_cast<v4u *>(to + S::kTile + ((2u * vg + 1u) * kDP + dim) * 16u) = bf16_of_codes(vr[j][2], vr[j][3]);
        }
      }
      float *scales = reinterpret_cast<float *>(to + 2u * S::kTile);
      if (thread < kKT) {
        scales[thread] = k_scale;
        // (of a tile that some rows do not see whole, see below)
        scales[kKT + thread] = whole || (__float_as_uint(v_scale) & 0x7F800000u) != 0x7F800000u ? v_scale : 0.0f;
        scales[2u * kKT + thread] = v_scale;
      }
    }
  };

  // (vector registers: with more scalar ones the loop loads arguments anew for each tile)
  float scale2 = a.scale2, cap2 = a.cap2, inv2 = a.cap_inv2;
  asm volatile("" : "+v"(scale2), "+v"(cap2), "+v"(inv2));
  float m = -INFINITY, l = 0.0f;
  v16f o[kDB];
#pragma unroll
  for (uint32_t b = 0; b < kDB; ++b)
#pragma unroll
    for (uint32_t i = 0; i < 16; ++i) o[b][i] = 0.0f;
  // the key of this lane's row of K in a half tile
  const uint32_t k_row = 16u * (r >> 4) + 8u * ((r >> 2) & 1u) + 4u * ((r >> 3) & 1u) + (r & 3u);
  const uint32_t k_at = (half * kKT + k_row) * 16u, v_at = (half * kDP + r) * 16u;

  // 0 * NaN must not reach a row that does not see the NaN's key.  Of tiles that not
  // every row of the workgroup sees whole, values that no row sees and values that
  // are not finite are zeroed in LDS; a second loop adds the latter where they are
  // seen.  Codes are finite, and their scales are made so: one that is not turns the
  // sum of the weights of a row that sees it into NaN.
  auto zero_some = [&](int32_t key0, uint32_t stage, uint64_t hole) {  // gives whether some are not finite
    bool bad = false;
#pragma unroll 1
    for (uint32_t i = thread; i < S::kTile / 16u; i += kThreads) {
      const uint32_t run = i / kDP;  // of eight keys
      const int32_t at = key0 + (int32_t)(8u * run), from = max(first - at, 0), to = min(end - 1 - at, 7);
      const uint32_t seen = hole >> (8u * run & ~15u) & 1u || from > to ? 0u : (0xFFu >> (7 - to)) & (0xFFu << from);
      v4u *u = reinterpret_cast<v4u *>(lds + stage * S::kStage + S::kTile + i * 16u), v = *u;
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) v[e] &= (seen >> (2u * e) & 1u ? 0xFFFFu : 0u) | (seen >> (2u * e + 1u) & 1u ? 0xFFFF0000u : 0u);
      bad |= any_not_finite(v);
      *u = finite_only(v);
    }
    return bad;
  };

  auto whole_at = [&](int32_t key0, uint64_t hole) { return !hole && key0 >= whole_low && key0 + (int32_t)kKT <= whole_end; };
  auto some_at = [&](int32_t key0) { return key0 < any_end && key0 + (int32_t)kKT > any_low; };
  // the keys 16 t.. of a tile that this row sees: of key0 + 16 t + 8 half + i, bit i
  auto seen_of = [&](int32_t key0, uint64_t hole, uint32_t t) {
    const int32_t at = key0 + (int32_t)(16u * t + 8u * half), from = max(low - at, 0), to = min(min(pos, p.keys - 1) - at, 7);
    return hole >> (16u * t) & 1u || from > to ? 0u : (0xFFu >> (7 - to)) & (0xFFu << from);
  };

  // One tile.  hole: bit 16 t where the tile's keys 16 t.. lie in no page; whole: all
  // rows of the wave see all of it, for_all: and those of the workgroup.
  auto compute = [&](int32_t key0, uint32_t stage, uint64_t hole, bool whole, bool for_all) {
    const uint8_t *kt = lds + stage * S::kStage + k_at, *vt = lds + stage * S::kStage + S::kTile + v_at;
    const float *scales = reinterpret_cast<const float *>(lds + stage * S::kStage + 2u * S::kTile) + 8u * half;
    // operands are read kAhead products before they are used, those of the second
    // product from before the softmax on
    // (products that follow each other belong to different sums: one has to wait for
    // the last one of its own)
    auto read_k = [&](uint32_t n) { return *reinterpret_cast<const v4u *>(kt + (2u * (n / kHalves) * kKT + 32u * (n % kHalves)) * 16u); };
    auto read_v = [&](uint32_t n) { return *reinterpret_cast<const v4u *>(vt + (2u * (n / kDB) * kDP + 32u * (n % kDB)) * 16u); };
    constexpr uint32_t kAhead = kDP > 128 ? 4 : 8, kFirst = kHalves * kDS, kSecond = kHalves * 2u * kDB;
    v16f x[kHalves];  // of keys 32 f + 16 (i / 8) + 8 half + i % 8
    v4u ring[kAhead];
#pragma unroll
    for (uint32_t n = 0; n < kAhead; ++n) ring[n] = read_k(n);
#pragma unroll
    for (uint32_t f = 0; f < kHalves; ++f)
#pragma unroll
      for (uint32_t i = 0; i < 16; ++i) x[f][i] = 0.0f;
#pragma unroll
    for (uint32_t n = 0; n < kFirst; ++n) {
      x[n % kHalves] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf(ring[n % kAhead]), as_bf(q[n / kHalves]), x[n % kHalves], 0, 0, 0);
      ring[n % kAhead] = n + kAhead < kFirst ? read_k(n + kAhead) : read_v(n + kAhead - kFirst);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (uint32_t f = 0; f < kHalves; ++f) {
      if constexpr (kBits == 8) {
#pragma unroll
        for (uint32_t i = 0; i < 16; i += 4) {
          const v4f s = *reinterpret_cast<const v4f *>(scales + 32u * f + 16u * (i / 8u) + i % 8u);
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) x[f][i + e] *= s[e];
        }
      }
      if constexpr (kCap != 0) {
#pragma unroll
        for (uint32_t i = 0; i < 16; ++i) x[f][i] = kCap == 1 ? capped(x[f][i], cap2, inv2) : capped_large(x[f][i], a);
      }
    }
    if (!whole) {
#pragma unroll
      for (uint32_t f = 0; f < kHalves; ++f)
#pragma unroll
        for (uint32_t kk = 0; kk < 2; ++kk) {
          uint32_t seen = seen_of(key0, hole, 2u * f + kk);
          asm volatile("" : "+v"(seen));  // (keeps this a branch: selects in every tile cost a tenth of it)
#pragma unroll
          for (uint32_t i = 0; i < 8; ++i) x[f][8u * kk + i] = seen >> i & 1u ? x[f][8u * kk + i] : -INFINITY;
        }
    }
    float top = x[0][0];
#pragma unroll
    for (uint32_t f = 0; f < kHalves; ++f)
#pragma unroll
      for (uint32_t i = 0; i < 16; i += 2) top = fmaxf(fmaxf(x[f][i], x[f][i + 1]), top);
    top *= scale2;
    if (__ballot(top > m)) {
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float next = fmaxf(m, top + kSlack);
      const float keep = m == -INFINITY ? 0.0f : exp2_hw(m - next);
      m = next;
      l *= keep;
#pragma unroll
      for (uint32_t b = 0; b < kDB; ++b)
#pragma unroll
        for (uint32_t i = 0; i < 16; ++i) o[b][i] *= keep;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    // Weights, rounded to bf16 for the matrix cores: 2^-8 of each at most, as the
    // output is rounded.  Their sum is that of the rounded ones (bf16), so that weights
    // and sum are off together.
    v4u w[kHalves][2];
#pragma unroll
    for (uint32_t f = 0; f < kHalves; ++f)
#pragma unroll
      for (uint32_t i = 0; i < 16; i += 2) {
        float y0 = exp2_hw(fmaf(x[f][i], scale2, -base)), y1 = exp2_hw(fmaf(x[f][i + 1], scale2, -base));
        if constexpr (kBits == 8) {
          l += y0 + y1;
          const float2 s = *reinterpret_cast<const float2 *>(scales + kKT + 32u * f + 16u * (i / 8u) + i % 8u);
          y0 *= s.x;
          y1 *= s.y;
        }
        const uint32_t two = two_bf16(y0, y1);
        if constexpr (kBits == 16) l = add_two_bf16(two, l);
        w[f][i / 8u][i % 8u / 2u] = two;
      }
    if (kBits == 8 && !for_all) {
#pragma unroll 1
      for (uint32_t t = 0; t < kSubs; ++t) {
        const uint32_t seen = seen_of(key0, hole, t);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) l = seen >> i & 1u ? fmaf(scales[2u * kKT + 16u * t + i], 0.0f, l) : l;
      }
    }
#pragma unroll
    for (uint32_t n = 0; n < kSecond; ++n) {
      const uint32_t at = (kFirst + n) % kAhead, b = n % kDB, kk = n / kDB;
      o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf(ring[at]), as_bf(w[kk / 2u][kk % 2u]), o[b], 0, 0, 0);
      if (n + kAhead < kSecond) ring[at] = read_v(n + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // The groups take the tiles in turn; the loop is the same for all of the workgroup.
  constexpr int32_t kStep = (int32_t)(kKT * kGroups);
  const int32_t own = begin + (int32_t)(kKT * group);
  // (of both groups' tiles: whether some rows of the workgroup do not see a key of them)
  auto for_all_groups = [&](int32_t key0, uint32_t id, uint32_t other) {
    if (kGroups == 1) return whole_for_all(key0, __ballot(id >= a.pages));
    const int32_t base = key0 - (int32_t)(kKT * group);
    return !__ballot(id >= a.pages || other >= a.pages) && base >= all_low && base + kStep <= all_end;
  };
  auto other_of = [&](int32_t key0) { return kGroups == 1 ? 0u : id_of(group ? key0 - (int32_t)kKT : key0 + (int32_t)kKT); };
  bool later = false;
  uint32_t id = id_of(own), other = other_of(own);
  if (own < end) {
    bring_k(own, id, 0);
    bring_v(own, id, 0);
    settle(0, whole_for_all(own, __ballot(id >= a.pages)));
  }
  uint32_t next_id = id_of(own + kStep), next_other = other_of(own + kStep);
  uint32_t stage = 0;
  for (int32_t base = begin, key0 = own; base < end; base += kStep, key0 += kStep, stage ^= 1u) {
    // this tile has arrived, and nobody reads the other stage any more
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    const uint64_t hole = __ballot(id >= a.pages);
    const bool more = key0 + kStep < end;
    if (more) {
      bring_k(key0 + kStep, next_id, stage ^ 1u);
      bring_v(key0 + kStep, next_id, stage ^ 1u);
    }
    // (each group its own tile, and only where the second loop comes to it again)
    if (kBits == 16 && !for_all_groups(key0, id, other))
      later |= __syncthreads_or(key0 < end && !whole_for_all(key0, hole) && zero_some(key0, stage, hole)) != 0;
    id = next_id;
    other = next_other;
    next_id = id_of(key0 + 2 * kStep);
    next_other = other_of(key0 + 2 * kStep);
    if (key0 < end && some_at(key0)) compute(key0, stage, hole, whole_at(key0, hole), whole_for_all(key0, hole));
    if (more) settle(stage ^ 1u, whole_for_all(key0 + kStep, __ballot(id >= a.pages)));
  }
  if constexpr (kGroups == 2) {
    // the second group's sums to the first, through LDS
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    constexpr uint32_t kRuns = kDB * 4u;
    v4f *const sums = reinterpret_cast<v4f *>(all_lds) + wave * (kRuns * 64u) + lane;
    float2 *const stats = reinterpret_cast<float2 *>(all_lds + kRuns * 16u * kThreads) + thread;
    if (group == 1u) {
      *stats = make_float2(m, l);
#pragma unroll
      for (uint32_t i = 0; i < kRuns; ++i) sums[i * 64u] = v4f{o[i / 4u][i % 4u * 4u], o[i / 4u][i % 4u * 4u + 1u], o[i / 4u][i % 4u * 4u + 2u], o[i / 4u][i % 4u * 4u + 3u]};
    }
    __syncthreads();
    if (group == 0u) {
      const float2 theirs = *stats;
      const float next = fmaxf(m, theirs.x);
      const float f = m == -INFINITY ? 0.0f : exp2_hw(m - next), g2 = theirs.x == -INFINITY ? 0.0f : exp2_hw(theirs.x - next);
      l = l * f + theirs.y * g2;
#pragma unroll
      for (uint32_t i = 0; i < kRuns; ++i) {
        const v4f y = sums[i * 64u];
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) o[i / 4u][i % 4u * 4u + e] = o[i / 4u][i % 4u * 4u + e] * f + y[e] * g2;
      }
    }
  }
  if constexpr (kBits == 16) {
    if (later) {  // (the same for the whole workgroup)
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
#pragma unroll 1
      for (int32_t key0 = begin; key0 < end; key0 += (int32_t)kKT) {
        id = id_of(key0);
        const uint64_t hole = __ballot(id >= a.pages);
        if (whole_for_all(key0, hole)) continue;
        bring_v(key0, id, 0);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
#pragma unroll 1
        for (uint32_t t = 0; t < kSubs; ++t) {
          const uint32_t seen = seen_of(key0, hole, t);
          v4u ones;  // 1 for the keys that are seen
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) ones[i] = (seen >> (2u * i) & 1u ? 0x3F80u : 0u) | (seen >> (2u * i + 1u) & 1u ? 0x3F800000u : 0u);
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b) {
            const v4u u = *reinterpret_cast<const v4u *>(lds + S::kTile + v_at + (2u * t * kDP + 32u * b) * 16u);
            v16f marks;
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i) marks[i] = 0.0f;
            marks = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf(not_finite_marks(u)), as_bf(ones), marks, 0, 0, 0);
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i) o[b][i] += of_marks(marks[i]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        __syncthreads();
      }
    }
  }

  // rows leave through LDS, where the stages were (each wave's own part)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  l += __shfl_xor(l, 32, 64);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (group != 0u) return;
  uint8_t *mine = all_lds + wave * 32u * S::kOutPitch;
#pragma unroll
  for (uint32_t b = 0; b < kDB; ++b)
#pragma unroll
    for (uint32_t i = 0; i < 16; i += 4)
      *reinterpret_cast<uint2 *>(mine + r * S::kOutPitch + (32u * b + 2u * i + 4u * half) * 2u) =
          make_uint2(two_bf16(o[b][i] * inv, o[b][i + 1] * inv), two_bf16(o[b][i + 2] * inv, o[b][i + 3] * inv));
  __builtin_amdgcn_wave_barrier();  // (a wave's own rows: LDS is in order)
  const uint32_t pieces = d / 8u;
  for (uint32_t i = lane; i < 32u * pieces; i += 64u) {
    const uint32_t at = i / pieces, piece = i % pieces, to = wrow0 + at;
    if (to >= rows) break;
    *reinterpret_cast<uint4 *>(a.out + ((uint64_t)(p.first + to / g) * a.hq + head * g + to % g) * d + piece * 8u) =
        *reinterpret_cast<const uint4 *>(mine + at * S::kOutPitch + piece * 16u);
  }
}

template <uint32_t kDP, uint32_t kBits, bool kExact, int kCap, uint32_t kGroups>
hipError_t launch(const PagedArgs &a, uint32_t groups, hipStream_t s) {
  using S = Shape<kDP, kBits>;
  constexpr uint32_t kSums = (kDP * 2u + 8u) * kThreads;  // of the second group
  constexpr uint32_t kLds = kGroups == 1 ? S::kLds : std::max(4u * S::kStage, kSums);
  auto *kernel = paged_prefill_kernel<kDP, kBits, kExact, kCap, kGroups>;
  if (kLds > 65536u) {
    const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void *>(kernel), (int)kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3(groups), dim3(kThreads * kGroups), kLds, s, a);
  return hipGetLastError();
}

template <uint32_t kDP, uint32_t kBits, bool kExact, int kCap>
hipError_t launch_groups(const PagedArgs &a, hipStream_t s) {
  // (of a sequence with rows: at most one tile that is not full)
  const uint64_t rows = (uint64_t)a.tokens * (a.hq / a.hk), tiles = (rows + (kRows - 1ull) * std::min(a.count, a.tokens)) / kRows;
  const uint32_t groups = (uint32_t)(tiles * a.hk);
  return groups <= kFew ? launch<kDP, kBits, kExact, kCap, 2>(a, groups, s) : launch<kDP, kBits, kExact, kCap, 1>(a, groups, s);
}

template <uint32_t kDP, uint32_t kBits>
hipError_t launch_exact(const PagedArgs &a, hipStream_t s) {
  const bool exact = a.d == kDP && (1u << a.page_shift) >= Shape<kDP, kBits>::kKT;
  if (a.cap == 0.0f) return exact ? launch_groups<kDP, kBits, true, 0>(a, s) : launch_groups<kDP, kBits, false, 0>(a, s);
  if (a.cap <= kShortCap) return exact ? launch_groups<kDP, kBits, true, 1>(a, s) : launch_groups<kDP, kBits, false, 1>(a, s);
  return launch_groups<kDP, kBits, false, 2>(a, s);  // (rare: for all heads and pages alike)
}

template <uint32_t kBits>
hipError_t launch_heads(const PagedArgs &a, hipStream_t s) {
  if (a.d <= 64u) return launch_exact<64, kBits>(a, s);
  if (a.d <= 96u) return launch_exact<96, kBits>(a, s);
  if (a.d <= 128u) return launch_exact<128, kBits>(a, s);
  return launch_exact<256, kBits>(a, s);
}

}  // namespace

hipError_t launch_paged_prefill(const PagedArgs &a, hipStream_t s) {
  return a.bits == 16u ? launch_heads<16>(score_args(a), s) : launch_heads<8>(score_args(a), s);
}

}  // namespace bqmm
