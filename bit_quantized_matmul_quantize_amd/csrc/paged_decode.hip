// Attention of a few new tokens of each sequence over the paged key-value cache:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - max s),  s_j = scale q . k_j, capped,
// in one pass over the cache with the running maximum and sum of the softmax.
//
// Bound by the cache's bytes: 64 tokens of 64 sequences up to 8192, 32 heads over 8 of
// 128, read 1.1 GB in 201 us, 5.5 TB/s; one token behind 130000 in int8 274 MB in 61 us,
// 4.5 TB/s; and a join of 5 to 6 us.  With several rows over an int8 cache, by the codes'
// way to bf16 between the loads and the products of two waves a SIMD: 8 sequences of 4
// tokens, 16 heads over 2 of 256, 74 MB in 38 us.  The rows of one product are the new tokens' heads
// that share a key head, 16 to a column block of the matrix instruction, so that
// keys and values are read once for all of them.  Both come from memory straight
// into the operands: S^T = K Q^T takes 16 keys by 32 values, which are units of
// the cache as they lie there, and gives a lane four keys of one row; two or four
// exchanges between the lanes of a wave turn these into the keys of a unit of v,
// which O^T = V^T P^T takes as it lies.  No operand passes through LDS.
//
// Work: the 64-key blocks of all sequences form one row, which a launch of a fixed
// size cuts into equal runs, whatever the lengths are: as many workgroups as the
// device holds at once, each with one run that may end and begin inside a sequence.
// What such a sequence's parts give is joined by a second launch.  Where the table
// has room for short sequences only, a workgroup takes one, and nothing is joined.
#include "paged_common.h"

namespace bqmm {
namespace {

constexpr uint32_t kBlock = 64;   // keys: the unit of the division of work
constexpr uint32_t kLeast = 4;    // blocks of a run: one token behind 5000 16.2 us, with 8 17.5, with 1 16.3
// Keys: where the table has room for up to so many, sequences are not cut: one token behind
// 700 11.5 us, cut and joined (behind a table for 8192) 14.6.
constexpr uint32_t kShort = 1024;
constexpr uint32_t kCus = 256;

// ---- division of the work ------------------------------------------------------

// Of sequence i: its tiles of rows, and the blocks of keys that any row sees (at
// least one, so that rows that see none are written too).
struct Job {
  uint32_t rows, tiles, blocks;
  int32_t first;  // the first of the blocks
};
__device__ __forceinline__ Job job_of(const PagedArgs &a, const PagedSpan &p, uint32_t tile_rows) {
  Job j;
  j.rows = p.n * (a.hq / a.hk);
  j.tiles = (j.rows + tile_rows - 1u) / tile_rows;
  const int32_t end = min(p.keys, max(p.at + (int32_t)p.n, 0));
  const int32_t begin = a.window ? max(min(p.at + 1 - (int32_t)a.window, end), 0) : 0;
  j.first = begin / (int32_t)kBlock;
  j.blocks = max((uint32_t)((end + (int32_t)kBlock - 1) / (int32_t)kBlock - j.first), 1u);
  return j;
}

// The blocks of all jobs together.
__device__ __forceinline__ uint32_t all_blocks(const PagedArgs &a, uint32_t tile_rows) {
  uint32_t blocks = 0;
  for (uint32_t i = __lane_id(); i < a.count; i += 64u) {
    const Job j = job_of(a, paged_span(a, i), tile_rows);
    blocks += j.tiles * j.blocks;
  }
  if (a.count > 1u) {
#pragma unroll
    for (uint32_t d = 1; d < 64u; d *= 2u) blocks += (uint32_t)__shfl_xor((int)blocks, (int)d, 64);
  }
  return __builtin_amdgcn_readfirstlane(blocks);
}

// A run: per blocks.
__device__ __forceinline__ uint32_t run_blocks(uint32_t blocks, uint32_t slots) { return max(kLeast, (blocks + slots - 1u) / slots); }

// A run leaves at most two parts of tiles: one that begins with it (0), and one that
// ends with it (1).
struct Parts {
  float *sums;    // [slots][2][hk][tile_rows][d]
  float2 *stats;  // [slots][2][hk][tile_rows]: maximum (base 2) and sum
  uint2 *where;   // [tokens][hq / hk]: a row's first part (slot, and 2^31 for a second part); its parts, and 2^16 its place in the tile
};
Parts parts_of(uint8_t *workspace, uint32_t slots, uint32_t hk, uint32_t tile_rows, uint32_t d) {
  const uint64_t rows = 2ull * slots * hk * tile_rows;
  uint8_t *stats = workspace + rows * d * 4u;
  return {reinterpret_cast<float *>(workspace), reinterpret_cast<float2 *>(stats), reinterpret_cast<uint2 *>(stats + rows * 8u)};
}

// The bits of the next binary32 towards 0, of 0 itself.
__device__ __forceinline__ uint32_t below(float w) { return __builtin_elementwise_sub_sat(__float_as_uint(w), 1u); }

// ---- a run ------------------------------------------------------------------------

// Waves of a SIMD that the registers are to suffice for.  Two where they do with few spills:
// one token of 96 sequences, heads of 80: 93 us, with three waves and spills 105; 8 tokens of
// 16 sequences up to 16384, int8 heads of 128: 103 us, with one wave 114, bf16 heads of 96 103
// and 115.  (32 rows of these spill up to 28 registers, nearly all outside the loop; of bf16
// heads between 128 and 256 they spill 155 with one wave, too.)  One wave for a run of
// 32 rows of bf16 heads of 128, where two spill 80 to 94: those 16 sequences 137 us, with two
// 148, 64 of up to 8192 258 and 280 (128 of up to 2000: 192 and 186); a whole short sequence
// spills 20 with two: 64 of up to 900 47.5 us, with one 58.  One for bf16 heads of 256: one
// token of 16 sequences 68 us, with two and spills 111.
constexpr int waves_of(uint32_t dp, uint32_t bits, uint32_t nt, bool cut) {
  return bits == 16u && (dp > 128u || (dp > 96u && nt > 1u && cut)) ? 1 : 2;
}

// kDP: values of a head, rounded up (kExact: as they are); kNT: column blocks of 16
// rows.
// kCut: a workgroup takes a run of blocks, else one tile of rows and its sequence.
template <uint32_t kDP, uint32_t kBits, uint32_t kNT, bool kExact, uint32_t kWaves, bool kCut>
__global__ __launch_bounds__(64 * kWaves, waves_of(kDP, kBits, kNT, kCut)) void paged_decode_kernel(PagedArgs a, uint32_t slots, Parts parts) {
  constexpr uint32_t kUnit = 128u / kBits;        // values of a unit
  constexpr uint32_t kKeys = kBits == 8u && kDP <= 128u ? 64 : 32;  // keys of a step
  constexpr uint32_t kKT = kKeys / 16u;           // their tiles
  constexpr uint32_t kOwn = kKeys / 4u;           // keys of a group of 16 lanes: a unit of v, or half of one
  typedef uint32_t Run __attribute__((ext_vector_type(kOwn * kBits / 32u)));  // its values of one dimension
  constexpr uint32_t kKS = (kDP / kUnit + 3u) / 4u;  // steps of a product over a head's values: four units each
  constexpr uint32_t kHalves = kBits == 16u ? 1u : 2u;  // operands of a unit of k
  constexpr uint32_t kHalvesV = kOwn / 8u;        // and of a group's keys of v
  constexpr uint32_t kDB = kDP / 16u;             // blocks of a head's values
  constexpr uint32_t kRows = 16u * kNT;
  constexpr uint32_t kPitch = kDP + 4u;           // of a row of sums in LDS
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15u, c = lane >> 4;
  const uint32_t slot = blockIdx.x / a.hk, head = blockIdx.x % a.hk, g = a.hq / a.hk;
  uint32_t at_block = 0, end_block = 1, run_begin = 0, per = 1;
  if constexpr (kCut) {
    const uint32_t all = all_blocks(a, kRows);
    per = run_blocks(all, slots);
    if ((uint64_t)slot * per >= all) return;
    run_begin = at_block = slot * per;
    end_block = min(at_block + per, all);
  }
  while (at_block < end_block) {
    uint32_t seq, inside;
    if (!paged_find(kCut ? at_block : slot, a.count, [&](uint32_t i) {
          const Job j = job_of(a, paged_span(a, i), kRows);
          return kCut ? j.tiles * j.blocks : j.tiles;
        }, &seq, &inside))
      return;
    const PagedSpan p = paged_span(a, seq);
    const Job job = job_of(a, p, kRows);
    const uint32_t tile = kCut ? inside / job.blocks : inside, skip = kCut ? inside % job.blocks : 0u;
    const uint32_t take = kCut ? min(job.blocks - skip, end_block - at_block) : job.blocks;
    const int32_t key_begin = (job.first + (int32_t)skip) * (int32_t)kBlock;
    const int32_t key_end = min((job.first + (int32_t)(skip + take)) * (int32_t)kBlock, p.keys);
    if constexpr (kCut) __syncthreads();  // LDS of the last part has been read

    // this lane's rows: places, and the operand of q
    const uint32_t page = 1u << a.page_shift, d = kExact ? kDP : a.d, block = paged_block_bytes(page, d, kBits), units = d / kUnit;
    int32_t pos[kNT], low[kNT];
    constexpr bool kShared = kDP > 128 || kNT > 1;  // q in LDS, where a lane's registers do not suffice
    v4u q[kNT][kKS * kHalves];
#pragma unroll
    for (uint32_t t = 0; t < kNT; ++t) {
      const uint32_t row = tile * kRows + t * 16u + r, token = row / g, hh = row % g;
      const bool live = row < job.rows;
      pos[t] = live ? p.at + (int32_t)token : -1;
      low[t] = a.window && live ? (int32_t)max((int64_t)pos[t] + 1 - (int64_t)a.window, (int64_t)0) : 0;
      const uint16_t *from = a.q + (uint64_t)(p.first + (live ? token : 0u)) * a.q_token + (uint64_t)(head * g + hh) * a.q_head;
#pragma unroll
      for (uint32_t s = 0; s < kKS; ++s)
#pragma unroll
        for (uint32_t h = 0; h < kHalves; ++h) {
          v4u v = {0, 0, 0, 0};
          const uint32_t unit = 4u * s + c;
          const uint32_t i = t * kKS * kHalves + s * kHalves + h;
          if (kShared && i % kWaves != wave) continue;
          if (live && unit < units) v = *reinterpret_cast<const v4u *>(from + unit * kUnit + h * 8u);
          if constexpr (kShared)
            *reinterpret_cast<v4u *>(lds + (i * 64u + lane) * 16u) = v;
          else
            q[t][s * kHalves + h] = v;
        }
    }
    if constexpr (kShared) __syncthreads();
    auto q_of = [&](uint32_t n, uint32_t i) {
      if constexpr (kShared) return *reinterpret_cast<const v4u *>(lds + ((n * kKS * kHalves + i) * 64u + lane) * 16u);
      return q[n][i];
    };
    // keys that all of the tile's rows see lie in [all_low, all_pos], those that any
    // does in [any_low, any_pos]
    int32_t all_pos, all_low, any_pos, any_low;
    {
      const uint32_t row0 = tile * kRows, row1 = min(row0 + kRows, job.rows) - 1u;
      all_pos = p.at + (int32_t)(row0 / g);
      any_pos = p.at + (int32_t)(row1 / g);
      any_low = a.window ? (int32_t)max((int64_t)all_pos + 1 - (int64_t)a.window, (int64_t)0) : 0;
      all_low = a.window ? (int32_t)max((int64_t)any_pos + 1 - (int64_t)a.window, (int64_t)0) : 0;
    }

    float scale2 = a.scale2, cap2 = a.cap2, inv2 = a.cap_inv2;
    asm volatile("" : "+v"(scale2), "+v"(cap2), "+v"(inv2));  // (else loaded anew in each step)
    float m[kNT], l[kNT];
    v4f o[kNT][kDB];
#pragma unroll
    for (uint32_t t = 0; t < kNT; ++t) {
      m[t] = -INFINITY;
      l[t] = 0.0f;
#pragma unroll
      for (uint32_t b = 0; b < kDB; ++b) o[t][b] = v4f{0, 0, 0, 0};
    }

    const int32_t *table = a.table + (uint64_t)seq * a.width;
    const uint8_t *kc = a.k_cache + (uint64_t)head * block, *vc = a.v_cache + (uint64_t)head * block;
    const uint64_t page_bytes = (uint64_t)block * a.hk;

    // A step: 32 keys (int8: 64).  Values are on their way while the scores are made,
    // the next step's keys while the softmax is.
    constexpr int32_t kStride = (int32_t)(kWaves * kKeys);
    auto ids_of = [&](int32_t key0, v4u &ids) {  // the pages of its tiles of 16 keys
#pragma unroll
      for (uint32_t t = 0; t < kKT; ++t) {
        const uint32_t at = (uint32_t)(key0 + (int32_t)(16u * t)) >> a.page_shift;
        ids[t] = __builtin_amdgcn_readfirstlane(at < a.width ? (uint32_t)table[at] : ~0u);
      }
    };
    v4u k[kKT][kKS];
    v4f ks[kKT];
    auto load_k = [&](int32_t key0, const v4u &ids) {
#pragma unroll
      for (uint32_t t = 0; t < kKT; ++t) {
        const uint32_t id = ids[t] < a.pages ? ids[t] : 0u, off = (uint32_t)(key0 + (int32_t)(16u * t)) & (page - 1u);
        const uint8_t *base = kc + id * page_bytes + off * 16u;
#pragma unroll
        for (uint32_t s = 0; s < kKS; ++s) {
          if (kExact && 4u * s + 4u <= kDP / kUnit) {
            k[t][s] = *reinterpret_cast<const v4u *>(base + (uint64_t)(4u * s) * page * 16u + (c * page + r) * 16u);
          } else {  // (beyond the head's units: the first again, as zeros)
            const bool has = 4u * s + c < units;
            k[t][s] = *reinterpret_cast<const v4u *>(base + ((has ? 4u * s + c : 0u) * page + r) * 16u);
            if (!has) k[t][s] = v4u{0, 0, 0, 0};
          }
        }
        if constexpr (kBits == 8u) ks[t] = *reinterpret_cast<const v4f *>(kc + id * page_bytes + page * d + (off + 4u * c) * 4u);
      }
    };

    Run v[kDB];  // of keys kOwn c.. of the step
    v4f vs[kKT];
    auto load_v = [&](int32_t key0, const v4u &ids) {
      const uint32_t t = c * kOwn / 16u;
      uint32_t id = ids[0];
#pragma unroll
      for (uint32_t i = 1; i < kKT; ++i) id = t == i ? ids[i] : id;
      id = id < a.pages ? id : 0u;
      const uint32_t off = (uint32_t)(key0 + (int32_t)(c * kOwn)) & (page - 1u);
      const uint8_t *base = vc + id * page_bytes + ((uint64_t)(off / kUnit) * d + r) * 16u + (kOwn < kUnit ? off % kUnit * (kBits / 8u) : 0u);
#pragma unroll
      for (uint32_t b = 0; b < kDB; ++b) {
        // (beyond the head's values: the first again, whose sums are not taken)
        v[b] = *reinterpret_cast<const Run *>(base + (kExact || 16u * b < d ? b : 0u) * 256u);
      }
      if constexpr (kBits == 8u) {
#pragma unroll
        for (uint32_t i = 0; i < kKT; ++i) {
          const uint32_t at = ids[i] < a.pages ? ids[i] : 0u, to = (uint32_t)(key0 + (int32_t)(16u * i)) & (page - 1u);
          vs[i] = *reinterpret_cast<const v4f *>(vc + at * page_bytes + page * d + (to + 4u * c) * 4u);
        }
      }
    };
    v4f x[kNT][kKT];
    auto scores = [&] {
#pragma unroll
      for (uint32_t t = 0; t < kKT; ++t)
#pragma unroll
        for (uint32_t n = 0; n < kNT; ++n) x[n][t] = v4f{0, 0, 0, 0};
      if constexpr (kBits == 8u) {  // (else the loop carries every code in a register of its own)
#pragma unroll
        for (uint32_t t = 0; t < kKT; ++t)
#pragma unroll
          for (uint32_t i = 0; i < kKS; ++i) asm volatile("" : "+v"(k[t][i]));
      }
      auto product = [&](uint32_t t, uint32_t s, uint32_t h, const v4u (&qq)[kNT]) {
        const v4u kk = kBits == 16u ? k[t][s] : bf16_of_codes(k[t][s][2 * h], k[t][s][2 * h + 1]);
#pragma unroll
        for (uint32_t n = 0; n < kNT; ++n) x[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(kk), as_bf(qq[n]), x[n][t], 0, 0, 0);
        if constexpr (kBits == 8u) __builtin_amdgcn_sched_barrier(0);  // (else all codes are unpacked at once)
      };
      if constexpr (kShared) {
#pragma unroll
        for (uint32_t i = 0; i < kKS * kHalves; ++i) {
          v4u qq[kNT];
#pragma unroll
          for (uint32_t n = 0; n < kNT; ++n) qq[n] = q_of(n, i);
#pragma unroll
          for (uint32_t t = 0; t < kKT; ++t) product(t, i / kHalves, i % kHalves, qq);
        }
      } else {
#pragma unroll
        for (uint32_t t = 0; t < kKT; ++t)
#pragma unroll
          for (uint32_t i = 0; i < kKS * kHalves; ++i) {
            v4u qq[kNT];
#pragma unroll
            for (uint32_t n = 0; n < kNT; ++n) qq[n] = q_of(n, i);
            product(t, i / kHalves, i % kHalves, qq);
          }
      }
      if constexpr (kBits == 8u) {
#pragma unroll
        for (uint32_t n = 0; n < kNT; ++n)
#pragma unroll
          for (uint32_t t = 0; t < kKT; ++t) x[n][t] *= ks[t];
      }
    };
    // scores to weights, where the lanes' units of v want them.  hole: bit t where the
    // step's keys 16 t.. lie in no page; whole: all rows see all keys.
    v4u ph[kNT][kHalvesV], pl[kNT][kHalvesV];
    auto weigh = [&](int32_t key0, uint32_t hole, bool whole) {
#pragma unroll
      for (uint32_t n = 0; n < kNT; ++n) {
        if (a.cap != 0.0f) {
          if (a.cap <= kShortCap) {
#pragma unroll
            for (uint32_t t = 0; t < kKT; ++t)
#pragma unroll
              for (uint32_t e = 0; e < 4; ++e) x[n][t][e] = capped(x[n][t][e], cap2, inv2);
          } else {
#pragma unroll
            for (uint32_t t = 0; t < kKT; ++t)
#pragma unroll
              for (uint32_t e = 0; e < 4; ++e) x[n][t][e] = capped_large(x[n][t][e], a);
          }
        }
        if (!whole) {
#pragma unroll
          for (uint32_t t = 0; t < kKT; ++t)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const int32_t key = key0 + (int32_t)(16u * t + 4u * c + e);
              const bool seen = key <= pos[n] && key >= low[n] && key < key_end && !(hole >> t & 1u);
              x[n][t][e] = seen ? x[n][t][e] : -INFINITY;
            }
        }
        float top = x[n][0][0];
#pragma unroll
        for (uint32_t t = 0; t < kKT; ++t) top = fmaxf(fmaxf(fmaxf(x[n][t][0], x[n][t][1]), top), fmaxf(x[n][t][2], x[n][t][3]));
        top *= scale2;
        if (__ballot(top > m[n])) {
          top = fmaxf(top, __shfl_xor(top, 16, 64));
          top = fmaxf(top, __shfl_xor(top, 32, 64));
          const float next = fmaxf(m[n], top + kSlack);
          const float keep = m[n] == -INFINITY ? 0.0f : exp2_hw(m[n] - next);
          m[n] = next;
          l[n] *= keep;
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b) o[n][b] *= keep;
        }
        const float base = m[n] == -INFINITY ? 0.0f : m[n];
        // the sum of two bf16: one would be off by 2^-8 of each weight.  Over a bf16 cache the
        // first is below the weight, so that the second is above 0 too, and an infinity of v
        // times both stays one (by 2^-15 off, to the nearest by 2^-16; the same time).
        uint32_t hi[kKT][2], lo[kKT][2];
#pragma unroll
        for (uint32_t t = 0; t < kKT; ++t) {
          float w[4];
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            const float s = x[n][t][e];
            w[e] = exp2_hw(fmaf(s, scale2, -base));
            l[n] += w[e];
            if constexpr (kBits == 8u) w[e] = s == -INFINITY ? 0.0f : w[e] * vs[t][e];
          }
#pragma unroll
          for (uint32_t e = 0; e < 2; ++e) {
            if constexpr (kBits == 16u)
              hi[t][e] = __builtin_amdgcn_perm(below(w[2 * e + 1]), below(w[2 * e]), 0x07060302u);
            else
              hi[t][e] = two_bf16(w[2 * e], w[2 * e + 1]);
            lo[t][e] = two_bf16(w[2 * e] - __uint_as_float(hi[t][e] << 16), w[2 * e + 1] - __uint_as_float(hi[t][e] & 0xFFFF0000u));
          }
        }
        // lanes of group c have keys 4 c.. of every tile, and want the keys of their unit
        auto turn = [&](uint32_t (&w)[kKT][2], v4u *out) {
#pragma unroll
          for (uint32_t e = 0; e < 2; ++e) {
            if constexpr (kKT == 2u) {
              const v2u s = __builtin_amdgcn_permlane32_swap(w[0][e], w[1][e], false, false);
              const v2u f = __builtin_amdgcn_permlane16_swap(s.x, s.y, false, false);
              out[0][e] = f.x;
              out[0][2 + e] = f.y;
            } else {
              const v2u s0 = __builtin_amdgcn_permlane32_swap(w[0][e], w[2][e], false, false);
              const v2u s1 = __builtin_amdgcn_permlane32_swap(w[1][e], w[3][e], false, false);
              const v2u f0 = __builtin_amdgcn_permlane16_swap(s0.x, s1.x, false, false);
              const v2u f1 = __builtin_amdgcn_permlane16_swap(s0.y, s1.y, false, false);
              out[0][e] = f0.x;
              out[0][2 + e] = f0.y;
              out[kHalvesV - 1][e] = f1.x;
              out[kHalvesV - 1][2 + e] = f1.y;
            }
          }
        };
        turn(hi, ph[n]);
        turn(lo, pl[n]);
      }
    };
    auto add_products = [&] {
#pragma unroll
      for (uint32_t b = 0; b < kDB; ++b)
#pragma unroll
        for (uint32_t h = 0; h < kHalvesV; ++h) {
          v4u u;
          if constexpr (kBits == 16u)
            u = v[b];
          else
            u = bf16_of_codes(v[b][2 * h], v[b][2 * h + 1]);
#pragma unroll
          for (uint32_t n = 0; n < kNT; ++n) {
            o[n][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(u), as_bf(ph[n][h]), o[n][b], 0, 0, 0);
            o[n][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(u), as_bf(pl[n][h]), o[n][b], 0, 0, 0);
          }
          if constexpr (kBits == 8u) __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Of a unit's eight keys (bf16), those in [from, to] that lie in a page: bit e.
    auto seen_in = [&](int32_t key0, uint32_t hole, int32_t from, int32_t to) {
      const int32_t at = key0 + (int32_t)(8u * c), lo = max(from - at, 0), hi = min(min(to, key_end - 1) - at, 7);
      return hole >> (c / 2u) & 1u || lo > hi ? 0u : (0xFFu >> (7 - hi)) & (0xFFu << lo);
    };
    auto holes_of = [&](const v4u &ids) {
      uint32_t hole = 0;
#pragma unroll
      for (uint32_t t = 0; t < kKT; ++t) hole |= ids[t] >= a.pages ? 1u << t : 0u;
      return hole;
    };
    // 0 * NaN must not reach a row that does not see the NaN's key.  Codes are finite;
    // of bf16, values that no row sees count as zero, and steps with keys that some
    // rows see and others do not are left for the second loop.
    auto mixed = [&](int32_t key0) {
      const int32_t last = key0 + (int32_t)kKeys - 1;
      return kBits == 16u && ((any_low < all_low && key0 < all_low && last >= any_low) || (all_pos < any_pos && key0 <= any_pos && last > all_pos));
    };

    v4u ids, next_ids;
    const int32_t key_first = key_begin + (int32_t)(wave * kKeys);
    if (key_first < key_end) {
      ids_of(key_first, ids);
      load_k(key_first, ids);
      ids_of(key_first + kStride, next_ids);
    }
    for (int32_t key0 = key_first; key0 < key_end; key0 += kStride) {
      const uint32_t hole = holes_of(ids);
      load_v(key0, ids);
      __builtin_amdgcn_sched_barrier(0);
      scores();
      __builtin_amdgcn_sched_barrier(0);
      if (key0 + kStride < key_end) load_k(key0 + kStride, next_ids);
      ids = next_ids;
      ids_of(key0 + 2 * kStride, next_ids);
      __builtin_amdgcn_sched_barrier(0);
      if (mixed(key0)) continue;
      const bool whole = !hole && key0 + (int32_t)kKeys - 1 <= all_pos && key0 >= all_low && key0 + (int32_t)kKeys <= key_end;
      weigh(key0, hole, whole);
      if constexpr (kBits == 16u) {
        if (!whole) {
          uint32_t seen = seen_in(key0, hole, any_low, any_pos);
          asm volatile("" : "+v"(seen));  // (keeps this a branch)
          v4u mask;
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) mask[i] = (seen >> (2u * i) & 1u ? 0xFFFFu : 0u) | (seen >> (2u * i + 1u) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b) v[b] &= mask;
        }
      }
      add_products();
    }
    if constexpr (kBits == 16u) {
      if (any_low < all_low || all_pos < any_pos) {
#pragma unroll 1
        for (int32_t key0 = key_first; key0 < key_end; key0 += kStride) {
          if (!mixed(key0)) continue;
          ids_of(key0, ids);
          const uint32_t hole = holes_of(ids);
          load_k(key0, ids);
          load_v(key0, ids);
          scores();
          __builtin_amdgcn_sched_barrier(0);
          weigh(key0, hole, false);
          bool bad = false;
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b) bad |= any_not_finite(v[b]);
          if (__ballot(bad)) {
            // a NaN or an infinity is added where it is seen, and counts as zero in the product
#pragma unroll
            for (uint32_t b = 0; b < kDB; ++b) {
              const v4u mark = not_finite_marks(v[b]);
              v[b] = finite_only(v[b]);
#pragma unroll
              for (uint32_t n = 0; n < kNT; ++n) {
                const uint32_t seen = seen_in(key0, hole, low[n], pos[n]);
                v4u ones;
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                  ones[i] = (seen >> (2u * i) & 1u ? 0x3F80u : 0u) | (seen >> (2u * i + 1u) & 1u ? 0x3F800000u : 0u);
                v4f marks = {0, 0, 0, 0};
                marks = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(mark), as_bf(ones), marks, 0, 0, 0);
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) o[n][b][i] += of_marks(marks[i]);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          add_products();
        }
      }
    }

    // the waves' results, two and two
#pragma unroll
    for (uint32_t n = 0; n < kNT; ++n) {
      l[n] += __shfl_xor(l[n], 16, 64);
      l[n] += __shfl_xor(l[n], 32, 64);
    }
    float *const shared = reinterpret_cast<float *>(lds);
    float2 *const shared_stats = reinterpret_cast<float2 *>(lds + (kWaves / 2u) * kRows * kPitch * 4u);
#pragma unroll
    for (uint32_t half = kWaves / 2u; half >= 1u; half /= 2u) {
      __syncthreads();
      if (wave >= half && wave < 2u * half) {
        const uint32_t at = wave - half;
#pragma unroll
        for (uint32_t n = 0; n < kNT; ++n) {
          const uint32_t row = at * kRows + n * 16u + r;
          if (c == 0u) shared_stats[row] = make_float2(m[n], l[n]);
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b) *reinterpret_cast<v4f *>(shared + row * kPitch + 16u * b + 4u * c) = o[n][b];
        }
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (uint32_t n = 0; n < kNT; ++n) {
          const uint32_t row = wave * kRows + n * 16u + r;
          const float2 other = shared_stats[row];
          const float next = fmaxf(m[n], other.x);
          const float mine = m[n] == -INFINITY ? 0.0f : exp2_hw(m[n] - next);
          const float theirs = other.x == -INFINITY ? 0.0f : exp2_hw(other.x - next);
          l[n] = l[n] * mine + other.y * theirs;
          m[n] = next;
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b) {
            const v4f y = *reinterpret_cast<const v4f *>(shared + row * kPitch + 16u * b + 4u * c);
            o[n][b] = o[n][b] * mine + y * theirs;
          }
        }
      }
    }
    if (wave == 0u) {
#pragma unroll
      for (uint32_t n = 0; n < kNT; ++n) {
        const uint32_t row = tile * kRows + n * 16u + r;
        if (row >= job.rows) continue;
        if (!kCut || take == job.blocks) {
          const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];
          uint16_t *to = a.out + ((uint64_t)(p.first + row / g) * a.hq + head * g + row % g) * d;
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b)
            if (16u * b < d)
              *reinterpret_cast<uint2 *>(to + 16u * b + 4u * c) =
                  make_uint2(pack_bf16x2(o[n][b][0] * inv, o[n][b][1] * inv), pack_bf16x2(o[n][b][2] * inv, o[n][b][3] * inv));
        } else {
          const uint64_t at = ((uint64_t)(2u * slot + (at_block != run_begin)) * a.hk + head) * kRows + n * 16u + r;
          if (c == 0u) parts.stats[at] = make_float2(m[n], l[n]);
#pragma unroll
          for (uint32_t b = 0; b < kDB; ++b)
            if (16u * b < d) *reinterpret_cast<v4f *>(parts.sums + at * d + 16u * b + 4u * c) = o[n][b];
        }
      }
    }
    if (kCut && head == 0u && skip + take == job.blocks && threadIdx.x < kRows) {
      // the tile's rows: where their parts begin, for the second launch
      const uint32_t job_begin = at_block - skip, slot0 = job_begin / per, row = tile * kRows + threadIdx.x;
      if (row < job.rows)
        parts.where[(uint64_t)p.first * g + row] =
            make_uint2(slot0 | (job_begin != slot0 * per ? 1u << 31 : 0u), (slot - slot0 + 1u) | threadIdx.x << 16);
    }
    at_block += kCut ? take : 1u;
  }
}

// ---- joining the runs ----------------------------------------------------------------

// A workgroup takes one row: lanes hold four of its values, groups of lanes share
// the parts.
constexpr uint32_t kJoinThreads = 256;

__global__ __launch_bounds__(kJoinThreads) void paged_join_kernel(PagedArgs a, uint32_t tile_rows, uint32_t slots, Parts parts) {
  __shared__ v4f part[kJoinThreads];
  __shared__ float part_sum[kJoinThreads / 4];
  const uint32_t g = a.hq / a.hk, token = blockIdx.x, h = blockIdx.y, head = h / g;
  const uint2 where = parts.where[(uint64_t)token * g + h % g];
  const int32_t first = a.starts[0], last = a.starts[a.count];
  const uint32_t slot0 = where.x & 0x7FFFFFFFu, runs = where.y & 0xFFFFu, row = where.y >> 16;
  // One part: the row is written.  (Of a row of no sequence nobody has written
  // where it is; nor do starts that do not ascend lead outside the parts.)
  if (runs <= 1u || (int64_t)token < first || (int64_t)token >= last || slot0 >= slots || runs > slots - slot0 || row >= tile_rows)
    return;
  auto at_of = [&](uint32_t i) {
    return ((uint64_t)(2u * (slot0 + i) + (i == 0u ? where.x >> 31 : 0u)) * a.hk + head) * tile_rows + row;
  };

  float top = -INFINITY;
  for (uint32_t i = threadIdx.x & 63u; i < runs; i += 64u) top = fmaxf(top, parts.stats[at_of(i)].x);
#pragma unroll
  for (uint32_t d = 1; d < 64u; d *= 2u) top = fmaxf(top, __shfl_xor(top, (int)d, 64));

  const uint32_t lanes = a.d / 4u, groups = kJoinThreads / lanes, lane = threadIdx.x % lanes, group = threadIdx.x / lanes;
  v4f sum = {0, 0, 0, 0};
  float weight = 0.0f;
  if (group < groups) {
#pragma unroll 4
    for (uint32_t i = group; i < runs; i += groups) {
      const uint64_t at = at_of(i);
      const float2 s = parts.stats[at];
      const float w = s.x == -INFINITY ? 0.0f : exp2_hw(s.x - top);
      weight += s.y * w;
      sum += *reinterpret_cast<const v4f *>(parts.sums + at * a.d + 4u * lane) * w;
    }
    part[threadIdx.x] = sum;
    if (lane == 0u) part_sum[group] = weight;
  }
  __syncthreads();
  if (group != 0u) return;
  weight = part_sum[0];
  for (uint32_t i = 1; i < groups; ++i) {
    sum += part[i * lanes + lane];
    weight += part_sum[i];
  }
  const float inv = weight == 0.0f ? 0.0f : 1.0f / weight;
  *reinterpret_cast<uint2 *>(a.out + ((uint64_t)token * a.hq + h) * a.d + 4u * lane) =
      make_uint2(pack_bf16x2(sum[0] * inv, sum[1] * inv), pack_bf16x2(sum[2] * inv, sum[3] * inv));
}

// ---- the launch ------------------------------------------------------------------

struct Plan {
  uint32_t blocks, slots, tiles;  // column blocks of a tile; runs; tiles at most
};

constexpr uint32_t kMostBlocks = 2;  // column blocks of 16 rows

Plan plan_of(const PagedArgs &a) {
  const uint32_t g = a.hq / a.hk;
  const uint64_t rows = (uint64_t)a.tokens * g, mean = (rows + a.count - 1u) / a.count;
  Plan p;
  // (16 sequences up to 16384 keys, 8 tokens of 4 heads of 128 each: by 32 rows bf16 147 us,
  // int8 103, by 16 rows 177 and 112; 4 tokens of 8 heads of 256, bf16: 91 and 102)
  // (wide int8 heads by 16 rows: 8 sequences of 4 tokens and 8 heads 46 us, by 32 53,
  // both with a join 3 us longer)
  p.blocks = mean <= 16u || (a.d > 128u && a.bits == 8u) ? 1u : kMostBlocks;
  const uint32_t tile = 16u * p.blocks, dp = a.d <= 64u ? 64u : a.d <= 96u ? 96u : a.d <= 128u ? 128u : 256u;
  // (of a sequence with rows: at most one tile that is not full)
  p.tiles = (uint32_t)std::min<uint64_t>(rows / tile + std::min(a.count, a.tokens), (uint64_t)a.tokens * ((g + tile - 1u) / tile));
  // as many workgroups as the device holds at once (four waves: one to a SIMD)
  p.slots = std::max(kCus * (uint32_t)waves_of(dp, a.bits, p.blocks, true) / a.hk, 1u);
  return p;
}

template <uint32_t kDP, uint32_t kBits, uint32_t kNT, bool kExact, uint32_t kWaves, bool kCut>
hipError_t launch(const PagedArgs &a, const Plan &plan, hipStream_t s) {
  const Parts parts = parts_of(a.workspace, plan.slots, a.hk, 16u * kNT, a.d);
  constexpr uint32_t kLds = (kWaves / 2u) * 16u * kNT * ((kDP + 4u) * 4u + 8u);  // (more than a shared q takes)
  auto *kernel = paged_decode_kernel<kDP, kBits, kNT, kExact, kWaves, kCut>;
  if (kLds > 65536u) {
    const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void *>(kernel), (int)kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((kCut ? plan.slots : plan.tiles) * a.hk), dim3(64 * kWaves), kLds, s, a, plan.slots, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !kCut) return e;
  hipLaunchKernelGGL(paged_join_kernel, dim3(a.tokens, a.hq), dim3(kJoinThreads), 0, s, a, 16u * kNT, plan.slots, parts);
  return hipGetLastError();
}

template <uint32_t kDP, uint32_t kBits, uint32_t kNT>
hipError_t launch_rows(const PagedArgs &a, const Plan &plan, hipStream_t s) {
  constexpr uint32_t kWide = kDP * kNT <= 128u ? 8 : 4;  // waves for a whole sequence
  if (((uint64_t)a.width << a.page_shift) <= kShort)
    return a.d == kDP ? launch<kDP, kBits, kNT, true, kWide, false>(a, plan, s) : launch<kDP, kBits, kNT, false, kWide, false>(a, plan, s);
  return a.d == kDP ? launch<kDP, kBits, kNT, true, 4, true>(a, plan, s) : launch<kDP, kBits, kNT, false, 4, true>(a, plan, s);
}

template <uint32_t kDP, uint32_t kBits>
hipError_t launch_heads(const PagedArgs &a, const Plan &plan, hipStream_t s) {
  if constexpr (kDP <= 128u || kBits == 16u)
    if (plan.blocks != 1u) return launch_rows<kDP, kBits, kMostBlocks>(a, plan, s);
  return launch_rows<kDP, kBits, 1>(a, plan, s);
}

template <uint32_t kBits>
hipError_t launch_bits(const PagedArgs &a, const Plan &plan, hipStream_t s) {
  if (a.d <= 64u) return launch_heads<64, kBits>(a, plan, s);
  if (a.d <= 96u) return launch_heads<96, kBits>(a, plan, s);
  if (a.d <= 128u) return launch_heads<128, kBits>(a, plan, s);
  return launch_heads<256, kBits>(a, plan, s);
}

}  // namespace

hipError_t launch_paged_decode(const PagedArgs &a, hipStream_t s) {
  const Plan plan = plan_of(a);
  return a.bits == 16u ? launch_bits<16>(score_args(a), plan, s) : launch_bits<8>(score_args(a), plan, s);
}

// The two parts of each run, for tiles of the most rows and as many runs as any form
// of the kernel has, and where each row's are.
uint64_t paged_workspace_bytes(uint32_t tokens, uint32_t hq, uint32_t hk, uint32_t d) {
  const uint64_t slots = std::max(kCus * 2u / hk, 1u);
  return 2u * slots * hk * 16u * kMostBlocks * (4ull * d + 8u) + 8ull * tokens * (hq / hk);
}

}  // namespace bqmm
