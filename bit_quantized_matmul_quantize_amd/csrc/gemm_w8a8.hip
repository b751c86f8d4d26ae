// Matrix product of 8-bit integers with a scale per token and per channel:
//   out[i][j] = bf16_rne(float(sum_t a[i][t] w[j][t]) * sa[i] * sw[j] + bias[j]),
// the sum exact in int32 on the int8 matrix cores, so no tile, split or order
// changes a bit of it.
//
// Two kernels.  Few rows (a decoded token, a verified batch) are bound by the
// weight's bytes: w8a8_rows_kernel streams it once.  Prompts are bound by the
// matrix cores: w8a8_tile_kernel.
//
// In both the weight is the A operand, so that a lane's accumulators share one
// output row and are runs of four columns.  Rows past m or n load the last
// valid row and are not stored.
#include "bqmm_internal.h"

#include <type_traits>

namespace bqmm {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr uint32_t kRowPad = 128;  // rows are padded to it

// Four columns j.. of output row i.
struct Scales {
  const float *sa, *sw;
  const uint16_t *bias;
  uint16_t *out;
  uint32_t m, n;
};
__device__ __forceinline__ void store4(const Scales &s, uint32_t i, uint32_t j, int a, int b, int c, int d, float sa) {
  if (i >= s.m || j >= s.n) return;
  const int v[4] = {a, b, c, d};
  uint16_t *p = s.out + (uint64_t)i * s.n + j;
  if (j + 4u <= s.n && (s.n & 3u) == 0u) {
    const float4 w = *reinterpret_cast<const float4 *>(s.sw + j);
    float y[4] = {(float)a * sa * w.x, (float)b * sa * w.y, (float)c * sa * w.z, (float)d * sa * w.w};
    if (s.bias) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] += bf16_to_f32(s.bias[j + e]);
    }
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  } else {
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e)
      if (j + e < s.n) {
        float y = (float)v[e] * sa * s.sw[j + e];
        if (s.bias) y += bf16_to_f32(s.bias[j + e]);
        p[e] = (uint16_t)f32_to_bf16_rne(y);
      }
  }
}

// 16 bytes a lane straight from memory into LDS: lane i's go to the wave's
// destination + 16 i.  Not a builtin, because the compiler waits for all such
// loads before any read of LDS; here the kernel waits itself, where a stage is
// complete.  (M0 holds the destination; a wait state lies between its write and
// its use.)  No register is written, so nothing can be overwritten in flight.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t offset, const uint8_t *base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base)
               : "memory", "m0");
}

// Waits until at most n of a wave's loads into LDS are on their way (for the n
// of a unit of few rows: 5 to 8).
__device__ __forceinline__ void wait_for_loads(uint32_t n) {
  switch (n) {
    case 8u: asm volatile("s_waitcnt vmcnt(8)" ::: "memory"); return;
    case 7u: asm volatile("s_waitcnt vmcnt(7)" ::: "memory"); return;
    case 6u: asm volatile("s_waitcnt vmcnt(6)" ::: "memory"); return;
    case 5u: asm volatile("s_waitcnt vmcnt(5)" ::: "memory"); return;
    default: asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
}

// ---- few rows ---------------------------------------------------------------------

// A workgroup takes 16 output columns and at most 16 rows; its waves split k in
// units of 256 bytes and add their sums in LDS.  A wave brings its units of the
// weight rows and the activations straight into LDS, two at a time and
// without a barrier (nobody else reads them), 256 consecutive bytes per row:
// memory serves such runs, while operands loaded as the matrix cores want them
// (16 rows x 64 bytes at once) stream at two thirds of the rate.  The 16 pieces
// of a row lie in the order piece ^ (row % 16), which spreads a column of
// pieces over the banks.
constexpr uint32_t kUnit = 256;  // bytes of k

template <int kWaves>
__global__ __launch_bounds__(64 * kWaves) void w8a8_rows_kernel(const uint8_t *__restrict__ act,
                                                                const uint8_t *__restrict__ w, Scales s, uint32_t kp,
                                                                uint32_t stages) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15u, q = lane >> 4;
  // the row blocks of a column block follow each other: they share its weight rows
  const uint32_t row_blocks = (s.m + 15u) / 16u, n0 = blockIdx.x / row_blocks * 16u, m0 = blockIdx.x % row_blocks * 16u;
  const uint32_t units = (kp + kUnit - 1u) / kUnit, u0 = units * wave / kWaves, u1 = units * (wave + 1u) / kWaves;
  const uint32_t act_loads = (min(s.m - m0, 16u) + 3u) / 4u, stage_bytes = (4u + act_loads) * 1024u;
  uint8_t *mine = lds + wave * stages * stage_bytes;
  const uint32_t mine0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)mine;

  // a load: 4 rows of 256 bytes.  kp is a multiple of 128: of a last half unit
  // the second half takes the first half's bytes again, and is not used.
  const uint8_t *wbase = w + (uint64_t)n0 * kp, *abase = act + (uint64_t)m0 * kp;
  auto load = [&](uint32_t u, uint32_t stage) {
    const uint32_t in_unit = min(kp - u * kUnit, kUnit);
    const uint32_t at = mine0 + stage * stage_bytes;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t row = 4u * i + q, piece = (r ^ row) * 16u;
      load_to_lds(at + i * 1024u, min(row, s.n - 1u - n0) * kp + (piece < in_unit ? piece : piece - 128u), wbase + u * kUnit);
    }
    for (uint32_t i = 0; i < act_loads; ++i) {
      const uint32_t row = 4u * i + q, piece = (r ^ row) * 16u;
      load_to_lds(at + (4u + i) * 1024u, min(row, s.m - 1u - m0) * kp + (piece < in_unit ? piece : piece - 128u), abase + u * kUnit);
    }
  };

  v4i acc = {0, 0, 0, 0};
  // rows of the activations past the loaded ones take the first: their columns of the result are not stored
  const uint8_t *w_at = mine + r * kUnit, *a_at = mine + 4096u + (r < 4u * act_loads ? r : 0u) * kUnit;
  const uint32_t a_row = r < 4u * act_loads ? r : 0u;
  for (uint32_t u = u0; u < min(u0 + stages, u1); ++u) load(u, u - u0);
  uint32_t stage = 0;
  for (uint32_t u = u0; u < u1; ++u) {
    // this unit has arrived; the next may be on its way
    wait_for_loads(stages == 2u && u1 - u >= 2u ? 4u + act_loads : 0u);
    const uint32_t parts = min(kp - u * kUnit, kUnit) / 64u;
    v4i A[4], B[4];
#pragma unroll
    for (uint32_t d = 0; d < 4; ++d) {
      A[d] = *reinterpret_cast<const v4i *>(w_at + stage * stage_bytes + ((d * 4u + q) ^ r) * 16u);
      B[d] = *reinterpret_cast<const v4i *>(a_at + stage * stage_bytes + ((d * 4u + q) ^ a_row) * 16u);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the stage is filled again
    if (u + stages < u1) load(u + stages, stage);
#pragma unroll
    for (uint32_t d = 0; d < 4; ++d)
      if (d < 2u || parts == 4u) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[d], B[d], acc, 0, 0, 0);
    stage = stage + 1u == stages ? 0u : stage + 1u;
  }

  __syncthreads();  // the stages' place takes the sums
  v4i *part = reinterpret_cast<v4i *>(lds);
  part[threadIdx.x] = acc;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int v = 1; v < kWaves; ++v) acc += part[64 * v + lane];
  store4(s, m0 + r, n0 + q * 4u, acc[0], acc[1], acc[2], acc[3], s.sa[min(m0 + r, s.m - 1u)]);
}

// ---- tiles ------------------------------------------------------------------------

// min(a, b) that the compiler does not see through: it would cut the loop over
// the steps in three where the min changes sides, and the copies spill.
__device__ __forceinline__ uint32_t at_most(uint32_t a, uint32_t b) {
  uint32_t x;
  asm("s_min_u32 %0, %1, %2" : "=s"(x) : "s"(a), "s"(b) : "scc");
  return x;
}

// Four waves, two by two, each of 32 kTm rows x 32 kTn columns: 64 kTm x 64 kTn
// outputs.  k runs in steps of 128 bytes (whole cache lines: with 64 the
// weight streams from memory a tenth to a quarter slower) through kStages LDS
// stages.  The eight 16-byte pieces of a row lie in the order piece ^ (row % 8),
// which spreads a column of pieces over the banks; the loads that fill the stage
// write LDS in order and take the pieces from memory in that order instead.
//
// Per step once for each 32 bytes of k: its matrix products, and between them
// the reads of the next 32 bytes.  With the last of them the stage has been
// read: the waves meet once, then the next stage's first reads and the loads
// that refill this one go between the products too (half of them; the other
// half goes with the first products of the step after).
constexpr uint32_t kStep = 128;  // bytes of k per step

template <int kTm, int kTn, int kStages>
struct Tile {
  static constexpr uint32_t BM = 64 * kTm, BN = 64 * kTn;
  static constexpr uint32_t kStage = (BM + BN) * kStep;
  static constexpr uint32_t kRowsAtOnce = 1024 / kStep;            // rows of one load of a wave, 1 KB
  static constexpr int kLoadsN = kTn * kStep / 64, kLoads = (kTm + kTn) * kStep / 64;  // per wave and step
  // stages, scales and biases; the results take the stages' place at the end
  static constexpr uint32_t kLds = (kStages * kStage > BM * BN * 2 ? kStages * kStage : BM * BN * 2) + (2 * BN + BM) * 4;
};

struct __attribute__((packed, aligned(2))) Row8 {  // eight results of a row, which starts at any even address
  uint32_t w[4];
};

template <int kTm, int kTn, int kStages>
__device__ __forceinline__ void run_tile(const uint8_t *act, const uint8_t *w, const Scales &s, uint32_t kp, uint32_t m0,
                                         uint32_t n0, uint8_t *lds) {
  using T = Tile<kTm, kTn, kStages>;
  constexpr uint32_t kInRow = kStep / 16;  // pieces of a row
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wn = wave & 1u, wm = wave >> 1, r = lane & 31u, half = lane >> 5;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

  // what this wave loads: kRowsAtOnce rows from row (wave + 4 i) kRowsAtOnce on of the stage, weight rows first
  const uint8_t *wbase = w + (uint64_t)n0 * kp, *abase = act + (uint64_t)m0 * kp;
  uint32_t off[T::kLoads];
  {
    const uint32_t lr = lane / kInRow, piece = ((lane % kInRow) ^ (lr & 7u)) * 16u;
#pragma unroll
    for (uint32_t i = 0; i < (uint32_t)T::kLoads; ++i) {
      const uint32_t row = T::kRowsAtOnce * (wave + 4u * i) + lr;
      off[i] = (i < (uint32_t)T::kLoadsN ? min(row, s.n - 1u - n0) : min(row - T::BN, s.m - 1u - m0)) * kp + piece;
    }
  }
  auto load = [&](int i, uint32_t stage, uint32_t k0) {
    load_to_lds(lds0 + stage * T::kStage + (wave + 4u * i) * 1024u, off[i], (i < T::kLoadsN ? wbase : abase) + k0);
  };
  // this lane's place in a row block of 32, for the pieces of a step
  constexpr int kParts = kStep / 32;
  uint32_t at[kParts];
#pragma unroll
  for (uint32_t kk = 0; kk < (uint32_t)kParts; ++kk) at[kk] = r * kStep + (((kk * 2u + half) ^ (r & 7u)) * 16u);
  auto read = [&](uint32_t stage, int kk, int t) -> v4i {  // t < kTn: weight rows, then activation rows
    const uint32_t row = t < kTn ? wn * (32u * kTn) + 32u * t : T::BN + wm * (32u * kTm) + 32u * (t - kTn);
    return *reinterpret_cast<const v4i *>(lds + stage * T::kStage + row * kStep + at[kk]);
  };

  v16i acc[kTn][kTm];
#pragma unroll
  for (int i = 0; i < kTn; ++i)
#pragma unroll
    for (int j = 0; j < kTm; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  constexpr int kHalf = T::kLoads / 2, kProducts = kTn * kTm, kReads = kTn + kTm;
  constexpr int kSpread = kProducts > 1 ? kProducts / 2 : 1;
  const uint32_t steps = kp / kStep;
  // the tile's scales and biases, for the end
  float *scale_w = reinterpret_cast<float *>(lds + T::kLds - (2 * T::BN + T::BM) * 4);
  float *biases = scale_w + T::BN, *scale_a = biases + T::BN;
  for (uint32_t i = threadIdx.x; i < T::BN; i += 256u) {
    const uint32_t j = min(n0 + i, s.n - 1u);
    scale_w[i] = s.sw[j];
    biases[i] = s.bias ? bf16_to_f32(s.bias[j]) : 0.0f;
  }
  for (uint32_t i = threadIdx.x; i < T::BM; i += 256u) scale_a[i] = s.sa[min(m0 + i, s.m - 1u)];
  v4i f[2][kReads];
  auto step = [&](uint32_t n, auto last) {
    constexpr bool kLast = decltype(last)::value;
    const uint32_t stage = n % kStages, next = (n + 1u) % kStages;
#pragma unroll
    for (int kk = 0; kk < kParts; ++kk) {
      // the next stage has arrived (those after it may be on their way), this one has been read
      if (kk == kParts - 1 && !kLast)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kStages - 2) * T::kLoads) : "memory");
#pragma unroll
      for (int p = 0; p < kProducts; ++p) {
        const int i = p % kTn, j = p / kTn;
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f[kk & 1][i], f[kk & 1][kTn + j], acc[i][j], 0, 0, 0);
        // reads of the next piece between the first half of the products, loads between the second
        if (p < kSpread && (kk < kParts - 1 || !kLast)) {
#pragma unroll
          for (int t = p * kReads / kSpread; t < (p + 1) * kReads / kSpread; ++t)
            f[(kk + 1) & 1][t] = kk < kParts - 1 ? read(stage, kk + 1, t) : read(next, 0, t);
        }
        // (past the end the last step's are loaded again, so that no step has a branch)
        if (p >= kProducts - kSpread && (kk == 0 || kk == kParts - 1) && !kLast) {
          const int q = p - (kProducts - kSpread);
          if (kk == 0) {
#pragma unroll
            for (int l = q * (T::kLoads - kHalf) / kSpread; l < (q + 1) * (T::kLoads - kHalf) / kSpread; ++l)
              load(kHalf + l, (n + kStages - 1u) % kStages, at_most(n + kStages - 1u, steps - 1u) * kStep);
          } else {
#pragma unroll
            for (int l = q * kHalf / kSpread; l < (q + 1) * kHalf / kSpread; ++l)
              load(l, stage, at_most(n + kStages, steps - 1u) * kStep);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
#pragma unroll
  for (uint32_t n = 0; n < (uint32_t)kStages; ++n)
#pragma unroll
    for (int i = 0; i < (n + 1u < (uint32_t)kStages ? T::kLoads : kHalf); ++i) load(i, n, min(n, steps - 1u) * kStep);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 2) * T::kLoads + kHalf) : "memory");
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kReads; ++t) f[0][t] = read(0u, 0, t);
  for (uint32_t n = 0; n + 1u < steps; ++n) step(n, std::false_type{});
  step(steps - 1u, std::true_type{});
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way into LDS any more

  // The results go through LDS, where the stages were (each wave's own part):
  // a lane has runs of four columns of one row, memory wants whole rows.  The
  // 16-byte pieces of a row are spread over the banks as in the stages.
  __syncthreads();
  constexpr uint32_t kPieces = 4 * kTn, kRowsAtOnce = 64 / kPieces;  // per row of the wave; rows per store
  uint8_t *mine = lds + wave * (32 * kTm * 64 * kTn);
#pragma unroll
  for (int i = 0; i < kTn; ++i)
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const uint32_t c = wn * (32u * kTn) + 32u * i + 2u * e + 4u * half;
      const float4 sw = *reinterpret_cast<const float4 *>(scale_w + c), bias = *reinterpret_cast<const float4 *>(biases + c);
#pragma unroll
      for (int j = 0; j < kTm; ++j) {
        const uint32_t row = 32u * j + r;
        const float sa = scale_a[wm * (32u * kTm) + row];
        const v16i &v = acc[i][j];
        const uint2 y = make_uint2(
            pack_bf16x2((float)v[e] * sa * sw.x + bias.x, (float)v[e + 1] * sa * sw.y + bias.y),
            pack_bf16x2((float)v[e + 2] * sa * sw.z + bias.z, (float)v[e + 3] * sa * sw.w + bias.w));
        const uint32_t piece = (4u * i + e / 4u) ^ (row & (kPieces - 1u));
        *reinterpret_cast<uint2 *>(mine + row * (64u * kTn) + piece * 16u + half * 8u) = y;
      }
    }
  const uint32_t piece = lane % kPieces, col = n0 + wn * (32u * kTn) + piece * 8u;
#pragma unroll 4
  for (uint32_t row = lane / kPieces; row < 32u * kTm; row += kRowsAtOnce) {
    const uint4 y = *reinterpret_cast<const uint4 *>(mine + row * (64u * kTn) + ((piece ^ (row & (kPieces - 1u))) * 16u));
    const uint32_t mm = m0 + wm * (32u * kTm) + row;
    if (mm >= s.m) continue;
    uint16_t *p = s.out + (uint64_t)mm * s.n + col;
    if (col + 8u <= s.n) {
      *reinterpret_cast<Row8 *>(p) = Row8{{y.x, y.y, y.z, y.w}};
    } else {
      const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q)
        if (col + q < s.n) p[q] = (uint16_t)(v[q / 2] >> (16u * (q & 1u)));
    }
  }
}

// Place of a tile among tiles_m x tiles_n: eight rows of tiles at a time,
// column by column, so that tiles that follow each other share operands.
__device__ __forceinline__ void tile_place(uint32_t tile, uint32_t tiles_m, uint32_t tiles_n, uint32_t &tm, uint32_t &tn) {
  const uint32_t group = tile / (8u * tiles_n), in = tile - group * 8u * tiles_n;
  const uint32_t rows = min(8u, tiles_m - group * 8u);
  tm = group * 8u + in % rows;
  tn = in / rows;
}

// Workgroups go round the eight XCDs; each XCD takes a run of `each` tiles.
// Workgroups from `whole` on take a quarter of a tile of 256 x 256 each.
template <int kTm, int kTn, int kStages, bool kQuarters>
__global__ __launch_bounds__(256, 1) void w8a8_tile_kernel(const uint8_t *__restrict__ act,
                                                           const uint8_t *__restrict__ w, Scales s, uint32_t kp,
                                                           uint32_t tiles_m, uint32_t tiles_n, uint32_t whole) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint32_t tm, tn;
  if (kQuarters && blockIdx.x >= whole) {
    const uint32_t q = blockIdx.x - whole;
    tile_place(whole + q / 4u, tiles_m, tiles_n, tm, tn);
    const uint32_t m0 = tm * 256u + (q & 1u) * 128u, n0 = tn * 256u + (q >> 1 & 1u) * 128u;
    if (m0 < s.m && n0 < s.n) run_tile<2, 2, 4>(act, w, s, kp, m0, n0, lds);
    return;
  }
  const uint32_t each = (whole + 7u) / 8u, tile = (blockIdx.x & 7u) * each + (blockIdx.x >> 3);
  if (tile >= whole) return;
  tile_place(tile, tiles_m, tiles_n, tm, tn);
  run_tile<kTm, kTn, kStages>(act, w, s, kp, tm * 64u * kTm, tn * 64u * kTn, lds);
}

template <int kTm, int kTn, int kStages, bool kQuarters>
hipError_t launch_tile_kernel(const uint8_t *act, const uint8_t *w, const Scales &s, uint32_t kp, uint32_t tm, uint32_t tn,
                              uint32_t whole, uint32_t blocks, hipStream_t st) {
  constexpr int lds = Tile<kTm, kTn, kStages>::kLds;
  const auto kernel = w8a8_tile_kernel<kTm, kTn, kStages, kQuarters>;
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void *>(kernel), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), lds, st, act, w, s, kp, tm, tn, whole);
  return hipGetLastError();
}

template <int kTm, int kTn, int kStages>
hipError_t launch_tiles(const uint8_t *act, const uint8_t *w, const Scales &s, uint32_t kp, hipStream_t st) {
  const uint32_t tm = (s.m + 64u * kTm - 1u) / (64u * kTm), tn = (s.n + 64u * kTn - 1u) / (64u * kTn);
  return launch_tile_kernel<kTm, kTn, kStages, false>(act, w, s, kp, tm, tn, tm * tn, (tm * tn + 7u) / 8u * 8u, st);
}

// Tiles of 256 x 256, one per CU at a time.  kQuarters: whole rounds of them, and what is
// left over in quarters where at most two rounds of those suffice (4096 x 4352,
// k = 4096: 16 of 272 tiles are left over; 85.3 us, and 118.8 with a second round;
// 4096 x 5120, k = 17408: 64 of 320; 297, and 384).
bool quarters(uint32_t total, uint32_t cus) {
  const uint32_t left = total % cus;
  return total > cus && cus % 8u == 0u && left > 0u && 2u * left <= cus;
}
template <bool kQuarters>
hipError_t launch_big_tiles(const uint8_t *act, const uint8_t *w, const Scales &s, uint32_t kp, uint32_t cus, hipStream_t st) {
  const uint32_t tm = (s.m + 255u) / 256u, tn = (s.n + 255u) / 256u, total = tm * tn, whole = total / cus * cus;
  if (kQuarters)
    return launch_tile_kernel<4, 4, 2, true>(act, w, s, kp, tm, tn, whole, whole + 4u * (total - whole), st);
  return launch_tile_kernel<4, 4, 2, false>(act, w, s, kp, tm, tn, total, (total + 7u) / 8u * 8u, st);
}

template <int kWaves>
hipError_t launch_rows(const uint8_t *act, const uint8_t *w, const Scales &s, uint32_t kp, hipStream_t st) {
  const uint32_t units = (kp + kUnit - 1u) / kUnit, per_wave = (units + kWaves - 1u) / kWaves;
  // Two units at a time: a third measured 1 to 5% slower (fewer workgroups fit a CU).
  const uint32_t stages = per_wave < 2u ? per_wave : 2u;
  const uint32_t rows = s.m < 16u ? s.m : 16u, need = kWaves * stages * (4u + (rows + 3u) / 4u) * 1024u;
  const uint32_t lds = need > 1024u * kWaves ? need : 1024u * kWaves;  // the stages, then a sum per lane
  const auto kernel = w8a8_rows_kernel<kWaves>;
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void *>(kernel), 65536 * 2);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((s.n + 15u) / 16u * ((s.m + 15u) / 16u)), dim3(64 * kWaves), lds, st, act, w, s, kp, stages);
  return hipGetLastError();
}

// What the forms take, in microseconds, as measured over m = 16 to 4096, n = 64
// to 17408, k = 200 to 5120: a fixed part, and per 128 bytes of k a part for
// each round of workgroups that fills the chip (a smaller one for a last round
// that leaves half the CUs, or half of two workgroups' places, empty).
struct Form {
  uint32_t bm, bn, per_cu;
  float base, round, half;
};
enum { kRows, kT11, kT12, kT21, kT22, kT22Pair, kBig, kForms };
constexpr Form kFormCosts[kForms] = {
    {16, 16, 0, 2.6f, 0.0003f, 0.0f},  // per workgroup: m 64, n 1000, k 1000: 3.2, against 5.0 of the next
    {64, 64, 2, 3.2f, 0.43f, 0.245f},  // 256 x 4096, k 4096: 11.2, 13.5 of the next two
    {64, 128, 1, 3.8f, 0.37f, 0.32f},  // 512 x 4096, k 4096: 15.7, 16.9 of 64 x 64, 18.4 of 128 x 128
    {128, 64, 1, 3.8f, 0.37f, 0.32f},
    {128, 128, 1, 4.0f, 0.62f, 0.43f},  // four stages; 1024 x 4096, k 4096: 25.0, 30.2 with two, 55.5 of 256 x 256
    {128, 128, 2, 4.0f, 1.13f, 0.79f},  // two stages, two workgroups a CU; 2048 x 4096, k 4096: 40.0, 47.1 with four, 60.6 of 256 x 256
    // 8192 x 4096, k 4096: 139.9, 145.4 of 128 x 128 with two stages; at 4096 x 4096 a tie for the model, which takes those (77.4, and 75.0)
    {256, 256, 1, 6.0f, 2.2f, 2.2f},
};

float cost(int form, uint32_t m, uint32_t n, uint32_t steps, uint32_t cus) {
  const Form &f = kFormCosts[form];
  const uint64_t tiles = (uint64_t)((m + f.bm - 1u) / f.bm) * ((n + f.bn - 1u) / f.bn);
  if (form == kRows) return f.base + f.round * (float)tiles * (float)steps;
  const uint64_t slots = (uint64_t)f.per_cu * cus, rounds = tiles / slots, left = tiles % slots;
  float last = left == 0u ? 0.0f : 2u * left <= slots ? f.half : f.round;
  if (form == kBig && tiles <= 0xFFFFFFFFu && quarters((uint32_t)tiles, cus))
    last = 4u * left <= cus ? kFormCosts[kT22].round : 2.0f * kFormCosts[kT22].round;
  return f.base + (float)steps * ((float)rounds * f.round + last);
}

// The form that a call takes: one of the above, or what two of them run otherwise.
enum { kRows4 = kForms, kQuartered };
int form_of(uint32_t m, uint32_t n, uint32_t k, uint32_t cus) {
  const uint32_t steps = (k + kRowPad - 1u) / kRowPad;
  int form = kRows;
  if (m > 16u)
    for (int f = kRows + 1; f < kForms; ++f)
      if (cost(f, m, n, steps, cus) < cost(form, m, n, steps, cus)) form = f;
  // Few workgroups leave most CUs idle: eight waves each then, four otherwise (one row, k = 5120: n = 1000
  // takes 4.0 us against 4.5, n = 17408 18.1 against 17.5).
  if (form == kRows && (m + 15u) / 16u * ((n + 15u) / 16u) > 128u) form = kRows4;
  if (form == kBig && quarters((m + 255u) / 256u * ((n + 255u) / 256u), cus)) form = kQuartered;
  return form;
}

}  // namespace

int w8a8_form(uint32_t m, uint32_t n, uint32_t k, uint32_t cus) { return form_of(m, n, k, cus); }

hipError_t launch_w8a8_gemm(const void *act, const void *w, const void *bias, void *out, uint32_t m, uint32_t n,
                            uint32_t k, hipStream_t st) {
  const uint32_t kp = (k + kRowPad - 1u) / kRowPad * kRowPad;
  const uint8_t *ap = static_cast<const uint8_t *>(act), *wp = static_cast<const uint8_t *>(w);
  const Scales s = {reinterpret_cast<const float *>(ap + (uint64_t)m * kp),
                    reinterpret_cast<const float *>(wp + (uint64_t)n * kp), static_cast<const uint16_t *>(bias),
                    static_cast<uint16_t *>(out), m, n};
  int cus = 0;
  const hipError_t e = device_cu_count(&cus);
  if (e != hipSuccess) return e;
  const uint32_t c = (uint32_t)(cus > 0 ? cus : 1);
  switch (form_of(m, n, k, c)) {
    case kRows: return launch_rows<8>(ap, wp, s, kp, st);
    case kRows4: return launch_rows<4>(ap, wp, s, kp, st);
    case kT11: return launch_tiles<1, 1, 4>(ap, wp, s, kp, st);
    case kT12: return launch_tiles<1, 2, 4>(ap, wp, s, kp, st);
    case kT21: return launch_tiles<2, 1, 4>(ap, wp, s, kp, st);
    case kT22: return launch_tiles<2, 2, 4>(ap, wp, s, kp, st);
    case kT22Pair: return launch_tiles<2, 2, 2>(ap, wp, s, kp, st);
    case kBig: return launch_big_tiles<false>(ap, wp, s, kp, c, st);
    default: return launch_big_tiles<true>(ap, wp, s, kp, c, st);
  }
}

}  // namespace bqmm
