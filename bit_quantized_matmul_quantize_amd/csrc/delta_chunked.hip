// The gated delta rule over prompts, in chunks of 64 tokens.
//
// Within a chunk that starts from state S0, with G_t the sum of g up to token
// t of the chunk (its last: G_L), unit keys k and queries q, b = beta:
//   A_ts = b_t e^(G_t - G_s) k_t.k_s  (s < t),   R_t = b_t (v_t - e^(G_t) k_t^T S0),
//   U = T R,  T = (1 + A)^-1  (unit lower triangle),
//   o_t = scale (e^(G_t) q_t^T S0 + sum_{s <= t} e^(G_t - G_s) (q_t.k_s) u_s),
//   S = e^(G_L) S0 + sum_t e^(G_L - G_t) k_t u_t^T.
//
// Two launches.  The first takes every chunk of every value head at once and
// leaves what does not depend on the state in the workspace: T, the decayed
// q.k triangle and a few factors per token.  The second
// walks each head's chunks in order, a workgroup for 16 columns of the state
// (columns do not depend on each other); long sequences of few heads it cuts
// into segments, and a third launch follows.
//
// Numbers.  The matrix cores multiply bf16 and add in binary32.  q and k are
// bf16 as they are: their norms, decays and beta are factors per token that
// are applied in binary32 outside the products.  A binary32 operand (T, R, U,
// S, the q.k triangle) enters as the sum of three bf16 (8 + 8 + 8 bits, nothing
// lost); a product of two such operands keeps the six products above 2^-24.
// That holds for the output too: where large terms cancel, what is left is
// right (with two parts there, 2^-16, both launches took 67.5 us for 2048 tokens
// of 32 heads, and take 71.7).  T is computed in binary32 throughout, the sums
// G in binary64: differences of G stay exact next to a strong decay.
#include "delta_common.h"

#include <cmath>
#include <type_traits>

namespace bqmm {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr int kChunk = 64;
constexpr int kThreads = 256;
constexpr uint32_t kCus = 256;  // of a whole card; on a part of it the choices that go by it are as right, and less fast
constexpr float kNormEps = 1e-6f;
constexpr float kNoDecay = -1e6f;  // exp of it is zero; sums of 64 of them stay exact to 2^-26

// Workspace.  A fragment is what a wave's 64 lanes load as one matrix
// operand, 16 bytes each, 1 KB.  Rows 16w..16w+15 of a lower triangle need
// only the 32 columns up to w = 1 and all 64 from w = 2: six fragments.
constexpr uint32_t kFragment = 1024;
constexpr uint32_t kTriangle = 6;
constexpr uint32_t kTBytes = kTriangle * 3 * kFragment;
constexpr uint32_t kInnerBytes = kTriangle * 3 * kFragment;
constexpr uint32_t kFactorRow = kChunk * 4;  // rows b, b e^G rk, e^(G_L - G) rk, scale e^G rq of 64 tokens, then e^G_L
constexpr uint32_t kFactorBytes = 4 * kFactorRow + 256;
constexpr uint32_t kHeadBytes = kTBytes + kInnerBytes + kFactorBytes;

__device__ __forceinline__ uint32_t triangle_fragment(uint32_t w, uint32_t ks) { return w < 2u ? w : 2u * w - 2u + ks; }

// Chunk places: a sequence that begins at token b as the s-th has its chunks
// from b / 64 + s on.  Places of different sequences never meet, and all lie
// below tokens / 64 + count.
__device__ __forceinline__ uint32_t first_place(uint32_t begin, uint32_t seq) { return begin / kChunk + seq; }

// Segments have places likewise, per `segment` chunks.
__host__ __device__ __forceinline__ uint32_t segment_places(uint32_t tokens, uint32_t count, uint32_t segment) {
  return tokens / (segment * kChunk) + count;
}

// How many sequences have their first place, of places of so many tokens, at or
// below this one: the last of them is the one that the place belongs to.
template <int kThreads>
__device__ __forceinline__ int sequences_up_to(const DeltaArgs &a, uint32_t place, uint32_t tokens) {
  int before = 0;
  for (uint32_t s0 = 0; s0 < a.count; s0 += kThreads) {
    const uint32_t s = s0 + threadIdx.x;
    bool at = false;
    if (s < a.count) at = min((uint32_t)max(a.starts[s], 0), a.tokens) / tokens + s <= place;
    before += __syncthreads_count(at);
  }
  return before;
}

// Row r of 16 of the state's tile T, among its dk: a wave's result rows are
// then the rows of a matrix operand of 32 in their natural order.
__device__ __forceinline__ uint32_t state_row(uint32_t tile, uint32_t r) {
  return 32u * (tile >> 1) + (r >> 2) * 8u + (tile & 1u) * 4u + (r & 3u);
}

// x = sum of N bf16 parts, for two values side by side (each part one packed register).
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const v2f f = {x, y};
    p[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, v2bf));
    x -= __uint_as_float(p[i] << 16);
    y -= __uint_as_float(p[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ v4f mfma32(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Between what lanes of a wave write to LDS and what others of the same wave read
// there (or the other way round).  The hardware keeps a wave's accesses of LDS in
// order; this keeps the compiler's order, which sees one lane's addresses only.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

struct __attribute__((packed, aligned(2))) Bf16x8 {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(2))) Bf16x4 {
  uint32_t w[2];
};

// ---- first launch: what a chunk has of its own ----------------------------------

constexpr int kStride = kChunk + 4;  // floats per row of the 64 x 64 buffers

// D += A B of 16 x 16 blocks in LDS (binary32).  The sum over k runs in the
// order in which a lane's results lie, so a result can be the next B without
// being moved: step i takes k = 4 (lane / 16) + i.
__device__ __forceinline__ v4f block_product(const float *a, const float *b, v4f d, uint32_t lr, uint32_t lq) {
  const float4 f = *reinterpret_cast<const float4 *>(a + lr * kStride + lq * 4);
  d = __builtin_amdgcn_mfma_f32_16x16x4f32(f.x, b[(lq * 4 + 0) * kStride + lr], d, 0, 0, 0);
  d = __builtin_amdgcn_mfma_f32_16x16x4f32(f.y, b[(lq * 4 + 1) * kStride + lr], d, 0, 0, 0);
  d = __builtin_amdgcn_mfma_f32_16x16x4f32(f.z, b[(lq * 4 + 2) * kStride + lr], d, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(f.w, b[(lq * 4 + 3) * kStride + lr], d, 0, 0, 0);
}
__device__ __forceinline__ v4f block_product(const float *a, v4f b, v4f d, uint32_t lr, uint32_t lq) {
  const float4 f = *reinterpret_cast<const float4 *>(a + lr * kStride + lq * 4);
  d = __builtin_amdgcn_mfma_f32_16x16x4f32(f.x, b[0], d, 0, 0, 0);
  d = __builtin_amdgcn_mfma_f32_16x16x4f32(f.y, b[1], d, 0, 0, 0);
  d = __builtin_amdgcn_mfma_f32_16x16x4f32(f.z, b[2], d, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(f.w, b[3], d, 0, 0, 0);
}

// A fragment of a lower triangle in LDS (rows 16w.., columns 32ks..), split into N parts.
template <int N>
__device__ __forceinline__ void put_triangle(const float *m, uint8_t *out, uint32_t w, uint32_t ks, uint32_t lane) {
  const uint32_t row = 16u * w + (lane & 15u), c0 = 32u * ks + (lane >> 4) * 8u;
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const float4 f = *reinterpret_cast<const float4 *>(m + row * kStride + c0 + j);
    x[j] = f.x; x[j + 1] = f.y; x[j + 2] = f.z; x[j + 3] = f.w;
  }
  uint32_t parts[4][N];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    split2<N>(c0 + 2u * j <= row ? x[2 * j] : 0.0f, c0 + 2u * j + 1u <= row ? x[2 * j + 1] : 0.0f, parts[j]);
  uint8_t *p = out + triangle_fragment(w, ks) * N * kFragment + lane * 16u;
#pragma unroll
  for (int i = 0; i < N; ++i)
    *reinterpret_cast<uint4 *>(p + i * kFragment) = make_uint4(parts[0][i], parts[1][i], parts[2][i], parts[3][i]);
}

// x added over the 8 or 16 lanes of a row of kDk values (eight to a lane).
template <int kLanes>
__device__ __forceinline__ float add_lanes(float x) {
  auto moved = [](float v, auto how) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(how)::value, 0xF, 0xF, true));
  };
  x += moved(x, std::integral_constant<int, 0xB1>{});              // the neighbour
  x += moved(x, std::integral_constant<int, 0x4E>{});              // the other pair of four
  x += moved(x, std::integral_constant<int, 0x141>{});             // the other four of eight
  if (kLanes == 16) x += moved(x, std::integral_constant<int, 0x140>{});  // the other eight
  return x;
}

// A workgroup takes a chunk, a key head, and kHeads of its value heads, side by
// side: they share the keys, the queries and their products, and each step's
// waits.  Bound by those waits, not by memory (2048 tokens of 32 heads leave 39
// MB in 17 us, one workgroup alone takes 9), so four workgroups share a CU: A
// lies where the keys and queries were, T in A's place, 128 registers a lane do.
// (With places of their own, two a CU, packed prompts of 2322 tokens took 84.8
// us in both launches where they took 78.4 so.)
template <int kDk, int kHeads, bool kWhole>
__global__ __launch_bounds__(kThreads, 4) void delta_chunk_kernel(const DeltaArgs a) {
  constexpr int kRow = 2 * kStride;  // bf16 per staged row, which a row of A takes the place of
  static_assert(kDk <= 2 * kChunk && kHeads <= 2, "a row fits, its pad holds two norms and two betas; a matrix for each staged one");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][kChunk * kStride * 4];
  __shared__ __attribute__((aligned(16))) double sum_g[kHeads][kChunk];  // of g log2(e): decays are powers of two
  uint16_t *keys = reinterpret_cast<uint16_t *>(lds[0]), *queries = reinterpret_cast<uint16_t *>(lds[1]);
  // A of each value head, where the keys and queries were, and T in its place
  auto lower = [&](uint32_t h) { return reinterpret_cast<float *>(lds[h]); };
  // a token's norms and betas lie in the pad of the first one's rows
  auto norm_k = [&](uint32_t t) -> float & { return lower(0)[t * kStride + kChunk]; };
  auto norm_q = [&](uint32_t t) -> float & { return lower(0)[t * kStride + kChunk + 1]; };
  auto betas = [&](uint32_t h, uint32_t t) -> float & { return lower(0)[t * kStride + kChunk + 2 + h]; };

  const uint32_t tid = threadIdx.x, lane = tid & 63u, w = __builtin_amdgcn_readfirstlane(tid >> 6), lr = lane & 15u, lq = lane >> 4;
  const uint32_t sets = a.hv / kHeads;  // of value heads
  // From the last chunk to the first, so that what the second launch begins with was written last and is still in the
  // caches (16384 tokens of 32 heads leave 313 MB: both launches 520 us, and 527 from the first on).
  const uint32_t place = gridDim.x / sets - 1u - blockIdx.x / sets, head0 = blockIdx.x % sets * kHeads, khead = head0 / (a.hv / a.hk);

  // the sequence that the place belongs to: the last whose first place is at or below it
  __shared__ uint32_t found[3];
  bool any = false;
  for (uint32_t s0 = 0; s0 < a.count; s0 += kThreads) {
    const uint32_t s = s0 + tid;
    bool at = false;
    if (s < a.count) {
      const uint32_t begin = min((uint32_t)max(a.starts[s], 0), a.tokens), end = min((uint32_t)max(a.starts[s + 1u], 0), a.tokens);
      at = first_place(begin, s) <= place;
      if (at && (s + 1u == a.count || first_place(end, s + 1u) > place)) {
        found[0] = begin;
        found[1] = end;
        found[2] = first_place(begin, s);
      }
    }
    any |= __syncthreads_or(at) != 0;
  }
  if (!any) return;
  const uint32_t t0 = found[0] + (place - found[2]) * kChunk, t_end = found[1];
  if (t0 >= t_end) return;
  const uint32_t n = min(t_end - t0, (uint32_t)kChunk);

  // keys and queries into LDS, zeros past the chunk's end and past dk; their
  // norms on the way (the lanes of a row lie side by side)
  {
    constexpr uint32_t kVecs = kDk / 8;
    // a wave for each value head: its sums of g, its betas (ahead of the keys, whose way it shares)
    float gt = 0.0f, beta = 0.0f;
    if (w < (uint32_t)kHeads) {
      const uint64_t at = (uint64_t)(t0 + min(lane, n - 1u)) * a.hv + head0 + w;
      gt = a.g[at];
      beta = a.beta[at];
    }
    const uint16_t *kbase = a.k + (uint64_t)t0 * a.k_token + (uint64_t)khead * a.k_head;
    const uint16_t *qbase = a.q + (uint64_t)t0 * a.q_token + (uint64_t)khead * a.q_head;
    uint4 kv[kVecs / 4], qv[kVecs / 4];
#pragma unroll
    for (uint32_t i = 0; i < kVecs / 4; ++i) {
      const uint32_t r = (i * kThreads + tid) / kVecs, c = tid % kVecs * 8u;
      kv[i] = qv[i] = make_uint4(0, 0, 0, 0);
      if constexpr (kWhole) {  // (no branch around the loads: they leave together)
        const uint32_t at = min(r, n - 1u);
        const Bf16x8 x = *reinterpret_cast<const Bf16x8 *>(kbase + (uint64_t)at * a.k_token + c);
        const Bf16x8 y = *reinterpret_cast<const Bf16x8 *>(qbase + (uint64_t)at * a.q_token + c);
        kv[i] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        qv[i] = make_uint4(y.w[0], y.w[1], y.w[2], y.w[3]);
      } else if (r < n) {
        const uint16_t *kp = kbase + (uint64_t)r * a.k_token + c, *qp = qbase + (uint64_t)r * a.q_token + c;
        if (c + 8u <= a.dk) {
          const Bf16x8 x = *reinterpret_cast<const Bf16x8 *>(kp), y = *reinterpret_cast<const Bf16x8 *>(qp);
          kv[i] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
          qv[i] = make_uint4(y.w[0], y.w[1], y.w[2], y.w[3]);
        } else {
          uint32_t x[8], y[8];
#pragma unroll
          for (uint32_t j = 0; j < 8; ++j) {
            x[j] = c + j < a.dk ? kp[j] : 0u;
            y[j] = c + j < a.dk ? qp[j] : 0u;
          }
          kv[i] = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
          qv[i] = make_uint4(y[0] | y[1] << 16, y[2] | y[3] << 16, y[4] | y[5] << 16, y[6] | y[7] << 16);
        }
      }
    }
    if (w < (uint32_t)kHeads) {
      if (lane >= n) gt = 0.0f;
      double g = (double)(gt < kNoDecay ? kNoDecay : gt) * 1.4426950408889634;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(g, d);
        g += lane >= (uint32_t)d ? o : 0.0;
      }
      sum_g[w][lane] = g;
      betas(w, lane) = lane < n ? beta : 0.0f;
    }
#pragma unroll
    for (uint32_t i = 0; i < kVecs / 4; ++i) {
      const uint32_t r = (i * kThreads + tid) / kVecs, c = tid % kVecs * 8u;
      if (kWhole && r >= n) kv[i] = qv[i] = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4 *>(keys + r * kRow + c) = kv[i];
      *reinterpret_cast<uint4 *>(queries + r * kRow + c) = qv[i];
      const uint32_t kw[4] = {kv[i].x, kv[i].y, kv[i].z, kv[i].w}, qw[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
      float sk = 0.0f, sq2 = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = __uint_as_float(kw[j] << 16), y = __uint_as_float(kw[j] & 0xFFFF0000u);
        const float u = __uint_as_float(qw[j] << 16), v = __uint_as_float(qw[j] & 0xFFFF0000u);
        sk = fmaf(x, x, fmaf(y, y, sk));
        sq2 = fmaf(u, u, fmaf(v, v, sq2));
      }
      sk = add_lanes<kVecs>(sk);
      sq2 = add_lanes<kVecs>(sq2);
      if (c == 0u) {
        norm_k(r) = sk;
        norm_q(r) = sq2;
      }
    }
  }
  __syncthreads();
  if (w < 2u) {  // a wave for the keys, one for the queries: the sums' roots
    float &x = w == 0u ? norm_k(lane) : norm_q(lane);
    x = (a.l2norm ? 1.0f / sqrtf(x + kNormEps) : 1.0f) * (w == 0u ? 1.0f : a.scale);
  }

  // k.k and k.q for tokens 16w.., the tiles of the lower triangle: a lane has
  // token 16w + lr and four keys 16j + 4 lq.. in each
  v4f kk[4], qk[4];
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) {
    kk[j] = v4f{0, 0, 0, 0};
    qk[j] = v4f{0, 0, 0, 0};
    if (j <= w) {
#pragma unroll
      for (int ks = 0; ks < kDk / 32; ++ks) {
        const v8bf kr = *reinterpret_cast<const v8bf *>(keys + (16 * w + lr) * kRow + 32 * ks + lq * 8);
        const v8bf qr = *reinterpret_cast<const v8bf *>(queries + (16 * w + lr) * kRow + 32 * ks + lq * 8);
        const v8bf kc = *reinterpret_cast<const v8bf *>(keys + (16 * j + lr) * kRow + 32 * ks + lq * 8);
        kk[j] = mfma32(kc, kr, kk[j]);
        qk[j] = mfma32(kc, qr, qk[j]);
      }
    }
  }
  __syncthreads();  // keys and queries have been read

  uint8_t *mine = a.workspace + ((uint64_t)place * a.hv + head0) * kHeadBytes;
  if (w < (uint32_t)kHeads) {
    const double g = sum_g[w][lane];
    const float e = __builtin_amdgcn_exp2f((float)g), beta = betas(w, lane);
    float *f = reinterpret_cast<float *>(mine + w * kHeadBytes + kTBytes + kInnerBytes) + lane;
    f[0] = beta;
    f[kChunk] = beta * e * norm_k(lane);
    f[2 * kChunk] = lane < n ? __builtin_amdgcn_exp2f((float)(sum_g[w][kChunk - 1] - g)) * norm_k(lane) : 0.0f;
    f[3 * kChunk] = lane < n ? e * norm_q(lane) : 0.0f;
    if (lane == kChunk - 1) f[3 * kChunk + 1] = e;
  }

  // A into LDS; the q.k triangle straight into the workspace: a lane's four
  // values lie side by side in its fragment.  (All four tiles, those above the
  // diagonal in vain: without branches between them their waits overlap.)
  {
    const uint32_t t = 16u * w + lr;
    const float tk = norm_k(t), tq = norm_q(t);
    float sk[4][4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) sk[j][i] = norm_k(16u * j + lq * 4u + i);
#pragma unroll
    for (uint32_t h = 0; h < (uint32_t)kHeads; ++h) {
      const double g = sum_g[h][t];
      const float row_k = betas(h, t) * tk;
      double gs[4][4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) gs[j][i] = sum_g[h][16u * j + lq * 4u + i];
      uint8_t *to = mine + h * kHeadBytes + kTBytes + triangle_fragment(w, 0) * 3u * kFragment + lr * 16u + (lq >> 1) * 256u + (lq & 1u) * 8u;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) {
        float x[4], y[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const uint32_t s = 16u * j + lq * 4u + i;
          // (keys after the token would grow: their power is not taken)
          const float decay = s <= t ? __builtin_amdgcn_exp2f((float)(g - gs[j][i])) * sk[j][i] : 0.0f;
          x[i] = s < t ? row_k * decay * kk[j][i] : 0.0f;
          y[i] = s <= t ? tq * decay * qk[j][i] : 0.0f;
        }
        *reinterpret_cast<float4 *>(lower(h) + t * kStride + 16u * j + lq * 4u) = make_float4(x[0], x[1], x[2], x[3]);
        if (j >= 2u && w < 2u) continue;  // no such fragment
        uint32_t lo[3], hi[3];
        split2<3>(y[0], y[1], lo);
        split2<3>(y[2], y[3], hi);
#pragma unroll
        for (uint32_t i = 0; i < 3; ++i)
          *reinterpret_cast<uint2 *>(to + ((j >> 1) * 3u + i) * kFragment + (j & 1u) * 512u) = make_uint2(lo[i], hi[i]);
      }
    }
  }

  wave_exchange();  // A's diagonal blocks: a wave's own rows, by other lanes

  // T: the 16 x 16 blocks on the diagonal by substitution (a wave has its own
  // rows' block of every head, a lane a column), then blocks of 16 and of 32
  // joined in pairs,
  //   [[a, 0], [c, b]]^-1 = [[a', 0], [-b' c a', b']],
  // each in the place of what it is the last to read.
  {
    const uint32_t h = lq & (kHeads - 1u);
    const float *block = lower(h) + 16u * w * kStride + 16u * w;
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x[4] = {(uint32_t)i == lr ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(block + i * kStride + m);
        x[0] = fmaf(-f.x, t[m], x[0]);
        if (m + 1 < i) x[1] = fmaf(-f.y, t[m + 1], x[1]);
        if (m + 2 < i) x[2] = fmaf(-f.z, t[m + 2], x[2]);
        if (m + 3 < i) x[3] = fmaf(-f.w, t[m + 3], x[3]);
      }
      t[i] = (x[0] + x[1]) + (x[2] + x[3]);
    }
    wave_exchange();  // (the blocks have been read)
    if (lq < (uint32_t)kHeads) {
#pragma unroll
      for (int i = 0; i < 16; ++i) lower(h)[(16u * w + i) * kStride + 16u * w + lr] = t[i];
    }
  }
  __syncthreads();
  if (w < 2u * kHeads) {
    float *v = lower(w >> 1);
    const uint32_t o = 32u * (w & 1u);
    const v4f x = block_product(v + (o + 16) * kStride + o, v + o * kStride + o, v4f{0, 0, 0, 0}, lr, lq);
    const v4f y = block_product(v + (o + 16) * kStride + o + 16, x, v4f{0, 0, 0, 0}, lr, lq);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[(o + 16 + lq * 4 + i) * kStride + o + lr] = -y[i];
  }
  __syncthreads();
  {
    const uint32_t jt = w & 1u, rt = w >> 1;
    v4f x[kHeads][2], y[kHeads];
#pragma unroll
    for (uint32_t h = 0; h < (uint32_t)kHeads; ++h)
#pragma unroll
      for (uint32_t r = 0; r < 2; ++r) {
        x[h][r] = v4f{0, 0, 0, 0};
        if (r > rt) continue;
        for (uint32_t kt = jt; kt < 2; ++kt)
          x[h][r] = block_product(lower(h) + (32 + 16 * r) * kStride + 16 * kt, lower(h) + 16 * kt * kStride + 16 * jt, x[h][r], lr, lq);
      }
#pragma unroll
    for (uint32_t h = 0; h < (uint32_t)kHeads; ++h) {
      y[h] = block_product(lower(h) + (32 + 16 * rt) * kStride + 32, x[h][0], v4f{0, 0, 0, 0}, lr, lq);
      if (rt == 1u) y[h] = block_product(lower(h) + 48 * kStride + 48, x[h][1], y[h], lr, lq);
    }
    __syncthreads();  // c has been read
#pragma unroll
    for (uint32_t h = 0; h < (uint32_t)kHeads; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) lower(h)[(32 + 16 * rt + lq * 4 + i) * kStride + 16 * jt + lr] = -y[h][i];
  }
  __syncthreads();
#pragma unroll
  for (uint32_t i0 = 0; i0 < kTriangle * kHeads; i0 += 4) {
    const uint32_t i = i0 + w, h = i / kTriangle, f = i % kTriangle;
    if (i >= kTriangle * kHeads) break;
    put_triangle<3>(lower(h), mine + h * kHeadBytes, f < 2u ? f : f / 2u + 1u, f < 2u ? 0u : f & 1u, lane);
  }
}

// ---- second launch: the state along the chunks ------------------------------------

// Eight waves.  The first four carry the state: wave w keeps rows of it
// (32 for dk 128, 16 for 64) in registers, multiplies them by the chunk's keys,
// the four partial sums meet in LDS, and tokens 16w.. of R and U are its own
// from there on.  The other four make the output of tokens 16w.. from the
// state's parts and U, which they find in LDS, beside that chain.  The operands
// of the next chunk are loaded into the registers of this one's as soon as
// those have been used: the loads are spread over the step and have most of
// its time to arrive.
//
// What bounds it is the chain itself, 1.45 us per chunk of one head alone: three
// exchanges through LDS, and the latency of what lies between them (1.8 with a
// workgroup on every CU, 2048 tokens of 32 heads; 1.8 where the operands pass
// through the caches, 16384 tokens).  So where there are more workgroups than CUs
// two should share one: 128 registers per lane allow it (the kernels of odd sizes
// are not held to it; all but one fit too).
constexpr int kScanThreads = 512;

// Where a few long sequences leave most CUs without work, the chunks of a
// sequence are cut into segments that run side by side.  The state after a
// segment is M S + N of the state S before it, with N what the segment makes of
// an empty state, and M's columns what it makes of the unit vectors without
// values.  A launch (kParts) runs the first segment of every sequence, and for
// the others but the last N and M; the next (kRest) finds each segment's state
// from N and M of those before it, and runs it.
//
// That is up to three times the work, for a chain of two segments and a product
// per segment instead of all chunks: one sequence of 9000 tokens takes 79 us with
// one head (211 in one chain), 101 with four (221).
enum { kChain = 0, kParts = 1, kRest = 2 };

// What both kinds of waves know of their work.
struct ScanPlace {
  DeltaSeq sq;  // (the tokens of the segment)
  uint32_t head, khead, col, place0, chunks, last;  // last: tokens of the last chunk
  bool col_in;
  bool keep;          // of segments: the state after this one is the sequence's
  bool unit, output;  // kParts: M's columns; the segment's output is made
  float *parts;       // kParts: where M's or N's columns go, null: nowhere
};

// M and N of a segment and head: kDk rows each of kDk and of dv (in 16s) values.
template <int kTiles>
__device__ __forceinline__ float *segment_parts(const DeltaArgs &a, uint32_t place, uint32_t head) {
  constexpr uint32_t kDk = 64 * kTiles;
  return a.parts + ((uint64_t)place * a.hv + head) * kDk * (kDk + (a.dv + 15u) / 16u * 16u);
}

// Loads of 16 (or 8) bytes from a uniform base and a lane's 32-bit offset.
__device__ __forceinline__ uint4 load16(const uint8_t *base, uint32_t off) {
  const Bf16x8 x = *reinterpret_cast<const Bf16x8 *>(base + off);
  return make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
}
__device__ __forceinline__ uint4 fragment(const uint8_t *base, uint32_t off) {
  return *reinterpret_cast<const uint4 *>(base + off);
}

// N bf16 (8 or 4) of a row of q or k from value d0 on, zeros past dk; off in bytes.
template <int N, bool kWhole>
__device__ __forceinline__ uint4 load_row(const uint8_t *base, uint32_t off, uint32_t d0, uint32_t dk) {
  if (!kWhole && d0 >= dk) return make_uint4(0u, 0u, 0u, 0u);
  if (!kWhole && d0 + N > dk) {
    uint32_t x[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
      x[i] = i < (uint32_t)N && d0 + i < dk ? *reinterpret_cast<const uint16_t *>(base + off + 2u * i) : 0u;
    return make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
  }
  if constexpr (N == 8) {
    return load16(base, off);
  } else {
    const Bf16x4 x = *reinterpret_cast<const Bf16x4 *>(base + off);
    return make_uint4(x.w[0], x.w[1], 0u, 0u);
  }
}

// bytes per token of a wave's rows of the keys; the pad spreads banks
template <int kTiles>
constexpr int kKeyRow = 32 * kTiles + 16;

// Whether four neighbouring lanes load neighbouring pieces of a row of q or k,
// so that one access of the CU's cache serves them; the keys then go through
// LDS before their first product, the queries change lanes.  As the operands lie
// in the lanes each lane's 16 bytes are an access: 2900 a chunk, which is what
// two workgroups on a CU wait for (prompts of up to 927 tokens, 16 heads: 59.6 us
// by quads, and 62.7 without; packed prompts of 2322 tokens 79.8 and 81.5; 16384
// tokens 520 and 535).  A chain of 64 values has fewer, and the way through LDS is
// longer (2048 tokens, packed, 1 head: 25.5 us by quads, and 24.2); nor do they
// pay in segments (8192 tokens, 1 head: 72.9 by quads, and 72.3).
template <int kTiles, bool kWhole, int kMode>
constexpr bool kQuads = kTiles == 2 && kWhole && kMode == 0;
// values per column of the state before a segment, likewise
template <int kTiles>
constexpr int kJoinedRow = 64 * kTiles + 4;

template <int kTiles>
struct ScanLds {
  float4 part[16][64];          // partial K S0: [token tile * 4 + wave][lane]
  uint8_t r[3][2][1024];        // R, decayed U and U as operands: [part][32 tokens][lane]
  uint8_t decayed[3][2][1024];
  uint8_t u[3][2][1024];
  struct __attribute__((aligned(16))) {
    float value[kChunk][16];    // b v
    float factor[3][kChunk];    // b e^G rk, e^(G_L - G) rk, scale e^G rq
    float decay;                // e^G_L
  } tokens[2];                  // of this chunk and of the next
  uint8_t keys[4][kChunk][kKeyRow<kTiles>];
  uint8_t s[3][2 * kTiles][1024];  // the state's parts: [part][32 rows][lane]

  // the state before a segment, column by column; it and its predecessor lie where the chain's operands come later
  __device__ float *joined(bool other = false) { return reinterpret_cast<float *>(other ? &keys[0][0][0] : reinterpret_cast<uint8_t *>(part)); }
  static_assert(16 * kJoinedRow<kTiles> * 4 <= 4 * kChunk * kKeyRow<kTiles> && 16 * kJoinedRow<kTiles> * 4 <= 16 * 64 * 16, "");
};

__device__ __forceinline__ v8bf as_bf(uint4 x) { return __builtin_bit_cast(v8bf, x); }

template <int kTiles, bool kWhole, int kMode>
__device__ __forceinline__ void carry_state(const DeltaArgs &a, const ScanPlace &pl, ScanLds<kTiles> &lds, uint32_t w,
                                            uint32_t lane) {
  const uint32_t lr = lane & 15u, lq = lane >> 4;
  const v4f zero = {0, 0, 0, 0};
  float *state = a.state + ((uint64_t)max(pl.sq.slot, 0) * a.hv + pl.head) * a.dk * a.dv + pl.col;
  v4f s[kTiles];
#pragma unroll
  for (uint32_t t = 0; t < kTiles; ++t)
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t r = state_row(w * kTiles + t, lq * 4u + i);
      if constexpr (kMode == kRest)
        s[t][i] = lds.joined()[lr * kJoinedRow<kTiles> + r];
      else
        s[t][i] = pl.sq.slot >= 0 && !pl.sq.fresh && (kWhole || (pl.col_in && r < a.dk)) ? state[(uint64_t)r * a.dv] : 0.0f;
      if constexpr (kMode == kParts)
        if (pl.unit && r == pl.col) s[t][i] = 1.0f;
    }
  if constexpr (kMode == kRest) __syncthreads();  // read before its place is filled

  // bases of the next chunk to load, and this lane's offsets in bytes
  const uint8_t *mine = a.workspace + ((uint64_t)pl.place0 * a.hv + pl.head) * kHeadBytes;
  const uint8_t *keys = reinterpret_cast<const uint8_t *>(a.k + (uint64_t)pl.khead * a.k_head + (uint64_t)pl.sq.begin * a.k_token);
  // the token (of 16) and the piece of its row that this lane loads
  constexpr bool kByQuads = kQuads<kTiles, kWhole, kMode>;
  const uint32_t load_t = kByQuads ? lane >> 2 : lr, load_p = kByQuads ? lane & 3u : lq;
  const uint32_t dk0 = state_row(w * kTiles, load_p * 4u), lane16 = lane * 16u;
  const uint32_t t_at[2] = {triangle_fragment(w, 0) * 3u * kFragment, triangle_fragment(w, 1) * 3u * kFragment};
  uint32_t k_off[4];
  // rows past the sequence's end read its last token: their factors are zero
  auto token_offsets = [&](uint32_t n) {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) k_off[i] = 2u * (min(16u * i + load_t, n - 1u) * a.k_token + dk0);
  };

  uint4 op_k[4], op_t[2][3];
  auto load_keys = [&]() {
#pragma unroll
    for (int m = 0; m < 4; ++m) op_k[m] = load_row<4 * kTiles, kWhole>(keys, k_off[m], dk0, a.dk);
  };
  auto load_inverse = [&]() {
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i) op_t[0][i] = fragment(mine + t_at[0] + i * kFragment, lane16);
    if (w >= 2u) {
#pragma unroll
      for (uint32_t i = 0; i < 3; ++i) op_t[1][i] = fragment(mine + t_at[1] + i * kFragment, lane16);
    }
  };

  // place of this lane's four rows in an operand of 64 tokens
  const uint32_t put = (w >> 1) * 1024u + ((w & 1u) * 2u + (lq >> 1)) * 256u + lr * 16u + (lq & 1u) * 8u;
  token_offsets(pl.chunks == 1u ? pl.last : (uint32_t)kChunk);
  load_keys();
  load_inverse();
  // The keys go through LDS, where each wave keeps its own rows of all tokens:
  // the product with the state takes them with tokens as rows, the update with
  // dk as rows, read back transposed (a group of 16 lanes reads 4 tokens x 16
  // rows, and lane i gets row i's 4).
  uint8_t *keys_put = &lds.keys[w][load_t][0] + load_p * (8u * kTiles);
  const uint8_t *keys_rows = &lds.keys[w][lr][0] + lq * (8u * kTiles);
  auto put_keys = [&]() {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if constexpr (kTiles == 2)
        *reinterpret_cast<uint4 *>(keys_put + 16 * m * kKeyRow<kTiles>) = op_k[m];
      else
        *reinterpret_cast<uint2 *>(keys_put + 16 * m * kKeyRow<kTiles>) = make_uint2(op_k[m].x, op_k[m].y);
    }
  };
  const uint8_t *keys_get = &lds.keys[w][lq * 8u + (lr >> 2)][0] + (lr & 3u) * (8u * kTiles);
  auto transposed = [&](int t, int ks) -> v8bf {
    const uint8_t *from = keys_get + 32 * ks * kKeyRow<kTiles> + t * 8;
    const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)from);
    const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)(from + 4 * kKeyRow<kTiles>));
    return __builtin_bit_cast(v8bf, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  for (uint32_t c = 0; c < pl.chunks; ++c) {
    // past the end the last chunk is loaded again
    if (c + 1u < pl.chunks) {
      mine += (uint64_t)a.hv * kHeadBytes;
      keys += (uint64_t)kChunk * 2u * a.k_token;
      if (c + 2u == pl.chunks) token_offsets(pl.last);
    }
    // K S0 over the wave's rows of the state
    if constexpr (kByQuads) {
      wave_exchange();  // (the last chunk's have been read)
      put_keys();
      wave_exchange();
#pragma unroll
      for (int m = 0; m < 4; ++m) op_k[m] = *reinterpret_cast<const uint4 *>(keys_rows + 16 * m * kKeyRow<kTiles>);
    }
    uint32_t sp[kTiles][2][3];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      split2<3>(s[t][0], s[t][1], sp[t][0]);
      split2<3>(s[t][2], s[t][3], sp[t][1]);
    }
    v4f x[4];
    if constexpr (kTiles == 2) {
#pragma unroll
      for (int i = 2; i >= 0; --i) {
        const uint4 b = make_uint4(sp[0][0][i], sp[0][1][i], sp[1][0][i], sp[1][1][i]);
        *reinterpret_cast<uint4 *>(&lds.s[i][w][lane16]) = b;
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = mfma32(as_bf(op_k[m]), as_bf(b), i == 2 ? zero : x[m]);
      }
    } else {
      // 16 rows: two parts of the state side by side make an operand of 32
#pragma unroll
      for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint2 *>(&lds.s[i][w >> 1][lane16 + (w & 1u) * 8u]) = make_uint2(sp[0][0][i], sp[0][1][i]);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        x[m] = mfma32(as_bf(op_k[m]), as_bf(make_uint4(sp[0][0][2], sp[0][1][2], 0u, 0u)), zero);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        x[m] = mfma32(as_bf(make_uint4(op_k[m].x, op_k[m].y, op_k[m].x, op_k[m].y)),
                      as_bf(make_uint4(sp[0][0][1], sp[0][1][1], sp[0][0][0], sp[0][1][0])), x[m]);
    }
    if constexpr (!kByQuads) {
      wave_exchange();
      put_keys();
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) *reinterpret_cast<v4f *>(&lds.part[m * 4 + w][lane]) = x[m];
    __syncthreads();
    // R for tokens 16w..
    const auto &tok = lds.tokens[c & 1u];
    v4f p[4], r;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const v4f *>(&lds.part[w * 4 + i][lane]);
    const v4f from_state = *reinterpret_cast<const v4f *>(&tok.factor[0][16u * w + lq * 4u]);
    const v4f to_state = *reinterpret_cast<const v4f *>(&tok.factor[1][16u * w + lq * 4u]);
    const float keep = tok.decay;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = tok.value[16u * w + lq * 4u + i][lr];
    __builtin_amdgcn_sched_barrier(0);
    load_keys();
    __builtin_amdgcn_sched_barrier(0);
    p[0] = (p[0] + p[1]) + (p[2] + p[3]);
    uint32_t lo[3], hi[3];
    r -= from_state * p[0];
    split2<3>(r[0], r[1], lo);
    split2<3>(r[2], r[3], hi);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2 *>(&lds.r[i][0][0] + put) = make_uint2(lo[i], hi[i]);
    __syncthreads();
    // U = T R for tokens 16w..; columns past 16w + 15 of T are zero
    v8bf rb[3][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int i = 0; i < 3; ++i) rb[i][ks] = *reinterpret_cast<const v8bf *>(&lds.r[i][ks][lane16]);
    v4f u = mfma32(as_bf(op_t[0][2]), rb[0][0], zero), u1 = mfma32(as_bf(op_t[0][1]), rb[0][0], zero);
    if (w < 2u) {
      u = mfma32(as_bf(op_t[0][1]), rb[1][0], u);
      u1 = mfma32(as_bf(op_t[0][0]), rb[1][0], u1);
      u = mfma32(as_bf(op_t[0][0]), rb[2][0], u);
      u1 = mfma32(as_bf(op_t[0][0]), rb[0][0], u1);
      u += u1;
    } else {
      v4f u2 = mfma32(as_bf(op_t[1][2]), rb[0][1], zero), u3 = mfma32(as_bf(op_t[1][1]), rb[0][1], zero);
      u = mfma32(as_bf(op_t[0][1]), rb[1][0], u);
      u1 = mfma32(as_bf(op_t[0][0]), rb[1][0], u1);
      u2 = mfma32(as_bf(op_t[1][1]), rb[1][1], u2);
      u3 = mfma32(as_bf(op_t[1][0]), rb[1][1], u3);
      u = mfma32(as_bf(op_t[0][0]), rb[2][0], u);
      u1 = mfma32(as_bf(op_t[0][0]), rb[0][0], u1);
      u2 = mfma32(as_bf(op_t[1][0]), rb[2][1], u2);
      u3 = mfma32(as_bf(op_t[1][0]), rb[0][1], u3);
      u = (u + u2) + (u1 + u3);
    }
    split2<3>(u[0] * to_state[0], u[1] * to_state[1], lo);
    split2<3>(u[2] * to_state[2], u[3] * to_state[3], hi);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2 *>(&lds.decayed[i][0][0] + put) = make_uint2(lo[i], hi[i]);
    split2<3>(u[0], u[1], lo);
    split2<3>(u[2], u[3], hi);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2 *>(&lds.u[i][0][0] + put) = make_uint2(lo[i], hi[i]);
    __syncthreads();
    // the state
    v8bf sb[3][2];
#pragma unroll
    for (int i = 2; i >= 0; --i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) sb[i][ks] = *reinterpret_cast<const v8bf *>(&lds.decayed[i][ks][lane16]);
    v8bf kt[kTiles][2];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) kt[t][ks] = transposed(t, ks);
    __builtin_amdgcn_sched_barrier(0);
    load_inverse();
    __builtin_amdgcn_sched_barrier(0);
    v4f s1[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) s[t] *= keep;
#pragma unroll
    for (int i = 2; i >= 0; --i)
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        s1[t] = mfma32(kt[t][0], sb[i][0], i == 2 ? zero : s1[t]);
        s[t] = mfma32(kt[t][1], sb[i][1], s[t]);
      }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) s[t] += s1[t];
  }

  uint32_t r0 = lq * 4u;
  asm volatile("" : "+v"(r0));  // the places are worked out again, not kept in registers over the loop
  if constexpr (kMode == kParts)
    if (pl.parts != nullptr) {
      const uint32_t stride = pl.unit ? 64u * kTiles : (a.dv + 15u) / 16u * 16u;
#pragma unroll
      for (uint32_t t = 0; t < kTiles; ++t)
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) pl.parts[state_row(w * kTiles + t, r0 + i) * stride + pl.col] = s[t][i];
    }
  if (pl.sq.slot < 0 || !pl.col_in || (kMode != kChain && !pl.keep)) return;
#pragma unroll
  for (uint32_t t = 0; t < kTiles; ++t)
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t r = state_row(w * kTiles + t, r0 + i);
      if (kWhole || r < a.dk) state[(uint64_t)r * a.dv] = s[t][i];
    }
}

template <int kTiles, bool kWhole, int kMode>
__device__ __forceinline__ void make_output(const DeltaArgs &a, const ScanPlace &pl, ScanLds<kTiles> &lds,
                                            uint32_t w, uint32_t lane) {
  const bool output = kMode != kParts || pl.output;
  constexpr int kSteps = 2 * kTiles;  // dk in 32s
  const uint32_t lr = lane & 15u, lq = lane >> 4, lane16 = lane * 16u;
  const v4f zero = {0, 0, 0, 0};
  const uint8_t *mine = a.workspace + ((uint64_t)pl.place0 * a.hv + pl.head) * kHeadBytes;
  const uint8_t *queries = reinterpret_cast<const uint8_t *>(a.q + (uint64_t)pl.khead * a.q_head + (uint64_t)pl.sq.begin * a.q_token);
  uint8_t *out = reinterpret_cast<uint8_t *>(a.out + ((uint64_t)pl.sq.begin * a.hv + pl.head) * a.dv);
  const uint32_t in_at[2] = {kTBytes + triangle_fragment(w, 0) * 3u * kFragment, kTBytes + triangle_fragment(w, 1) * 3u * kFragment};
  // factors: a lane takes row lane / 16 of token 16w + lane % 16 (rows 1 to 3, and then the decay), and the b of token
  // 16w + lane / 4, of which it takes v's columns 4 (lane % 4)..
  const uint8_t *vals = reinterpret_cast<const uint8_t *>(a.v + (uint64_t)pl.head * a.v_head + (uint64_t)pl.sq.begin * a.v_token);
  const uint32_t f_off = kTBytes + kInnerBytes + (lq == 3u ? 4u * kFactorRow : (lq + 1u) * kFactorRow + (16u * w + lr) * 4u);
  const uint32_t b_off = kTBytes + kInnerBytes + (16u * w + (lane >> 2)) * 4u;
  const uint32_t v_col = pl.col - lr + (lane & 3u) * 4u;
  // Step k of the product takes 8 values of row lr: those from 32 k + 8 lq on.
  // By quads it takes those from 32 lq + 8 k on: lane lr loads them of the row
  // with k in place of its lowest bits, at these bits' place, and they change.
  constexpr bool kByQuads = kQuads<kTiles, kWhole, kMode>;
  uint32_t q_off[kByQuads ? kSteps : 1], v_off;
  const uint32_t out_row = 2u * a.hv * a.dv, out_off = (16u * w + lq * 4u) * out_row + 2u * pl.col;
  auto token_offsets = [&](uint32_t n) {
    if constexpr (kByQuads) {
#pragma unroll
      for (uint32_t k = 0; k < kSteps; ++k)
        q_off[k] = 2u * (min(16u * w + ((lr & ~3u) | k), n - 1u) * a.q_token + 32u * lq + (lr & 3u) * 8u);
    } else {
      q_off[0] = 2u * (min(16u * w + lr, n - 1u) * a.q_token + lq * 8u);
    }
    v_off = 2u * (min(16u * w + (lane >> 2), n - 1u) * a.v_token + v_col);
  };

  uint4 op_q[kSteps], op_in[2][3];
  uint4 val;
  float factor, beta;
  auto load_tokens = [&]() {
    if (kMode == kParts && pl.unit)
      val = make_uint4(0u, 0u, 0u, 0u);
    else
      val = load_row<4, kWhole>(vals, v_off, v_col, a.dv);
    factor = *reinterpret_cast<const float *>(mine + f_off);
    beta = *reinterpret_cast<const float *>(mine + b_off);
  };
  // the loaded tokens into LDS, for both kinds of waves
  auto put_tokens = [&](uint32_t c) {
    auto &tok = lds.tokens[c & 1u];
    const v4f v = {__uint_as_float(val.x << 16), __uint_as_float(val.x & 0xFFFF0000u), __uint_as_float(val.y << 16),
                   __uint_as_float(val.y & 0xFFFF0000u)};
    *reinterpret_cast<v4f *>(&tok.value[16u * w + (lane >> 2)][(lane & 3u) * 4u]) = v * beta;
    if (lq < 3u)
      tok.factor[lq][16u * w + lr] = factor;
    else if (lr == 0u && w == 0u)
      tok.decay = factor;
  };
  auto load_queries = [&]() {
    if (!output) return;
#pragma unroll
    for (uint32_t k = 0; k < kSteps; ++k) op_q[k] = kByQuads ? load16(queries, q_off[k]) : load_row<8, kWhole>(queries, q_off[0] + 64u * k, 32u * k + lq * 8u, a.dk);
  };
  // a bit of the lane and one of the step change places
  auto exchange = [&](auto bit) {
    constexpr uint32_t kBit = decltype(bit)::value;
    const bool set = (lane & kBit) != 0u;
    auto swap = [&](uint32_t &lo, uint32_t &hi) {
      const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(set ? lo : hi), kBit == 1u ? 0xB1 : 0x4E, 0xF, 0xF, true);
      if (set) lo = got; else hi = got;
    };
#pragma unroll
    for (uint32_t k = 0; k < kSteps; ++k) {
      if (k & kBit) continue;
      swap(op_q[k].x, op_q[k | kBit].x);
      swap(op_q[k].y, op_q[k | kBit].y);
      swap(op_q[k].z, op_q[k | kBit].z);
      swap(op_q[k].w, op_q[k | kBit].w);
    }
  };
  auto load_inner = [&]() {
    if (!output) return;
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i) op_in[0][i] = fragment(mine + in_at[0] + i * kFragment, lane16);
    if (w >= 2u) {
#pragma unroll
      for (uint32_t i = 0; i < 3; ++i) op_in[1][i] = fragment(mine + in_at[1] + i * kFragment, lane16);
    }
  };
  // The tokens run one chunk ahead of the rest: they are loaded in one step,
  // put into LDS at the end of the next, and used in the one after.
  auto advance = [&](uint32_t c) {  // bases of chunk c
    mine += (uint64_t)a.hv * kHeadBytes;
    queries += (uint64_t)kChunk * 2u * a.q_token;
    vals += (uint64_t)kChunk * 2u * a.v_token;
    if (c + 1u == pl.chunks) token_offsets(pl.last);
  };
  if constexpr (kMode == kRest) __syncthreads();
  // The column blocks of a head run side by side on one XCD.  Where the first
  // launch has left more than the caches hold beside q, k, v and the output,
  // each touches its share of the lines of the chunk after the next: two waves
  // the workspace's, two those of q, k and v.  From 80 MB of workspace on: 8000
  // tokens of 20 heads (95 MB) 216 us, and 233 without; 16000 of 12 (114 MB) 398,
  // and 494; 9000 of 16 (86 MB) 233, and 237; 2128 packed tokens of 8 heads (13
  // MB) 48.2, and 47.0.
  const uint8_t *touch = mine;
  uint64_t touch_step = (uint64_t)a.hv * kHeadBytes;
  bool touches = false;
  if (kMode == kChain && (uint64_t)(a.tokens / kChunk + a.count) * a.hv > (80u << 20) / kHeadBytes) {
    const uint32_t mine_of = __builtin_amdgcn_readfirstlane(pl.col >> 4) + (a.dv + 15u) / 16u * ((w & 1u) * 64u + lane);
    if (w < 2u) {
      touch += mine_of * 128u;
      touches = mine_of < kHeadBytes / 128u;
    } else {  // token, which of the three, half of the row
      const uint64_t t = pl.sq.begin + mine_of / 6u;
      const uint32_t what = mine_of % 6u / 2u, token = what == 0u ? a.q_token : what == 1u ? a.k_token : a.v_token;
      const uint16_t *row = what == 0u   ? a.q + (uint64_t)pl.khead * a.q_head
                            : what == 1u ? a.k + (uint64_t)pl.khead * a.k_head
                                         : a.v + (uint64_t)pl.head * a.v_head;
      touch = reinterpret_cast<const uint8_t *>(row + t * token + (mine_of & 1u) * min(64u, (what == 2u ? a.dv : a.dk) - 1u));
      touch_step = (uint64_t)kChunk * 2u * token;
      touches = mine_of < kChunk * 6u;
    }
    touch += 2u * touch_step;
  }
  uint32_t touched = 0;
  token_offsets(pl.chunks == 1u ? pl.last : (uint32_t)kChunk);
  load_tokens();
  load_queries();
  load_inner();
  put_tokens(0);
  if (pl.chunks > 1u) advance(1);
  load_tokens();
  for (uint32_t c = 0; c < pl.chunks; ++c) {
    __syncthreads();
    if constexpr (kMode == kChain) {
      asm volatile("" ::"v"(touched));  // (a step later, so that nothing waits for it)
      if (touches && c + 3u < pl.chunks) touched = *reinterpret_cast<const uint16_t *>(touch);  // (whole chunks alone; one value of a row, its last at most)
      touch += touch_step;
    }
    if constexpr (kByQuads) {
      exchange(std::integral_constant<uint32_t, 1>{});
      exchange(std::integral_constant<uint32_t, 2>{});
    }
    __syncthreads();
    if (!output) {  // the tokens alone
      __syncthreads();
      put_tokens(c + 1u);
      if (c + 2u < pl.chunks) advance(c + 2u);
      load_tokens();
      continue;
    }
    // Q S0 for tokens 16w.., beside the chain's longest phase
    const v4f scale = *reinterpret_cast<const v4f *>(&lds.tokens[c & 1u].factor[2][16u * w + lq * 4u]);
    v4f o = zero, o1 = zero;
#pragma unroll
    for (int i = 2; i >= 0; --i) {
#pragma unroll
      for (uint32_t k = 0; k < kSteps; ++k) {
        const v8bf sb = *reinterpret_cast<const v8bf *>(kByQuads ? &lds.s[i][lq][(k * 16u + lr) * 16u] : &lds.s[i][k][lane16]);
        if (i > 0)
          o = mfma32(as_bf(op_q[k]), sb, o);
        else
          o1 = mfma32(as_bf(op_q[k]), sb, o1);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    put_tokens(c + 1u);
    load_queries();
    o = (o + o1) * scale;
    // and the chunk's own part; columns past 16w + 15 of the triangle are zero
#pragma unroll
    for (uint32_t ks = 0; ks < 2; ++ks) {
      if (ks == 1u && w < 2u) continue;
      v8bf ub[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) ub[i] = *reinterpret_cast<const v8bf *>(&lds.u[i][ks][lane16]);
      o1 = mfma32(as_bf(op_in[ks][2]), ub[0], ks == 0u ? zero : o1);
      o = mfma32(as_bf(op_in[ks][1]), ub[0], o);
      o1 = mfma32(as_bf(op_in[ks][1]), ub[1], o1);
      o = mfma32(as_bf(op_in[ks][0]), ub[1], o);
      o1 = mfma32(as_bf(op_in[ks][0]), ub[2], o1);
      o = mfma32(as_bf(op_in[ks][0]), ub[0], o);
    }
    __builtin_amdgcn_sched_barrier(0);
    load_inner();
    if (c + 2u < pl.chunks) advance(c + 2u);
    load_tokens();
    o += o1;
    uint32_t lo[1], hi[1];
    split2<1>(o[0], o[1], lo);
    split2<1>(o[2], o[3], hi);
    const uint32_t n = c + 1u == pl.chunks ? pl.last : (uint32_t)kChunk, row = 16u * w + lq * 4u;
    uint32_t at = out_off;
    asm volatile("" : "+v"(at));  // (an offset to a uniform base: four addresses in the loop are eight registers)
    if (pl.col_in && row < n) *reinterpret_cast<uint16_t *>(out + at) = (uint16_t)lo[0];
    if (pl.col_in && row + 1u < n) *reinterpret_cast<uint16_t *>(out + at + out_row) = (uint16_t)(lo[0] >> 16);
    if (pl.col_in && row + 2u < n) *reinterpret_cast<uint16_t *>(out + at + 2u * out_row) = (uint16_t)hi[0];
    if (pl.col_in && row + 3u < n) *reinterpret_cast<uint16_t *>(out + at + 3u * out_row) = (uint16_t)(hi[0] >> 16);
    out += (uint64_t)kChunk * 2u * a.hv * a.dv;
  }
}

// The state before segment p > 0 of a sequence: N of the first, then M S + N of
// each in turn, in binary32.  A wave takes 16 rows; the sum over k runs in the
// order of block_product.  Bound by M, 64 KB that one CU fetches at 33 KB a us:
// 1.8 us a step.  (As three bf16 parts, 96 KB, 2.9 us; in a launch of its own,
// which reads each M once, and twice as far ahead, 5% slower at the best cut.)
template <int kTiles>
__device__ __forceinline__ void join_segments(const DeltaArgs &a, ScanLds<kTiles> &lds, uint32_t place0, uint32_t p,
                                              uint32_t head, uint32_t col0, uint32_t w, uint32_t lane) {
  constexpr uint32_t kDk = 64 * kTiles, kRow = kJoinedRow<kTiles>;
  const uint32_t lr = lane & 15u, lq = lane >> 4, n_stride = (a.dv + 15u) / 16u * 16u;
  const bool works = 16u * w < kDk;
  const uint32_t m_off = (16u * w + lr) * kDk + lq * 4u, n_off = kDk * kDk + (16u * w + lq * 4u) * n_stride + col0 + lr;
  float4 m[kDk / 16];
  v4f n;
  auto load = [&](uint32_t q) {
    const float *from = segment_parts<kTiles>(a, place0 + q, head);
    if (q > 0u) {
#pragma unroll
      for (uint32_t i = 0; i < kDk / 16; ++i) m[i] = *reinterpret_cast<const float4 *>(from + m_off + 16u * i);
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) n[i] = from[n_off + i * n_stride];
  };
  if (works) load(0);
  for (uint32_t q = 0; q < p; ++q) {
    // two places in turn; the last state lies where carry_state looks for it
    const float *before = lds.joined(((p - q) & 1u) != 0u);
    float *after = lds.joined(((p - q) & 1u) == 0u);
    if (works) {
      v4f x = n, y = {0, 0, 0, 0};
      if (q > 0u) {
#pragma unroll
        for (uint32_t i = 0; i < kDk / 16; ++i) {
          const float4 f = *reinterpret_cast<const float4 *>(before + lr * kRow + 16u * i + lq * 4u);
          x = __builtin_amdgcn_mfma_f32_16x16x4f32(m[i].x, f.x, x, 0, 0, 0);
          y = __builtin_amdgcn_mfma_f32_16x16x4f32(m[i].y, f.y, y, 0, 0, 0);
          x = __builtin_amdgcn_mfma_f32_16x16x4f32(m[i].z, f.z, x, 0, 0, 0);
          y = __builtin_amdgcn_mfma_f32_16x16x4f32(m[i].w, f.w, y, 0, 0, 0);
        }
      }
      if (q + 1u < p) load(q + 1u);
      *reinterpret_cast<v4f *>(after + lr * kRow + 16u * w + lq * 4u) = x + y;
    }
    __syncthreads();
  }
}

// The sequence (of at most 64) that stands at this place when they are ordered
// by length, the longest first, equal ones as they come.
__device__ __forceinline__ uint32_t by_length(const DeltaArgs &a, uint32_t place, uint32_t lane) {
  int length = -1;
  if (lane < a.count) {
    const DeltaSeq sq = delta_sequence(a, lane);
    length = (int)(sq.end - sq.begin);
  }
  uint32_t longer = 0;
  for (uint32_t s = 0; s < a.count; ++s) {
    const int other = __builtin_amdgcn_readlane(length, s);
    longer += other > length || (other == length && s < lane) ? 1u : 0u;
  }
  return (uint32_t)__builtin_ctzll(__ballot(lane < a.count && longer == place));
}

template <int kTiles, bool kWhole, int kMode>
__global__ __launch_bounds__(kScanThreads, kWhole ? 4 : 2) void delta_scan_kernel(const DeltaArgs a) {
  __shared__ __attribute__((aligned(16))) ScanLds<kTiles> lds;
  constexpr uint32_t kDk = 64 * kTiles;
  const uint32_t lane = threadIdx.x & 63u, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go round the eight XCDs: the column blocks of a head all to one,
  // so that its L2 serves the chunk's operands to all of them.
  const uint32_t v_blocks = (a.dv + 15u) / 16u, blocks = v_blocks + (kMode == kParts ? kDk / 16u : 0u);
  const uint32_t j = blockIdx.x >> 3, pair = (j / blocks) * 8u + (blockIdx.x & 7u), block = j % blocks;
  const uint32_t place = pair / a.hv;  // the sequence, or the segment's place
  ScanPlace pl;
  uint32_t seq = place, p = 0;
  if constexpr (kMode == kChain) {
    if (place >= a.count) return;
    // Where the workgroups do not all start at once, the longest chains go first (8 prompts of 2 to 927 tokens, 16
    // heads: 59 us, and 62 to 65 in their own order).
    if (a.count > 1u && a.count <= 64u && a.count * a.hv * v_blocks > kCus) seq = by_length(a, place, lane);
  } else {
    const uint32_t in = a.segment * kChunk;
    if (place >= segment_places(a.tokens, a.count, a.segment)) return;
    const int before = sequences_up_to<kScanThreads>(a, place, in);
    if (before == 0) return;
    seq = (uint32_t)before - 1u;
  }
  pl.sq = delta_sequence(a, seq);
  pl.head = pair - place * a.hv;
  pl.khead = pl.head / (a.hv / a.hk);
  pl.col = block * 16u + (lane & 15u);
  pl.col_in = pl.col < a.dv;
  pl.keep = pl.output = true;
  pl.unit = false;
  pl.parts = nullptr;
  const uint32_t tokens = pl.sq.end - pl.sq.begin;
  pl.chunks = (tokens + kChunk - 1u) / kChunk;
  pl.last = tokens - (pl.chunks - 1u) * kChunk;
  pl.place0 = first_place(pl.sq.begin, seq);
  if constexpr (kMode != kChain) {
    const uint32_t first = pl.sq.begin / (a.segment * kChunk) + seq;
    p = place - first;
    const uint32_t c0 = p * a.segment, all = pl.chunks;
    if (p > 0u && c0 >= all) return;  // a place of no segment
    const bool is_last = c0 + a.segment >= all;
    if (kMode == kParts && (block < v_blocks ? p > 0u && is_last : p == 0u || is_last)) return;
    if (kMode == kRest && p == 0u) return;
    if (!is_last) {
      pl.chunks = a.segment;
      pl.last = kChunk;
      pl.keep = false;
    } else {
      pl.chunks = all - c0;
    }
    if (kMode == kParts) {
      if (p > 0u) {
        pl.sq.fresh = true;  // from zeros
        pl.output = false;
        pl.unit = block >= v_blocks;
      }
      if (!is_last) {
        if (pl.unit) pl.col -= v_blocks * 16u;
        pl.parts = segment_parts<kTiles>(a, place, pl.head) + (pl.unit ? 0u : kDk * kDk);
      }
    } else {
      join_segments<kTiles>(a, lds, first, p, pl.head, block * 16u, w, lane);
    }
    pl.place0 += c0;
    pl.sq.begin += c0 * kChunk;
  }
  if (tokens == 0u) {  // an empty sequence keeps its state, or loses it
    if (pl.sq.fresh && pl.sq.slot >= 0 && pl.col_in)
      for (uint32_t r = threadIdx.x >> 4; r < a.dk; r += kScanThreads / 16)
        a.state[(((uint64_t)pl.sq.slot * a.hv + pl.head) * a.dk + r) * a.dv + pl.col] = 0.0f;
    return;
  }
  // both take part in every barrier: three per chunk
  if (w < 4u)
    carry_state<kTiles, kWhole, kMode>(a, pl, lds, w, lane);
  else
    make_output<kTiles, kWhole, kMode>(a, pl, lds, w - 4u, lane);
}

// How many times longer than one workgroup a CU so many workgroups take (two on a
// CU hide little of each other's waits).
double rounds(double groups) { return groups > kCus ? groups / kCus : 1.0; }

// The leading five bits of a number of chunks.  The rule below goes by them, so
// that it can be asked for every smaller number in a few steps.
uint32_t low_bits(uint32_t chunks) {
  uint32_t n = 0;
  while (chunks >> n >= 32u) ++n;
  return n;
}
uint32_t leading_bits(uint32_t chunks) { return chunks >> low_bits(chunks) << low_bits(chunks); }

// Whether the chains alone give every CU work; such sequences are never cut.
bool fills_the_chip(uint64_t count, uint32_t hv, uint32_t dv) { return 0.8 * count * hv * ((dv + 15u) / 16u) >= kCus; }

// Chunks of a segment; 0: the sequences are not cut.  From the sizes alone, as
// the lengths lie on the device: as if all sequences were equally long.  Whole
// segments are counted, as whole ones are run.  The constants are fitted to 136
// sizes, among them (us, not cut / cut in 8 / 16 / 32 / 64 chunks): 9000
// tokens of 1 head 211 / 79 / 84 / 128 / 230; of 4 heads 221 / 149 / 101 / 140 /
// 240; 16000 of 8 heads 390 / 497 / 308 / 257 / 278; of 12 heads 395 / 758 / 471 /
// 402 / 407; of 16 heads 413 / 986 / 610 / 512 / 476.  Over them the choice takes 1% longer than the best one does, and at the
// worst 3% longer than no cut (16000 tokens of 12 heads).
uint32_t segment_chunks(uint32_t all, uint32_t count, uint32_t hv, uint32_t dk, uint32_t dv) {
  if (count == 0u || fills_the_chip(count, hv, dv)) return 0u;
  const double chunks = (double)leading_bits(all) / count, heads = (double)count * hv;
  const double v = (dv + 15u) / 16u, m = dk <= 64u ? 4.0 : 8.0;
  constexpr double kPerChunk = 1.25;  // us
  double best = 0.85 * chunks * kPerChunk * rounds(0.93 * heads * v);
  uint32_t cut = 0;
  for (uint32_t n = 2; n <= 64; n *= 2) {
    if (chunks < 2.0 * n) break;
    const double parts = ceil(chunks / n);
    const double first = heads * (v + (parts - 2.0) * (v + m));  // workgroups: of the first segment, and N's and M's
    const double rest = heads * v * (parts - 1.0);               // of the next launch, which all read M's
    const double join = 1.95 * (m / 8.0) * (m / 8.0) * rounds(0.75 * rest);
    const double t = n * kPerChunk * (rounds(0.8 * first) + rounds(0.8 * rest)) + join * (parts - 2.0) + 10.5;
    if (t < best) {
      best = t;
      cut = n;
    }
  }
  return cut;
}

// M and N of all segments of so many chunks in all.
uint64_t parts_bytes(uint32_t all, uint32_t count, uint32_t hv, uint32_t dk, uint32_t dv) {
  const uint64_t rows = dk <= 64u ? 64u : 128u;
  const uint32_t segment = segment_chunks(all, count, hv, dk, dv);
  return segment ? (uint64_t)(all / segment + count) * hv * rows * (rows + (dv + 15u) / 16u * 16u) * 4u : 0u;
}

template <int kTiles, int kMode>
hipError_t launch_scan(const DeltaArgs &a, uint64_t places, hipStream_t s) {
  const uint32_t blocks = (a.dv + 15u) / 16u + (kMode == kParts ? 4u * kTiles : 0u);
  const dim3 grid((uint32_t)((places * a.hv + 7u) / 8u * 8u * blocks));
  if (a.dk == 64u * kTiles && a.dv % 16u == 0u)
    hipLaunchKernelGGL((delta_scan_kernel<kTiles, true, kMode>), grid, dim3(kScanThreads), 0, s, a);
  else
    hipLaunchKernelGGL((delta_scan_kernel<kTiles, false, kMode>), grid, dim3(kScanThreads), 0, s, a);
  return hipGetLastError();
}

template <int kTiles>
hipError_t launch_chunked(DeltaArgs a, hipStream_t s) {
  const uint64_t places = a.tokens / kChunk + (uint64_t)a.count;
  if (a.tokens > 0) {
    const auto launch = [&](auto heads) {
      constexpr int kHeads = decltype(heads)::value;
      const dim3 grid((uint32_t)(places * (a.hv / kHeads)));
      if (a.dk == 64u * kTiles)
        hipLaunchKernelGGL((delta_chunk_kernel<64 * kTiles, kHeads, true>), grid, dim3(kThreads), 0, s, a);
      else
        hipLaunchKernelGGL((delta_chunk_kernel<64 * kTiles, kHeads, false>), grid, dim3(kThreads), 0, s, a);
    };
    if (a.hv / a.hk % 2u == 0u)
      launch(std::integral_constant<int, 2>{});
    else
      launch(std::integral_constant<int, 1>{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  a.segment = segment_chunks(a.tokens / kChunk, a.count, a.hv, a.dk, a.dv);
  if (a.segment == 0u) return launch_scan<kTiles, kChain>(a, a.count, s);
  a.parts = reinterpret_cast<float *>(a.workspace + places * a.hv * kHeadBytes);
  const uint32_t segments = segment_places(a.tokens, a.count, a.segment);
  const hipError_t e = launch_scan<kTiles, kParts>(a, segments, s);
  return e != hipSuccess ? e : launch_scan<kTiles, kRest>(a, segments, s);
}

}  // namespace

uint64_t delta_workspace_needed(uint32_t tokens, uint32_t count, uint32_t hv, uint32_t dk, uint32_t dv) {
  return (tokens / kChunk + (uint64_t)count) * hv * kHeadBytes + parts_bytes(tokens / kChunk, count, hv, dk, dv);
}

// What every call of at most so many tokens and sequences needs at most.  Fewer
// tokens or sequences can be cut where these are not, or shorter: the largest
// of what any of them has of segments.
uint64_t delta_workspace_bytes(uint32_t tokens, uint32_t count, uint32_t hv, uint32_t dk, uint32_t dv) {
  const uint32_t all = tokens / kChunk;
  uint64_t parts = 0;
  for (uint32_t c = 1; c <= count && !fills_the_chip(c, hv, dv); ++c)
    for (uint64_t x = 0; x <= all;) {  // a run of numbers that the rule does not tell apart, by its last
      const uint64_t next = leading_bits((uint32_t)x) + (1ull << low_bits((uint32_t)x));
      const uint64_t bytes = parts_bytes((uint32_t)(next - 1u < all ? next - 1u : all), c, hv, dk, dv);
      parts = bytes > parts ? bytes : parts;
      x = next;
    }
  return (all + (uint64_t)count) * hv * kHeadBytes + parts;
}

hipError_t launch_delta_chunked(const DeltaArgs &a, hipStream_t s) {
  return a.dk <= 64u ? launch_chunked<1>(a, s) : launch_chunked<2>(a, s);
}

}  // namespace bqmm
