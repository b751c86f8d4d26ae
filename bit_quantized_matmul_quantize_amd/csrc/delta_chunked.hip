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
// q.k triangle, a few factors per token, and the keys transposed.  The second
// walks each head's chunks in order, a workgroup for 16 columns of the state
// (columns do not depend on each other).
//
// Numbers.  The matrix cores multiply bf16 and add in binary32.  q and k are
// bf16 as they are: their norms, decays and beta are factors per token that
// are applied in binary32 outside the products.  A binary32 operand (T, R, U,
// S) enters as the sum of three bf16 (8 + 8 + 8 bits, nothing lost) wherever
// the state depends on it; T R keeps the six products above 2^-24.  The output
// is rounded to bf16, so its products take the two leading parts (2^-16).
// T is computed in binary32 throughout, the sums G in binary64: differences of
// G stay exact next to a strong decay.
#include "delta_common.h"

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
constexpr float kNormEps = 1e-6f;
constexpr float kNoDecay = -1e6f;  // exp of it is zero; sums of 64 of them stay exact to 2^-26

// Workspace.  A fragment is what a wave's 64 lanes load as one matrix
// operand, 16 bytes each, 1 KB.  Rows 16w..16w+15 of a lower triangle need
// only the 32 columns up to w = 1 and all 64 from w = 2: six fragments.
constexpr uint32_t kFragment = 1024;
constexpr uint32_t kTriangle = 6;
constexpr uint32_t kTBytes = kTriangle * 3 * kFragment;
constexpr uint32_t kInnerBytes = kTriangle * 2 * kFragment;
constexpr uint32_t kFactorBytes = kChunk * 16 + 256;  // (b, b e^G rk, scale e^G rq, e^(G_L - G) rk) per token, then e^G_L
constexpr uint32_t kHeadBytes = kTBytes + kInnerBytes + kFactorBytes;
__host__ __device__ constexpr uint32_t key_bytes(int kd) { return kd * kChunk * 2; }  // the keys transposed

__device__ __forceinline__ uint32_t triangle_fragment(uint32_t w, uint32_t ks) { return w < 2u ? w : 2u * w - 2u + ks; }

// Chunk places: a sequence that begins at token b as the s-th has its chunks
// from b / 64 + s on.  Places of different sequences never meet, and all lie
// below tokens / 64 + count.
__device__ __forceinline__ uint32_t first_place(uint32_t begin, uint32_t seq) { return begin / kChunk + seq; }

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

// One workgroup for a chunk and value head; the first value head of a key head also transposes the keys.
template <int kDk>
__global__ __launch_bounds__(kThreads) void delta_chunk_kernel(const DeltaArgs a) {
  constexpr int kRow = kDk + 8;  // bf16 per staged row
  constexpr uint32_t kBuffer = kChunk * kStride * 4;
  static_assert(kChunk * kRow * 2 <= kBuffer, "the staged keys and queries fit the buffers that replace them");
  __shared__ __attribute__((aligned(16))) uint8_t lds[3 * kBuffer];
  __shared__ double sum_g[kChunk];
  __shared__ float norm_k[kChunk], norm_q[kChunk], betas[kChunk];
  uint16_t *keys = reinterpret_cast<uint16_t *>(lds), *queries = reinterpret_cast<uint16_t *>(lds + kBuffer);
  float *inverse = reinterpret_cast<float *>(lds);             // in the keys' place
  float *inner = reinterpret_cast<float *>(lds + kBuffer);     // in the queries' place
  float *lower = reinterpret_cast<float *>(lds + 2 * kBuffer);

  const uint32_t tid = threadIdx.x, lane = tid & 63u, w = tid >> 6, lr = lane & 15u, lq = lane >> 4;
  const uint32_t place = blockIdx.x / a.hv, head = blockIdx.x - place * a.hv;
  const uint32_t ratio = a.hv / a.hk, khead = head / ratio;

  // the sequence whose places hold this one: as many as begin at or before it, less one
  int before = 0;
  for (uint32_t s0 = 0; s0 < a.count; s0 += kThreads) {
    const uint32_t s = s0 + tid;
    bool at = false;
    if (s < a.count) at = first_place(min((uint32_t)max(a.starts[s], 0), a.tokens), s) <= place;
    before += __syncthreads_count(at);
  }
  if (before == 0) return;
  const uint32_t seq = (uint32_t)before - 1u;
  const DeltaSeq sq = delta_sequence(a, seq);
  const uint32_t t0 = sq.begin + (place - first_place(sq.begin, seq)) * kChunk;
  if (t0 >= sq.end) return;
  const uint32_t n = min(sq.end - t0, (uint32_t)kChunk);

  // keys and queries into LDS, zeros past the chunk's end and past dk
  {
    const uint32_t vecs = kDk / 8;
    for (uint32_t i = tid; i < kChunk * vecs; i += kThreads) {
      const uint32_t r = i / vecs, c = (i - r * vecs) * 8u;
      uint4 kv = make_uint4(0, 0, 0, 0), qv = kv;
      if (r < n) {
        const uint16_t *kp = a.k + (uint64_t)(t0 + r) * a.k_token + (uint64_t)khead * a.k_head + c;
        const uint16_t *qp = a.q + (uint64_t)(t0 + r) * a.q_token + (uint64_t)khead * a.q_head + c;
        if (c + 8u <= a.dk) {
          const Bf16x8 x = *reinterpret_cast<const Bf16x8 *>(kp), y = *reinterpret_cast<const Bf16x8 *>(qp);
          kv = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
          qv = make_uint4(y.w[0], y.w[1], y.w[2], y.w[3]);
        } else {
          uint32_t x[8], y[8];
#pragma unroll
          for (uint32_t j = 0; j < 8; ++j) {
            x[j] = c + j < a.dk ? kp[j] : 0u;
            y[j] = c + j < a.dk ? qp[j] : 0u;
          }
          kv = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
          qv = make_uint4(y[0] | y[1] << 16, y[2] | y[3] << 16, y[4] | y[5] << 16, y[6] | y[7] << 16);
        }
      }
      *reinterpret_cast<uint4 *>(keys + r * kRow + c) = kv;
      *reinterpret_cast<uint4 *>(queries + r * kRow + c) = qv;
    }
  }
  if (w == 0) {
    const float gt = lane < n ? a.g[(uint64_t)(t0 + lane) * a.hv + head] : 0.0f;
    double g = (double)(gt < kNoDecay ? kNoDecay : gt);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(g, d);
      g += lane >= (uint32_t)d ? o : 0.0;
    }
    sum_g[lane] = g;
    betas[lane] = lane < n ? a.beta[(uint64_t)(t0 + lane) * a.hv + head] : 0.0f;
  }
  __syncthreads();

  uint8_t *mine = a.workspace + ((uint64_t)place * a.hv + head) * kHeadBytes;
  // norms: four lanes per row
  {
    const uint32_t r = tid >> 2, c = (tid & 3u) * (kDk / 4);
    float sk = 0.0f, sq2 = 0.0f;
#pragma unroll
    for (int j = 0; j < kDk / 4; ++j) {
      const float x = bf16_to_f32(keys[r * kRow + c + j]), y = bf16_to_f32(queries[r * kRow + c + j]);
      sk = fmaf(x, x, sk);
      sq2 = fmaf(y, y, sq2);
    }
    sk += __shfl_xor(sk, 1);
    sk += __shfl_xor(sk, 2);
    sq2 += __shfl_xor(sq2, 1);
    sq2 += __shfl_xor(sq2, 2);
    if ((tid & 3u) == 0u) {
      norm_k[r] = a.l2norm ? 1.0f / sqrtf(sk + kNormEps) : 1.0f;
      norm_q[r] = (a.l2norm ? 1.0f / sqrtf(sq2 + kNormEps) : 1.0f) * a.scale;
    }
  }
  // the keys transposed: rows are dk as the state's lie in the second launch, columns tokens
  if (head == khead * ratio) {
    constexpr int kTiles = kDk / 64;
    uint8_t *out = a.workspace + (uint64_t)(a.tokens / kChunk + a.count) * a.hv * kHeadBytes +
                   ((uint64_t)place * a.hk + khead) * key_bytes(kDk) + w * (kTiles * 2 * kFragment) + lane * 16u;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const uint32_t row = kTiles == 2 ? 32u * w + (lr >> 2) * 8u + t * 4u + (lr & 3u) : 16u * w + lr;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = keys[(32 * ks + lq * 8 + j) * kRow + row];
        *reinterpret_cast<uint4 *>(out + (t * 2 + ks) * kFragment) =
            make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
      }
    }
  }
  // k.k and q.k: rows 16w.. by the wave, the tiles of the lower triangle
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
        kk[j] = mfma32(kr, kc, kk[j]);
        qk[j] = mfma32(qr, kc, qk[j]);
      }
    }
  }
  __syncthreads();  // the norms are there; keys and queries have been read

  if (w == 0) {
    const double g = sum_g[lane];
    const float e = expf((float)g);
    float4 f;
    f.x = betas[lane];
    f.y = betas[lane] * e * norm_k[lane];
    f.z = lane < n ? e * norm_q[lane] : 0.0f;
    f.w = lane < n ? expf((float)(sum_g[kChunk - 1] - g)) * norm_k[lane] : 0.0f;
    *reinterpret_cast<float4 *>(mine + kTBytes + kInnerBytes + lane * 16u) = f;
    if (lane == kChunk - 1) *reinterpret_cast<float *>(mine + kTBytes + kInnerBytes + kChunk * 16) = e;
  }
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) {
    if (j > w) continue;
    const uint32_t s = 16u * j + lr;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t t = 16u * w + lq * 4u + i;
      const float decay = s <= t ? expf((float)(sum_g[t] - sum_g[s])) * norm_k[s] : 0.0f;
      lower[t * kStride + s] = s < t ? betas[t] * norm_k[t] * decay * kk[j][i] : 0.0f;
      inner[t * kStride + s] = s <= t ? norm_q[t] * decay * qk[j][i] : 0.0f;
    }
  }
  __syncthreads();

  // T: the 16 x 16 blocks on the diagonal by substitution (a lane a column),
  // then blocks of 16 and of 32 joined in pairs,
  //   [[a, 0], [c, b]]^-1 = [[a', 0], [-b' c a', b']].
  if (w == 0) {
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float *row = lower + (16 * lq + i) * kStride + 16 * lq;
      float x = (uint32_t)i == lr ? 1.0f : 0.0f, y = 0.0f;
#pragma unroll
      for (int m = 0; m < i; ++m) {
        if (m & 1)
          y = fmaf(-row[m], t[m], y);
        else
          x = fmaf(-row[m], t[m], x);
      }
      t[i] = x + y;
      inverse[(16 * lq + i) * kStride + 16 * lq + lr] = t[i];
    }
  } else {
    // meanwhile the other waves put the q.k triangle away, two fragments each
    for (uint32_t f = 2u * w - 2u; f < 2u * w; ++f)
      put_triangle<2>(inner, mine + kTBytes, f < 2u ? f : f / 2u + 1u, f < 2u ? 0u : f & 1u, lane);
  }
  __syncthreads();
  if (w < 2) {
    const uint32_t o = 32u * w;
    const v4f x = block_product(lower + (o + 16) * kStride + o, inverse + o * kStride + o, v4f{0, 0, 0, 0}, lr, lq);
    const v4f y = block_product(inverse + (o + 16) * kStride + o + 16, x, v4f{0, 0, 0, 0}, lr, lq);
#pragma unroll
    for (int i = 0; i < 4; ++i) inverse[(o + 16 + lq * 4 + i) * kStride + o + lr] = -y[i];
  }
  __syncthreads();
  {
    const uint32_t jt = w & 1u, rt = w >> 1;
    v4f x[2], y = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r) {
      x[r] = v4f{0, 0, 0, 0};
      for (uint32_t kt = jt; kt < 2; ++kt)
        x[r] = block_product(lower + (32 + 16 * r) * kStride + 16 * kt, inverse + 16 * kt * kStride + 16 * jt, x[r], lr, lq);
    }
    y = block_product(inverse + (32 + 16 * rt) * kStride + 32, x[0], y, lr, lq);
    if (rt == 1u) y = block_product(inverse + 48 * kStride + 48, x[1], y, lr, lq);
#pragma unroll
    for (int i = 0; i < 4; ++i) inverse[(32 + 16 * rt + lq * 4 + i) * kStride + 16 * jt + lr] = -y[i];
  }
  __syncthreads();
  for (uint32_t f = w; f < kTriangle; f += 4)
    put_triangle<3>(inverse, mine, f < 2u ? f : f / 2u + 1u, f < 2u ? 0u : f & 1u, lane);
}

// ---- second launch: the state along the chunks ------------------------------------

// What a wave w needs of a chunk.  The state's rows are split over the waves
// (rows 32w.. for dk 128, 16w.. for 64): each multiplies its rows by the
// chunk's keys and queries, and the four partial sums meet in LDS.
template <int kTiles>
struct Operands {
  uint4 k[4], q[4];          // 64 tokens x the wave's rows (for one tile 8 bytes of each)
  uint4 t[2][3], inner[2][2];  // rows 16w.. of T and of the q.k triangle
  uint4 kt[kTiles][2];       // the wave's rows x 64 tokens
  float4 f[4];               // factors of tokens 16w + 4 (lane / 16) + i
  float decay;
  uint32_t v[4];
};

template <int kTiles, bool kWhole>
__global__ __launch_bounds__(kThreads) void delta_scan_kernel(const DeltaArgs a) {
  constexpr int kDk = 64 * kTiles;
  constexpr int kRows = 16 * kTiles;  // rows of the state per wave
  // partial sums [token tile][wave][lane], R and U as operands [part][32 tokens][lane]
  __shared__ __attribute__((aligned(16))) float4 part_k[16][64], part_q[16][64];
  __shared__ __attribute__((aligned(16))) uint8_t lds_r[3][2][1024], lds_u[2][2][1024], lds_s[3][2][1024];

  const uint32_t tid = threadIdx.x, lane = tid & 63u, lr = lane & 15u, lq = lane >> 4;
  const uint32_t w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroups go round the eight XCDs: the column blocks of a head all to one,
  // so that its L2 serves the chunk's operands to all of them.
  const uint32_t blocks = (a.dv + 15u) / 16u;
  const uint32_t j = blockIdx.x >> 3, pair = (j / blocks) * 8u + (blockIdx.x & 7u);
  if (pair >= a.count * a.hv) return;
  const uint32_t seq = pair / a.hv, head = pair - seq * a.hv, khead = head / (a.hv / a.hk);
  const uint32_t col = (j % blocks) * 16u + lr;
  const bool col_in = col < a.dv;
  const DeltaSeq sq = delta_sequence(a, seq);
  if (sq.begin >= sq.end && !sq.fresh) return;  // nothing changes

  // row of result register i of tile t, among the state's dk
  auto state_row = [&](int t, int i) -> uint32_t {
    return kTiles == 2 ? 32u * w + lq * 8u + t * 4u + i : 16u * w + lq * 4u + i;
  };
  float *state = a.state + ((uint64_t)max(sq.slot, 0) * a.hv + head) * a.dk * a.dv + col;
  v4f s[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = state_row(t, i);
      s[t][i] = sq.slot >= 0 && !sq.fresh && col_in && r < a.dk ? state[(uint64_t)r * a.dv] : 0.0f;
    }

  const uint32_t place0 = first_place(sq.begin, seq);
  const uint32_t chunks = (sq.end - sq.begin + kChunk - 1u) / kChunk;
  const uint8_t *key_base = a.workspace + (uint64_t)(a.tokens / kChunk + a.count) * a.hv * kHeadBytes;

  // Rows past the chunk's end read its last token: their factors are zero.
  auto load = [&](uint32_t c, Operands<kTiles> &o) {
    const uint32_t t0 = sq.begin + c * kChunk, n = min(sq.end - t0, (uint32_t)kChunk);
    const uint8_t *mine = a.workspace + ((uint64_t)(place0 + c) * a.hv + head) * kHeadBytes;
    const uint8_t *kt = key_base + ((uint64_t)(place0 + c) * a.hk + khead) * key_bytes(kDk) + w * (kTiles * 2 * kFragment);
    const uint32_t dk0 = kRows * w + lq * (kTiles * 4);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint64_t t = t0 + min(16u * m + lr, n - 1u);
      const uint16_t *kp = a.k + t * a.k_token + (uint64_t)khead * a.k_head + dk0;
      const uint16_t *qp = a.q + t * a.q_token + (uint64_t)khead * a.q_head + dk0;
      if constexpr (!kWhole) {
        uint32_t x[8], y[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
          const bool in = i < kTiles * 4u && dk0 + i < a.dk;
          x[i] = in ? kp[i] : 0u;
          y[i] = in ? qp[i] : 0u;
        }
        o.k[m] = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
        o.q[m] = make_uint4(y[0] | y[1] << 16, y[2] | y[3] << 16, y[4] | y[5] << 16, y[6] | y[7] << 16);
      } else if constexpr (kTiles == 2) {
        const Bf16x8 x = *reinterpret_cast<const Bf16x8 *>(kp), y = *reinterpret_cast<const Bf16x8 *>(qp);
        o.k[m] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        o.q[m] = make_uint4(y.w[0], y.w[1], y.w[2], y.w[3]);
      } else {
        const Bf16x4 x = *reinterpret_cast<const Bf16x4 *>(kp), y = *reinterpret_cast<const Bf16x4 *>(qp);
        o.k[m] = make_uint4(x.w[0], x.w[1], 0u, 0u);
        o.q[m] = make_uint4(y.w[0], y.w[1], 0u, 0u);
      }
    }
#pragma unroll
    for (uint32_t ks = 0; ks < 2; ++ks) {
      const uint32_t f = triangle_fragment(w, ks);  // the upper waves' second half is not used
#pragma unroll
      for (int i = 0; i < 3; ++i) o.t[ks][i] = *reinterpret_cast<const uint4 *>(mine + (f * 3 + i) * kFragment + lane * 16u);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        o.inner[ks][i] = *reinterpret_cast<const uint4 *>(mine + kTBytes + (f * 2 + i) * kFragment + lane * 16u);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) o.kt[t][ks] = *reinterpret_cast<const uint4 *>(kt + (t * 2 + ks) * kFragment + lane * 16u);
    }
    const float4 *factors = reinterpret_cast<const float4 *>(mine + kTBytes + kInnerBytes);
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t r = 16u * w + lq * 4u + i;
      o.f[i] = factors[r];
      o.v[i] = a.v[(uint64_t)(t0 + min(r, n - 1u)) * a.v_token + (uint64_t)head * a.v_head + min(col, a.dv - 1u)];
    }
    o.decay = *reinterpret_cast<const float *>(factors + kChunk);
  };

  // place of this lane's four rows in an operand of 64 tokens
  const uint32_t put = (w >> 1) * 1024u + ((w & 1u) * 2u + (lq >> 1)) * 256u + lr * 16u + (lq & 1u) * 8u;
  auto bf = [](uint4 x) { return __builtin_bit_cast(v8bf, x); };

  auto step = [&](uint32_t c, const Operands<kTiles> &o) {
    // K S0 and Q S0 over the wave's rows of the state
    uint32_t sp[kTiles][2][3];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      split2<3>(s[t][0], s[t][1], sp[t][0]);
      split2<3>(s[t][2], s[t][3], sp[t][1]);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      v4f x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
      for (int i = 2; i >= 0; --i) {
        if constexpr (kTiles == 2) {
          const v8bf b = bf(make_uint4(sp[0][0][i], sp[0][1][i], sp[1][0][i], sp[1][1][i]));
          x = mfma32(bf(o.k[m]), b, x);
          if (i < 2) y = mfma32(bf(o.q[m]), b, y);
        } else {
          const v4s b = __builtin_bit_cast(v4s, make_uint2(sp[0][0][i], sp[0][1][i]));
          x = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(v4s, make_uint2(o.k[m].x, o.k[m].y)), b, x, 0, 0, 0);
          if (i < 2)
            y = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(v4s, make_uint2(o.q[m].x, o.q[m].y)), b, y, 0, 0, 0);
        }
      }
      part_k[m * 4 + w][lane] = make_float4(x[0], x[1], x[2], x[3]);
      part_q[m * 4 + w][lane] = make_float4(y[0], y[1], y[2], y[3]);
    }
    __syncthreads();
    // R for tokens 16w..
    float r[4], qs[4];
    {
      float4 x = part_k[w * 4][lane], y = part_q[w * 4][lane];
#pragma unroll
      for (int p = 1; p < 4; ++p) {
        const float4 u = part_k[w * 4 + p][lane], v = part_q[w * 4 + p][lane];
        x.x += u.x; x.y += u.y; x.z += u.z; x.w += u.w;
        y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
      }
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = o.f[i].x * bf16_to_f32(o.v[i]) - o.f[i].y * xs[i];
        qs[i] = o.f[i].z * ys[i];
      }
    }
    uint32_t lo[3], hi[3];
    split2<3>(r[0], r[1], lo);
    split2<3>(r[2], r[3], hi);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2 *>(&lds_r[i][0][0] + put) = make_uint2(lo[i], hi[i]);
    __syncthreads();
    // U = T R for tokens 16w..; columns past 16w + 15 of T are zero
    v4f u = {0, 0, 0, 0};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (ks == 1 && w < 2u) continue;
      v8bf b[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) b[i] = *reinterpret_cast<const v8bf *>(&lds_r[i][ks][lane * 16u]);
      u = mfma32(bf(o.t[ks][2]), b[0], u);
      u = mfma32(bf(o.t[ks][1]), b[1], u);
      u = mfma32(bf(o.t[ks][0]), b[2], u);
      u = mfma32(bf(o.t[ks][1]), b[0], u);
      u = mfma32(bf(o.t[ks][0]), b[1], u);
      u = mfma32(bf(o.t[ks][0]), b[0], u);
    }
    split2<3>(u[0] * o.f[0].w, u[1] * o.f[1].w, lo);
    split2<3>(u[2] * o.f[2].w, u[3] * o.f[3].w, hi);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2 *>(&lds_s[i][0][0] + put) = make_uint2(lo[i], hi[i]);
    uint32_t ulo[2], uhi[2];
    split2<2>(u[0], u[1], ulo);
    split2<2>(u[2], u[3], uhi);
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<uint2 *>(&lds_u[i][0][0] + put) = make_uint2(ulo[i], uhi[i]);
    __syncthreads();
    // the state
#pragma unroll
    for (int t = 0; t < kTiles; ++t) s[t] *= o.decay;
#pragma unroll
    for (int i = 2; i >= 0; --i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const v8bf b = *reinterpret_cast<const v8bf *>(&lds_s[i][ks][lane * 16u]);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) s[t] = mfma32(bf(o.kt[t][ks]), b, s[t]);
      }
    // the output of tokens 16w..
    v4f y = {qs[0], qs[1], qs[2], qs[3]};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (ks == 1 && w < 2u) continue;
      const v8bf b0 = *reinterpret_cast<const v8bf *>(&lds_u[0][ks][lane * 16u]);
      const v8bf b1 = *reinterpret_cast<const v8bf *>(&lds_u[1][ks][lane * 16u]);
      y = mfma32(bf(o.inner[ks][1]), b0, y);
      y = mfma32(bf(o.inner[ks][0]), b1, y);
      y = mfma32(bf(o.inner[ks][0]), b0, y);
    }
    const uint32_t t0 = sq.begin + c * kChunk, n = min(sq.end - t0, (uint32_t)kChunk);
    uint16_t *out = a.out + ((uint64_t)(t0 + 16u * w + lq * 4u) * a.hv + head) * a.dv + col;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      if (col_in && 16u * w + lq * 4u + i < n) out[(uint64_t)i * a.hv * a.dv] = (uint16_t)f32_to_bf16_rne(y[i]);
  };

  // The next chunk's operands are on their way while one is computed.
  Operands<kTiles> even, odd;
  if (chunks > 0) load(0, even);
  for (uint32_t c = 0; c < chunks; c += 2) {
    if (c + 1 < chunks) load(c + 1, odd);
    step(c, even);
    if (c + 1 < chunks) {
      if (c + 2 < chunks) load(c + 2, even);
      step(c + 1, odd);
    }
  }

  if (sq.slot < 0 || !col_in) return;
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = state_row(t, i);
      if (r < a.dk) state[(uint64_t)r * a.dv] = s[t][i];
    }
}

template <int kTiles>
hipError_t launch_chunked(const DeltaArgs &a, hipStream_t s) {
  const uint64_t places = a.tokens / kChunk + (uint64_t)a.count;
  if (a.tokens > 0) {
    hipLaunchKernelGGL((delta_chunk_kernel<64 * kTiles>), dim3((uint32_t)(places * a.hv)), dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const uint64_t pairs = ((uint64_t)a.count * a.hv + 7u) / 8u * 8u;
  const dim3 grid((uint32_t)(pairs * ((a.dv + 15u) / 16u)));
  if (a.dk == 64u * kTiles)
    hipLaunchKernelGGL((delta_scan_kernel<kTiles, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((delta_scan_kernel<kTiles, false>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

uint64_t delta_workspace_bytes(uint32_t tokens, uint32_t count, uint32_t hk, uint32_t hv, uint32_t dk) {
  const uint64_t places = tokens / kChunk + (uint64_t)count;
  return places * ((uint64_t)hv * kHeadBytes + (uint64_t)hk * key_bytes(dk <= 64u ? 64 : 128));
}

hipError_t launch_delta_chunked(const DeltaArgs &a, hipStream_t s) {
  return a.dk <= 64u ? launch_chunked<1>(a, s) : launch_chunked<2>(a, s);
}

}  // namespace bqmm
