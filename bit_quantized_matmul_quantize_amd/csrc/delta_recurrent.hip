// The gated delta rule, token by token.
//
// Per value head, with the state S [dk][dv] in binary32 and for each token
// a = exp(g), b = beta (and with l2norm q, k divided by sqrt(|.|^2 + 1e-6)):
//   u = b (v - a k^T S),   S' = a S + k u,   o = scale q^T S'.
// With k^T S, q^T S and q.k from one look at S, o = scale (a q^T S + (q.k) u):
// S is read once and updated once per token.  The norms of q and k are common
// factors of those sums, so q and k stay as they were read (exact bf16).
//
// The columns of S are independent of each other, so a wave takes one head's
// 4 kQuads columns and all dk rows: a lane holds four columns (16-byte loads)
// of kRows consecutive rows, and the sums over rows end in a butterfly over
// the 64 / kQuads lanes that share the columns.  The state stays in registers
// over a sequence's tokens.
//
// Bound by memory where the batch is large: 8 dk dv bytes of state move for
// 6 dk dv operations per token.  96 sequences of 32 heads of 128 x 128 (405 MB):
// 72 us, 5.6 TB/s (part of it in the 256 MB cache); 83 us without the non-temporal
// hints (a state is not used again before the next token) and without a run of
// heads per XCD.  One sequence (4.2 MB) 4.7 us: a launch and three dependent trips
// to memory (the ranges; the state, q and k; g, beta and v, which the compiler
// issues after the sums where dk is 128), and one more or two per further token,
// whose loads wait for the stores of the one before.  16 columns per wave 5.0, 8 columns 7.6, 64 columns 5.5.
#include "delta_common.h"

namespace bqmm {
namespace {

constexpr float kNormEps = 1e-6f;
constexpr uint32_t kQuads = 8;  // quads of columns that a wave takes (add_eighths sums over the lanes that share them)

typedef float Float4 __attribute__((ext_vector_type(4), aligned(4)));
template <int N>
struct __attribute__((packed, aligned(2))) Bf16s {
  uint16_t v[N];
};

// N bf16 values from row r0 of dk; rows past dk are zero.
template <int N, bool kWhole>
__device__ __forceinline__ void load_rows(const uint16_t *p, uint32_t r0, uint32_t dk, float (&v)[N]) {
  if (kWhole || r0 + N <= dk) {
    const Bf16s<N> a = *reinterpret_cast<const Bf16s<N> *>(p + r0);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = bf16_to_f32(a.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = r0 + i < dk ? bf16_to_f32(p[r0 + i]) : 0.0f;
  }
}

// Four columns of a row of the state, those past dv zero.  kWhole: all four
// are inside, or none (its lanes then work on the first columns, and store nothing).
template <bool kWhole>
__device__ __forceinline__ float4 load_columns(const float *p, uint32_t cols) {
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (kWhole || cols == 4u) {
    const Float4 f = __builtin_nontemporal_load(reinterpret_cast<const Float4 *>(p));
    return make_float4(f[0], f[1], f[2], f[3]);
  }
  if (cols > 0u) s.x = p[0];
  if (cols > 1u) s.y = p[1];
  if (cols > 2u) s.z = p[2];
  return s;
}

// x added over the lanes that differ in bits 3 to 5 alone: the other eight of a
// row of 16 without a trip through LDS, then the rest.  (8 tokens of one
// sequence, heads of 64: 12.1 us, and 13.0 with three trips; with none, by lane
// swaps, 12.3, but 96 sequences 22.3 instead of 19.9: more instructions.)
__device__ __forceinline__ float add_eighths(float x) {
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xF, 0xF, true));
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

template <int kDk, bool kWhole>
__global__ __launch_bounds__(64) void delta_recurrent_kernel(const DeltaArgs a) {
  constexpr int kGroups = 64 / kQuads;
  constexpr int kRows = kDk / kGroups;
  const uint32_t quad = threadIdx.x % kQuads, r0 = threadIdx.x / kQuads * kRows;
  const uint32_t blocks = (a.dv + 4u * kQuads - 1u) / (4u * kQuads);
  // each XCD takes a run of heads, so that a head's columns share the lines of q, k and v
  const uint32_t unit = (blockIdx.x & 7u) * (gridDim.x >> 3) + (blockIdx.x >> 3), head_seq = unit / blocks;
  if (head_seq >= a.count * a.hv) return;
  const uint32_t hv = head_seq % a.hv, seq = head_seq / a.hv;
  const uint32_t hk = hv / (a.hv / a.hk);
  const uint32_t c0 = (unit - head_seq * blocks) * (4u * kQuads) + quad * 4u;
  const uint32_t cols = c0 < a.dv ? min(a.dv - c0, 4u) : 0u;

  const DeltaSeq sq = delta_sequence(a, seq);
  if (sq.begin >= sq.end && !sq.fresh) return;  // nothing changes

  float4 s[kRows];
  const uint32_t c = kWhole && cols == 0u ? 0u : c0;
  float *state = a.state + ((uint64_t)max(sq.slot, 0) * a.hv + hv) * a.dk * a.dv + c;
  if (sq.slot >= 0 && !sq.fresh) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (kWhole)  // no branch around the loads: they leave together
        s[i] = load_columns<true>(state + (uint64_t)(r0 + i) * a.dv, 4u);
      else
        s[i] = load_columns<false>(state + (uint64_t)(r0 + i) * a.dv, r0 + i < a.dk ? cols : 0u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }

  for (uint32_t t = sq.begin; t < sq.end; ++t) {
    float q[kRows], k[kRows], v[4];
    load_rows<kRows, kWhole>(a.q + (uint64_t)t * a.q_token + (uint64_t)hk * a.q_head, r0, a.dk, q);
    load_rows<kRows, kWhole>(a.k + (uint64_t)t * a.k_token + (uint64_t)hk * a.k_head, r0, a.dk, k);
    load_rows<4, kWhole>(a.v + (uint64_t)t * a.v_token + (uint64_t)hv * a.v_head, c, a.dv, v);
    const float decay = expf(a.g[(uint64_t)t * a.hv + hv]), beta = a.beta[(uint64_t)t * a.hv + hv];

    // k^T S, q^T S (four columns each), |k|^2, |q|^2, q.k
    float sum[11];
#pragma unroll
    for (int j = 0; j < 11; ++j) sum[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      sum[0] = fmaf(k[i], s[i].x, sum[0]);
      sum[1] = fmaf(k[i], s[i].y, sum[1]);
      sum[2] = fmaf(k[i], s[i].z, sum[2]);
      sum[3] = fmaf(k[i], s[i].w, sum[3]);
      sum[4] = fmaf(q[i], s[i].x, sum[4]);
      sum[5] = fmaf(q[i], s[i].y, sum[5]);
      sum[6] = fmaf(q[i], s[i].z, sum[6]);
      sum[7] = fmaf(q[i], s[i].w, sum[7]);
      sum[8] = fmaf(k[i], k[i], sum[8]);
      sum[9] = fmaf(q[i], q[i], sum[9]);
      sum[10] = fmaf(q[i], k[i], sum[10]);
    }
#pragma unroll
    for (int j = 0; j < 11; ++j) sum[j] = add_eighths(sum[j]);
    const float rk = a.l2norm ? 1.0f / sqrtf(sum[8] + kNormEps) : 1.0f;
    const float rq = (a.l2norm ? 1.0f / sqrtf(sum[9] + kNormEps) : 1.0f) * a.scale;

    float u[4], o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = rk * (beta * (v[j] - decay * (rk * sum[j])));  // with k's factor for the update
      o[j] = rq * fmaf(sum[10], u[j], decay * sum[4 + j]);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      s[i].x = fmaf(k[i], u[0], decay * s[i].x);
      s[i].y = fmaf(k[i], u[1], decay * s[i].y);
      s[i].z = fmaf(k[i], u[2], decay * s[i].z);
      s[i].w = fmaf(k[i], u[3], decay * s[i].w);
    }
    if (threadIdx.x < kQuads) {
      uint16_t *op = a.out + ((uint64_t)t * a.hv + hv) * a.dv + c0;
      if (cols == 4u) {
        *reinterpret_cast<Bf16s<4> *>(op) =
            __builtin_bit_cast(Bf16s<4>, make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])));
      } else {
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
          if (j < cols) op[j] = (uint16_t)f32_to_bf16_rne(o[j]);
      }
    }
  }

  if (sq.slot < 0 || cols == 0u) return;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (!kWhole && r0 + i >= a.dk) continue;
    float *p = state + (uint64_t)(r0 + i) * a.dv;
    if (kWhole || cols == 4u) {
      __builtin_nontemporal_store(Float4{s[i].x, s[i].y, s[i].z, s[i].w}, reinterpret_cast<Float4 *>(p));
    } else {
      p[0] = s[i].x;
      if (cols > 1u) p[1] = s[i].y;
      if (cols > 2u) p[2] = s[i].z;
    }
  }
}

template <int kDk>
hipError_t launch_recurrent(const DeltaArgs &a, hipStream_t s) {
  const uint64_t blocks = ((uint64_t)a.count * a.hv * ((a.dv + 4ull * kQuads - 1u) / (4ull * kQuads)) + 7u) / 8u * 8u;
  if (a.dk == (uint32_t)kDk && a.dv % 4u == 0u)
    hipLaunchKernelGGL((delta_recurrent_kernel<kDk, true>), dim3((uint32_t)blocks), dim3(64), 0, s, a);
  else
    hipLaunchKernelGGL((delta_recurrent_kernel<kDk, false>), dim3((uint32_t)blocks), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_recurrent(const DeltaArgs &a, hipStream_t s) {
  return a.dk <= 64u ? launch_recurrent<64>(a, s) : launch_recurrent<128>(a, s);
}

}  // namespace bqmm
