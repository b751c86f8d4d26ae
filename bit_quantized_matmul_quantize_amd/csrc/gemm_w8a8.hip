// Matrix product of 8-bit integers with a scale per token and per channel:
//   out[i][j] = bf16_rne(float(sum_t a[i][t] w[j][t]) * sa[i] * sw[j] + bias[j]),
// the sum exact in int32 on the int8 matrix cores.
//
// Tile 128 x 128, four waves of 64 x 64; k is staged 128 at a time through two
// LDS stages.  The weight is the A operand, so that a lane's accumulators
// share one output row and are stored as runs of four columns.  Rows past m or
// n load the last valid row and are not stored.
#include "bqmm_internal.h"

namespace bqmm {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int BM = 128, BN = 128, KS = 128;
constexpr int kStride = KS + 16;  // bytes per staged row; the pad spreads banks
constexpr int kThreads = 256;
constexpr int kTileBytes = BM * kStride;

__global__ __launch_bounds__(kThreads, 2) void w8a8_tile_kernel(const uint8_t *__restrict__ act,
                                                                const uint8_t *__restrict__ w,
                                                                const uint16_t *__restrict__ bias,
                                                                uint16_t *__restrict__ out, uint32_t m, uint32_t n,
                                                                uint32_t kp) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  const uint32_t wn = wave & 1u, wm = wave >> 1;
  const uint32_t n_base = blockIdx.y * BN, m_base = blockIdx.x * BM;
  const uint32_t r0 = tid >> 3, col = (tid & 7u) * 16u;
  v16i acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  for (uint32_t k0 = 0; k0 < kp; k0 += KS) {
    uint4 ra[4], rw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ra[i] = *reinterpret_cast<const uint4 *>(act + (uint64_t)min(m_base + r0 + 32u * i, m - 1u) * kp + k0 + col);
      rw[i] = *reinterpret_cast<const uint4 *>(w + (uint64_t)min(n_base + r0 + 32u * i, n - 1u) * kp + k0 + col);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<uint4 *>(lds + (r0 + 32 * i) * kStride + col) = ra[i];
      *reinterpret_cast<uint4 *>(lds + kTileBytes + (r0 + 32 * i) * kStride + col) = rw[i];
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < KS / 32; ++kk) {
      v4i A[2], B[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        A[t] = *reinterpret_cast<const v4i *>(lds + kTileBytes + (wn * 64 + t * 32 + (lane & 31)) * kStride + 32 * kk + 16 * (lane >> 5));
        B[t] = *reinterpret_cast<const v4i *>(lds + (wm * 64 + t * 32 + (lane & 31)) * kStride + 32 * kk + 16 * (lane >> 5));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(A[i], B[j], acc[i][j], 0, 0, 0);
    }
  }

  const float *sa = reinterpret_cast<const float *>(act + (uint64_t)m * kp);
  const float *sw = reinterpret_cast<const float *>(w + (uint64_t)n * kp);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t mm = m_base + wm * 64 + j * 32 + (lane & 31);
    if (mm >= m) continue;
    const float s = sa[mm];
    uint16_t *row = out + (uint64_t)mm * n;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t nn = n_base + wn * 64 + i * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (nn < n) {
          float y = (float)acc[i][j][r] * s * sw[nn];
          if (bias) y += bf16_to_f32(bias[nn]);
          row[nn] = (uint16_t)f32_to_bf16_rne(y);
        }
      }
  }
}

}  // namespace

hipError_t launch_w8a8_gemm(const void *act, const void *w, const void *bias, void *out, uint32_t m, uint32_t n,
                            uint32_t k, hipStream_t s) {
  const uint32_t kp = (k + 127u) / 128u * 128u;
  constexpr int lds = 2 * kTileBytes;
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void *>(w8a8_tile_kernel), lds);
  if (e != hipSuccess) return e;
  const dim3 grid((uint32_t)(((uint64_t)m + BM - 1) / BM), (uint32_t)(((uint64_t)n + BN - 1) / BN));
  hipLaunchKernelGGL(w8a8_tile_kernel, grid, dim3(kThreads), lds, s, static_cast<const uint8_t *>(act),
                     static_cast<const uint8_t *>(w), static_cast<const uint16_t *>(bias),
                     static_cast<uint16_t *>(out), m, n, kp);
  return hipGetLastError();
}

}  // namespace bqmm
