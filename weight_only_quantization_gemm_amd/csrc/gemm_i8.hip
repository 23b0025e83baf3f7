// The product in 8-bit integers: y = (x codes) (w codes)^T in exact 32-bit sums,
// times a scale for each token and each channel.
//
// Tiles of 128 bytes of K go from global memory straight into LDS (the layout of
// mfma_pipe.h, a pair of codes in the place of a half) and feed
// v_mfma_i32_32x32x32_i8; the weights are the A operand, so a lane's accumulators
// hold four consecutive channels of one token.
#include "awq_internal.h"
#include "mfma_pipe.h"

namespace awq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

// Output tile BM tokens x BN channels by 2 x 2 waves, two stages.
template <int BM, int BN, typename Y>
__global__ __launch_bounds__(256) void gemm_i8_kernel(const int8_t* __restrict__ x, const float* __restrict__ xs,
                                                      const int8_t* __restrict__ w, const float* __restrict__ ws,
                                                      Y* __restrict__ y, int64_t M, int64_t N, int64_t K,
                                                      int64_t mtiles) {
  constexpr int TM = BM / 2, TN = BN / 2, AM = TM / 32, AN = TN / 32;
  __shared__ __align__(16) f16 lds[2][(BM + BN) * 64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t m0 = (blockIdx.x % mtiles) * BM, n0 = (blockIdx.x / mtiles) * BN;
  const int wm = (wave & 1) * TM, wn = (wave >> 1) * TN;
  TilePlan<BM, 4, 64> px;
  TilePlan<BN, 4, 64> pw;
  px.init(reinterpret_cast<const f16*>(x), K / 2, m0, M, wave, lane);
  pw.init(reinterpret_cast<const f16*>(w), K / 2, n0, N, wave, lane);
  i32x16 acc[AN][AM];
#pragma unroll
  for (int i = 0; i < AN; ++i)
#pragma unroll
    for (int j = 0; j < AM; ++j) acc[i][j] = i32x16{};
  const int steps = (int)(K / 128);
  px.issue(lds[0], 0);
  pw.issue(lds[0] + BM * 64, 0);
  for (int s = 0; s < steps; ++s) {
    wait_vmcnt<0>();
    lds_barrier();  // stage s is in LDS, and every wave is done with the other stage
    if (s + 1 < steps) {
      px.issue(lds[(s + 1) & 1], (int64_t)(s + 1) * 64);
      pw.issue(lds[(s + 1) & 1] + BM * 64, (int64_t)(s + 1) * 64);
    }
    const f16* tx = lds[s & 1];
    const f16* tw = tx + BM * 64;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      i32x4 a[AN], b[AM];
#pragma unroll
      for (int i = 0; i < AN; ++i)
        a[i] = __builtin_bit_cast(i32x4, frag(tw, wn + i * 32 + (lane & 31), 2 * c + (lane >> 5)));
#pragma unroll
      for (int j = 0; j < AM; ++j)
        b[j] = __builtin_bit_cast(i32x4, frag(tx, wm + j * 32 + (lane & 31), 2 * c + (lane >> 5)));
#pragma unroll
      for (int i = 0; i < AN; ++i)
#pragma unroll
        for (int j = 0; j < AM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < AM; ++j) {
    const int64_t m = m0 + wm + j * 32 + (lane & 31);
    if (m >= M) continue;
    const float sm = xs[m];
#pragma unroll
    for (int i = 0; i < AN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t n = n0 + wn + i * 32 + 8 * q + 4 * (lane >> 5) + u;
          if (n < N) y[m * N + n] = (Y)((float)acc[i][j][4 * q + u] * sm * ws[n]);
        }
  }
}

static size_t rows_bytes(int64_t M, int64_t K) { return ((size_t)M * (size_t)K + 255) / 256 * 256; }

size_t gemm_i8_workspace(int64_t M, int64_t N, int64_t K, bool quantized) {
  return quantized ? 0 : rows_bytes(M, K) + ((size_t)M * 4 + 255) / 256 * 256;
}

hipError_t launch_gemm_i8(const void* x, const float* x_scales, const float* s, const void* codes, const float* scales,
                          void* y, int y_bytes, int64_t M, int64_t N, int64_t K, void* ws, hipStream_t st) {
  const int64_t mtiles = (M + 127) / 128, ntiles = (N + 127) / 128;
  const dim3 grid((unsigned)(mtiles * ntiles)), block(256);
  if (KernelPlan* p = active_plan())
    return plan_record(p, "gemm_i8_kernel<128,128> block=%u grid=%u", block.x, grid.x);
  if (x_scales == nullptr) {
    int8_t* xc = reinterpret_cast<int8_t*>(ws);
    float* sc = reinterpret_cast<float*>(xc + rows_bytes(M, K));
    const hipError_t e = launch_rows_i8(x, K, s, true, M, K, xc, sc, st);
    if (e != hipSuccess) return e;
    x = xc;
    x_scales = sc;
  }
  const int8_t *xp = reinterpret_cast<const int8_t*>(x), *wp = reinterpret_cast<const int8_t*>(codes);
  if (y_bytes == 2)
    gemm_i8_kernel<128, 128><<<grid, block, 0, st>>>(xp, x_scales, wp, scales, reinterpret_cast<f16*>(y), M, N, K, mtiles);
  else
    gemm_i8_kernel<128, 128><<<grid, block, 0, st>>>(xp, x_scales, wp, scales, reinterpret_cast<float*>(y), M, N, K, mtiles);
  return hipGetLastError();
}

}  // namespace awq
