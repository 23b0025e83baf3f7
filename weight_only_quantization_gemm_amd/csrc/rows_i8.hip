// Rows in 8 bits: activations (x, or x / s) and weights (W, or W * s) to int8
// codes with one scale a row.
//
// Two passes over a row by one block: the largest magnitude, then the codes; the
// second pass finds the row in the caches.  Bound by memory.
#include "awq_internal.h"
#include "row_common.h"

namespace awq {

constexpr int kRowThreads = 256;

enum RowScaling { kPlainRow, kDividedRow, kMultipliedRow };

// Eight consecutive values of a row from channel k on.
template <int SCALING>
__device__ __forceinline__ f32x8 row_values(const f16* __restrict__ row, const float* __restrict__ s, int64_t k) {
  f32x8 v = widen(*reinterpret_cast<const f16x8*>(row + k));
  if constexpr (SCALING != kPlainRow) {
    const f32x8 f = *reinterpret_cast<const f32x8*>(s + k);
    v = SCALING == kDividedRow ? v / f : v * f;
  }
  return v;
}

template <int SCALING>
__global__ __launch_bounds__(kRowThreads) void rows_i8_kernel(const f16* __restrict__ x, int64_t stride,
                                                              const float* __restrict__ s, int64_t M, int64_t K,
                                                              int8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float part[kRowThreads / 64];
  const int64_t m = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (m >= M) return;
  const f16* row = x + m * stride;
  float top = 0.f;
  for (int64_t k = threadIdx.x * 8; k < K; k += kRowThreads * 8) {
    const f32x8 v = row_values<SCALING>(row, s, k);
#pragma unroll
    for (int u = 0; u < 8; ++u) top = fmaxf(top, fabsf(v[u]));
  }
  top = row_join<kRowThreads>(top, part, MaxOp());
  const float by = 127.f / top;
  for (int64_t k = threadIdx.x * 8; k < K; k += kRowThreads * 8) {
    const f32x8 v = row_values<SCALING>(row, s, k);
    float c[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) c[u] = code_of(v[u], by, top);
    *reinterpret_cast<u32x2*>(codes + m * K + k) =
        u32x2{code_word(c[0], c[1], c[2], c[3]), code_word(c[4], c[5], c[6], c[7])};
  }
  if (threadIdx.x == 0) scales[m] = top / 127.f;
}

hipError_t launch_rows_i8(const void* x, int64_t stride, const float* s, bool divide, int64_t M, int64_t K, void* codes,
                          float* scales, hipStream_t st) {
  const unsigned wide = M < 65536 ? (unsigned)M : 65536u;
  const dim3 grid(wide, (unsigned)((M + wide - 1) / wide)), block(kRowThreads);
  const f16* xp = reinterpret_cast<const f16*>(x);
  int8_t* cp = reinterpret_cast<int8_t*>(codes);
  if (s == nullptr) rows_i8_kernel<kPlainRow><<<grid, block, 0, st>>>(xp, stride, s, M, K, cp, scales);
  else if (divide) rows_i8_kernel<kDividedRow><<<grid, block, 0, st>>>(xp, stride, s, M, K, cp, scales);
  else rows_i8_kernel<kMultipliedRow><<<grid, block, 0, st>>>(xp, stride, s, M, K, cp, scales);
  return hipGetLastError();
}

}  // namespace awq
