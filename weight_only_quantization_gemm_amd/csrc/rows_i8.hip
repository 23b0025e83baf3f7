// Rows in 8 bits: activations (x, or x / s) and weights (W, or W * s) to int8
// codes with one scale a row.
//
// A row of up to 16384 values stays in the registers of one block from its read to
// its codes' write, so every byte moves once; a longer one is read twice, the
// second time from the caches.  Bound by memory, for few rows by the chain load -
// join - store.
#include "awq_internal.h"
#include "row_common.h"

namespace awq {

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

__device__ __forceinline__ void store_codes(int8_t* __restrict__ to, const f32x8& v, float by, float top) {
  float c[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) c[u] = code_of(v[u], by, top);
  *reinterpret_cast<u32x2*>(to) = u32x2{code_word(c[0], c[1], c[2], c[3]), code_word(c[4], c[5], c[6], c[7])};
}

// PER: eights of a row a thread holds; 0: the row is read twice.
template <int SCALING, int THREADS, int PER>
__global__ __launch_bounds__(THREADS) void rows_i8_kernel(const f16* __restrict__ x, int64_t stride,
                                                          const float* __restrict__ s, int64_t M, int64_t K,
                                                          int8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float part[THREADS / 64];
  const int64_t m = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (m >= M) return;
  const f16* row = x + m * stride;
  int8_t* to = codes + m * K;
  float top = 0.f;
  if constexpr (PER > 0) {
    f32x8 v[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int64_t k = (p * THREADS + (int)threadIdx.x) * 8;
      v[p] = f32x8{};
      if (k < K) v[p] = row_values<SCALING>(row, s, k);
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) top = largest_of(top, v[p]);
    top = row_join<THREADS>(top, part, MaxOp());
    const float by = 127.f / top;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int64_t k = (p * THREADS + (int)threadIdx.x) * 8;
      if (k < K) store_codes(to + k, v[p], by, top);
    }
  } else {
    for (int64_t k = threadIdx.x * 8; k < K; k += THREADS * 8) top = largest_of(top, row_values<SCALING>(row, s, k));
    top = row_join<THREADS>(top, part, MaxOp());
    const float by = 127.f / top;
    for (int64_t k = threadIdx.x * 8; k < K; k += THREADS * 8)
      store_codes(to + k, row_values<SCALING>(row, s, k), by, top);
  }
  if (threadIdx.x == 0) scales[m] = top / 127.f;
}

template <int THREADS, int PER>
static hipError_t rows_launch(const f16* x, int64_t stride, const float* s, bool divide, int64_t M, int64_t K,
                              int8_t* codes, float* scales, hipStream_t st) {
  const unsigned wide = M < 65536 ? (unsigned)M : 65536u;
  const dim3 grid(wide, (unsigned)((M + wide - 1) / wide)), block(THREADS);
  if (s == nullptr) rows_i8_kernel<kPlainRow, THREADS, PER><<<grid, block, 0, st>>>(x, stride, s, M, K, codes, scales);
  else if (divide) rows_i8_kernel<kDividedRow, THREADS, PER><<<grid, block, 0, st>>>(x, stride, s, M, K, codes, scales);
  else rows_i8_kernel<kMultipliedRow, THREADS, PER><<<grid, block, 0, st>>>(x, stride, s, M, K, codes, scales);
  return hipGetLastError();
}

hipError_t launch_rows_i8(const void* x, int64_t stride, const float* s, bool divide, int64_t M, int64_t K, void* codes,
                          float* scales, hipStream_t st) {
  const f16* xp = reinterpret_cast<const f16*>(x);
  int8_t* cp = reinterpret_cast<int8_t*>(codes);
  // many rows: small blocks, more of which run at once (8192 x 8192: 37 us; 75 with 1024 threads a row; 4000 x
  // 4096: 12 and 20 with 512); few: a short chain (77 x 11008: 3.5 us, 6.1 with 256 threads)
  const bool many = M >= 1024;
  if (K <= 2048) return rows_launch<256, 1>(xp, stride, s, divide, M, K, cp, scales, st);
  if (many && K <= 4096) return rows_launch<256, 2>(xp, stride, s, divide, M, K, cp, scales, st);
  if (many && K <= 8192) return rows_launch<512, 2>(xp, stride, s, divide, M, K, cp, scales, st);
  if (K <= 4096) return rows_launch<512, 1>(xp, stride, s, divide, M, K, cp, scales, st);
  if (K <= 8192) return rows_launch<1024, 1>(xp, stride, s, divide, M, K, cp, scales, st);
  if (K <= 16384) return rows_launch<1024, 2>(xp, stride, s, divide, M, K, cp, scales, st);
  return rows_launch<1024, 0>(xp, stride, s, divide, M, K, cp, scales, st);
}

}  // namespace awq
