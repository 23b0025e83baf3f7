// Rows held in registers: sums and maxima over the threads that share a row,
// and the rounding of a row to 8 bits.
#pragma once

#include "awq_common.h"

namespace awq {

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 widen(f16x8 v) { return __builtin_convertvector(v, f32x8); }

// A wave's join of v by `op` (0 its neutral element), in every lane: shifts within
// rows of 16 lanes, then each row's last lane broadcast to the rows above.
template <typename Op>
__device__ __forceinline__ float wave_join(float v, Op op) {
  auto step = [&](int other) { v = op(v, __int_as_float(other)); };
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xF, 0xF, false));  // row_shr 1, 2, 4, 8
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xA, 0xF, false));  // row_bcast 15, 31
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xC, 0xF, false));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
struct AddOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {  // NaN where either is
  __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_elementwise_maximum(a, b); }
};
// The largest of most and the |v|, NaN where one is.
__device__ __forceinline__ float largest_of(float most, const f32x8& v) {
  const f32x8 m = __builtin_elementwise_abs(v);
  const MaxOp max;
  return max(max(max(most, max(m[0], m[1])), max(m[2], m[3])), max(max(m[4], m[5]), max(m[6], m[7])));
}

// The same over the L threads of a row (L = 64: a wave, otherwise the whole block)
// by way of part [L / 64], which no thread may still be reading: callers take
// another part for each join between two barriers of their own.
template <int L, typename Op>
__device__ __forceinline__ float row_join(float v, float* part, Op op) {
  v = wave_join(v, op);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    lds_barrier();
    if constexpr (L <= 256) {
      v = part[0];
#pragma unroll
      for (int w = 1; w < L / 64; ++w) v = op(v, part[w]);
    } else {  // a lane for each wave's: one access and six steps instead of an access for each
      const int lane = threadIdx.x & 63;
      v = wave_join(lane < L / 64 ? part[lane] : 0.f, op);
    }
  }
  return v;
}

// rint(127 v / top) exactly, for top = max |v| over the row; by = 127 / top rounded.
// The product v * by is within 2^-15 of 127 v / top, so its nearest whole number
// is the wanted one unless it lies closer than that to a half; within 10^-4 of one (one
// value in five thousand) the quotient is formed in 64 bits.  With v = a 2^i and
// top = b 2^(i + d), a and b whole and below 2^24, it differs from a half h / 2 by
// (254 a - h b 2^d) / (b 2^(d + 1)).  A whole numerator that is not 0 is at least 1, and 2
// where d > 0, as both of its terms are even then; d is at most 8 (254 a < 2^32, b >= 2^23,
// and with h >= 1 a quotient next to a half has b 2^d near 254 a).  So what is no half is at least
// 2^-32 away from one, and the 64-bit quotient's error, 127 2^-53, makes and misses none.
// A row with an infinity or a NaN has codes 0, and its scale says what it had.
__device__ __forceinline__ float code_of(float v, float by, float top) {
  const float q = v * by, r = rintf(q);
  if (fabsf(q - r) <= 0.4999f) return r;  // false for a NaN too: by overflows where top is tiny
  return top > 0.f && top < INFINITY ? (float)rint(127.0 * (double)v / (double)top) : 0.f;
}

// Four codes as the bytes of a word.
__device__ __forceinline__ uint32_t code_word(float a, float b, float c, float d) {
  return ((uint32_t)(int)a & 255u) | ((uint32_t)(int)b & 255u) << 8 | ((uint32_t)(int)c & 255u) << 16 |
         (uint32_t)(int)d << 24;
}

}  // namespace awq
