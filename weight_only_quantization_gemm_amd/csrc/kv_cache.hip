// Keys and values quantised as they are written into a paged cache, and read
// back: the group quantizer of awq_pack on the D channels of one (token, head)
// row, at 4 or 8 bits.
//
// Both kernels move D / 8 lanes x 16 bytes of fp16 per row and half; they read
// and write every byte once and are bound by memory (launch latency at a
// decoding step's sizes).
#include "awq_common.h"
#include "awq_internal.h"
#include "kv_common.h"

namespace awq {

constexpr int kKvThreads = 256;

// Largest of v over the L lanes of a row (L = 8, 16 or 32 consecutive lanes),
// in every lane.  The first four steps pair lanes through DPP: neighbours,
// pairs, quads (mirror of 8) and eights (mirror of 16).
template <int L>
__device__ inline f16x2 row_max(f16x2 v) {
  auto step = [&](uint32_t other) { v = __builtin_elementwise_max(v, as_f16x2(other)); };
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u32(v), 0xB1, 0xF, 0xF, true));   // quad_perm 1 0 3 2
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u32(v), 0x4E, 0xF, 0xF, true));   // quad_perm 2 3 0 1
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u32(v), 0x141, 0xF, 0xF, true));  // row_half_mirror
  if (L >= 16) step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u32(v), 0x140, 0xF, 0xF, true));  // row_mirror
  if (L >= 32) step((uint32_t)__shfl_xor((int)as_u32(v), 16, kWave));
  return v;
}

// v / scale rounded once, from inv = 1 / scale rounded once: a quotient one or
// two units off, then one correction by its exact remainder (Markstein, "IBM
// Journal of Research and Development" 34, 1990).  v and scale have 11-bit
// significands, so the corrected quotient is the rounded one.
__device__ inline float quotient(float v, float scale, float inv) {
  const float q = v * inv;
  return fmaf(fmaf(-q, scale, v), inv, q);
}

template <int D, int BITS>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(const f16* __restrict__ k, const f16* __restrict__ v,
                                                              int64_t k_stride, int64_t v_stride,
                                                              const int32_t* __restrict__ slots, KvHalf kc, KvHalf vc,
                                                              int64_t T, KvShape sh) {
  constexpr int L = D / 8, W = D * BITS / 32;
  constexpr float kTop = BITS == 4 ? 15.f : 255.f;
  const int64_t i = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / L;  // row of this half: t * H + h
  const int lane = threadIdx.x % L;
  if (i >= T * sh.heads) return;  // whole rows leave together
  const int64_t t = i / sh.heads;
  const int h = (int)(i - t * sh.heads);
  const bool values = blockIdx.y != 0;
  const int64_t slot = slots[t];
  if (!kv_slot_ok(sh, slot)) return;
  const f16* src = (values ? v + t * v_stride : k + t * k_stride) + h * D + lane * 8;
  const f16x8 x = *reinterpret_cast<const f16x8*>(src);
  // (max v, max -v), both at least 0: the range always holds 0
  f16x2 m = {(f16)0.f, (f16)0.f};
#pragma unroll
  for (int j = 0; j < 8; ++j) m = __builtin_elementwise_max(m, f16x2{x[j], -x[j]});
  m = row_max<L>(m);
  const float hi = (float)m.x, lo = -(float)m.y;
  const float step = fmaxf((hi - lo) / kTop, 6.103515625e-05f);
  const f16 sc = (f16)fminf(step, 65504.f);
  const float scale = (float)sc, inv = 1.0f / scale;
  const float zero = fminf(fmaxf(rintf(quotient(-lo, scale, inv)), 0.f), kTop);
  uint32_t w[BITS / 4] = {};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float c = fminf(fmaxf(rintf(quotient((float)x[j], scale, inv)) + zero, 0.f), kTop);
    if (BITS == 4) w[0] |= (uint32_t)c << (4 * nibble_pos(j));
    else w[j / 4] |= (uint32_t)c << (8 * (j % 4));
  }
  const KvHalf c = values ? vc : kc;
  const int64_t row = kv_row(sh, slot, h);
  uint32_t* dst = c.codes + row * W + lane * (W / L);
  if constexpr (BITS == 4) dst[0] = w[0];
  else *reinterpret_cast<u32x2*>(dst) = u32x2{w[0], w[1]};
  if (lane == 0) c.params[row] = as_u32(f16x2{sc, (f16)zero});
}

template <int D, int BITS>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvHalf kc, KvHalf vc, const int32_t* __restrict__ slots,
                                                             f16* __restrict__ k, f16* __restrict__ v, int64_t T,
                                                             KvShape sh) {
  constexpr int L = D / 8, W = D * BITS / 32;
  const int64_t i = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / L;
  const int lane = threadIdx.x % L;
  if (i >= T * sh.heads) return;
  const int64_t t = i / sh.heads;
  const int h = (int)(i - t * sh.heads);
  const bool values = blockIdx.y != 0;
  const int64_t slot = slots[t];
  f16x8 x = {};
  if (kv_slot_ok(sh, slot)) {
    const KvHalf c = values ? vc : kc;
    const int64_t row = kv_row(sh, slot, h);
    const uint32_t* src = c.codes + row * W + lane * (W / L);
    const f16x2 p = as_f16x2(c.params[row]);
    const float scale = (float)p.x, zero = (float)p.y;
    uint32_t w[BITS / 4];
    if constexpr (BITS == 4) {
      w[0] = src[0];
    } else {
      const u32x2 u = *reinterpret_cast<const u32x2*>(src);
      w[0] = u.x;
      w[1] = u.y;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c8 = BITS == 4 ? (w[0] >> (4 * nibble_pos(j))) & 15u : (w[j / 4] >> (8 * (j % 4))) & 255u;
      x[j] = (f16)(((float)c8 - zero) * scale);  // exact in fp32, rounded once
    }
  }
  *reinterpret_cast<f16x8*>((values ? v : k) + i * D + lane * 8) = x;
}

template <typename F>
static hipError_t kv_dispatch(int D, int bits, F&& f) {
  if (bits == 4) {
    if (D == 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    if (D == 128) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 4>{});
    if (D == 256) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
  } else if (bits == 8) {
    if (D == 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
    if (D == 128) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 8>{});
    if (D == 256) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 8>{});
  }
  return hipErrorInvalidValue;
}

hipError_t launch_kv_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* slots,
                           KvHalf kc, KvHalf vc, int64_t T, int D, int bits, KvShape sh, hipStream_t st) {
  return kv_dispatch(D, bits, [&](auto d, auto b) {
    const int64_t lanes = T * sh.heads * (d.value / 8);
    const dim3 grid((unsigned)((lanes + kKvThreads - 1) / kKvThreads), 2);
    kv_write_kernel<d.value, b.value><<<grid, dim3(kKvThreads), 0, st>>>(
        reinterpret_cast<const f16*>(k), reinterpret_cast<const f16*>(v), k_stride, v_stride, slots, kc, vc, T, sh);
    return hipGetLastError();
  });
}

hipError_t launch_kv_read(KvHalf kc, KvHalf vc, const int32_t* slots, void* k, void* v, int64_t T, int D, int bits,
                          KvShape sh, hipStream_t st) {
  return kv_dispatch(D, bits, [&](auto d, auto b) {
    const int64_t lanes = T * sh.heads * (d.value / 8);
    const dim3 grid((unsigned)((lanes + kKvThreads - 1) / kKvThreads), 2);
    kv_read_kernel<d.value, b.value><<<grid, dim3(kKvThreads), 0, st>>>(
        kc, vc, slots, reinterpret_cast<f16*>(k), reinterpret_cast<f16*>(v), T, sh);
    return hipGetLastError();
  });
}

}  // namespace awq
