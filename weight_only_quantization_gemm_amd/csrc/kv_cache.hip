// Keys and values quantised as they are written into a paged cache, and read
// back: the group quantizer of awq_pack on the D channels of one (token, head)
// row, at 4 or 8 bits.
//
// Both kernels move D / 8 lanes x 16 bytes of fp16 per row; they read and write
// every byte once and are bound by memory (launch latency at a decoding step's
// sizes).
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

// v / d rounded once, from inv = 1 / d rounded once: a quotient one or two units
// off, then one correction by its exact remainder (Markstein, "IBM Journal of
// Research and Development" 34, 1990), off by 2^-23 of a unit before it is
// rounded.  The quotients here stay further from a rounding border than that: of
// a 24-bit number by 15 or 255 at least 1/510 of a unit, of two 11-bit numbers at
// least 2^-12.
__device__ inline float quotient(float v, float d, float inv) {
  const float q = v * inv;
  return fmaf(fmaf(-q, d, v), inv, q);
}

// 1 / d of an 11-bit number d, rounded once, by the same argument: one Newton
// step from the hardware's reciprocal (good to a unit).
__device__ inline float reciprocal(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return fmaf(fmaf(-d, r, 1.f), r, r);
}

// One row's eight channels of a lane: quantised, and written to the cache.
template <int D, int BITS>
__device__ __forceinline__ void write_row(f16x8 x, KvHalf c, int64_t row, int lane) {
  constexpr int L = D / 8, W = D * BITS / 32;
  constexpr float kTop = BITS == 4 ? 15.f : 255.f;
  const f16x2 p[4] = {{x[0], x[1]}, {x[2], x[3]}, {x[4], x[5]}, {x[6], x[7]}};
  f16x2 hi2 = p[0], lo2 = p[0];
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    hi2 = __builtin_elementwise_max(hi2, p[j]);
    lo2 = __builtin_elementwise_min(lo2, p[j]);
  }
  // (max v, max -v) in one register, both at least 0: the range always holds 0
  const f16x2 none = {(f16)0.f, (f16)0.f};
  f16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(f16x2{hi2.x, -lo2.x}, f16x2{hi2.y, -lo2.y}), none);
  m = row_max<L>(m);
  const float hi = (float)m.x, lo = -(float)m.y;
  const float step = fmaxf(quotient(hi - lo, kTop, 1.f / kTop), 6.103515625e-05f);
  const f16 sc = (f16)fminf(step, 65504.f);
  const float scale = (float)sc, inv = reciprocal(scale);
  const float zero = fminf(fmaxf(rintf(quotient(-lo, scale, inv)), 0.f), kTop);
  // bytes in the order 0 4 1 5 / 2 6 3 7 at 4 bits (the second word then goes to the upper nibbles)
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float code = fminf(fmaxf(rintf(quotient((float)x[j], scale, inv)) + zero, 0.f), kTop);
    const int byte = BITS == 4 ? 2 * (j & 1) + (j >> 2) : j & 3, word = BITS == 4 ? (j >> 1) & 1 : j >> 2;
    w[word] = __builtin_amdgcn_cvt_pk_u8_f32(code, byte, w[word]);
  }
  uint32_t* dst = c.codes + row * W + lane * (W / L);
  if constexpr (BITS == 4) dst[0] = w[0] | (w[1] << 4);
  else *reinterpret_cast<u32x2*>(dst) = u32x2{w[0], w[1]};
  if (lane == 0) c.params[row] = as_u32(f16x2{sc, (f16)zero});
}

template <int D, int BITS>
__device__ __forceinline__ f16x8 read_row(KvHalf c, int64_t row, int lane) {
  constexpr int L = D / 8, W = D * BITS / 32;
  const uint32_t* src = c.codes + row * W + lane * (W / L);
  uint32_t w[2];
  if constexpr (BITS == 4) {
    w[0] = src[0];
    w[1] = w[0] >> 4;
  } else {
    const u32x2 u = *reinterpret_cast<const u32x2*>(src);
    w[0] = u.x;
    w[1] = u.y;
  }
  const f16x2 p = as_f16x2(c.params[row]);
  const float scale = (float)p.x, zero = (float)p.y;
  f16x8 x;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int byte = BITS == 4 ? 2 * (j & 1) + (j >> 2) : j & 3, word = BITS == 4 ? (j >> 1) & 1 : j >> 2;
    const uint32_t code = (w[word] >> (8 * byte)) & (BITS == 4 ? 15u : 255u);
    x[j] = (f16)(((float)code - zero) * scale);  // exact in fp32, rounded once
  }
  return x;
}

// A run of D / 8 lanes takes one (token, head): its key row and its value row.  A
// block takes consecutive tokens of one head (the next block the next head): the
// division by the number of heads is the block's own, and a prompt's parameters,
// 4 bytes a row, leave a block side by side.  8000 tokens x 32 heads of 128 to 8
// bits: 198 MB in 41 to 46 us (4.3 to 4.8 TB/s; 50 us with loads that stay in the caches, 47
// with the quantizer left out), read back in 30 us (6.6 TB/s).
template <int D, int BITS>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(const f16* __restrict__ k, const f16* __restrict__ v,
                                                              int64_t k_stride, int64_t v_stride,
                                                              const int32_t* __restrict__ slots, KvHalf kc, KvHalf vc,
                                                              int64_t T, KvShape sh) {
  constexpr int L = D / 8;
  const uint32_t group = blockIdx.x / (uint32_t)sh.heads, h = blockIdx.x - group * sh.heads;
  const int64_t t = (int64_t)group * (kKvThreads / L) + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  if (t >= T) return;  // whole rows leave together
  const f16x8 kx = __builtin_nontemporal_load(reinterpret_cast<const f16x8*>(k + t * k_stride + h * D + lane * 8));
  const f16x8 vx = __builtin_nontemporal_load(reinterpret_cast<const f16x8*>(v + t * v_stride + h * D + lane * 8));
  const int64_t slot = slots[t];
  if (!kv_slot_ok(sh, slot)) return;
  const int64_t row = kv_row(sh, slot, h);
  write_row<D, BITS>(kx, kc, row, lane);
  write_row<D, BITS>(vx, vc, row, lane);
}

template <int D, int BITS>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvHalf kc, KvHalf vc, const int32_t* __restrict__ slots,
                                                             f16* __restrict__ k, f16* __restrict__ v, int64_t T,
                                                             KvShape sh) {
  constexpr int L = D / 8;
  const uint32_t group = blockIdx.x / (uint32_t)sh.heads, h = blockIdx.x - group * sh.heads;
  const int64_t t = (int64_t)group * (kKvThreads / L) + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  if (t >= T) return;
  const int64_t slot = slots[t];
  f16x8 kx = {}, vx = {};
  if (kv_slot_ok(sh, slot)) {
    const int64_t row = kv_row(sh, slot, h);
    kx = read_row<D, BITS>(kc, row, lane);
    vx = read_row<D, BITS>(vc, row, lane);
  }
  *reinterpret_cast<f16x8*>(k + (t * sh.heads + h) * D + lane * 8) = kx;
  *reinterpret_cast<f16x8*>(v + (t * sh.heads + h) * D + lane * 8) = vx;
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
    constexpr int per = kKvThreads / (d.value / 8);  // tokens of a block
    const dim3 grid((unsigned)((T + per - 1) / per * sh.heads));
    kv_write_kernel<d.value, b.value><<<grid, dim3(kKvThreads), 0, st>>>(
        reinterpret_cast<const f16*>(k), reinterpret_cast<const f16*>(v), k_stride, v_stride, slots, kc, vc, T, sh);
    return hipGetLastError();
  });
}

hipError_t launch_kv_read(KvHalf kc, KvHalf vc, const int32_t* slots, void* k, void* v, int64_t T, int D, int bits,
                          KvShape sh, hipStream_t st) {
  return kv_dispatch(D, bits, [&](auto d, auto b) {
    constexpr int per = kKvThreads / (d.value / 8);  // tokens of a block
    const dim3 grid((unsigned)((T + per - 1) / per * sh.heads));
    kv_read_kernel<d.value, b.value><<<grid, dim3(kKvThreads), 0, st>>>(
        kc, vc, slots, reinterpret_cast<f16*>(k), reinterpret_cast<f16*>(v), T, sh);
    return hipGetLastError();
  });
}

}  // namespace awq
