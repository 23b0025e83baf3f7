// The norm between two blocks: the block's output enters the residual stream,
// and the next block's input is normed from that, as fp16 or as rows of 8 bits.
//
// A row stays in the registers of the L threads that share it from its one read to
// its last write, so every byte moves once; two statistics (post-norm) make two
// joins over the row, a layer norm's mean and variance two each, the second from
// the differences to the mean, so nothing cancels.  A row of more than 8192 is kept in
// its own types and widened where it is used: half the registers, so that two blocks
// share a compute unit up to 16384 (4000 rows of it 111 us, 131 as fp32) and rows of
// 32768 fit at all (2000 rows 130 us; 1045 with registers spilled to memory).  Open:
// fp32 rows above 32768 still spill some (1000 x 65536 235 us, a copy's time 152).
// Bound by memory: fp16 rows with y and post-norm, out of the caches, take 28 us
// (8000 x 2048), 106 (16384 x 4096), 234 (16384 x 8192 with a gate), 111 (4000 x
// 16384), i.e. 4.5 to 5.1 TB/s where a copy reaches 5.2; at a decoding step's sizes by the launch and the chain load - join - store
// (4 x 4096 2.7 us).
#include <type_traits>

#include "awq.h"
#include "awq_internal.h"
#include "row_common.h"

namespace awq {

template <typename H>
struct RowVec;
template <>
struct RowVec<f16> {
  typedef f16x8 type;
};
template <>
struct RowVec<float> {
  typedef f32x8 type;
};

__device__ __forceinline__ f32x8 as_f32(f16x8 v) { return widen(v); }
__device__ __forceinline__ f32x8 as_f32(f32x8 v) { return v; }

// Widened numbers of v are not kept past this: for long rows they would not fit beside the next step's.
template <typename V, int PER>
__device__ __forceinline__ void narrow(V (&v)[PER]) {
  if constexpr (PER >= 4 && sizeof(V) == 16)
#pragma unroll
    for (int p = 0; p < PER; ++p) __asm__("" : "+v"(v[p]));
}

// mean (0 unless layer) and 1 / sqrt(variance + eps) of the row v.
template <int L, typename V, int PER>
__device__ __forceinline__ void statistics(V (&v)[PER], const bool (&live)[PER], int64_t N, bool layer,
                                           float eps, float* part, float* mean, float* r) {
  constexpr int W = L / 64;
  float sum = 0.f;
  *mean = 0.f;
  if (layer) {
#pragma unroll
    for (int p = 0; p < PER; ++p)
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += (float)v[p][u];  // 0 beyond the row
    *mean = row_join<L>(sum, part, AddOp()) / (float)N;
    narrow(v);
  }
  sum = 0.f;
#pragma unroll
  for (int p = 0; p < PER; ++p)
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float d = live[p] ? (float)v[p][u] - *mean : 0.f;
      sum = fmaf(d, d, sum);
    }
  narrow(v);
  sum = row_join<L>(sum, part + W, AddOp());
  *r = 1.f / sqrtf(sum / (float)N + eps);
}

template <typename H, int L, int PER>
__global__ __launch_bounds__(L < 256 ? 256 : L) void norm_kernel(NormArgs a) {
  typedef typename RowVec<H>::type HV;
  constexpr int ROWS = L < 256 ? 256 / L : 1, W = L / 64;
  __shared__ float part[5 * W];
  const int lane = threadIdx.x % L;
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * ROWS + threadIdx.x / L;
  if (t >= a.T) return;  // a whole wave of its own row (L = 64) or the whole block
  const bool layer = a.kind == AWQ_NORM_LAYER;
  // With one eight a thread and wide rows everything is under way before the first join: 16384 x 8192 with
  // post-norm and gate 232 us, 247 with each vector read where it is used (x 4096: 106 and 111).  Narrower
  // rows do not gain by it (16000 x 1024: 28.0, and 26.1 without), and longer ones have no registers for it.
  constexpr bool EARLY = PER == 1 && L >= 512;
  constexpr bool HELD = PER * sizeof(H) <= 8;  // the weights in registers before the first store, where they fit
  bool live[PER];
  int at[PER];
  // Long rows stay in their own types, half the registers of fp32; one eight is widened at once (16384 x 8192
  // with post-norm and gate: 233 us, 247 kept as it is).
  typedef typename std::conditional<PER == 1, f32x8, HV>::type KeptH;
  typedef typename std::conditional<PER == 1, f32x8, f16x8>::type KeptY;
  KeptH h[PER];
  f16x8 w_early[PER], pw_early[PER], g_early[PER];
  auto part_of = [&](const f16* v, int p) {
    return v != nullptr && live[p] ? *reinterpret_cast<const f16x8*>(v + at[p]) : f16x8{};
  };
  int64_t row = a.gates > 1 ? t : 0;
  if (a.gate_rows != nullptr) row = a.gate_rows[t];
  const bool adds = a.gate == nullptr || (row >= 0 && row < a.gates);
  const f16* gate = adds && a.gate != nullptr ? a.gate + row * a.N : nullptr;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    at[p] = (p * L + lane) * 8;
    live[p] = at[p] < a.N;
    h[p] = KeptH{};
    if (live[p])
      h[p] = __builtin_convertvector(
          *reinterpret_cast<const HV*>(reinterpret_cast<const H*>(a.h) + t * a.h_stride + at[p]), KeptH);
  }
  float mean, r;
  if (a.y != nullptr) {
    KeptY y[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      y[p] = KeptY{};
      if (live[p])
        y[p] = __builtin_convertvector(*reinterpret_cast<const f16x8*>(a.y + t * a.y_stride + at[p]), KeptY);
    }
    if constexpr (EARLY)
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        pw_early[p] = part_of(a.post_weight, p);
        g_early[p] = part_of(gate, p);
        w_early[p] = part_of(a.weight, p);
      }
    if (a.post_weight != nullptr) {
      statistics<L>(y, live, a.N, layer, a.eps, part, &mean, &r);
    }
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (live[p]) {
        if (PER * sizeof(H) >= 16) __asm__ volatile("" ::: "memory");  // the vectors of one step at a time, likewise
        f32x8 v = as_f32(y[p]), g = f32x8{} + a.scale;
        if (a.post_weight != nullptr) {
          v = (v - mean) * r * widen(EARLY ? pw_early[p] : part_of(a.post_weight, p));
          if (a.post_bias != nullptr) v += widen(part_of(a.post_bias, p));
        }
        if (gate != nullptr) g *= widen(EARLY ? g_early[p] : part_of(gate, p));
        if (adds) h[p] = __builtin_convertvector(__builtin_convertvector(as_f32(h[p]) + v * g, HV), KeptH);
      }
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (live[p]) *reinterpret_cast<HV*>(reinterpret_cast<H*>(a.h_out) + t * a.N + at[p]) = __builtin_convertvector(h[p], HV);
  } else if constexpr (EARLY) {
#pragma unroll
    for (int p = 0; p < PER; ++p) w_early[p] = part_of(a.weight, p);
  }
  if (a.weight == nullptr) return;
  narrow(h);
  statistics<L>(h, live, a.N, layer, a.eps, part + 2 * W, &mean, &r);
  f16x8 w_held[PER];
  if constexpr (!EARLY && HELD)
#pragma unroll
    for (int p = 0; p < PER; ++p) w_held[p] = part_of(a.weight, p);
  auto w = [&](int p) { return widen(EARLY ? w_early[p] : HELD ? w_held[p] : part_of(a.weight, p)); };
  if (a.x_scales == nullptr) {
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (live[p]) {
        f32x8 x = (as_f32(h[p]) - mean) * r * w(p);
        if (a.bias != nullptr) x += widen(part_of(a.bias, p));
        *reinterpret_cast<f16x8*>(reinterpret_cast<f16*>(a.x) + t * a.N + at[p]) = __builtin_convertvector(x, f16x8);
      }
    return;
  }
  float top = 0.f;
#pragma unroll
  for (int p = 0; p < PER; ++p) top = largest_of(top, as_f32(h[p]) * w(p));
  narrow(h);
  top = row_join<L>(top, part + 4 * W, MaxOp());
  const float by = 127.f / top;
#pragma unroll
  for (int p = 0; p < PER; ++p)
    if (live[p]) {
      const f32x8 v = as_f32(h[p]) * w(p);
      float c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] = code_of(v[u], by, top);
      *reinterpret_cast<u32x2*>(reinterpret_cast<int8_t*>(a.x) + t * a.N + at[p]) =
          u32x2{code_word(c[0], c[1], c[2], c[3]), code_word(c[4], c[5], c[6], c[7])};
    }
  if (lane == 0) a.x_scales[t] = top == 0.f ? 0.f : r * (top / 127.f);  // without eps r is infinite where h is 0
}

template <int L, int PER>
static hipError_t norm_launch(const NormArgs& a, int h_bytes, hipStream_t st) {
  constexpr int THREADS = L < 256 ? 256 : L, ROWS = THREADS / L;
  const int64_t blocks = (a.T + ROWS - 1) / ROWS;
  const unsigned wide = blocks < 65536 ? (unsigned)blocks : 65536u;
  const dim3 grid(wide, (unsigned)((blocks + wide - 1) / wide)), block(THREADS);
  if (h_bytes == 2) norm_kernel<f16, L, PER><<<grid, block, 0, st>>>(a);
  else norm_kernel<float, L, PER><<<grid, block, 0, st>>>(a);
  return hipGetLastError();
}

// By the row's length alone, so that a row's sums, and its result, do not depend on the rows beside it.  With post-norm,
// beside the nearest other layout: 16000 x 512 16 us (31 with 256 threads a row); x 1024 27 (39; but 300 rows 4.2 and
// 3.4); 8000 x 2048 27 (30 with a wave a row, and 4 rows 3.0 and 5.3); x 4096 52 (48 with 256 threads and two eights;
// 4 rows 3.4 and 4.0); x 8192 107 (106 with 512; 4 rows 4.3 and 4.4); 4000 x 16384 112 (118 with 512).
hipError_t launch_norm(const NormArgs& a, int h_bytes, hipStream_t st) {
  if (a.N <= 512) return norm_launch<64, 1>(a, h_bytes, st);
  if (a.N <= 1024) return norm_launch<64, 2>(a, h_bytes, st);
  if (a.N <= 2048) return norm_launch<256, 1>(a, h_bytes, st);
  if (a.N <= 4096) return norm_launch<512, 1>(a, h_bytes, st);
  if (a.N <= 8192) return norm_launch<1024, 1>(a, h_bytes, st);
  if (a.N <= 16384) return norm_launch<1024, 2>(a, h_bytes, st);
  if (a.N <= 32768) return norm_launch<1024, 4>(a, h_bytes, st);
  return norm_launch<1024, 8>(a, h_bytes, st);
}

}  // namespace awq
