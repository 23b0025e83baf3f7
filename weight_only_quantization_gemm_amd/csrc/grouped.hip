// W4A16 / W3A16 products grouped by expert: rows offsets[e] .. offsets[e+1] - 1
// of the ragged batch are multiplied by expert e's packed matrix.
//
// The group sizes are on the device, so the grid covers the most row tiles
// the sizes could make and every block finds its own: a wave counts each
// expert's tiles, 64 experts at a time, and takes the expert in which the
// block's tile number falls.  Blocks past the last tile leave at once.
//
// Arithmetic (as the decode kernels of the single product): code - zero exact
// in fp16, fp32 sums per 128-channel group on the matrix cores, the group's
// scale applied in fp32, one rounding of y to fp16.
#include "awq_common.h"
#include "awq_internal.h"

namespace awq {

struct RowTile {
  int expert, row, rows;  // first row of the ragged batch, rows of the tile; rows = 0: no such tile
};

// Tile number `tile` (of BM rows) of the ragged batch; the same in every lane.
// Offsets are clamped to [0, R] and to order, so a tile never leaves the batch.
__device__ inline RowTile find_tile(const int32_t* __restrict__ offsets, int E, int R, int tile, int BM) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int a = 0, n = 0;
    if (e < E) {
      a = offsets[e];
      a = a < 0 ? 0 : (a > R ? R : a);
      int z = offsets[e + 1];
      z = z < a ? a : (z > R ? R : z);
      n = z - a;
    }
    const int mine = (n + BM - 1) / BM;
    int upto = mine;  // inclusive scan over the lanes
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(upto, off, kWave);
      if (lane >= off) upto += o;
    }
    const uint64_t past = __ballot(upto > tile);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      const int first = (tile - __builtin_amdgcn_readlane(upto - mine, at)) * BM;
      const int left = __builtin_amdgcn_readlane(n, at) - first;
      return {e0 + at, __builtin_amdgcn_readlane(a, at) + first, left < BM ? left : BM};
    }
    tile -= __builtin_amdgcn_readlane(upto, 63);
  }
  return {0, 0, 0};
}

// Row of x that row i of the ragged batch reads.
__device__ inline int64_t x_row(const int32_t* __restrict__ rows, int i, int top_k, int64_t x_rows) {
  int64_t r = rows == nullptr ? i : rows[i] / top_k;
  return r < 0 ? 0 : (r < x_rows ? r : x_rows - 1);
}

// xs[i] = fp16(fp32(x of row i) / s of its expert): the input side of the
// per-channel scaling, one block per row of the ragged batch.
__global__ __launch_bounds__(256) void scale_rows_kernel(const f16* __restrict__ x, int64_t x_rows,
                                                         const int32_t* __restrict__ rows, int top_k,
                                                         const int32_t* __restrict__ offsets,
                                                         const float* __restrict__ s, int E, int R, int64_t K,
                                                         f16* __restrict__ xs) {
  const int i = (int)blockIdx.x;
  const RowTile t = find_tile(offsets, E, R, i, 1);
  if (t.rows == 0) return;
  const f16* src = x + x_row(rows, t.row, top_k, x_rows) * K;
  const float* sc = s + (int64_t)t.expert * K;
  f16* dst = xs + (int64_t)t.row * K;
  for (int64_t k = threadIdx.x * 8; k < K; k += 256 * 8) {
    const f16x8 v = *reinterpret_cast<const f16x8*>(src + k);
    f16x8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (f16)((float)v[j] / sc[k + j]);
    *reinterpret_cast<f16x8*>(dst + k) = o;
  }
}

// 16 rows of the batch x 16 weight rows per block; four waves take the
// 128-channel groups in turn and are summed through LDS in a fixed order.
constexpr int kGrpWaves = 4;

template <int BITS>
__global__ __launch_bounds__(64 * kGrpWaves) void grouped_kernel(
    const f16* __restrict__ x, int64_t x_rows, const int32_t* __restrict__ rows, int top_k,
    const int32_t* __restrict__ offsets, const uint32_t* __restrict__ packed, const f16* __restrict__ scales,
    const uint8_t* __restrict__ zeros, f16* __restrict__ y, int R, int E, int64_t N, int64_t K) {
  __shared__ float red[kGrpWaves][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nl = lane & 15, kq = lane >> 4;
  const int nt = (int)((N + 15) / 16), mb = (int)blockIdx.x / nt;
  const RowTile tile = find_tile(offsets, E, R, mb, 16);
  if (tile.rows == 0) return;
  const int64_t G = K / kGroup, P2 = (G + 1) / 2, W = BITS == 4 ? K / 8 : 3 * (K / 32);
  const int64_t n0 = (int64_t)((int)blockIdx.x - mb * nt) * 16;
  const int64_t n = (int64_t)tile.expert * N + (n0 + nl < N ? n0 + nl : N - 1);
  const f16* xr = x + x_row(rows, tile.row + (nl < tile.rows ? nl : tile.rows - 1), top_k, x_rows) * K + kq * 32;
  const uint32_t bias = bias_in_vgpr();
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t g = wave; g < G; g += kGrpWaves) {
    const ZeroForms zf = zero_forms((zeros[n * P2 + (g >> 1)] >> (4 * (g & 1))) & 0xFu);
    const float sc = (float)scales[n * G + g];
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    f16x8 b[4];
    if constexpr (BITS == 4) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(packed + n * W + g * 16 + kq * 4);
#pragma unroll
      for (int s = 0; s < 4; ++s) b[s] = word_minus_zero(w[s], bias, zf);
    } else {
      const uint32_t* wp = packed + n * W + g * 12 + kq * 3;
      const uint32_t w[3] = {wp[0], wp[1], wp[2]};
      f16x2 q[16];
#pragma unroll
      for (int p = 0; p < 15; ++p) q[p] = as_f16x2(((w[p / 5] >> (3 * (p % 5))) & 0x00070007u) | bias) - zf.zb1;
      q[15] = as_f16x2(((w[0] >> 15) & 0x00010001u) | ((w[1] >> 14) & 0x00020002u) | ((w[2] >> 13) & 0x00040004u) |
                       bias) -
              zf.zb1;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        b[s] = f16x8{q[4 * s].x,     q[4 * s].y,     q[4 * s + 1].x, q[4 * s + 1].y,
                     q[4 * s + 2].x, q[4 * s + 2].y, q[4 * s + 3].x, q[4 * s + 3].y};
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
      d = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const f16x8*>(xr + g * kGroup + 8 * s), b[s], d, 0,
                                                 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(sc, d[r], acc[r]);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) red[wave][4 * kq + r][nl] = acc[r];
  __syncthreads();
  const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (m < tile.rows && n0 + c < N) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kGrpWaves; ++w) v += red[w][m][c];
    y[(int64_t)(tile.row + m) * N + n0 + c] = (f16)v;
  }
}

// The most tiles of BM rows that R rows in E groups can make.
static int64_t row_tiles(int64_t R, int64_t E, int64_t BM) { return (R + (E < R ? E : R) * (BM - 1)) / BM; }

bool gemm_grouped_fits(int64_t R, int64_t E, int64_t N) {
  return (N + 15) / 16 * row_tiles(R, E, 16) * (64 * kGrpWaves) < (int64_t(1) << 32);  // a grid's threads
}

hipError_t launch_gemm_grouped(const void* x, int64_t x_rows, const int32_t* rows, int top_k, const int32_t* offsets,
                               const float* s, const void* packed, const void* scales, const void* zeros, void* y,
                               int64_t R, int E, int64_t N, int64_t K, int bits, void* ws, hipStream_t st) {
  const f16* xp = reinterpret_cast<const f16*>(x);
  if (s != nullptr) {
    scale_rows_kernel<<<dim3((unsigned)R), dim3(256), 0, st>>>(xp, x_rows, rows, top_k, offsets, s, E, (int)R, K,
                                                               reinterpret_cast<f16*>(ws));
    if (hipError_t e = hipGetLastError()) return e;
    xp = reinterpret_cast<const f16*>(ws);
    x_rows = R;
    rows = nullptr;
  }
  const dim3 grid((unsigned)((N + 15) / 16 * row_tiles(R, E, 16))), block(64 * kGrpWaves);
  auto pp = reinterpret_cast<const uint32_t*>(packed);
  auto sp = reinterpret_cast<const f16*>(scales);
  auto zp = reinterpret_cast<const uint8_t*>(zeros);
  auto yp = reinterpret_cast<f16*>(y);
  if (bits == 4)
    grouped_kernel<4><<<grid, block, 0, st>>>(xp, x_rows, rows, top_k, offsets, pp, sp, zp, yp, (int)R, E, N, K);
  else
    grouped_kernel<3><<<grid, block, 0, st>>>(xp, x_rows, rows, top_k, offsets, pp, sp, zp, yp, (int)R, E, N, K);
  return hipGetLastError();
}

}  // namespace awq
