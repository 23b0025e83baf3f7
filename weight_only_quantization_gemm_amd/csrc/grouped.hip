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
#include "awq.h"
#include "awq_common.h"
#include "awq_internal.h"
#include "mfma_pipe.h"

#include <type_traits>

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
    const int upto = wave_scan(mine);
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

// The zero point in the forms the unpacking subtracts: of 4-bit codes those of
// word_minus_zero; of 3-bit codes 1024 + zero, -(128 + zero) and -(16 + zero).
template <int BITS>
struct Zero;
template <>
struct Zero<4> {
  ZeroForms f;
  __device__ __forceinline__ void set(uint32_t z) { f = zero_forms(z); }
};
template <>
struct Zero<3> {
  f16x2 zb1, nz128, nz16;
  __device__ __forceinline__ void set(uint32_t z) {
    zb1 = zero_biased(z);
    nz128 = as_f16x2(0xD800D800u | (z << 3) | (z << 19));  // 128 has spacing 1/8
    nz16 = as_f16x2(0xCC00CC00u | (z << 6) | (z << 22));   // 16 has spacing 1/64
  }
};

// Eight channels' code - zero, exact, as a matrix-core operand: 8 s .. 8 s + 7 of
// the 32 channels in `w` (four words, or three).
template <typename Words>
__device__ __forceinline__ f16x8 unpack8(const Words& w, int s, uint32_t bias, const Zero<4>& z) {
  return word_minus_zero(w[s], bias, z.f);
}
// 3 bits: fields 0, 1, 2 of a word, or of the word shifted by nine (fields 3, 4),
// masked where they stand are 1024 + code, 1024 + 8 code and 1024 + 64 code once
// the bias is or-ed in; a packed subtraction or fma leaves code - zero, exactly.
template <typename Words>
__device__ __forceinline__ f16x8 unpack8(const Words& w, int s, uint32_t bias, const Zero<3>& z) {
  const f16x2 eighth = {(f16)0.125f, (f16)0.125f}, sixty_fourth = {(f16)0.015625f, (f16)0.015625f};
  f16x2 q[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int p = 4 * s + u, j = p % 5;
    if (p == 15) {
      const uint32_t bits = ((w[0] >> 15) & 0x00010001u) | ((w[1] >> 14) & 0x00020002u) | ((w[2] >> 13) & 0x00040004u);
      q[u] = as_f16x2(bits | bias) - z.zb1;
    } else {
      const uint32_t v = j < 3 ? w[p / 5] : w[p / 5] >> 9;
      if (j % 3 == 0) q[u] = as_f16x2((v & 0x00070007u) | bias) - z.zb1;
      else if (j % 3 == 1) q[u] = __builtin_elementwise_fma(as_f16x2((v & 0x00380038u) | bias), eighth, z.nz128);
      else q[u] = __builtin_elementwise_fma(as_f16x2((v & 0x01C001C0u) | bias), sixty_fourth, z.nz16);
    }
  }
  return f16x8{q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
}

// Row of x that row i of the ragged batch reads.
__device__ inline int64_t x_row(const int32_t* __restrict__ rows, int i, int top_k, int64_t x_rows) {
  int64_t r = rows == nullptr ? i : rows[i] / top_k;
  return r < 0 ? 0 : (r < x_rows ? r : x_rows - 1);
}

// xs[i] = fp16(fp32(x of row i) / s of its expert), the input side of the
// per-channel scaling, and where `lo` is given what that rounding took off (0 of an
// infinity), rounded to fp16 too: one block per row of the ragged batch.
__global__ __launch_bounds__(256) void scale_rows_kernel(const f16* __restrict__ x, int64_t x_rows,
                                                         const int32_t* __restrict__ rows, int top_k,
                                                         const int32_t* __restrict__ offsets,
                                                         const float* __restrict__ s, int E, int R, int64_t K,
                                                         f16* __restrict__ xs, f16* __restrict__ lo) {
  const int i = (int)blockIdx.x;
  const RowTile t = find_tile(offsets, E, R, i, 1);
  if (t.rows == 0) return;
  const f16* src = x + x_row(rows, t.row, top_k, x_rows) * K;
  const float* sc = s + (int64_t)t.expert * K;
  f16* dst = xs + (int64_t)t.row * K;
  for (int64_t k = threadIdx.x * 8; k < K; k += 256 * 8) {
    const f16x8 v = *reinterpret_cast<const f16x8*>(src + k);
    f16x8 o, rest;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = (float)v[j] / sc[k + j];
      o[j] = (f16)q;
      const float r = q - (float)o[j];
      rest[j] = (f16)(fabsf(r) < INFINITY ? r : 0.f);
    }
    *reinterpret_cast<f16x8*>(dst + k) = o;
    if (lo != nullptr) *reinterpret_cast<f16x8*>(lo + (int64_t)t.row * K + k) = rest;
  }
}

// Bytes [at, at + len) of src into LDS, byte at + i at the returned offset + i
// of dst: whole 16-byte pieces of src by direct loads, the rest by plain ones.
// src is 16-byte aligned; `waves` waves share the work, and a direct load may
// not be waited for here.
__device__ __forceinline__ int stage_bytes(unsigned char* dst, const unsigned char* __restrict__ src, int64_t at,
                                           int64_t len, ScaleSwizzle sw, int waves, int wave,
                                           int lane, int tid) {
  const int skew = (int)(at & 15);
  src += at - skew;
  len += skew;
  const int64_t n16 = len / 16;
  if (tid < len - n16 * 16) dst[n16 * 16 + tid] = src[n16 * 16 + tid];
  __asm__ volatile("" ::: "memory");
  for (int64_t base = (int64_t)wave * 64; base < n16; base += 64 * waves) {
    const int64_t i = base + lane;
    if (i < n16)
      __builtin_amdgcn_global_load_lds((global_ptr_t)(src + 16 * sw.piece_src(i)),
                                       (lds_ptr_t)(dst + 16 * base), 16, 0, 0);
  }
  return skew;
}

// ---------------------------------------------------------------------------
// Few rows per expert (decoding): tiles of 16 rows x 16 RW weight rows, all of K
// per block, its 128-channel groups dealt to the block's waves in turn.  The
// kernel is bound by reading the weights once.  A wave owns a ring of S stages
// in LDS: a stage is one group of the weight rows (RW tiles of 16 rows x 64 or
// 48 bytes), moved there directly, S - 1 stages ahead, with the x fragments of
// that group in registers; the block's scales and zeros go to LDS once.  (Reading
// them and the weights row by row into registers instead asks the L1 for 16 lines
// per instruction, which alone takes longer than the memory: 20 us against 13
// below.)  The waves' tiles are summed through LDS in a fixed order.
// One token through 2 of 8 experts of 11008 x 4096: 47 MB in 13 us (3.6 TB/s); 45
// tokens x 6 over 64 3-bit experts of 2048 x 1408: 73 MB in 22 us (3.3 TB/s), 24 with a
// scaled x (PAIRS below), the vector ALU 28 % and the address units 57 % busy: latency.
// PAIRS: a scaled x of few rows is two fp16 numbers, the second at x + lo (x / s
// rounded to one adds an error of the size of y's own rounding, more where a few
// channels of few rows make most of the sums).  The tile is then 8 rows, the second
// numbers its rows 8 .. 15, and the two products of a row are added at the end.
template <int BITS, int RW, int S>
struct RingShape {
  static constexpr int NW = BITS == 4 ? RW : (3 * RW + 3) / 4;  // 1 KB loads of a stage
  static constexpr int STAGE = NW * 1024, LOADS = NW + 4;        // and the x fragment's four
  // scales and zeros, each with room for the bytes before them in their first 16
  static __host__ __device__ constexpr int scales_at(int waves) { return waves * S * STAGE; }
  static __host__ __device__ constexpr int zeros_at(int waves, int G) {
    return scales_at(waves) + (RW * 32 * G + 15 + 1024) / 1024 * 1024;
  }
  static __host__ __device__ constexpr int bytes(int waves, int G) {
    const int ring = zeros_at(waves, G) + (RW * 16 * ((G + 1) / 2) + 15 + 1024) / 1024 * 1024;
    const int sum = waves * 16 * (16 * RW + 1) * 4;  // the sum over the waves takes the rings' place
    return ring > sum ? ring : sum;
  }
};

template <int BITS, int RW, int S, bool PAIRS>
__global__ __launch_bounds__(512) void grouped_ring_kernel(
    const f16* __restrict__ x, int64_t lo, int64_t x_rows, const int32_t* __restrict__ rows, int top_k,
    const int32_t* __restrict__ offsets, const uint32_t* __restrict__ packed, const f16* __restrict__ scales,
    const uint8_t* __restrict__ zeros, f16* __restrict__ y, int R, int E, int64_t N, int64_t K, int nt, int waves) {
  using Q = RingShape<BITS, RW, S>;
  constexpr int kRows = PAIRS ? 8 : 16;  // of a tile
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int G = (int)(K / kGroup), P2 = (G + 1) / 2;
  const int lane = threadIdx.x & 63, nl = lane & 15, kq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mb = (int)blockIdx.x / nt;
  const RowTile tile = find_tile(offsets, E, R, mb, kRows);
  if (tile.rows == 0) return;
  const int64_t W = BITS == 4 ? K / 8 : 3 * (K / 32);
  const int64_t n0 = (int64_t)((int)blockIdx.x - mb * nt) * (16 * RW), first = (int64_t)tile.expert * N + n0;
  const int cols = N - n0 < 16 * RW ? (int)(N - n0) : 16 * RW;

  // Sources of this lane's 16-byte pieces, less the group's offset.  4 bits: piece
  // slot ^ (r / 4 % 4) of row r, so that 16 rows at one piece lie in all banks;
  // 3 bits: rows of three pieces back to back do so by themselves.  Rows past N
  // and past the tile repeat the last; they are never stored.
  const uint32_t* ws[Q::NW];
#pragma unroll
  for (int q = 0; q < Q::NW; ++q) {
    int r, word;
    if (BITS == 4) {
      r = 16 * q + (lane >> 2);
      word = 4 * ((lane & 3) ^ ((r >> 2) & 3));
    } else {
      const int pc = q * 64 + lane < 48 * RW ? q * 64 + lane : 48 * RW - 1;
      r = pc / 3;
      word = 4 * (pc % 3);
    }
    ws[q] = packed + (first + (r < cols ? r : cols - 1)) * W + word;
  }
  unsigned char* ring = smem + wave * (S * Q::STAGE);

  const ScaleSwizzle ssw(G);
  unsigned char* sl = smem + Q::scales_at(waves);
  unsigned char* zl = smem + Q::zeros_at(waves, G);
  sl += stage_bytes(sl, reinterpret_cast<const unsigned char*>(scales), first * G * 2, (int64_t)cols * G * 2,
                    ssw, waves, wave, lane, threadIdx.x);
  zl += stage_bytes(zl, zeros, first * P2, (int64_t)cols * P2, ScaleSwizzle(0), waves, wave, lane, threadIdx.x);
  const int xr = nl & (kRows - 1);
  const f16* xs = x + x_row(rows, tile.row + (xr < tile.rows ? xr : tile.rows - 1), top_k, x_rows) * K + kq * 32;
  if (PAIRS && nl >= kRows) xs += lo;
  struct Fragment {
    f16x8 a[4];
  };
  auto issue = [&](int g, int slot, Fragment& f) {
    g = g < G ? g : G - 1;  // past the last group: reloaded, not used
    unsigned char* st = ring + slot * Q::STAGE;
#pragma unroll
    for (int q = 0; q < Q::NW; ++q)
      __builtin_amdgcn_global_load_lds((global_ptr_t)(ws[q] + g * (4 * BITS)), (lds_ptr_t)(st + q * 1024), 16, 0, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) f.a[s] = *reinterpret_cast<const f16x8*>(xs + g * kGroup + 8 * s);
  };
  Fragment f[S];
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(wave + s * waves, s, f[s]);

  int row[RW], sx[RW];
#pragma unroll
  for (int t = 0; t < RW; ++t) {
    row[t] = 16 * t + nl < cols ? 16 * t + nl : cols - 1;
    sx[t] = ssw.xor_of(row[t]);
  }
  const uint32_t bias = bias_in_vgpr();
  f32x4 acc[RW];
#pragma unroll
  for (int t = 0; t < RW; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  wait_vmcnt<(S - 2) * Q::LOADS>();  // the scales and zeros (issued first), and the first stage
  lds_barrier();
  const int turns = (G - wave + waves - 1) / waves;  // stages of this wave
  for (int j0 = 0; j0 < turns; j0 += S)
#pragma unroll
    for (int u = 0; u < S; ++u) {  // slot u
      if (j0 + u >= turns) break;
      const int g = wave + (j0 + u) * waves;
      __builtin_amdgcn_s_waitcnt(0xC07F);  // this wave's LDS reads of the slot refilled now are done
      __builtin_amdgcn_sched_barrier(0);
      issue(g + (S - 1) * waves, (u + S - 1) % S, f[(u + S - 1) % S]);
      wait_vmcnt<(S - 1) * Q::LOADS>();
      __builtin_amdgcn_sched_barrier(0);
      const unsigned char* st = ring + u * Q::STAGE;
      uint32_t w[RW][BITS], z[RW];
      float sc[RW];
#pragma unroll
      for (int t = 0; t < RW; ++t) {
        if constexpr (BITS == 4) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(st + t * 1024 + nl * 64 + ((kq ^ ((nl >> 2) & 3)) << 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) w[t][i] = v[i];
        } else {
          const uint32_t* v = reinterpret_cast<const uint32_t*>(st + (16 * t + nl) * 48 + kq * 12);
#pragma unroll
          for (int i = 0; i < 3; ++i) w[t][i] = v[i];
        }
        z[t] = (zl[row[t] * P2 + (g >> 1)] >> (4 * (g & 1))) & 0xFu;
        sc[t] = (float)reinterpret_cast<const f16*>(sl)[row[t] * G + (g ^ sx[t])];
      }
#pragma unroll
      for (int t = 0; t < RW; ++t) {
        Zero<BITS> zf;
        zf.set(z[t]);
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[u].a[s], unpack8(w[t], s, bias, zf), d, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(sc[t], d[r], acc[t][r]);
      }
    }
  // the rings become the place of the sum: lane holds rows 4 kq + r of column 16 t + nl
  wait_vmcnt<0>();  // the reloads past the end have landed
  __syncthreads();
  constexpr int NC = 16 * RW, PITCH = NC + 1;
  float* red = reinterpret_cast<float*>(smem);  // [waves][16][PITCH]
#pragma unroll
  for (int t = 0; t < RW; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      red[(wave * 16 + 4 * kq + r) * PITCH + 16 * t + nl] = acc[t][r];
  __syncthreads();
  for (int i = threadIdx.x; i < tile.rows * NC; i += waves * 64) {
    const int m = i / NC, c = i - m * NC;
    float v = 0.f;
    for (int u = 0; u < waves; ++u) {
      v += red[(u * 16 + m) * PITCH + c];
      if (PAIRS) v += red[(u * 16 + m + kRows) * PITCH + c];
    }
    if (n0 + c < N) y[(int64_t)(tile.row + m) * N + n0 + c] = (f16)v;
  }
}

// ---------------------------------------------------------------------------
// Many rows per expert: output tiles of BM x 256 on the 32 x 32 x 16 matrix
// instructions.  Four waves side by side along N (times WMW along M) each own
// a 32 AB x 64 tile of it.  A stage is 64 channels (half a group): the x tile
// (rows gathered from x, BM x 128 bytes) and the packed weights (256 rows of 32
// or 24 bytes) go straight into an LDS ring, the tile's group scales and zeros
// once before the loop.  A weight fragment is unpacked by the wave that uses
// it, to the exact code - zero, and feeds AB matrix instructions.  The
// accumulators are kept in units of the current group's scale, in fp32: where a
// group begins they are multiplied by the ratio of the scales.  (Adding each half
// group's sum times its scale takes twice the vector instructions beside the
// unpacking: 1150 us against 1010 below; weights rounded to fp16 1092.)
// 6000 tokens x 2 of 8 experts of 11008 x 4096: 1.08e12 operations in 1010 us (1.07
// PFLOP/s; a plain fp16 product of 8192 cubed reaches 1.15 on this card), the
// matrix cores busy 56 % of the cycles of a clock that their power holds down.
constexpr int kGBN = 256, kGXcds = 8;

template <int BITS, int AB, int WMW, int STAGES>
struct GroupedShape {
  static constexpr int NW = 4 * WMW, BM = 32 * AB * WMW, JB = 2;
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = kGBN * (BITS == 4 ? 32 : 24);
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int XL = BM / 8 / NW;                     // x loads per wave per stage (1 KB each)
  static constexpr int WL = BITS == 4 ? B_BYTES / 1024 / NW : B_BYTES / 256 / NW;  // weight loads (1 KB / 256 B)
  static_assert(BM % (8 * NW) == 0 && XL >= 1 && WL >= 1, "tile rows must split over the waves");
  static constexpr int LOADS = XL + WL;
};

__host__ __device__ constexpr int64_t grouped_meta_bytes(int64_t G) {
  return ((int64_t)kGBN * G * 2 + 31) / 16 * 16 + ((int64_t)kGBN * ((G + 1) / 2) + 31) / 16 * 16;
}

// Word w of 32 channels whose codes all are z.
template <int BITS>
__device__ inline uint32_t zero_word(uint32_t z, int w) {
  if (BITS == 4) return z * 0x11111111u;
  return z * 0x12491249u + ((z >> w) & 1u) * 0x80008000u;  // five fields in either half, then bit w of the last pair
}

template <int BITS, int AB, int WMW, int STAGES>
__global__ __launch_bounds__(256 * WMW) void grouped_pipe_kernel(
    const f16* __restrict__ x, int64_t x_rows, const int32_t* __restrict__ rows, int top_k,
    const int32_t* __restrict__ offsets, const uint32_t* __restrict__ packed, const f16* __restrict__ scales,
    const uint8_t* __restrict__ zeros, f16* __restrict__ y, int R, int E, int64_t N, int64_t K, int nt, int tiles) {
  using S = GroupedShape<BITS, AB, WMW, STAGES>;
  constexpr int D = STAGES - 1;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, h = lane >> 5, l32 = lane & 31;

  // Blocks b, b + 8, ... run on one XCD and take runs of 16 tiles, n fastest.
  constexpr int kRun = 16;
  const int b = (int)blockIdx.x, xcd = b % kGXcds, i = b / kGXcds;
  const int t = (i / kRun * kGXcds + xcd) * kRun + i % kRun;
  if (t >= tiles) return;
  const int mb = t / nt, nb = t - mb * nt;
  const RowTile tile = find_tile(offsets, E, R, mb, S::BM);
  if (tile.rows == 0) return;

  const int G = (int)(K / kGroup), P2 = (G + 1) / 2;
  const int64_t W = BITS == 4 ? K / 8 : 3 * (K / 32);  // words per weight row
  const int64_t n0 = (int64_t)nb * kGBN, e0 = (int64_t)tile.expert * N;
  const int ncols = N - n0 < kGBN ? (int)(N - n0) : kGBN;

  // this lane's source of every load of a stage (rows past the tile's end repeat its last)
  const f16* xsrc[S::XL];
#pragma unroll
  for (int j = 0; j < S::XL; ++j) {
    const int r = (wave * S::XL + j) * 8 + (lane >> 3), chunk = (lane & 7) ^ ((r >> 1) & 7);
    const int64_t xr = x_row(rows, tile.row + (r < tile.rows ? r : tile.rows - 1), top_k, x_rows);
    xsrc[j] = x + xr * K + chunk * 8;
  }
  const uint32_t* wsrc[S::WL];
#pragma unroll
  for (int j = 0; j < S::WL; ++j) {
    int r, word;
    if (BITS == 4) {  // 32 rows of two 16-byte pieces per load
      r = (wave * S::WL + j) * 32 + (lane >> 1);
      word = 4 * ((lane & 1) ^ ((r >> 3) & 1));
    } else {  // 64 words of rows of six
      const int at = (wave * S::WL + j) * 64 + lane;
      r = at / 6;
      word = at - 6 * r;
    }
    wsrc[j] = packed + (e0 + n0 + (r < ncols ? r : ncols - 1)) * W + word;
  }
  const int last = 2 * G - 1;  // last stage
  auto issue = [&](int g, int slot) {
    g = g < last ? g : last;  // past the end: reloaded into a free slot, so every step issues the same loads
    unsigned char* st = smem + slot * S::STAGE;
#pragma unroll
    for (int j = 0; j < S::XL; ++j)
      __builtin_amdgcn_global_load_lds((global_ptr_t)(xsrc[j] + (int64_t)g * 64),
                                       (lds_ptr_t)(st + (wave * S::XL + j) * 1024), 16, 0, 0);
#pragma unroll
    for (int j = 0; j < S::WL; ++j) {
      if constexpr (BITS == 4)
        __builtin_amdgcn_global_load_lds((global_ptr_t)(wsrc[j] + (int64_t)g * 8),
                                         (lds_ptr_t)(st + S::A_BYTES + (wave * S::WL + j) * 1024), 16, 0, 0);
      else
        __builtin_amdgcn_global_load_lds((global_ptr_t)(wsrc[j] + (int64_t)g * 6),
                                         (lds_ptr_t)(st + S::A_BYTES + (wave * S::WL + j) * 256), 4, 0, 0);
    }
  };

  const ScaleSwizzle ssw(G);
  unsigned char* msc = smem + STAGES * S::STAGE;
  unsigned char* mz = msc + ((int64_t)kGBN * G * 2 + 31) / 16 * 16;
  msc += stage_bytes(msc, reinterpret_cast<const unsigned char*>(scales), (e0 + n0) * G * 2,
                            (int64_t)ncols * G * 2, ssw, S::NW, wave, lane, tid);
  mz += stage_bytes(mz, zeros, (e0 + n0) * P2, (int64_t)ncols * P2, ScaleSwizzle(0), S::NW, wave, lane, tid);
#pragma unroll
  for (int s = 0; s < D; ++s) issue(s, s);

  int mrow[S::JB], msx[S::JB];  // staged row of the lane's weight rows, its scale xor
#pragma unroll
  for (int j = 0; j < S::JB; ++j) {
    const int r = wn * 64 + j * 32 + l32;
    mrow[j] = r < ncols ? r : ncols - 1;
    msx[j] = ssw.xor_of(mrow[j]);
  }
  f32x16 acc[AB][S::JB];
#pragma unroll
  for (int a = 0; a < AB; ++a)
#pragma unroll
    for (int j = 0; j < S::JB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][j][r] = 0.f;
  const uint32_t magic = bias_in_vgpr();
  Zero<BITS> zf[S::JB];
  uint32_t zz[S::JB];
  bool empty[S::JB];
  float sc[S::JB] = {1.f, 1.f};  // scale of the group the accumulators are in units of
  const int blocks = (tile.rows + 31) / 32;  // 32-row blocks that hold a row; wave wm takes blocks wm, wm + WMW, ...

  // NA: the wave's row blocks that hold a row.  Every wave loads and meets the
  // barriers alike; which products it makes is settled outside the loop (a
  // branch around them inside it costs the accumulators their registers).
  auto multiply = [&](auto count) {
  constexpr int NA = decltype(count)::value;
  int cur = 0, nxt = D;
  for (int g = 0; g <= last; ++g) {
    wait_vmcnt<(D - 1) * S::LOADS>();  // stage g (and, at g = 0, the scales and zeros) has landed
    lds_barrier();                     // for every wave; stage g - 1 is no longer read
    issue(g + D, nxt);
    nxt = nxt + 1 == STAGES ? 0 : nxt + 1;
    const unsigned char* st = smem + cur * S::STAGE;
    cur = cur + 1 == STAGES ? 0 : cur + 1;
    const f16* At = reinterpret_cast<const f16*>(st);
    const unsigned char* Bt = st + S::A_BYTES;
    u32x4 wv[S::JB];
#pragma unroll
    for (int j = 0; j < S::JB; ++j) {
      const int r = wn * 64 + j * 32 + l32;
      if constexpr (BITS == 4) {
        wv[j] = *reinterpret_cast<const u32x4*>(Bt + r * 32 + ((h ^ ((r >> 3) & 1)) << 4));
      } else {
        const uint32_t* wp = reinterpret_cast<const uint32_t*>(Bt) + r * 6 + h * 3;
        wv[j] = u32x4{wp[0], wp[1], wp[2], 0u};
      }
    }
    if ((g & 1) == 0) {
      const int gr = g >> 1;
#pragma unroll
      for (int j = 0; j < S::JB; ++j) {
        zz[j] = (mz[mrow[j] * P2 + (gr >> 1)] >> (4 * (gr & 1))) & 0xFu;
        zf[j].set(zz[j]);
        const float was = sc[j], now = (float)reinterpret_cast<const f16*>(msc)[mrow[j] * G + (gr ^ msx[j])];
        sc[j] = now != 0.f ? now : was;
        empty[j] = now == 0.f;
        const float ratio = was * __builtin_amdgcn_rcpf(sc[j]);
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[a][j][r] *= ratio;
      }
    }
    // a group of scale 0 adds nothing: its codes become its zero point
    if (__ballot(empty[0] || empty[1])) {
#pragma unroll
      for (int j = 0; j < S::JB; ++j)
#pragma unroll
        for (int w = 0; w < (BITS == 4 ? 4 : 3); ++w) wv[j][w] = empty[j] ? zero_word<BITS>(zz[j], w) : wv[j][w];
    }
    auto unpack = [&](int s, f16x8(&bq)[S::JB]) {
#pragma unroll
      for (int j = 0; j < S::JB; ++j) {
        bq[j] = unpack8(wv[j], s, magic, zf[j]);
      }
    };
    f16x8 av[2][NA > 0 ? NA : 1], bq[2][S::JB];
#pragma unroll
    for (int a = 0; a < NA; ++a) av[0][a] = frag(At, (a * WMW + wm) * 32 + l32, 4 * h);
    if (NA > 0) unpack(0, bq[0]);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = s & 1, n = c ^ 1;
      if (s < 3) {
#pragma unroll
        for (int a = 0; a < NA; ++a) av[n][a] = frag(At, (a * WMW + wm) * 32 + l32, 4 * h + s + 1);
      }
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int j = 0; j < S::JB; ++j)
          acc[a][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av[c][a], bq[c][j], acc[a][j], 0, 0, 0);
      if (s < 3 && NA > 0) unpack(s + 1, bq[n]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  };
  const int mine = (blocks - wm + WMW - 1) / WMW;
  if (mine >= AB) multiply(std::integral_constant<int, AB>{});
  else if (AB > 3 && mine == 3) multiply(std::integral_constant<int, AB < 3 ? AB : 3>{});
  else if (AB > 2 && mine == 2) multiply(std::integral_constant<int, AB < 2 ? AB : 2>{});
  else if (AB > 1 && mine == 1) multiply(std::integral_constant<int, 1>{});
  else multiply(std::integral_constant<int, 0>{});
  wait_vmcnt<0>();  // the tail's reloads have landed before the block's LDS is given back

  // register r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
#pragma unroll
  for (int a = 0; a < AB; ++a)
#pragma unroll
    for (int j = 0; j < S::JB; ++j) {
      const int64_t n = n0 + wn * 64 + j * 32 + l32;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = (a * WMW + wm) * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
        if (m < tile.rows && n < N) y[(tile.row + m) * N + n] = (f16)(acc[a][j][r] * sc[j]);
      }
    }
}

// The most tiles of BM rows that R rows in E groups can make.
static int64_t row_tiles(int64_t R, int64_t E, int64_t BM) { return (R + (E < R ? E : R) * (BM - 1)) / BM; }

constexpr int64_t kGrpLds = 160 * 1024;

template <int BITS, int AB, int WMW, int STAGES>
static hipError_t pipe_stages(const f16* x, int64_t x_rows, const int32_t* rows, int top_k, const int32_t* offsets,
                              const void* packed, const void* scales, const void* zeros, void* y, int64_t R, int E,
                              int64_t N, int64_t K, hipStream_t st) {
  using S = GroupedShape<BITS, AB, WMW, STAGES>;
  const int64_t nt = (N + kGBN - 1) / kGBN, tiles = nt * row_tiles(R, E, S::BM);
  const size_t lds = (size_t)(STAGES * S::STAGE + grouped_meta_bytes(K / kGroup));
  const dim3 grid((unsigned)((tiles + 127) / 128 * 128)), block(256 * WMW);
  if (KernelPlan* p = active_plan())
    return plan_record(p, "grouped_pipe_kernel<%d,%d,%d,%d> block=%u grid=%u", BITS, AB, WMW, STAGES, block.x, grid.x);
  grouped_pipe_kernel<BITS, AB, WMW, STAGES><<<grid, block, lds, st>>>(
      x, x_rows, rows, top_k, offsets, reinterpret_cast<const uint32_t*>(packed), reinterpret_cast<const f16*>(scales),
      reinterpret_cast<const uint8_t*>(zeros), reinterpret_cast<f16*>(y), (int)R, E, N, K, (int)nt, (int)tiles);
  return hipGetLastError();
}

// Stages of the ring that leave LDS for the tile's scales and zeros (below 2: the tile cannot run).
template <int AB, int WMW>
static int pipe_stages_that_fit(int64_t G, int bits) {
  const int64_t stage = bits == 4 ? GroupedShape<4, AB, WMW, 2>::STAGE : GroupedShape<3, AB, WMW, 2>::STAGE;
  const int64_t n = (kGrpLds - grouped_meta_bytes(G)) / stage;
  return n < 3 ? (int)n : 3;
}

template <int BITS, int AB, int WMW>
static hipError_t pipe_launch(const f16* x, int64_t, int64_t x_rows, const int32_t* rows, int top_k, const int32_t* offsets,
                              const void* packed, const void* scales, const void* zeros, void* y, int64_t R, int E,
                              int64_t N, int64_t K, hipStream_t st) {
  if (pipe_stages_that_fit<AB, WMW>(K / kGroup, BITS) == 3)
    return pipe_stages<BITS, AB, WMW, 3>(x, x_rows, rows, top_k, offsets, packed, scales, zeros, y, R, E, N, K, st);
  return pipe_stages<BITS, AB, WMW, 2>(x, x_rows, rows, top_k, offsets, packed, scales, zeros, y, R, E, N, K, st);
}

template <int BITS, int RW>
static hipError_t ring_launch(const f16* x, int64_t lo, int64_t x_rows, const int32_t* rows, int top_k, const int32_t* offsets,
                              const void* packed, const void* scales, const void* zeros, void* y, int64_t R, int E,
                              int64_t N, int64_t K, hipStream_t st) {
  constexpr int S = 2;  // deeper rings cost blocks per compute unit: 3 and 4 stages were 2 .. 30 % slower
  const int G = (int)(K / kGroup);
  const int64_t nt = (N + 16 * RW - 1) / (16 * RW), blocks = nt * row_tiles(R, E, lo ? 8 : 16);
  // Waves per block: ten for each compute unit in all, or eight a block.  One token through 2 of 8
  // experts of 11008 x 4096: 17.2, 14.8, 12.6, 13.1 us with 1, 2, 4, 8; 45 tokens x 6 over 64 3-bit
  // experts of 2048 x 1408: 23.0, 23.5, 30.0, 36.7 us.
  int waves = 1;
  while (waves < 8 && 2 * waves <= G && blocks * waves < 2500) waves *= 2;
  if (KernelPlan* p = active_plan())
    return plan_record(p, "grouped_ring_kernel<%d,%d,%d> block=%d grid=%lld", BITS, RW, S, 64 * waves, (long long)blocks);
  auto kernel = lo ? grouped_ring_kernel<BITS, RW, S, true> : grouped_ring_kernel<BITS, RW, S, false>;
  kernel<<<dim3((unsigned)blocks), dim3(64 * waves), RingShape<BITS, RW, S>::bytes(waves, G), st>>>(
      x, lo, x_rows, rows, top_k, offsets, reinterpret_cast<const uint32_t*>(packed),
      reinterpret_cast<const f16*>(scales), reinterpret_cast<const uint8_t*>(zeros), reinterpret_cast<f16*>(y), (int)R, E,
      N, K, (int)nt, waves);
  return hipGetLastError();
}

// Which kernel, by the rows an expert has on average (the sizes themselves are
// on the device).  Measured over E = 8, 16, 64 experts of 2048 x 1408 (3 bits),
// 2048 x 2048, 11008 x 4096, 4096 x 11008 and 1000 x 4096 at 0.25 .. 700 rows an
// expert (us):
//   ring kernel, 4 weight tiles a wave against 2: 11.6 / 9.7, 17.4 / 15.4, 20.7 /
//     16.3 at 0.25 rows; 28.9 / 34.5, 26.1 / 28.7 at 1; 55 / 66, 72 / 86 at 16
//   ring against 64-row tiles: 43 / 41, 55 / 65, 50 / 101 at 8; 55 / 43, 72 / 63
//     at 16, but 69 / 101 and 19 / 38 where 256-column tiles are fewer than the
//     compute units (4096 x 11008, 8 experts; 1000 x 4096, 16), which at 32 is
//     122 / 114 and 26 / 48
//   64-row tiles against 256-row ones: 112 / 130, 154 / 180 at 128; 186 / 192,
//     252 / 281, 346 / 273 at 256; 465 / 429, 603 / 545, 718 / 566 at 700
enum class Kernel { ring2, ring4, rows64, rows256 };

static Kernel grouped_choice(int64_t R, int64_t E, int64_t N, int64_t K, int bits) {
  const int64_t G = K / kGroup, nt = (N + kGBN - 1) / kGBN;
  const bool few = R <= 10 * E || (R <= 40 * E && nt * E < 256);
  if (!few && R >= 384 * E && pipe_stages_that_fit<4, 2>(G, bits) >= 2) return Kernel::rows256;
  if (!few && pipe_stages_that_fit<2, 1>(G, bits) >= 2) return Kernel::rows64;
  return R > E && RingShape<4, 4, 2>::bytes(8, (int)G) <= kGrpLds ? Kernel::ring4 : Kernel::ring2;
}

// Whether a scaled x is two fp16 numbers, in tiles of half as many rows.  One number's rounding is
// as large an error as that of y (2.9e-4 of it in all, against 2.1e-4 with two).  Two cost, over the
// shapes above, 3 to 5 % at one row an expert, 4 to 6 at two, 7 to 19 at four (45 tokens x 6 over 64
// 3-bit experts of 2048 x 1408: 25.5 -> 28.6 us), 12 to 23 at five, 18 to 37 at seven, and the pipelined
// kernel would make every product twice: up to five rows an expert x / s enters with 22 bits,
// beyond rounded as awq_scale_input rounds it.  (Two numbers of more than 2048 rows have no room
// in the workspace.)
static bool paired(Kernel choice, int64_t R, int64_t E) {
  return (choice == Kernel::ring2 || choice == Kernel::ring4) && R <= 2 * AWQ_MAX_EXPERTS && (R <= 5 * E || R <= 16);
}

// Whether the chosen kernel's grid (2^32 threads at most) covers the batch.
bool gemm_grouped_fits(int64_t R, int64_t E, int64_t N, int64_t K, int bits, bool scaled) {
  if (scaled && R >= (int64_t(1) << 24)) return false;  // a block of 256 threads per row
  const int64_t nt = (N + kGBN - 1) / kGBN;
  const Kernel choice = grouped_choice(R, E, N, K, bits);
  const int64_t ring = row_tiles(R, E, scaled && paired(choice, R, E) ? 8 : 16);
  switch (choice) {
    case Kernel::ring2: return (N + 31) / 32 * ring < (int64_t(1) << 23);
    case Kernel::ring4: return (N + 63) / 64 * ring < (int64_t(1) << 23);
    case Kernel::rows64: return nt * row_tiles(R, E, 64) + 127 < (int64_t(1) << 24);
    case Kernel::rows256: return nt * row_tiles(R, E, 256) + 127 < (int64_t(1) << 23);
  }
  return false;
}

hipError_t launch_gemm_grouped(const void* x, int64_t x_rows, const int32_t* rows, int top_k, const int32_t* offsets,
                               const float* s, const void* packed, const void* scales, const void* zeros, void* y,
                               int64_t R, int E, int64_t N, int64_t K, int bits, void* ws, hipStream_t st) {
  const f16* xp = reinterpret_cast<const f16*>(x);
  const Kernel choice = grouped_choice(R, E, N, K, bits);
  int64_t lo = 0;  // elements from x to the second halves of a scaled one
  if (s != nullptr && active_plan() == nullptr) {
    f16* xs = reinterpret_cast<f16*>(ws);
    if (paired(choice, R, E)) lo = R * K;
    scale_rows_kernel<<<dim3((unsigned)R), dim3(256), 0, st>>>(xp, x_rows, rows, top_k, offsets, s, E, (int)R, K, xs,
                                                               lo ? xs + lo : nullptr);
    if (hipError_t e = hipGetLastError()) return e;
    xp = xs;
    x_rows = R;
    rows = nullptr;
  }
#define AWQ_GROUPED(launch, ...)                                                                          \
  return bits == 4                                                                                        \
             ? launch<4, __VA_ARGS__>(xp, lo, x_rows, rows, top_k, offsets, packed, scales, zeros, y, R, E, N, K, st) \
             : launch<3, __VA_ARGS__>(xp, lo, x_rows, rows, top_k, offsets, packed, scales, zeros, y, R, E, N, K, st)
  switch (choice) {
    case Kernel::ring2: AWQ_GROUPED(ring_launch, 2);
    case Kernel::ring4: AWQ_GROUPED(ring_launch, 4);
    case Kernel::rows64: AWQ_GROUPED(pipe_launch, 2, 1);
    case Kernel::rows256: AWQ_GROUPED(pipe_launch, 4, 2);
  }
#undef AWQ_GROUPED
  return hipErrorInvalidValue;
}

}  // namespace awq
