// The product in 8-bit integers: y = (x codes) (w codes)^T in exact 32-bit sums,
// times a scale for each token and each channel.
//
// Tile kernel: BM tokens x BN channels a block, K in stages of 2 W bytes (128, a whole
// line, where the weights come from memory: 32 x 50021 x 4096 49.6 us, 56.0 with 64;
// 64 for the largest tiles, whose stages would not fit).  Stages go from global memory
// straight into a ring of LDS buffers (the layouts of mfma_pipe.h, a pair of codes in
// the place of a half) and feed v_mfma_i32_32x32x32_i8.  A stage's first fragments are read before the barrier
// that opens it, so the matrix cores do not wait for the barrier or the LDS: the
// barrier of stage s only says that stage s + 1 has landed and stage s - 1 is free.
// The weights are the A operand, so a lane's accumulators hold four consecutive
// channels of one token; the results are turned over through LDS and stored as
// whole rows.
// Many tokens are bound by the matrix cores and the power they may take: 8192 x 28672
// x 8192 1.65 to 1.71 ms, 2250 to 2330 TOP/s (the library's product of 8192 cubed: 2080),
// the matrix cores busy for 60 % of the cycles at the 1.8 GHz that is left.  Waves of
// 128 tokens x 64 channels, 2 x 4 of them: 1645 us; 4 x 2 of 64 x 128 1688; four of
// 128 x 128 1860.  Few tokens are bound by the weights' one read: 32 x 50021 x 4096
// 50 us, 4.1 TB/s (a read alone: 6.3; 391 blocks for 256 units); 77 x 4096 x 11008 with 7 shares of K
// 14.3 us and 4 for their join, of which a block's start and end are the larger part (6 and 8 shares take as long).
#include <cmath>

#include "awq_internal.h"
#include "mfma_pipe.h"
#include "row_common.h"

namespace awq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

// A sum with its scales, rounded at each step.  The empty asm keeps the last product a number of its own:
// joined with the rounding to fp16 into one instruction it would be rounded once less, in some kernels.
template <typename Y>
__device__ __forceinline__ Y scaled(int32_t sum, float token, float channel) {
  float v = (float)sum * token * channel;
  __asm__("" : "+v"(v));
  return (Y)v;
}

struct I8Args {
  const int8_t* x;
  const float* xs;
  const int8_t* w;
  const float* ws;
  void* y;
  int64_t M, N, K;
  const float* s;     // input scales, where x is fp16
  int mtiles, ntiles, splits;
  int32_t* partial;   // [splits][M][partial_pitch(N)] sums of each share of K, where splits > 1
};
static __host__ __device__ constexpr int64_t partial_pitch(int64_t N) { return (N + 3) / 4 * 4; }

// Block b's tile.  Blocks are dispatched to the 8 XCDs in turn; each XCD takes a run of
// tiles, in groups of up to 8 token tiles by all channel tiles, so that the blocks of an XCD
// share panels of both operands in its L2.
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(int b, int mtiles, int ntiles) {
  const int tiles = mtiles * ntiles, per = tiles / 8, more = tiles % 8, xcd = b % 8, i = b / 8;
  const int t = xcd * per + (xcd < more ? xcd : more) + i;
  const int group = t / (8 * ntiles), in = t - group * 8 * ntiles;
  const int rows = mtiles - group * 8 < 8 ? mtiles - group * 8 : 8;
  return {group * 8 + in % rows, in / rows};
}

template <int BM, int BN, int WM, int WN, int STAGES, int W>
struct I8Shape {
  static constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, AM = TM / 32, AN = TN / 32;
  static constexpr int SUB = W / 16;            // matrix instructions along K of a stage
  static constexpr int STAGE = (BM + BN) * W;   // halfs
  static constexpr int LOADS = (BM + BN) * W / 512 / NW;
  static constexpr int PITCH = TN + 4;          // words of a row of the turned-over tile (fp32; fp16 uses half)
  static constexpr int RING = STAGES * STAGE * 2, TURN = NW * 32 * PITCH * 4;
  static constexpr int LDS = RING > TURN ? RING : TURN;
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <int BM, int BN, int WM, int WN, int STAGES, int W, typename Y>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_kernel(I8Args a) {
  typedef I8Shape<BM, BN, WM, WN, STAGES, W> S;
  constexpr int AM = S::AM, AN = S::AN;
  __shared__ __align__(16) unsigned char lds[S::LDS];
  f16* ring = reinterpret_cast<f16*>(lds);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tiles = a.mtiles * a.ntiles, share = blockIdx.x / tiles;
  const TileAt at = tile_at(blockIdx.x - share * tiles, a.mtiles, a.ntiles);
  const int64_t m0 = (int64_t)at.m * BM, n0 = (int64_t)at.n * BN;
  const int wm = (wave % WM) * S::TM, wn = (wave / WM) * S::TN;
  TilePlan<BM, S::NW, W> px;
  TilePlan<BN, S::NW, W> pw;
  px.init(reinterpret_cast<const f16*>(a.x), a.K / 2, m0, a.M, wave, lane);
  pw.init(reinterpret_cast<const f16*>(a.w), a.K / 2, n0, a.N, wave, lane);
  const int all = (int)(a.K / (2 * W)), first = (int)((int64_t)all * share / a.splits);
  const int steps = (int)((int64_t)all * (share + 1) / a.splits) - first;  // splits <= all
  auto issue = [&](int s) {
    f16* stage = ring + (s % STAGES) * S::STAGE;
    const int64_t k = (int64_t)(first + (s < steps ? s : steps - 1)) * W;  // past the end: counted, never used
    px.issue(stage, k);
    pw.issue(stage + BM * W, k);
  };
  i32x16 acc[AN][AM];
#pragma unroll
  for (int i = 0; i < AN; ++i)
#pragma unroll
    for (int j = 0; j < AM; ++j) acc[i][j] = i32x16{};
  i32x4 fa[2][AN], fb[2][AM];
  auto piece = [](const f16* tile, int r, int c) {
    return __builtin_bit_cast(i32x4, W == 32 ? frag32(tile, r, c) : frag(tile, r, c));
  };
  auto read = [&](int s, int c, int into) {
    const f16* tx = ring + (s % STAGES) * S::STAGE;
    const f16* tw = tx + BM * W;
#pragma unroll
    for (int i = 0; i < AN; ++i)
      fa[into][i] = piece(tw, wn + i * 32 + (lane & 31), 2 * c + (lane >> 5));
#pragma unroll
    for (int j = 0; j < AM; ++j)
      fb[into][j] = piece(tx, wm + j * 32 + (lane & 31), 2 * c + (lane >> 5));
  };
  auto multiply = [&](int from) {
#pragma unroll
    for (int i = 0; i < AN; ++i)
#pragma unroll
      for (int j = 0; j < AM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[from][i], fb[from][j], acc[i][j], 0, 0, 0);
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s);
  wait_vmcnt<(STAGES - 2) * S::LOADS>();
  lds_barrier();
  read(0, 0, 0);
  for (int s = 0; s < steps; ++s) {
    wait_vmcnt<(STAGES - 3) * S::LOADS>();  // stage s + 1
    lds_barrier();
    issue(s + STAGES - 1);  // into stage s - 1
#pragma unroll
    for (int c = 0; c < S::SUB; ++c) {
      if (c + 1 < S::SUB) read(s, c + 1, (c + 1) & 1);
      else read(s + 1, 0, 0);
      multiply(c & 1);
    }
  }
  wait_vmcnt<0>();  // the loads past the end
  lds_barrier();

  // each wave turns its tile over, 32 tokens at a time
  float* turn = reinterpret_cast<float*>(lds) + wave * 32 * S::PITCH;
  Y* turn_y = reinterpret_cast<Y*>(turn);
  constexpr int PITCH = sizeof(Y) == 4 ? S::PITCH : 2 * S::PITCH;  // elements
  constexpr int PER = 16 / sizeof(Y), LANES = S::TN / PER, ROWS = 64 / LANES;
  constexpr bool kPartial = __is_same(Y, int32_t);
  const int64_t pitch = kPartial ? partial_pitch(a.N) : a.N;
  Y* y = kPartial ? reinterpret_cast<Y*>(a.partial) + share * a.M * pitch : reinterpret_cast<Y*>(a.y);
  const bool whole = pitch % PER == 0 && n0 + wn + S::TN <= a.N;
#pragma unroll
  for (int j = 0; j < AM; ++j) {
    const int64_t mj = m0 + wm + j * 32, m = mj + (lane & 31);
    float sm = 0.f;
    if constexpr (!kPartial) sm = a.xs[m < a.M ? m : a.M - 1];
#pragma unroll
    for (int i = 0; i < AN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        typedef Y yx4 __attribute__((ext_vector_type(4)));
        const int n = i * 32 + 8 * q + 4 * (lane >> 5);
        yx4 v;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t ng = n0 + wn + n + u;
          if constexpr (kPartial) v[u] = acc[i][j][4 * q + u];
          else v[u] = scaled<Y>(acc[i][j][4 * q + u], sm, a.ws[ng < a.N ? ng : a.N - 1]);
        }
        *reinterpret_cast<yx4*>(turn_y + (lane & 31) * PITCH + n) = v;
      }
    __asm__ volatile("" ::: "memory");  // the wave's own tile: its LDS accesses are done in order
    if (whole) {
#pragma unroll
      for (int r = 0; r < 32; r += ROWS) {
        const int row = r + lane / LANES, n = (lane % LANES) * PER;
        const u32x4 v = *reinterpret_cast<const u32x4*>(turn_y + row * PITCH + n);
        if (mj + row < a.M) *reinterpret_cast<u32x4*>(y + (mj + row) * pitch + n0 + wn + n) = v;
      }
    } else {
      for (int r = 0; r < 32; ++r)
        for (int n = lane; n < S::TN; n += 64)
          if (mj + r < a.M && n0 + wn + n < a.N) y[(mj + r) * pitch + n0 + wn + n] = turn_y[r * PITCH + n];
    }
    __asm__ volatile("" ::: "memory");
  }
}

// The shares' sums joined, scaled and rounded: four channels of a token a thread.
template <typename Y>
__global__ __launch_bounds__(256) void gemm_i8_join_kernel(I8Args a) {
  const int64_t pitch = partial_pitch(a.N), per = pitch / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * per) return;
  const int64_t m = i / per, n = (i - m * per) * 4;
  i32x4 v = {};
  for (int s = 0; s < a.splits; ++s) v += *reinterpret_cast<const i32x4*>(a.partial + (s * a.M + m) * pitch + n);
  const float sm = a.xs[m];
  typedef Y yx4 __attribute__((ext_vector_type(4)));
  Y* y = reinterpret_cast<Y*>(a.y) + m * a.N + n;
  yx4 o;
#pragma unroll
  for (int u = 0; u < 4; ++u) o[u] = scaled<Y>(v[u], sm, a.ws[n + u < a.N ? n + u : a.N - 1]);
  if (a.N % 4 == 0) *reinterpret_cast<yx4*>(y) = o;
  else
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (n + u < a.N) y[u] = o[u];
}

// Few tokens: a block takes 16 channels at a time (gridDim.x groups apart), its NW waves every NW-th
// 128 bytes of K, and their sums are joined through LDS.  A lane of v_mfma_i32_16x16x64_i8 holds 16 bytes
// of one of 16 rows: lane l reads row l % 16, bytes 16 (l / 16) on of each half of a chunk, so four lanes read
// 64 bytes side by side and both operands agree on the order of K.  Bound by the weights' one read: DEPTH chunks
// of a wave are under way while DEPTH are multiplied, across the groups' ends; TT tiles of 16 tokens come
// from the caches again for every group.
// FUSED: x is one fp16 row, which each block quantises to LDS itself (one launch instead of two), while its
// first weights are under way.  11008 x 4096: 15.4 us with the row's codes (28 with a launch for them and without DEPTH), 12.0
// for a row that is in 8 bits already; a bare kernel's read of these 45 MB that ends each block with a store takes 8.7.
// Open: more than one batch of weights under way while the row is quantised, and blocks of equal numbers of
// groups (688 of them on 256 units).  24 tokens x 4096 x 4096: 8.2 us.
template <int TT, int NW, int DEPTH, bool FUSED, typename Y>
__global__ __launch_bounds__(64 * NW) void gemm_i8_skinny_kernel(I8Args a) {
  extern __shared__ __align__(16) unsigned char rows[];  // FUSED: the row's codes
  __shared__ i32x4 sums[2][NW][TT][64];
  __shared__ float part[NW];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int chunks = (int)(a.K / 128), groups = (int)((a.N + 15) / 16), M = (int)a.M;
  const int row = lane & 15, off = (lane >> 4) * 16;
  const int batches = (chunks + NW * DEPTH - 1) / (NW * DEPTH);
  struct Batch {
    i32x4 w[DEPTH][2], x[FUSED ? 1 : TT][FUSED ? 1 : DEPTH][2];
  };
  int token[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) token[t] = t * 16 + row < M ? t * 16 + row : M - 1;  // the others' sums are not stored
  auto chunk = [&](int b, int d) { return wave + (b * DEPTH + d) * NW; };
  auto fetch = [&](int g, int b, Batch& to) {
    const int64_t n = (int64_t)g * 16 + row;
    const int8_t* w = a.w + (n < a.N ? n : a.N - 1) * a.K + off;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int c = chunk(b, d);
      if (c >= chunks) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        to.w[d][h] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(w + (int64_t)c * 128) + 4 * h);
      if constexpr (!FUSED)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            to.x[t][d][h] = reinterpret_cast<const i32x4*>(a.x + (int64_t)token[t] * a.K + (int64_t)c * 128 + off)[4 * h];
    }
  };
  Batch cur, next;
  int g = blockIdx.x, b = 0, buffer = 0;
  fetch(g, 0, cur);
  float top = 0.f;
  if constexpr (FUSED) {
    const f16* x = reinterpret_cast<const f16*>(a.x);
    auto values = [&](int k) {
      const f32x8 v = widen(*reinterpret_cast<const f16x8*>(x + k));
      return a.s ? v / *reinterpret_cast<const f32x8*>(a.s + k) : v;
    };
    float most = 0.f;
    for (int k = threadIdx.x * 8; k < (int)a.K; k += 512 * NW) most = largest_of(most, values(k));
    most = row_join<64 * NW>(most, part, MaxOp());
    top = most;
    const float by = 127.f / most;
    for (int k = threadIdx.x * 8; k < (int)a.K; k += 512 * NW) {
      const f32x8 v = values(k);
      float c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] = code_of(v[u], by, most);
      *reinterpret_cast<u32x2*>(rows + k) = u32x2{code_word(c[0], c[1], c[2], c[3]), code_word(c[4], c[5], c[6], c[7])};
    }
    lds_barrier();
  }
  i32x4 acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = i32x4{};
  while (g < groups) {
    const bool last = b + 1 == batches;
    const int g2 = last ? g + (int)gridDim.x : g, b2 = last ? 0 : b + 1;
    if (g2 < groups) fetch(g2, b2, next);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (chunk(b, d) < chunks) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            i32x4 xv;
            if constexpr (FUSED)
              xv = reinterpret_cast<const i32x4*>(rows + chunk(b, d) * 128 + off)[4 * h];
            else xv = cur.x[t][d][h];
            acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(cur.w[d][h], xv, acc[t], 0, 0, 0);
          }
      }
    if (last) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        sums[buffer][wave][t][lane] = acc[t];
        acc[t] = i32x4{};
      }
      lds_barrier();
      // tile t's sums by wave t, four channels of a token a lane; the buffers are taken in turn, and the next
      // group's barrier comes after these reads
      if (wave < TT) {
        i32x4 v = sums[buffer][0][wave][lane];
#pragma unroll
        for (int i = 1; i < NW; ++i) v += sums[buffer][i][wave][lane];
        const int m = wave * 16 + row;
        const int64_t n = (int64_t)g * 16 + 4 * (lane >> 4);
        if (m < M) {
          const float sm = FUSED ? top / 127.f : a.xs[m];
          typedef Y yx4 __attribute__((ext_vector_type(4)));
          Y* y = reinterpret_cast<Y*>(a.y) + (int64_t)m * a.N + n;
          yx4 o;
#pragma unroll
          for (int u = 0; u < 4; ++u) o[u] = scaled<Y>(v[u], sm, a.ws[n + u < a.N ? n + u : a.N - 1]);
          if (n + 4 <= a.N && a.N % 4 == 0) *reinterpret_cast<yx4*>(y) = o;
          else
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (n + u < a.N) y[u] = o[u];
        }
      }
      buffer ^= 1;
    }
    cur = next;
    g = g2;
    b = b2;
  }
}

static size_t rows_bytes(int64_t M, int64_t K) { return ((size_t)M * (size_t)K + 255) / 256 * 256; }

// One fp16 row is quantised by the product itself, up to this many codes (its LDS).
static bool i8_fused(int64_t M, int64_t K, bool quantized) { return !quantized && M == 1 && K <= 32768; }

// The kernel for these sizes: the one of least estimated time, in us.  The numbers are fitted to 1300
// times measured on an MI355X with the weights out of the caches, over N x K = 700 x 512 .. 50021 x 4096
// and 28672 x 8192, M = 1 .. 5000; the kernel picked is on average 2 % slower than the best.  E.g.
//   8 x 4096 x 4096:   few tokens' kernel 6.1, 32 x 64 tiles with 4 shares 10.0
//   32 x 50021 x 4096: few tokens' kernel 82, 32 x 128 tiles 49.6, 64 x 128 52.7
//   77 x 4096 x 11008: 64 x 64 tiles with 4 shares 20.5, 128 x 128 with 6 to 8 20, with 1 share 38
//   512 x 28672 x 8192: 256 x 256 tiles 135, 128 x 128 168
struct I8Plan {
  int tile;    // index of kI8Tiles; -1: the kernel for few tokens
  int splits;  // shares of K
};
struct I8Tile {
  int tokens, channels;
  double start, step;  // before the first and after the last stage; 128 bytes of K
};
constexpr I8Tile kI8Tiles[] = {{32, 64, 5.0, 0.28},   {32, 128, 4.6, 0.48},  {64, 64, 5.7, 0.32},
                               {64, 128, 6.4, 0.60}, {128, 128, 6.4, 0.68}, {256, 256, 9.0, 1.85}};
static I8Plan i8_estimate(int64_t M, int64_t N, int64_t K, bool quantized) {
  const double weights = (double)N * (double)K * 1e-6;  // MB, streamed at TB/s
  I8Plan best{-1, 1};
  double least = 1e30;
  if (M <= 64)  // the rows' codes come from the L2 once for each 16 channels
    least = 4.3 + fmax(weights / (M <= 8 ? 4.5 : M <= 16 ? 3.9 : M <= 32 ? 3.2 : 1.85),
                       (double)K / 1024 * 0.44 * (M <= 16 ? 1 : M <= 32 ? 2 : 4));
  const double rows = i8_fused(M, K, quantized) ? 3.0 : 0.0;  // the rows' own launch, which that kernel saves
  const int64_t steps = K / 128;
  for (int i = 0; i < (int)(sizeof(kI8Tiles) / sizeof(kI8Tiles[0])); ++i) {
    const I8Tile& t = kI8Tiles[i];
    const int64_t tiles = ((M + t.tokens - 1) / t.tokens) * ((N + t.channels - 1) / t.channels);
    for (int splits = 1; splits == 1 || (splits <= 8 && splits * 2 <= steps && tiles * splits <= 1024); ++splits) {
      // blocks of a compute unit one after the other; small ones share it more evenly
      const double blocks = (double)(tiles * splits) / 256.0;
      const double rounds = t.tokens == 256 ? ceil(blocks) : blocks <= 1.0 ? 1.0 : blocks + 0.3;
      double us = rows + t.start + fmax(weights / 4.7, rounds * (double)((steps + splits - 1) / splits) * t.step);
      if (splits > 1) us += 1.6 + 0.21 * (double)splits * (double)M * (double)N * 8e-6;  // the join
      if (us < least) {
        least = us;
        best = {i, splits};
      }
    }
  }
  return best;
}

// A call asks twice, for its workspace and for its launch.
static I8Plan i8_plan(int64_t M, int64_t N, int64_t K, bool quantized) {
  struct Last {
    int64_t M, N, K;
    bool quantized;
    I8Plan plan;
  };
  static thread_local Last last{0, 0, 0, false, {-1, 1}};
  if (last.M != M || last.N != N || last.K != K || last.quantized != quantized)
    last = {M, N, K, quantized, i8_estimate(M, N, K, quantized)};
  return last.plan;
}

size_t gemm_i8_workspace(int64_t M, int64_t N, int64_t K, bool quantized) {
  const I8Plan plan = i8_plan(M, N, K, quantized);
  size_t bytes = plan.splits > 1 ? (size_t)plan.splits * (size_t)M * (size_t)partial_pitch(N) * 4 : 0;
  if (!quantized && !(plan.tile < 0 && i8_fused(M, K, quantized)))
    bytes += rows_bytes(M, K) + ((size_t)M * 4 + 255) / 256 * 256;
  return (bytes + 255) / 256 * 256;
}

template <int BM, int BN, int WM, int WN, int STAGES, int W>
static hipError_t tile_launch(I8Args a, int y_bytes, hipStream_t st) {
  if (a.splits < 1 || a.splits > a.K / (2 * W)) return hipErrorInvalidValue;  // a share has a stage at least
  a.mtiles = (int)((a.M + BM - 1) / BM);
  a.ntiles = (int)((a.N + BN - 1) / BN);
  const dim3 grid((unsigned)(a.mtiles * a.ntiles * a.splits)), block(64 * WM * WN);
  if (KernelPlan* p = active_plan())
    return plan_record(p, "gemm_i8_kernel<%d,%d,%d,%d,%d,%d> block=%u grid=%u shares=%d", BM, BN, WM, WN, STAGES, W, block.x,
                       grid.x, a.splits);
  if (a.splits > 1) {
    gemm_i8_kernel<BM, BN, WM, WN, STAGES, W, int32_t><<<grid, block, 0, st>>>(a);
    const dim3 join((unsigned)((a.M * (partial_pitch(a.N) / 4) + 255) / 256));
    if (y_bytes == 2) gemm_i8_join_kernel<f16><<<join, dim3(256), 0, st>>>(a);
    else gemm_i8_join_kernel<float><<<join, dim3(256), 0, st>>>(a);
  } else if (y_bytes == 2) {
    gemm_i8_kernel<BM, BN, WM, WN, STAGES, W, f16><<<grid, block, 0, st>>>(a);
  } else {
    gemm_i8_kernel<BM, BN, WM, WN, STAGES, W, float><<<grid, block, 0, st>>>(a);
  }
  return hipGetLastError();
}

template <int TT, int NW, int DEPTH, bool FUSED>
static hipError_t skinny_launch(const I8Args& a, int y_bytes, int per_cu, hipStream_t st) {
  const int64_t groups = (a.N + 15) / 16, most = 256 * per_cu;
  const dim3 grid((unsigned)(groups < most ? groups : most)), block(64 * NW);
  const size_t lds = FUSED ? (size_t)a.K : 0;
  if (KernelPlan* p = active_plan())
    return plan_record(p, "gemm_i8_skinny_kernel<%d,%d,%d,%d> block=%u grid=%u", TT, NW, DEPTH, (int)FUSED, block.x, grid.x);
  if (y_bytes == 2) gemm_i8_skinny_kernel<TT, NW, DEPTH, FUSED, f16><<<grid, block, lds, st>>>(a);
  else gemm_i8_skinny_kernel<TT, NW, DEPTH, FUSED, float><<<grid, block, lds, st>>>(a);
  return hipGetLastError();
}

static hipError_t skinny_dispatch(const I8Args& a, bool fused, int y_bytes, hipStream_t st) {
  const bool narrow = a.N <= 16 * 512;  // few groups: more waves on each
  if (fused) return narrow ? skinny_launch<1, 8, 4, true>(a, y_bytes, 2, st) : skinny_launch<1, 4, 4, true>(a, y_bytes, 4, st);
  if (a.M <= 16) return narrow ? skinny_launch<1, 8, 4, false>(a, y_bytes, 2, st) : skinny_launch<1, 4, 4, false>(a, y_bytes, 4, st);
  if (a.M <= 32) return narrow ? skinny_launch<2, 8, 2, false>(a, y_bytes, 2, st) : skinny_launch<2, 4, 2, false>(a, y_bytes, 4, st);
  return narrow ? skinny_launch<4, 8, 2, false>(a, y_bytes, 2, st) : skinny_launch<4, 4, 2, false>(a, y_bytes, 4, st);
}

hipError_t launch_gemm_i8(const void* x, const float* x_scales, const float* s, const void* codes, const float* scales,
                          void* y, int y_bytes, int64_t M, int64_t N, int64_t K, void* ws, hipStream_t st) {
  const I8Plan plan = i8_plan(M, N, K, x_scales != nullptr);
  const bool fused = plan.tile < 0 && i8_fused(M, K, x_scales != nullptr);
  int8_t* scratch = reinterpret_cast<int8_t*>(ws);
  if (x_scales == nullptr && !fused && active_plan() == nullptr) {
    float* sc = reinterpret_cast<float*>(scratch + rows_bytes(M, K));
    const hipError_t e = launch_rows_i8(x, K, s, true, M, K, scratch, sc, st);
    if (e != hipSuccess) return e;
    x = scratch;
    x_scales = sc;
    scratch += rows_bytes(M, K) + ((size_t)M * 4 + 255) / 256 * 256;
  }
  const I8Args a{reinterpret_cast<const int8_t*>(x), x_scales, reinterpret_cast<const int8_t*>(codes), scales, y, M, N, K, s,
                 0, 0, plan.splits, reinterpret_cast<int32_t*>(scratch)};
  switch (plan.tile) {
    case -1: return skinny_dispatch(a, fused, y_bytes, st);
    case 0: return tile_launch<32, 64, 1, 2, 6, 64>(a, y_bytes, st);
    case 1: return tile_launch<32, 128, 1, 4, 4, 64>(a, y_bytes, st);
    case 2: return tile_launch<64, 64, 1, 2, 5, 64>(a, y_bytes, st);
    case 3: return tile_launch<64, 128, 1, 4, 3, 64>(a, y_bytes, st);
    case 4: return tile_launch<128, 128, 2, 4, 4, 64>(a, y_bytes, st);
    default: return tile_launch<256, 256, 2, 4, 4, 32>(a, y_bytes, st);
  }
}

}  // namespace awq
