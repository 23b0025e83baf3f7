// The product in 8-bit integers: y = (x codes) (w codes)^T in exact 32-bit sums,
// times a scale for each token and each channel.
//
// Tile kernel: BM tokens x BN channels a block, K in stages of 64 bytes.  Stages go
// from global memory straight into a ring of LDS buffers (the 64-byte-row layout
// of mfma_pipe.h, a pair of codes in the place of a half) and feed
// v_mfma_i32_32x32x32_i8.  A stage's first fragments are read before the barrier
// that opens it, so the matrix cores do not wait for the barrier or the LDS: the
// barrier of stage s only says that stage s + 1 has landed and stage s - 1 is free.
// The weights are the A operand, so a lane's accumulators hold four consecutive
// channels of one token; the results are turned over through LDS and stored as
// whole rows.
#include "awq_internal.h"
#include "mfma_pipe.h"

namespace awq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

struct I8Args {
  const int8_t* x;
  const float* xs;
  const int8_t* w;
  const float* ws;
  void* y;
  int64_t M, N, K;
  int mtiles, ntiles;
};

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

template <int BM, int BN, int WM, int WN, int STAGES>
struct I8Shape {
  static constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, AM = TM / 32, AN = TN / 32;
  static constexpr int STAGE = (BM + BN) * 32;  // halfs
  static constexpr int LOADS = (BM + BN) / 16 / NW;
  static constexpr int PITCH = TN + 4;          // words of a row of the turned-over tile (fp32; fp16 uses half)
  static constexpr int RING = STAGES * STAGE * 2, TURN = NW * 32 * PITCH * 4;
  static constexpr int LDS = RING > TURN ? RING : TURN;
  static_assert((BM / 16) % NW == 0 && (BN / 16) % NW == 0, "whole loads a wave");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <int BM, int BN, int WM, int WN, int STAGES, typename Y>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_kernel(I8Args a) {
  typedef I8Shape<BM, BN, WM, WN, STAGES> S;
  constexpr int AM = S::AM, AN = S::AN;
  __shared__ __align__(16) unsigned char lds[S::LDS];
  f16* ring = reinterpret_cast<f16*>(lds);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const TileAt at = tile_at(blockIdx.x, a.mtiles, a.ntiles);
  const int64_t m0 = (int64_t)at.m * BM, n0 = (int64_t)at.n * BN;
  const int wm = (wave % WM) * S::TM, wn = (wave / WM) * S::TN;
  TilePlan<BM, S::NW, 32> px;
  TilePlan<BN, S::NW, 32> pw;
  px.init(reinterpret_cast<const f16*>(a.x), a.K / 2, m0, a.M, wave, lane);
  pw.init(reinterpret_cast<const f16*>(a.w), a.K / 2, n0, a.N, wave, lane);
  const int steps = (int)(a.K / 64);  // even
  auto issue = [&](int s) {
    f16* stage = ring + (s % STAGES) * S::STAGE;
    const int64_t k = (int64_t)(s < steps ? s : steps - 1) * 32;  // past the end: counted, never used
    px.issue(stage, k);
    pw.issue(stage + BM * 32, k);
  };
  i32x16 acc[AN][AM];
#pragma unroll
  for (int i = 0; i < AN; ++i)
#pragma unroll
    for (int j = 0; j < AM; ++j) acc[i][j] = i32x16{};
  i32x4 fa[2][AN], fb[2][AM];
  auto read = [&](int s, int c, int into) {
    const f16* tx = ring + (s % STAGES) * S::STAGE;
    const f16* tw = tx + BM * 32;
#pragma unroll
    for (int i = 0; i < AN; ++i)
      fa[into][i] = __builtin_bit_cast(i32x4, frag32(tw, wn + i * 32 + (lane & 31), 2 * c + (lane >> 5)));
#pragma unroll
    for (int j = 0; j < AM; ++j)
      fb[into][j] = __builtin_bit_cast(i32x4, frag32(tx, wm + j * 32 + (lane & 31), 2 * c + (lane >> 5)));
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
    read(s, 1, 1);
    multiply(0);
    read(s + 1, 0, 0);
    multiply(1);
  }
  wait_vmcnt<0>();  // the loads past the end
  lds_barrier();

  // each wave turns its tile over, 32 tokens at a time
  float* turn = reinterpret_cast<float*>(lds) + wave * 32 * S::PITCH;
  Y* turn_y = reinterpret_cast<Y*>(turn);
  constexpr int PITCH = sizeof(Y) == 4 ? S::PITCH : 2 * S::PITCH;  // elements
  constexpr int PER = 16 / sizeof(Y), LANES = S::TN / PER, ROWS = 64 / LANES;
  Y* y = reinterpret_cast<Y*>(a.y);
  const bool whole = a.N % PER == 0 && n0 + wn + S::TN <= a.N;
#pragma unroll
  for (int j = 0; j < AM; ++j) {
    const int64_t mj = m0 + wm + j * 32, m = mj + (lane & 31);
    const float sm = a.xs[m < a.M ? m : a.M - 1];
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
          v[u] = (Y)((float)acc[i][j][4 * q + u] * sm * a.ws[ng < a.N ? ng : a.N - 1]);
        }
        *reinterpret_cast<yx4*>(turn_y + (lane & 31) * PITCH + n) = v;
      }
    __asm__ volatile("" ::: "memory");  // the wave's own tile: its LDS accesses are done in order
    if (whole) {
#pragma unroll
      for (int r = 0; r < 32; r += ROWS) {
        const int row = r + lane / LANES, n = (lane % LANES) * PER;
        const u32x4 v = *reinterpret_cast<const u32x4*>(turn_y + row * PITCH + n);
        if (mj + row < a.M) *reinterpret_cast<u32x4*>(y + (mj + row) * a.N + n0 + wn + n) = v;
      }
    } else {
      for (int r = 0; r < 32; ++r)
        for (int n = lane; n < S::TN; n += 64)
          if (mj + r < a.M && n0 + wn + n < a.N) y[(mj + r) * a.N + n0 + wn + n] = turn_y[r * PITCH + n];
    }
    __asm__ volatile("" ::: "memory");
  }
}

static size_t rows_bytes(int64_t M, int64_t K) { return ((size_t)M * (size_t)K + 255) / 256 * 256; }

size_t gemm_i8_workspace(int64_t M, int64_t N, int64_t K, bool quantized) {
  return quantized ? 0 : rows_bytes(M, K) + ((size_t)M * 4 + 255) / 256 * 256;
}

template <int BM, int BN, int WM, int WN, int STAGES>
static hipError_t tile_launch(I8Args a, int y_bytes, hipStream_t st) {
  a.mtiles = (int)((a.M + BM - 1) / BM);
  a.ntiles = (int)((a.N + BN - 1) / BN);
  const dim3 grid((unsigned)(a.mtiles * a.ntiles)), block(64 * WM * WN);
  if (KernelPlan* p = active_plan())
    return plan_record(p, "gemm_i8_kernel<%d,%d,%d,%d,%d> block=%u grid=%u", BM, BN, WM, WN, STAGES, block.x, grid.x);
  if (y_bytes == 2) gemm_i8_kernel<BM, BN, WM, WN, STAGES, f16><<<grid, block, 0, st>>>(a);
  else gemm_i8_kernel<BM, BN, WM, WN, STAGES, float><<<grid, block, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_gemm_i8(const void* x, const float* x_scales, const float* s, const void* codes, const float* scales,
                          void* y, int y_bytes, int64_t M, int64_t N, int64_t K, void* ws, hipStream_t st) {
  if (x_scales == nullptr && active_plan() == nullptr) {
    int8_t* xc = reinterpret_cast<int8_t*>(ws);
    float* sc = reinterpret_cast<float*>(xc + rows_bytes(M, K));
    const hipError_t e = launch_rows_i8(x, K, s, true, M, K, xc, sc, st);
    if (e != hipSuccess) return e;
    x = xc;
    x_scales = sc;
  }
  const I8Args a{reinterpret_cast<const int8_t*>(x), x_scales, reinterpret_cast<const int8_t*>(codes), scales, y, M, N, K, 0, 0};
  if (M > 128) return tile_launch<256, 256, 4, 2, 4>(a, y_bytes, st);
  return tile_launch<128, 128, 2, 2, 4>(a, y_bytes, st);
}

}  // namespace awq
