// Attention of one new token of each sequence over the paged low-bit cache.
//
// For a sequence of n tokens, a query head's row q and the key-value head it
// belongs to:  s_t = a q . k_t,  out = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m)
// over t < n, with k_t = scale_t (code_t - zero_t) and v_t alike.  The codes are
// never expanded to fp16 values.  A 4- or 8-bit whole number c in the low bits
// of a half is the fp16 subnormal c 2^-24, which the matrix cores take exactly,
// so unpacking is one mask (and a shift for every second pair); scale and zero
// point, one of each per token, stay outside the products:
//   q . k_t = scale_t (2^24 q . [c_t] - zero_t sum(q)),
//   sum_t p_t v_t = 2^24 sum_t (p_t scale_t) [c_t] - sum_t (p_t scale_t) zero_t.
// Everything but the operands q (fp16 as given) and w_t = p_t scale_t is kept in
// fp32; w_t enters the products as the sum of two fp16 numbers, which leaves
// 2^-22 of it (one would add an error of the size of the output's own rounding).
//
// A block takes one chunk of the sequence's tokens for one key-value head and
// up to 16 of its query heads; its waves take 32-token steps in turn, each
// wave with its own running maximum, sum and output, and are joined through
// LDS.  Chunks of one sequence are joined by kv_join_kernel in the order of
// the chunks, so results do not depend on timing.
//
// Lanes.  With l = 16 b + n, the products are 16 x 16 x 32:
//   scores  A = codes of 16 tokens (row n: token; lane's channels D/4 b ..),
//           B = q (column n: head): lane gets head n, tokens 4 b .. 4 b + 3
//   output  A = codes of 16 channels (row n) of 32 tokens, B = w (column n:
//           head; the lane's tokens are those whose scores it already holds),
//           so w goes from the scores to the products without leaving its lane,
//           and the lane gets channels of head n: rescaling is per lane.
#include "awq_common.h"
#include "awq_internal.h"
#include "kv_common.h"

namespace awq {

constexpr int kAttWaves = 4;
constexpr int kAttStep = 32;       // tokens a wave takes at a time
constexpr int kAttHeads = 16;      // query heads of a block: columns of a product
constexpr float kSlack = 8.f;      // a score may pass the running maximum by this (log2) before all is rescaled
constexpr float kTwo24 = 16777216.f;

// Channel of the cache row that product row n of tile c of the output stands for.
template <int D, int BITS>
__host__ __device__ constexpr int att_channel(int n, int c) {
  // 4-bit halves of words hold channels 0 2 4 6 / 1 3 5 7 of 8
  if (BITS == 4 && D == 64) return 8 * (n >> 1) + 2 * c + (n & 1);
  if (BITS == 4) return n * (D / 16) + 8 * (c / 8) + 2 * (c % 4) + (c % 8) / 4;
  return n * (D / 16) + c;
}

// Whether tile c's codes come times 16 (the upper nibble of each byte).
template <int BITS>
__host__ __device__ constexpr bool att_times16(int c) {
  return BITS == 4 && (c & 1);
}

__device__ inline uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); }

template <int D, int BITS>
struct AttStep {
  static constexpr int KW = D * BITS / 128;              // words of a lane's K row quarter
  static constexpr int VW = D * BITS / 512 > 0 ? D * BITS / 512 : 1;  // words of a lane's channels of a V row
  uint32_t k[2][KW];
  uint32_t v[8][VW];
  u32x4 kp[2], vp[2];
};

template <int D, int BITS>
__global__ __launch_bounds__(64 * kAttWaves) void kv_attention_kernel(
    const f16* __restrict__ q, int64_t q_stride, KvHalf kc, KvHalf vc, const int32_t* __restrict__ table, int width,
    const int32_t* __restrict__ lengths, int64_t max_len, KvShape sh, int ratio, float scale_log2, int chunk,
    int chunks, f16* __restrict__ out, float* __restrict__ part_o, float* __restrict__ part_ml) {
  constexpr int W = D * BITS / 32, TILES = D / 16;
  using Step = AttStep<D, BITS>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];

  const int lane = threadIdx.x & 63, n = lane & 15, b = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row_tiles = (ratio + kAttHeads - 1) / kAttHeads;
  const int hk = (int)blockIdx.x / row_tiles, h0 = ((int)blockIdx.x - hk * row_tiles) * kAttHeads;
  const int seq = (int)blockIdx.z;
  const int heads = ratio - h0 < kAttHeads ? ratio - h0 : kAttHeads;  // query heads of this block
  const int Hq = sh.heads * ratio;

  const int64_t len = kv_length(sh, lengths[seq], width, max_len);
  const int64_t t0 = (int64_t)blockIdx.y * chunk;
  if (t0 >= len && blockIdx.y > 0) return;  // the first chunk of an empty sequence stores its zeros
  const int count = (int)(len - t0 < chunk ? (len - t0 > 0 ? len - t0 : 0) : chunk);

  // Pages of the chunk: lane i holds that of the chunk's tokens 16 i .. 16 i + 15
  // (a chunk has at most 64 such tiles), -1 where there is none.
  int page_of = -1;
  if (16 * lane < count) page_of = kv_page(sh, table[(int64_t)seq * width + ((t0 + 16 * lane) >> sh.ps)]);

  // q: columns past the block's heads repeat the last one and are never stored
  const int hn = n < heads ? n : heads - 1;
  const f16* qrow = q + seq * q_stride + (int64_t)(hk * ratio + h0 + hn) * D;
  f16x8 qf[D / 32];
  float qsum = 0.f;
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    const f16x8 x = *reinterpret_cast<const f16x8*>(qrow + b * (D / 4) + 8 * s);
#pragma unroll
    for (int j = 0; j < 8; ++j) qsum += (float)x[j];
    const f16 t = (f16)0.0625f;
    if (BITS == 4) qf[s] = f16x8{x[0], x[1], x[2] * t, x[3] * t, x[4], x[5], x[6] * t, x[7] * t};
    else qf[s] = f16x8{x[0], x[2], x[1], x[3], x[4], x[6], x[5], x[7]};
  }
  qsum += __shfl_xor(qsum, 16, kWave);
  qsum += __shfl_xor(qsum, 32, kWave);
  const float qz = qsum * (1.f / kTwo24);
  const float sfac = scale_log2 * kTwo24;

  f32x4 o[TILES], oz = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < TILES; ++c) o[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  float F = 0.f;  // power of two that brings the largest scale seen so far to 2^6 .. 2^7; 0: none seen

  const int steps = (count + kAttStep - 1) / kAttStep;
  auto load = [&](int i, Step& st) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int tile = 2 * i + u;
      const int64_t row = kv_tile_row(sh, __builtin_amdgcn_readlane(page_of, tile & 63), t0 + 16 * tile, hk);
      const uint32_t* ks = kc.codes + row * W + n * W + b * Step::KW;
      if constexpr (Step::KW == 2) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(ks);
        st.k[u][0] = x.x;
        st.k[u][1] = x.y;
      } else {
#pragma unroll
        for (int j = 0; j < Step::KW / 4; ++j) {
          const u32x4 x = reinterpret_cast<const u32x4*>(ks)[j];
#pragma unroll
          for (int e = 0; e < 4; ++e) st.k[u][4 * j + e] = x[e];
        }
      }
      const uint32_t* vs = vc.codes + (row + 4 * b) * W;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = 4 * u + j;
        if constexpr (D * BITS == 256) {
          st.v[at][0] = reinterpret_cast<const uint16_t*>(vs + j * W)[n];
        } else if constexpr (Step::VW == 1) {
          st.v[at][0] = (vs + j * W)[n];
        } else if constexpr (Step::VW == 2) {
          const u32x2 x = reinterpret_cast<const u32x2*>(vs + j * W)[n];
          st.v[at][0] = x.x;
          st.v[at][1] = x.y;
        } else {
          const u32x4 x = reinterpret_cast<const u32x4*>(vs + j * W)[n];
#pragma unroll
          for (int e = 0; e < 4; ++e) st.v[at][e] = x[e];
        }
      }
      st.kp[u] = *reinterpret_cast<const u32x4*>(kc.params + row + 4 * b);
      st.vp[u] = *reinterpret_cast<const u32x4*>(vc.params + row + 4 * b);
    }
  };

  auto compute = [&](int i, Step& st) {
    // tokens past the chunk's end or of a page that is none: no score, scale and zero point 0
    bool live[8];
    const bool page0 = __builtin_amdgcn_readlane(page_of, (2 * i) & 63) >= 0;
    const bool page1 = __builtin_amdgcn_readlane(page_of, (2 * i + 1) & 63) >= 0;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        live[4 * u + r] = (u ? page1 : page0) && kAttStep * i + 16 * u + 4 * b + r < count;

    float s[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        u32x4 a;
        if (BITS == 4) {
          const uint32_t w = st.k[u][t], w8 = w >> 8;
          a = u32x4{w & 0x000F000Fu, w & 0x00F000F0u, w8 & 0x000F000Fu, w8 & 0x00F000F0u};
        } else {
          const uint32_t w0 = st.k[u][2 * t], w1 = st.k[u][2 * t + 1];
          a = u32x4{w0 & 0x00FF00FFu, (w0 >> 8) & 0x00FF00FFu, w1 & 0x00FF00FFu, (w1 >> 8) & 0x00FF00FFu};
        }
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), qf[t], acc, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f16x2 p = as_f16x2(st.kp[u][r]);
        const float x = fmaf(-(float)p.y, qz, acc[r]) * ((float)p.x * sfac);
        s[4 * u + r] = live[4 * u + r] ? x : -INFINITY;
      }
    }
    float vscale[8];
    float top = s[0], wide = 0.f;
    uint32_t vz[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t p = live[j] ? st.vp[j >> 2][j & 3] : 0u;
      vscale[j] = (float)as_f16x2(p).x;
      vz[j] = p;
      top = fmaxf(top, s[j]);
      wide = fmaxf(wide, vscale[j]);
    }
    // rarely: a new maximum or a larger scale; every lane then rescales what it holds
    if (__ballot((top > m + kSlack) || (wide * F > 128.f) || (wide > 0.f && F == 0.f))) {
      top = fmaxf(top, __shfl_xor(top, 16, kWave));
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) wide = fmaxf(wide, __shfl_xor(wide, off, kWave));
      const float m2 = fmaxf(m, top);
      const float alpha = m == m2 ? 1.f : exp2f(m - m2);  // m = -inf: 0
      m = m2;
      float f2 = F;
      if (wide > 0.f) {
        int e;
        frexpf(wide, &e);  // wide in [2^(e - 1), 2^e)
        const float fw = ldexpf(1.f, 7 - e);
        f2 = F == 0.f ? fw : fminf(F, fw);
      }
      const float beta = F == 0.f ? alpha : alpha * (f2 / F);
      F = f2;
      l *= alpha;
#pragma unroll
      for (int c = 0; c < TILES; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[c][r] *= beta;
#pragma unroll
      for (int r = 0; r < 4; ++r) oz[r] *= beta;
    }
    const float mm = m == -INFINITY ? 0.f : m;
    f16x8 whi, wlo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float p = __builtin_amdgcn_exp2f(s[j] - mm);
      l += p;
      const float w = p * (vscale[j] * F);
      whi[j] = (f16)w;
      wlo[j] = (f16)(w - (float)whi[j]);
    }
    auto mac = [&](u32x4 a, f32x4& acc) {
      const f16x8 af = __builtin_bit_cast(f16x8, a);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, whi, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, wlo, acc, 0, 0, 0);
    };
    {
      u32x4 a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = perm(vz[2 * j + 1], vz[2 * j], 0x07060302u);  // the upper halves
      mac(a, oz);
    }
    if constexpr (BITS == 4) {
#pragma unroll
      for (int g = 0; g < (D * BITS == 256 ? 1 : 2 * Step::VW); ++g) {  // halves of the lane's words
        u32x4 x, x8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = perm(st.v[2 * j + 1][g / 2], st.v[2 * j][g / 2], g % 2 ? 0x07060302u : 0x05040100u);
          x8[j] = x[j] >> 8;
        }
        mac(x & 0x000F000Fu, o[4 * g]);
        mac(x & 0x00F000F0u, o[4 * g + 1]);
        mac(x8 & 0x000F000Fu, o[4 * g + 2]);
        mac(x8 & 0x00F000F0u, o[4 * g + 3]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < TILES; ++c) {
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a[j] = perm(st.v[2 * j + 1][c / 4], st.v[2 * j][c / 4], 0x0C040C00u + 0x00010001u * (c % 4));
        mac(a, o[c]);
      }
    }
  };

  Step cur;
  for (int i = wave; i < steps; i += kAttWaves) {
    load(i, cur);
    compute(i, cur);
  }

  // join the waves: largest maximum, then the sums in the order of the waves
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  float* red_o = reinterpret_cast<float*>(smem);               // [waves][heads][D]
  float* red_m = red_o + kAttWaves * heads * D;                // [waves][16]
  float* red_l = red_m + kAttWaves * kAttHeads;
  if (b == 0) {
    red_m[wave * kAttHeads + n] = m;
    red_l[wave * kAttHeads + n] = l;
  }
  if (n < heads) {
    const float back = F > 0.f ? 1.f / F : 0.f;
#pragma unroll
    for (int c = 0; c < TILES; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red_o[(wave * heads + n) * D + att_channel<D, BITS>(4 * b + r, c)] =
            (o[c][r] * (att_times16<BITS>(c) ? kTwo24 / 16.f : kTwo24) - oz[r]) * back;
  }
  __syncthreads();
  const bool whole = len <= chunk;  // the sequence's only chunk: store the result itself
  for (int i = threadIdx.x; i < heads * D; i += 64 * kAttWaves) {
    const int h = i / D, d = i - h * D;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttWaves; ++w) mx = fmaxf(mx, red_m[w * kAttHeads + h]);
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kAttWaves; ++w) {
      const float mw = red_m[w * kAttHeads + h];
      const float f = mw == -INFINITY ? 0.f : exp2f(mw - mx);
      sum += f * red_l[w * kAttHeads + h];
      acc = fmaf(f, red_o[(w * heads + h) * D + d], acc);
    }
    const int64_t head = (int64_t)seq * Hq + hk * ratio + h0 + h;
    if (whole) {
      out[head * D + d] = (f16)(sum > 0.f ? acc / sum : 0.f);
    } else {
      const int64_t at = head * chunks + blockIdx.y;
      part_o[at * D + d] = acc;
      if (d == 0) {
        part_ml[2 * at] = mx;
        part_ml[2 * at + 1] = sum;
      }
    }
  }
}

// Joins the chunks of one query head of one sequence: D threads.
__global__ void kv_join_kernel(const float* __restrict__ part_o, const float* __restrict__ part_ml,
                               const int32_t* __restrict__ lengths, int64_t max_len, int width, KvShape sh, int Hq,
                               int chunk, int chunks, f16* __restrict__ out) {
  const int64_t head = blockIdx.x;
  const int D = (int)blockDim.x, d = (int)threadIdx.x;
  const int64_t len = kv_length(sh, lengths[head / Hq], width, max_len);
  if (len <= chunk) return;  // stored by its only block
  const int used = (int)((len + chunk - 1) / chunk);
  const float* ml = part_ml + head * chunks * 2;
  const float* po = part_o + head * chunks * D + d;
  float mx = -INFINITY;
  for (int c = 0; c < used; ++c) mx = fmaxf(mx, ml[2 * c]);
  float sum = 0.f, acc = 0.f;
  for (int c = 0; c < used; ++c) {
    const float f = ml[2 * c] == -INFINITY ? 0.f : exp2f(ml[2 * c] - mx);
    sum = fmaf(f, ml[2 * c + 1], sum);
    acc = fmaf(f, po[(int64_t)c * D], acc);
  }
  out[head * D + d] = (f16)(sum > 0.f ? acc / sum : 0.f);
}

// Tokens of a chunk: as many as leave about eight blocks for each of the 256
// compute units, from one step of every wave (128) to what a wave's lanes
// hold the pages of (1024).
static int att_chunk(int64_t B, int64_t Hkv, int ratio, int64_t max_len) {
  const int64_t rows = B * Hkv * ((ratio + kAttHeads - 1) / kAttHeads);
  int chunk = kAttStep * kAttWaves;
  while (chunk < 1024 && rows * ((max_len + chunk - 1) / chunk) > 2048) chunk *= 2;
  return chunk;
}

size_t kv_attention_workspace(int64_t B, int64_t Hkv, int ratio, int D, int64_t max_len) {
  const int chunk = att_chunk(B, Hkv, ratio, max_len);
  const int64_t chunks = (max_len + chunk - 1) / chunk;
  return chunks > 1 ? (size_t)(B * Hkv * ratio * chunks * (D + 2)) * sizeof(float) : 0;
}

template <int D, int BITS>
static hipError_t attention_launch(const void* q, int64_t q_stride, KvHalf kc, KvHalf vc, const int32_t* table,
                                   int64_t width, const int32_t* lengths, int64_t B, int ratio, float scale,
                                   int64_t max_len, KvShape sh, void* out, float* ws, hipStream_t st) {
  const int chunk = att_chunk(B, sh.heads, ratio, max_len);
  const int chunks = max_len > 0 ? (int)((max_len + chunk - 1) / chunk) : 1;
  const int heads = ratio < kAttHeads ? ratio : kAttHeads;
  const size_t lds = (size_t)(kAttWaves * (heads * D + 2 * kAttHeads)) * sizeof(float);
  const dim3 grid((unsigned)(sh.heads * ((ratio + kAttHeads - 1) / kAttHeads)), (unsigned)chunks, (unsigned)B);
  float* part_ml = ws == nullptr ? nullptr : ws + B * sh.heads * ratio * chunks * D;
  kv_attention_kernel<D, BITS><<<grid, dim3(64 * kAttWaves), lds, st>>>(
      reinterpret_cast<const f16*>(q), q_stride, kc, vc, table, (int)width, lengths, max_len, sh, ratio,
      scale * 1.4426950408889634f, chunk, chunks, reinterpret_cast<f16*>(out), ws, part_ml);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks == 1) return e;
  kv_join_kernel<<<dim3((unsigned)(B * sh.heads * ratio)), dim3(D), 0, st>>>(
      ws, part_ml, lengths, max_len, (int)width, sh, sh.heads * ratio, chunk, chunks, reinterpret_cast<f16*>(out));
  return hipGetLastError();
}

hipError_t launch_kv_attention(const void* q, int64_t q_stride, KvHalf kc, KvHalf vc, const int32_t* table,
                               int64_t width, const int32_t* lengths, int64_t B, int ratio, int D, int bits,
                               float scale, int64_t max_len, KvShape sh, void* out, void* ws, hipStream_t st) {
  float* w = reinterpret_cast<float*>(ws);
#define AWQ_ATT(d, b)       \
  if (D == d && bits == b) \
    return attention_launch<d, b>(q, q_stride, kc, vc, table, width, lengths, B, ratio, scale, max_len, sh, out, w, st)
  AWQ_ATT(64, 4);
  AWQ_ATT(128, 4);
  AWQ_ATT(256, 4);
  AWQ_ATT(64, 8);
  AWQ_ATT(128, 8);
  AWQ_ATT(256, 8);
#undef AWQ_ATT
  return hipErrorInvalidValue;
}

}  // namespace awq
