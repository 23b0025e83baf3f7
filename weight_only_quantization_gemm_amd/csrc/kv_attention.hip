// Attention of one new token of each sequence over the paged low-bit cache.
//
// For a sequence of n tokens, a query head's row q and the key-value head it
// belongs to:  s_t = a q . k_t,  out = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m)
// over t < n, with k_t = scale_t (code_t - zero_t) and v_t alike.  The codes are
// never expanded to fp16 values.  A whole number c below 2^10 in the bits of a half is
// the fp16 subnormal c 2^-24, which the matrix cores take, so unpacking is a shift and
// a mask.  (The products of a subnormal operand are cut off as if it had no leading
// zeros, at 2^-24 of the largest of a sum: codes are therefore brought to the top, 4-bit
// ones to bits 6 .. 9 and 8-bit ones to bits 2 .. 9.  Of long sequences, whose output is
// a small difference, codes two bits lower made errors of up to 0.7 of the output's
// rounding, with a mean; the shifts cost 1 to 2 % of the time.)  Scale and zero
// point, one of each per token, stay outside the products; u = 2^18 or 2^22:
//   q . k_t = scale_t (u q . [c_t] - zero_t sum(q)),
//   sum_t p_t v_t = u sum_t (p_t scale_t) [c_t] - sum_t (p_t scale_t) zero_t.
// Everything but the operands q (fp16 as given) and w_t = p_t scale_t is kept in
// fp32; w_t enters the products as the sum of two fp16 numbers, which leaves
// 2^-22 of it (one would add an error of the size of the output's own rounding).
//
// A block takes one piece of a sequence's tokens for one key-value head and up to
// 16 of its query heads; its waves take 32-token steps in turn, each wave with its
// own running maximum, sum and output, and are joined through LDS.  The pieces of
// one sequence are joined by kv_join_kernel in their order, so results do not
// depend on timing.
//
// Bound by reading the cache: 64 sequences of 4096 tokens x 8 heads of 128 at 4
// bits, 285 MB in 62 us (4.6 TB/s); 32 of 2000 to 6000 at 8 bits, 269 MB in 64 us;
// 64 ragged ones of 2000 to 6000 tokens at 4 bits 279 MB in 69 us, the last blocks
// leaving units idle; one of 2000 tokens 10 us, launches and latency.  The vector
// ALU is busy 55 % of the time.
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
#include "mfma_pipe.h"

#include <cmath>

namespace awq {

constexpr int kAttWaves = 4;
constexpr int kAttStep = 32;       // tokens a wave takes at a time
constexpr int kAttHeads = 16;      // query heads of a block: columns of a product
constexpr float kSlack = 8.f;      // a score may pass the running maximum by this (log2) before all is rescaled
constexpr int kNonTemporal = 2;    // cache policy of the code loads: every line is used once (54 us against 61)
constexpr int kAttWindow = 1024;   // tokens whose pages a wave's lanes hold, 16 each

// Codes enter the products divided by this.
constexpr float att_unit(int bits) { return bits == 4 ? 262144.f : 4194304.f; }

// Channel of the cache row that product row n of tile c of the output stands for.
template <int D, int BITS>
__host__ __device__ constexpr int att_channel(int n, int c) {
  // 4-bit halves of words hold channels 0 2 4 6 / 1 3 5 7 of 8
  if (BITS == 4 && D == 64) return 8 * (n >> 1) + 2 * c + (n & 1);
  if (BITS == 4) return n * (D / 16) + 8 * (c / 8) + 2 * (c % 4) + (c % 8) / 4;
  return n * (D / 16) + c;
}

// Four words of halves whose bits 0 .. 15 are four 4-bit codes: code k of each times 64.
template <int k>
__device__ __forceinline__ u32x4 nibbles(u32x4 x) {
  return (k == 0 ? x << 6 : (k == 1 ? x << 2 : (k == 2 ? x >> 2 : x >> 6))) & 0x03C003C0u;
}

__device__ inline uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); }

// A stage of a wave's ring: 32 tokens' keys, values and parameters, moved
// straight into LDS.  Keys: rows of RB bytes, piece c (16 bytes) of row r in slot
// c ^ f(r), so that 16 rows at one piece lie in all banks.  Values: within a
// tile of 16, token 4 b + j in row 4 j + b, so that one read of the four lane
// groups b is contiguous.  Parameters: keys' of 32 tokens, then values'.
template <int D, int BITS>
struct AttStage {
  static constexpr int RB = D * BITS / 8, PIECES = RB / 16;
  static constexpr int HALF = kAttStep * RB, NI = HALF / 1024;  // bytes, 1 KB loads of keys (and of values)
  static constexpr int BYTES = 2 * HALF + 256, LOADS = 2 * NI + 1;
  static constexpr int KW = RB / 16;                     // words of a lane's quarter of a key row
  static constexpr int RING = 2 * BYTES;                  // (three stages cost a block per compute unit: 75 us against 70)
  static __host__ __device__ constexpr int slot_xor(int r) { return (r / (256 / RB)) & (PIECES - 1); }
};

// How a call's tokens are cut into pieces, one (sequence, run of tokens) each.
// By the bound on the lengths (chunk > 0): `chunk` tokens of sequence blockIdx.z.
// By the lengths themselves (chunk = 0): piece blockIdx.y of those of all sequences,
// which PieceSplit counts from the lengths on the device.
struct AttSplit {
  const int32_t* lengths;
  int64_t max_len;
  int width;   // entries of a page table's row
  int batch;
  int chunk, chunks;
  int heads;   // blocks' heads: key-value heads x tiles of query heads
  int most;    // pieces of all heads that keep the chip full
};

static_assert(kKvUnit == kAttStep * kAttWaves, "a unit is a step of every wave");
constexpr int kPieceWindows = 4, kPieceRun = 64 * kPieceWindows, kPieceBatch = 1024;

// The sequence of piece `slot`, counted from the lengths; lane i of window k holds
// sequence s0 + 64 k + i of a run of sequences.
struct PieceSplit {
  int seq, len;       // the piece's sequence and its length
  int first, pieces;  // its first piece and their number

  // False where there are fewer pieces.
  __device__ __forceinline__ bool find(const AttSplit& sp, const KvShape& sh, int lane, int slot) {
    int held[kPieceWindows];
    auto read = [&](int s0) {
#pragma unroll
      for (int k = 0; k < kPieceWindows; ++k) {  // (sequences past the batch repeat its last and do not count)
        const int s = s0 + 64 * k + lane;
        held[k] = (int)kv_length(sh, sp.lengths[s < sp.batch ? s : sp.batch - 1], sp.width, sp.max_len);
      }
    };
    int64_t units = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < sp.batch; s0 += kPieceRun) {
      read(s0);
#pragma unroll
      for (int k = 0; k < kPieceWindows; ++k)
        if (s0 + 64 * k < sp.batch)
          units += __builtin_amdgcn_readlane(wave_scan(s0 + 64 * k + lane < sp.batch ? kv_units(held[k]) : 0), 63);
    }
    const int shift = kv_piece_shift(units, sp.heads, sp.most);
    int total = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < sp.batch; s0 += kPieceRun) {
      if (sp.batch > kPieceRun) read(s0);
#pragma unroll
      for (int k = 0; k < kPieceWindows; ++k)
        if (s0 + 64 * k < sp.batch) {
          const int upto = total + wave_scan(s0 + 64 * k + lane < sp.batch ? kv_pieces(kv_units(held[k]), shift) : 0);
          total = __builtin_amdgcn_readlane(upto, 63);
          const uint64_t past = __ballot(upto > slot);
          if (past) {
            const int at = __ffsll((unsigned long long)past) - 1;
            seq = s0 + 64 * k + at;
            len = __builtin_amdgcn_readlane(held[k], at);
            pieces = kv_pieces(kv_units(len), shift);
            first = __builtin_amdgcn_readlane(upto, at) - pieces;
            return true;
          }
        }
    }
    return false;
  }
};

template <int D, int BITS>
__global__ __launch_bounds__(64 * kAttWaves, D * BITS <= 512 ? 4 : 1) void kv_attention_kernel(
    const f16* __restrict__ q, int64_t q_stride, KvHalf kc, KvHalf vc, const int32_t* __restrict__ table, AttSplit sp,
    KvShape sh, int ratio, float signed_factor, f16* __restrict__ out, float* __restrict__ part_o,
    float* __restrict__ part_ml, int32_t* __restrict__ meta) {
  using A = AttStage<D, BITS>;
  constexpr int TILES = D / 16, RB = A::RB;
  constexpr float kUnit = att_unit(BITS);
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row_tiles = (ratio + kAttHeads - 1) / kAttHeads;
  const int hk = (int)blockIdx.x / row_tiles, h0 = ((int)blockIdx.x - hk * row_tiles) * kAttHeads;
  const int heads = ratio - h0 < kAttHeads ? ratio - h0 : kAttHeads;  // query heads of this block
  const int Hq = sh.heads * ratio;

  const int tid = threadIdx.x;
  const int lane = tid & 63, n = lane & 15, b = lane >> 4;
  int seq, slot, count;  // the piece: tokens t0 .. t0 + count - 1 of sequence seq
  int64_t t0;
  bool whole;  // all of them
  // Pages: lane i holds that of tile 64 w + i of 16 tokens, w the window of 1024 tokens
  // under way, -1 where there is none.  The table's entries are fetched whatever the
  // count (one load always: the waits below count it), and dropped by it afterwards.
  auto entry = [&](int w) {
    const int64_t e = (t0 + kAttWindow * w + 16 * lane) >> sh.ps;
    return table + (int64_t)seq * sp.width + (e < sp.width ? e : sp.width - 1);
  };
  auto page_of = [&](int w, int entry) { return kAttWindow * w + 16 * lane < count ? kv_page(sh, entry) : -1; };
  int pages, next = -1;
  if (sp.chunk == 0) {
    PieceSplit split;
    slot = (int)blockIdx.y;
    if (!split.find(sp, sh, lane, slot)) return;
    seq = split.seq;
    const int len = split.len, pieces = split.pieces, first = split.first;
    const int span = (kv_units(len) + pieces - 1) / pieces * kKvUnit;
    if (slot == first && blockIdx.x == 0 && tid == 0) {
      meta[2 * seq] = first;
      meta[2 * seq + 1] = pieces;
    }
    t0 = (int64_t)(slot - first) * span;
    count = len - (int)t0 < span ? len - (int)t0 : span;
    whole = pieces == 1;
    pages = *entry(0);
  } else {
    seq = (int)blockIdx.z;
    t0 = (int64_t)blockIdx.y * sp.chunk;
    pages = *entry(0);  // along with the length
    const int64_t len = kv_length(sh, sp.lengths[seq], sp.width, sp.max_len);
    if (t0 >= len && blockIdx.y > 0) return;  // the first piece of an empty sequence stores its zeros
    count = (int)(len - t0 < sp.chunk ? (len - t0 > 0 ? len - t0 : 0) : sp.chunk);
    whole = len <= sp.chunk;
    slot = seq * sp.chunks + (int)blockIdx.y;
  }
  pages = page_of(0, pages);
  auto page = [&](int tile) { return __builtin_amdgcn_readlane(pages, tile & 63); };

  unsigned char* ring = smem + wave * A::RING;
  int* ahead = reinterpret_cast<int*>(smem + kAttWaves * A::RING) + wave * 64;  // the next window's entries
  auto issue = [&](int i, int slot, int pages_of_i) {
    unsigned char* st = ring + slot * A::BYTES;
    int64_t row[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      row[u] = kv_tile_row(sh, __builtin_amdgcn_readlane(pages_of_i, (2 * i + u) & 63), t0 + 16 * (2 * i + u), hk);
#pragma unroll
    for (int k = 0; k < A::NI; ++k) {
      const int r = (k * 64 + lane) / A::PIECES, slot_of = lane % A::PIECES;  // row of the step, 16-byte slot
      const int64_t base = RB == 32 ? (lane < 32 ? row[0] : row[1]) : row[k * 1024 / RB / 16];
      const int tr = r & 15;
      const unsigned char* ks = reinterpret_cast<const unsigned char*>(kc.codes) + base * RB;
      const unsigned char* vs = reinterpret_cast<const unsigned char*>(vc.codes) + base * RB;
      __builtin_amdgcn_global_load_lds((global_ptr_t)(ks + tr * RB + ((slot_of ^ A::slot_xor(tr)) << 4)),
                                       (lds_ptr_t)(st + k * 1024), 16, 0, kNonTemporal);
      __builtin_amdgcn_global_load_lds((global_ptr_t)(vs + (4 * (tr & 3) + (tr >> 2)) * RB + (slot_of << 4)),
                                       (lds_ptr_t)(st + A::HALF + k * 1024), 16, 0, kNonTemporal);
    }
    const uint32_t* ps = (lane < 32 ? kc.params : vc.params) + (lane & 16 ? row[1] : row[0]) + n;
    __builtin_amdgcn_global_load_lds((global_ptr_t)ps, (lds_ptr_t)(st + 2 * A::HALF), 4, 0, 0);
  };
  const int steps = (count + kAttStep - 1) / kAttStep;
  const int turns = steps > wave ? (steps - wave + kAttWaves - 1) / kAttWaves : 0;
  if (turns > 0) issue(wave, 0, pages);

  // q: columns past the block's heads repeat the last one and are never stored.  A negative
  // factor goes to q's sign, so that larger sums are larger scores.
  const float factor = fabsf(signed_factor);
  const int hn = n < heads ? n : heads - 1;
  const f16* qrow = q + seq * q_stride + (int64_t)(hk * ratio + h0 + hn) * D;
  f16x8 qf[D / 32];
  float qz = 0.f;
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    f16x8 x = *reinterpret_cast<const f16x8*>(qrow + b * (D / 4) + 8 * s);
    if (signed_factor < 0.f) x = -x;
#pragma unroll
    for (int j = 0; j < 8; ++j) qz += (float)x[j];
    if (BITS == 4) qf[s] = x;
    else qf[s] = f16x8{x[0], x[2], x[1], x[3], x[4], x[6], x[5], x[7]};
  }
  qz += __shfl_xor(qz, 16, kWave);
  qz += __shfl_xor(qz, 32, kWave);
  qz *= -1.f / kUnit;

  // Weights are kept as 2^(factor (s - top) + F), top following the largest sum and F the
  // exponent that brings the largest weight times its value scale to 2^6 .. 2^7 (and on to 2^15
  // before all is rescaled): of any other, two fp16 numbers then leave at most 2^-31 of that one.
  // (Not the largest value scale alone: one of a token of no weight would push all others off
  // fp16's lower end.)  Sums are subtracted before they are multiplied:
  // the difference is exact near the top, so the weight of the top itself is 2^F whatever the
  // size of the scores (factor s - (factor top - F) would be off by half a unit of factor top,
  // in the exponent).
  f32x4 o[TILES], oz = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < TILES; ++c) o[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  float top_seen = -INFINITY, base = 0.f;         // the top, and what is subtracted (0 while there is none)
  float F = 0.f, most = 0.f;                      // most: the largest weight times value scale when last rescaled

  auto compute = [&](int i, const unsigned char* st) {
    float s[8];
    uint32_t vp[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const u32x4 kp = *reinterpret_cast<const u32x4*>(st + 2 * A::HALF + u * 64 + b * 16);
      const u32x4 vq = *reinterpret_cast<const u32x4*>(st + 2 * A::HALF + 128 + u * 64 + b * 16);
      uint32_t w[A::KW];
      if constexpr (A::KW == 2) {
        const int at = n * RB + b * 8;  // the lane's half of piece b / 2
        const u32x2 x = *reinterpret_cast<const u32x2*>(st + u * 16 * RB + (at ^ (A::slot_xor(n) << 4)));
        w[0] = x.x;
        w[1] = x.y;
      } else {
#pragma unroll
        for (int j = 0; j < A::KW / 4; ++j) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(
              st + u * 16 * RB + n * RB + (((b * (A::KW / 4) + j) ^ A::slot_xor(n)) << 4));
#pragma unroll
          for (int e = 0; e < 4; ++e) w[4 * j + e] = x[e];
        }
      }
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        u32x4 a;
        if (BITS == 4) {
          const uint32_t x = w[t];
          a = u32x4{(x << 6) & 0x03C003C0u, (x << 2) & 0x03C003C0u, (x >> 2) & 0x03C003C0u, (x >> 6) & 0x03C003C0u};
        } else {
          a = u32x4{(w[2 * t] << 2) & 0x03FC03FCu, (w[2 * t] >> 6) & 0x03FC03FCu, (w[2 * t + 1] << 2) & 0x03FC03FCu,
                    (w[2 * t + 1] >> 6) & 0x03FC03FCu};
        }
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), qf[t], acc, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f16x2 p = as_f16x2(kp[r]);
        s[4 * u + r] = fmaf(fmaf((float)p.y, qz, acc[r]), (float)p.x, 0.f);  // (fma takes the fp16 operand as it is)
        vp[4 * u + r] = vq[r];
      }
    }
    // tokens past the piece's end or of a page that is none: no score, value scale and zero point 0
    const bool page0 = page(2 * i) >= 0, page1 = page(2 * i + 1) >= 0;
    if (!page0 || !page1 || kAttStep * (i + 1) > count) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool live = (j < 4 ? page0 : page1) && kAttStep * i + 16 * (j >> 2) + 4 * b + (j & 3) < count;
        s[j] = live ? s[j] : -INFINITY;
        vp[j] = live ? vp[j] : 0u;
      }
    }
    float top = s[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, s[j]);
    // rarely: a new maximum
    const bool moved = __ballot((top - top_seen) * factor > kSlack) != 0;
    float alpha = 1.f;
    if (moved) {
      top = fmaxf(top, __shfl_xor(top, 16, kWave));
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
      const float was = top_seen;
      top_seen = fmaxf(top_seen, top);
      base = top_seen == -INFINITY ? 0.f : top_seen;
      alpha = was == -INFINITY ? 0.f : exp2f((was - base) * factor);
    }
    float w[8], sum = 0.f, big = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float p = __builtin_amdgcn_exp2f(fmaf(s[j] - base, factor, F));
      sum += p;
      w[j] = fmaf(p, (float)as_f16x2(vp[j]).x, 0.f);
      big = fmaxf(big, w[j]);
    }
    // then, or where a weight times its value scale grows too large: what a lane holds is rescaled
    if (moved || __ballot(big > 32768.f)) {
      big = fmaxf(big, __shfl_xor(big, 16, kWave));
      big = fmaxf(big, __shfl_xor(big, 32, kWave));
      most = fmaxf(most * alpha, big);
      int e;
      frexpf(most, &e);  // most in [2^(e - 1), 2^e)
      const float now = most > 0.f ? fminf(fmaxf(F + (float)(7 - e), -40.f), 40.f) : F;
      const float by = ldexpf(1.f, (int)(now - F));  // exact
      F = now;
      most *= by;
      sum *= by;
      alpha *= by;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= by;
      l *= alpha;
#pragma unroll
      for (int c = 0; c < TILES; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[c][r] *= alpha;
#pragma unroll
      for (int r = 0; r < 4; ++r) oz[r] *= alpha;
    }
    l += sum;
    f16x8 whi, wlo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      whi[j] = (f16)w[j];
      wlo[j] = (f16)fmaf((float)whi[j], -1.f, w[j]);
    }
    auto mac = [&](u32x4 a, f32x4& acc) {
      const f16x8 af = __builtin_bit_cast(f16x8, a);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, whi, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, wlo, acc, 0, 0, 0);
    };
    {
      u32x4 a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = perm(vp[2 * j + 1], vp[2 * j], 0x07060302u);  // the zero points
      mac(a, oz);
    }
    constexpr int LB = RB / 16;  // bytes of a lane's channels of a value row: 2, 4, 8 or 16
    uint32_t v[8][LB < 4 ? 1 : LB / 4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned char* src = st + A::HALF + (16 * (j >> 2) + 4 * (j & 3) + b) * RB + n * LB;
      if constexpr (LB == 2) {
        v[j][0] = *reinterpret_cast<const uint16_t*>(src);
      } else if constexpr (LB == 4) {
        v[j][0] = *reinterpret_cast<const uint32_t*>(src);
      } else if constexpr (LB == 8) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(src);
        v[j][0] = x.x;
        v[j][1] = x.y;
      } else {
        const u32x4 x = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = x[e];
      }
    }
    if constexpr (BITS == 4) {
#pragma unroll
      for (int g = 0; g < TILES / 4; ++g) {  // halves of the lane's words
        u32x4 x;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[j] = perm(v[2 * j + 1][g / 2], v[2 * j][g / 2], g % 2 ? 0x07060302u : 0x05040100u);
        mac(nibbles<0>(x), o[4 * g]);
        mac(nibbles<1>(x), o[4 * g + 1]);
        mac(nibbles<2>(x), o[4 * g + 2]);
        mac(nibbles<3>(x), o[4 * g + 3]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < TILES; ++c) {
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a[j] = perm(v[2 * j + 1][c / 4], v[2 * j][c / 4], 0x0C040C00u + 0x00010001u * (c % 4)) << 2;
        mac(a, o[c]);
      }
    }
  };

  constexpr int kTurns = kAttWindow / kKvUnit;
  for (int j = 0; j < turns; ++j) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this wave's LDS reads of the stage refilled now are done
    __builtin_amdgcn_sched_barrier(0);
    const int i = wave + j * kAttWaves, w = j / kTurns;
    const bool last = j % kTurns == kTurns - 1;  // the next step lies in the next window
    if (j + 1 < turns) {
      if (last) next = page_of(w + 1, ahead[lane]);
      issue(i + kAttWaves, (j + 1) & 1, last ? next : pages);
      if (j % kTurns == 0) {  // the next window's entries, a window ahead (in a register each turn would wait for them)
        __builtin_amdgcn_global_load_lds((global_ptr_t)entry(w + 1), (lds_ptr_t)ahead, 4, 0, 0);
        wait_vmcnt<A::LOADS + 1>();
      } else {
        wait_vmcnt<A::LOADS>();
      }
    } else {
      wait_vmcnt<0>();
    }
    __builtin_amdgcn_sched_barrier(0);
    compute(i, ring + (j & 1) * A::BYTES);
    if (last) pages = next;
  }
  __syncthreads();  // the rings become the place of the sum

  // Join the waves: each output in LDS [wave][head][D], then its share of the sum,
  // 2^(factor (top - largest top) - F), and the sums in the order of the waves.
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  float* red_o = reinterpret_cast<float*>(smem);
  float* red_m = red_o + kAttWaves * heads * D;  // [wave][16]
  float* red_l = red_m + kAttWaves * kAttHeads;
  float* red_f = red_l + kAttWaves * kAttHeads;
  float* share = red_f + kAttWaves * kAttHeads;  // [wave][16], then the head's sum [16]
  if (b == 0) {
    red_m[wave * kAttHeads + n] = top_seen;
    red_l[wave * kAttHeads + n] = l;
    red_f[wave * kAttHeads + n] = (float)F;
  }
  if (n < heads) {
#pragma unroll
    for (int c = 0; c < TILES; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red_o[(wave * heads + n) * D + att_channel<D, BITS>(4 * b + r, c)] =
            o[c][r] * kUnit - oz[r];
  }
  __syncthreads();
  const int64_t head0 = (int64_t)seq * Hq + hk * ratio + h0;
  if (tid < kAttHeads) {
    float mx = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kAttWaves; ++w) mx = fmaxf(mx, red_m[w * kAttHeads + n]);
#pragma unroll
    for (int w = 0; w < kAttWaves; ++w) {
      const float mw = red_m[w * kAttHeads + n];
      const float f = mw == -INFINITY ? 0.f : exp2f(fmaf(mw - mx, factor, -red_f[w * kAttHeads + n]));
      share[w * kAttHeads + n] = f;
      sum = fmaf(f, red_l[w * kAttHeads + n], sum);
    }
    share[kAttWaves * kAttHeads + n] = sum == 0.f ? 0.f : 1.f / sum;  // (the top's own weight is 1: 0 is no token)
    if (!whole && n < heads) {
      const int64_t at = (int64_t)slot * Hq + hk * ratio + h0 + n;
      part_ml[2 * at] = mx;
      part_ml[2 * at + 1] = sum;
    }
  }
  __syncthreads();
  for (int i = tid; i < heads * D / 4; i += 64 * kAttWaves) {
    const int h = i / (D / 4), d = (i - h * (D / 4)) * 4;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kAttWaves; ++w) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(red_o + (w * heads + h) * D + d);
      const float f = share[w * kAttHeads + h];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(f, v[e], acc[e]);
    }
    if (whole) {
      const float f = share[kAttWaves * kAttHeads + h];
      *reinterpret_cast<u32x2*>(out + (head0 + h) * D + d) =
          u32x2{as_u32(f16x2{(f16)(acc[0] * f), (f16)(acc[1] * f)}), as_u32(f16x2{(f16)(acc[2] * f), (f16)(acc[3] * f)})};
    } else {
      *reinterpret_cast<f32x4*>(part_o + ((int64_t)slot * Hq + hk * ratio + h0 + h) * D + d) = acc;
    }
  }
}

// Joins the pieces of one query head of one sequence: D x parts threads, part p
// taking pieces p, p + parts, ...; the parts are summed in order.
__global__ __launch_bounds__(1024) void kv_join_kernel(const float* __restrict__ part_o,
                                                       const float* __restrict__ part_ml,
                                                       const int32_t* __restrict__ meta, AttSplit sp, KvShape sh,
                                                       int Hq, float factor, f16* __restrict__ out) {
  __shared__ float red[2 * 1024], top[16];
  const int64_t head = blockIdx.x;
  const int D = (int)blockDim.x, d = (int)threadIdx.x, part = (int)threadIdx.y, parts = (int)blockDim.y;
  const int tid = part * D + d, threads = parts * D;
  const int seq = (int)blockIdx.x / Hq;
  int used, slot0;
  if (sp.chunk == 0) {
    slot0 = meta[2 * seq];
    used = meta[2 * seq + 1];
  } else {
    used = (int)((kv_length(sh, sp.lengths[seq], sp.width, sp.max_len) + sp.chunk - 1) / sp.chunk);
    slot0 = seq * sp.chunks;
  }
  if (used <= 1) return;  // stored by its only block
  const int64_t row0 = (int64_t)slot0 * Hq + (head - (int64_t)seq * Hq);
  const float* ml = part_ml + row0 * 2;
  const float* po = part_o + row0 * D + d;
  float mx = -INFINITY;
  for (int c = tid; c < used; c += threads) mx = fmaxf(mx, ml[(int64_t)c * Hq * 2]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, kWave));
  if ((tid & 63) == 0) top[tid >> 6] = mx;
  __syncthreads();
  for (int w = 0; w < threads / 64; ++w) mx = fmaxf(mx, top[w]);
  float sum = 0.f, acc = 0.f;
#pragma unroll 4
  for (int c = part; c < used; c += parts) {
    const float m = ml[(int64_t)c * Hq * 2];
    const float f = m == -INFINITY ? 0.f : exp2f((m - mx) * factor);
    sum = fmaf(f, ml[(int64_t)c * Hq * 2 + 1], sum);
    acc = fmaf(f, po[(int64_t)c * Hq * D], acc);
  }
  red[2 * tid] = acc;
  red[2 * tid + 1] = sum;
  __syncthreads();
  if (part > 0) return;
  for (int p = 1; p < parts; ++p) {
    acc += red[2 * (p * D + d)];
    sum += red[2 * (p * D + d) + 1];
  }
  out[head * D + d] = (f16)(sum == 0.f ? 0.f : acc / sum);  // no token: 0 (a NaN stays one)
}

// The split.  By the bound alone, chunks are a power of two of at least 128 tokens: a
// piece costs a block's start (dependent loads) and end (the joins) beside its steps, so
// chunks grow to 512 tokens while there are more than 512 blocks, and on to 4096 while
// there are more than about one and a half times what the compute units hold at once (by
// the rows' bytes, which size the ring; one at 256 bytes).  Measured, us at chunks of 128 /
// 256 / 512 / 1024 / 2048 / 4096 tokens: one sequence of 30000, 8 heads: 31.2 / 22.5 /
// 19.1 / 19.6; 16 of up to 2000: 20.0 / 18.7 / 16.8 / 17.8 / 22.0 / 21.9; 4 of up to 5000, 32
// heads: 32.0 / 25.0 / 22.8 / 25.3 / 32.5 / 41.2; 64 of up to 6000, 8 heads: 161 / 110 / 91.3 /
// 74.4 / 72.0 / 95.8; 8-bit rows of 256 channels, 4 of up to 9000: 63.7 / 45.8 / 35.4 / 28.4.
// Up to 512 tokens one block does without a join: 9.8 us where four chunks and a second launch
// take 10.8.
// Where the bound leaves a choice (chunks above 128 tokens, several a sequence), batches of
// up to kPieceBatch make it by the lengths on the device instead, which costs a block's
// start up to 1 us and serves page tables made for longer sequences (bounds of 131072
// tokens, by the bound / by the lengths: 8 sequences of 2000 46.4 / 15.6 us, 64 of 2000 to
// 6000 162 / 70, 256 of 1000 196 / 64, 300 of 700 183 / 65) and ragged batches (32 of up to
// 30000 136 / 116); with tight bounds 64 of 4096 61.8 / 62.4, 16 of up to 2000 16.7 / 17.2,
// one of 30000 19.1 / 20.4.
static AttSplit att_split(int64_t B, int64_t Hkv, int ratio, int row_bytes, int64_t max_len) {
  AttSplit sp{};
  sp.max_len = max_len;
  sp.batch = (int)B;
  sp.heads = (int)(Hkv * ((ratio + kAttHeads - 1) / kAttHeads));
  sp.most = row_bytes <= 64 ? 1536 : (row_bytes == 128 ? 1024 : 256);
  auto blocks = [&](int chunk) { return B * sp.heads * ((max_len + chunk - 1) / chunk); };
  sp.chunk = max_len <= 512 ? 512 : kKvUnit;
  while (sp.chunk < 512 && blocks(sp.chunk) > 512) sp.chunk *= 2;
  while (sp.chunk >= 512 && sp.chunk < 4096 && blocks(sp.chunk) > sp.most) sp.chunk *= 2;
  sp.chunks = max_len > 0 ? (int)((max_len + sp.chunk - 1) / sp.chunk) : 1;
  const int64_t pieces = kv_most_pieces(B, (int)max_len, sp.heads, sp.most);
  if (sp.chunk > kKvUnit && sp.chunks > 1 && B <= kPieceBatch && pieces < 65536) {  // (blockIdx.y's limit)
    sp.chunk = 0;
    sp.chunks = (int)pieces;
  }
  return sp;
}

// Pieces that are joined (0: every sequence is one piece).
static int64_t att_slots(const AttSplit& sp) {
  if (sp.chunk == 0) return sp.chunks;
  return sp.chunks > 1 ? (int64_t)sp.batch * sp.chunks : 0;
}

// fp32 outputs and (maximum, sum) of every piece, then by the lengths each sequence's first piece and their number.
size_t kv_attention_workspace(int64_t B, int64_t Hkv, int ratio, int D, int bits, int64_t max_len) {
  const AttSplit sp = att_split(B, Hkv, ratio, D * bits / 8, max_len);
  return (size_t)(att_slots(sp) * Hkv * ratio * (D + 2) + (sp.chunk == 0 ? 2 * B : 0)) * sizeof(float);
}

template <int D, int BITS>
static hipError_t attention_launch(const void* q, int64_t q_stride, KvHalf kc, KvHalf vc, const int32_t* table,
                                   int64_t width, const int32_t* lengths, int64_t B, int ratio, float scale,
                                   int64_t max_len, KvShape sh, void* out, float* ws, hipStream_t st) {
  AttSplit sp = att_split(B, sh.heads, ratio, D * BITS / 8, max_len);
  sp.lengths = lengths;
  sp.width = (int)width;
  const int heads = ratio < kAttHeads ? ratio : kAttHeads;
  const size_t sum = (size_t)(kAttWaves * heads * D + (4 * kAttWaves + 1) * kAttHeads) * sizeof(float);
  const size_t ring = (size_t)kAttWaves * (AttStage<D, BITS>::RING + 64 * sizeof(int)), lds = ring > sum ? ring : sum;
  const dim3 grid((unsigned)sp.heads, (unsigned)sp.chunks, sp.chunk ? (unsigned)B : 1u);
  const int64_t slots = att_slots(sp), Hq = (int64_t)sh.heads * ratio;
  float* part_ml = ws == nullptr ? nullptr : ws + slots * Hq * D;
  int32_t* meta = ws == nullptr ? nullptr : reinterpret_cast<int32_t*>(part_ml + slots * Hq * 2);
  // A scale of 0 is taken as one that leaves a masked score (-infinity) what it is.
  const float factor = std::fmax(std::fabs(scale) * 1.4426950408889634f * att_unit(BITS), 7.888609e-31f);
  kv_attention_kernel<D, BITS><<<grid, dim3(64 * kAttWaves), lds, st>>>(
      reinterpret_cast<const f16*>(q), q_stride, kc, vc, table, sp, sh, ratio, std::copysign(factor, scale),
      reinterpret_cast<f16*>(out), ws, part_ml, meta);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || slots == 0) return e;
  const int64_t pieces = sp.chunk ? sp.chunks : (sp.most / sp.heads + B) / B;
  int parts = 1;  // about eight pieces a part
  while (parts * D < 1024 && 8 * parts < pieces) parts *= 2;
  kv_join_kernel<<<dim3((unsigned)(B * Hq)), dim3(D, parts), 0, st>>>(ws, part_ml, meta, sp, sh, (int)Hq, factor,
                                                                     reinterpret_cast<f16*>(out));
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
