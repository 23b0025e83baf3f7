// The next token of each row of logits: temperature, top-k, top-p and min-p, and
// the choice by a given random number, without sorting the row.
//
// One block takes one row.  The order of the tokens (logit descending, then index)
// only matters at the border of what is kept, which a search digit by digit over
// the logits' order-preserving images finds: by counts for top-k, by weights for
// top-p.  Weights are whole multiples of 2^-43, so their sums are the same in any
// order and the result does not depend on timing.  The choice itself walks the
// row's sums in index order.
#include "awq_internal.h"
#include "row_common.h"

namespace awq {

constexpr int kSampleThreads = 1024, kSampleWaves = kSampleThreads / 64;
constexpr double kWeightOne = 8796093022208.0;  // 2^43: a row of 2^20 tokens sums to at most 2^63

// Order-preserving image of a logit; 0: one that is never chosen (-inf, NaN).
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 becomes +0
  return v > -INFINITY ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__shfl((int)(uint32_t)v, lane, kWave) |
         (uint64_t)(uint32_t)__shfl((int)(uint32_t)(v >> 32), lane, kWave) << 32;
}
__device__ __forceinline__ uint64_t scan64(uint64_t v) {  // inclusive, over the wave
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t o = shfl64(v, lane >= d ? lane - d : lane);
    v += lane >= d ? o : 0;
  }
  return v;
}

// A row's 16-byte pieces: piece j holds the E elements from j E - lead on.
template <typename T>
struct LogitRow {
  static constexpr int E = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(E)));
  const T* base;  // 16-byte aligned, lead elements before the row
  int lead, V, pieces;
  __device__ LogitRow(const T* row, int V_) : V(V_) {
    lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    base = row - lead;
    pieces = (lead + V + E - 1) / E;
  }
  // keys of the piece's elements; 0 outside the row
  __device__ __forceinline__ void keys(int j, uint32_t (&k)[E]) const {
    const int first = j * E - lead;
    if (first >= 0 && first + E <= V) {
      const vec v = *reinterpret_cast<const vec*>(base + (int64_t)j * E);
#pragma unroll
      for (int u = 0; u < E; ++u) k[u] = logit_key((float)v[u]);
    } else {
#pragma unroll
      for (int u = 0; u < E; ++u)
        k[u] = first + u >= 0 && first + u < V ? logit_key((float)base[(int64_t)j * E + u]) : 0u;
    }
  }
};

// The kept part of a row: tokens above key, and of those equal to it the indices up to last.
struct Border {
  uint32_t key;
  int last;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= last); }
};

struct Weigher {
  double top, by;  // largest logit, 1 / temperature
  float topf;
  __device__ __forceinline__ double operator()(uint32_t key) const {
    const float v = key_logit(key);
    if (v == topf) return 1.0;
    const double z = ((double)v - top) * by;
    return z > -31.0 ? exp(z) : 0.0;  // below 2^-44; false for a NaN (infinite logits, infinite temperature)
  }
};
__device__ __forceinline__ uint64_t fixed(double w) { return (uint64_t)rint(w * kWeightOne); }

template <typename T>
struct SampleRow {
  LogitRow<T> row;
  uint64_t* sums;     // [chunks]: of each wave's 64 pieces
  uint64_t* weights;  // [256]
  uint32_t* counts;   // [256]
  uint64_t* found;    // [4]
  static constexpr int E = LogitRow<T>::E;

  // sums[c] of amount(key, index) over chunk c; returns the row's sum.
  template <typename F>
  __device__ uint64_t chunk_sums(F amount) {
    const int lane = threadIdx.x & 63, chunks = (row.pieces + 63) / 64;
    for (int c = threadIdx.x >> 6; c < chunks; c += kSampleWaves) {
      const uint64_t s = scan64(piece_sum(c * 64 + lane, amount));
      if (lane == 63) sums[c] = s;
    }
    __syncthreads();
    uint64_t total = 0;
    for (int c = lane; c < chunks; c += 64) total += sums[c];
    return shfl64(scan64(total), 63);
  }
  template <typename F>
  __device__ uint64_t piece_sum(int j, F amount) const {
    uint64_t s = 0;
    if (j < row.pieces) {
      uint32_t k[E];
      row.keys(j, k);
#pragma unroll
      for (int u = 0; u < E; ++u)
        if (k[u] != 0) s += amount(k[u], j * E - row.lead + u);
    }
    return s;
  }

  // After chunk_sums: the first index at which the sums exceed `target` (below the total), and
  // its key; by the first wave, returned to every thread.
  template <typename F>
  __device__ int locate(uint64_t target, F amount, uint32_t* key) {
    const int lane = threadIdx.x & 63, chunks = (row.pieces + 63) / 64;
    if (threadIdx.x < 64) {
      uint64_t before = 0;
      int c0 = 0;
      for (; c0 < chunks; c0 += 64) {
        const uint64_t upto = scan64(c0 + lane < chunks ? sums[c0 + lane] : 0);
        const uint64_t over = __ballot(before + upto > target);
        if (over != 0) {
          const int at = __builtin_ctzll(over);
          c0 += at;
          before += at == 0 ? 0 : shfl64(upto, at - 1);
          break;
        }
        before += shfl64(upto, 63);
      }
      const int j = c0 * 64 + lane;
      const uint64_t mine = piece_sum(j, amount), upto = before + scan64(mine);
      const uint64_t over = __ballot(upto > target);
      if (over != 0 && lane == __builtin_ctzll(over)) {
        uint64_t sum = upto - mine;
        uint32_t k[E];
        row.keys(j, k);
        bool done = false;
#pragma unroll
        for (int u = 0; u < E; ++u)
          if (!done && k[u] != 0) {
            sum += amount(k[u], j * E - row.lead + u);
            if (sum > target) {
              done = true;
              found[0] = (uint64_t)(uint32_t)(j * E - row.lead + u);
              found[1] = k[u];
            }
          }
      }
    }
    __syncthreads();
    const int index = (int)found[0];
    *key = (uint32_t)found[1];
    __syncthreads();
    return index;
  }

  // The border below which nothing is kept, searched within what `b` keeps: of the tokens in
  // order, the one at which count (rank_at > 0: the rank_at-th token) or weight (the first
  // token with the weight up to it at least `least`) is reached.  b stays where it is not reached.
  __device__ void cut(Border* b, const Weigher& weigher, uint64_t rank_at, double least) {
    const bool by_count = rank_at > 0;
    uint32_t prefix = 0;
    uint64_t above = 0;    // counts or weights of the tokens above the digits fixed so far
    uint64_t equal = 0;    // tokens with the key found
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSampleThreads) {
        counts[i] = 0;
        weights[i] = 0;
      }
      __syncthreads();
      for (int j = threadIdx.x; j < row.pieces; j += kSampleThreads) {
        uint32_t k[E];
        row.keys(j, k);
#pragma unroll
        for (int u = 0; u < E; ++u)
          if (k[u] != 0 && b->keeps(k[u], j * E - row.lead + u) &&
              (shift == 24 || (k[u] >> (shift + 8)) == prefix)) {
            const uint32_t d = (k[u] >> shift) & 255u;
            atomicAdd(&counts[d], 1u);
            if (!by_count) atomicAdd(reinterpret_cast<unsigned long long*>(&weights[d]), (unsigned long long)fixed(weigher(k[u])));
          }
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        found[0] = 256;
        uint64_t sum = above;
        for (int d = 255; d >= 0; --d) {
          if (counts[d] == 0) continue;
          const uint64_t next = sum + (by_count ? counts[d] : weights[d]);
          if (by_count ? next >= rank_at : (double)next >= least) {
            found[0] = d;
            found[1] = sum;
            found[2] = counts[d];
            break;
          }
          sum = next;
        }
      }
      __syncthreads();
      const uint32_t d = (uint32_t)found[0];
      above = found[1];
      equal = found[2];
      __syncthreads();
      if (d == 256) return;  // not reached: everything stays
      prefix = prefix << 8 | d;
    }
    // of the `equal` tokens with that key, the first ones
    uint64_t stay;
    if (by_count) {
      stay = rank_at - above;
    } else {
      const uint64_t one = fixed(weigher(prefix));
      stay = 1;
      while (stay < equal && (double)(above + stay * one) < least) {
        const double more = one > 0 ? floor((least - (double)(above + stay * one)) / (double)one) : 1.0;
        stay += more < 1.0 ? 1 : more < (double)(equal - stay) ? (uint64_t)more : equal - stay;
      }
    }
    int last = b->last;
    if (prefix > b->key) last = 0x7FFFFFFF;
    if (stay < equal) {
      const Border old = *b;
      const uint32_t key = prefix;
      auto is = [=](uint32_t k, int i) -> uint64_t { return k == key && old.keeps(k, i) ? 1 : 0; };
      chunk_sums(is);
      uint32_t unused;
      last = locate(stay - 1, is, &unused);
    }
    b->key = prefix;
    b->last = last;
  }
};

template <typename T>
__global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleArgs a) {
  extern __shared__ uint64_t sums[];
  __shared__ uint64_t weights[256], found[4], part[kSampleWaves];
  __shared__ uint32_t counts[256];
  const int64_t r = blockIdx.x;
  SampleRow<T> s{LogitRow<T>(reinterpret_cast<const T*>(a.logits) + r * a.stride, (int)a.V), sums, weights, counts, found};
  constexpr int E = SampleRow<T>::E;
  const float t = a.temperature ? a.temperature[r] : a.temperature_value;
  const int32_t k = a.top_k ? a.top_k[r] : a.top_k_value;
  const float p = a.top_p ? a.top_p[r] : a.top_p_value, m = a.min_p ? a.min_p[r] : a.min_p_value, u = a.u[r];

  uint64_t best = 0;  // the largest logit's image above the complement of its first index
  for (int j = threadIdx.x; j < s.row.pieces; j += kSampleThreads) {
    uint32_t key[E];
    s.row.keys(j, key);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint64_t c = (uint64_t)key[e] << 32 | (uint32_t)~(j * E - s.row.lead + e);
      best = key[e] != 0 && c > best ? c : best;
    }
  }
  for (int d = 32; d >= 1; d /= 2) {
    const uint64_t o = shfl64(best, (threadIdx.x & 63) ^ d);
    best = o > best ? o : best;
  }
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = best;
  __syncthreads();
  for (int i = 0; i < kSampleWaves; ++i) best = part[i] > best ? part[i] : best;

  const uint32_t top_key = (uint32_t)(best >> 32);
  const int first = (int)~(uint32_t)best;
  if (best == 0 || !(t > 0.f)) {
    if (threadIdx.x == 0) {
      a.tokens[r] = best == 0 ? -1 : first;
      if (a.probs) a.probs[r] = best == 0 ? 0.f : 1.f;
    }
    return;
  }
  const Weigher weigher{(double)key_logit(top_key), 1.0 / (double)t, key_logit(top_key)};
  Border b{0u, 0x7FFFFFFF};
  if (k >= 1 && k < a.V) s.cut(&b, weigher, (uint64_t)k, 0.0);
  if (p < 1.f) {
    const uint64_t all = s.chunk_sums([&](uint32_t key, int i) -> uint64_t { return b.keeps(key, i) ? fixed(weigher(key)) : 0; });
    __syncthreads();
    s.cut(&b, weigher, 0, (double)p * (double)all);
  }
  const double low = m > 0.f ? (double)m : 0.0;
  auto amount = [&](uint32_t key, int i) -> uint64_t {
    if (!b.keeps(key, i)) return 0;
    const double w = weigher(key);
    return w >= low || i == first ? fixed(w) : 0;
  };
  const uint64_t total = s.chunk_sums(amount);
  const double at = (u > 0.f ? (double)u : 0.0) * (double)total;
  const uint64_t target = at < (double)total ? (uint64_t)at : total - 1;
  uint32_t key;
  const int token = s.locate(target < total ? target : total - 1, amount, &key);
  if (threadIdx.x == 0) {
    a.tokens[r] = token;
    if (a.probs) a.probs[r] = (float)(weigher(key) * kWeightOne / (double)total);
  }
}

size_t sample_workspace(int64_t, int64_t, int) { return 0; }

hipError_t launch_sample(const SampleArgs& a, int logit_bytes, int64_t B, hipStream_t st) {
  const int per = 64 * 16 / logit_bytes;  // elements of a chunk
  const size_t lds = (size_t)((a.V + 16 + per - 1) / per) * sizeof(uint64_t);
  const dim3 grid((unsigned)B), block(kSampleThreads);
  if (logit_bytes == 2) sample_kernel<f16><<<grid, block, lds, st>>>(a);
  else sample_kernel<float><<<grid, block, lds, st>>>(a);
  return hipGetLastError();
}

}  // namespace awq
