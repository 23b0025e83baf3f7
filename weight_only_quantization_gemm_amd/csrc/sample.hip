// The next token of each row of logits: temperature, top-k, top-p and min-p, and
// the choice by a given random number, without sorting the row.
//
// One block takes one row.  A first pass finds the largest logit and leaves each
// thread the largest of its 16-byte pieces, so later steps read again only what
// they need.  What is kept is always a first part of the tokens in order (logit
// descending, then index), so all that has to be found is its border:
//   few tokens kept (top-k up to kListK, or min-p alone): a logit that at least k
//   threads' own maxima reach leaves a list short enough to sort;
//   otherwise: a histogram of the weights (or counts) over equal steps of the
//   logit finds the border's bin; a further pass lists that bin's tokens, which are
//   sorted, and sums the weights of those above it by chunks of 64 pieces.  A bin
//   with more tokens than the list holds (ties) is searched digit by digit instead.
// The choice walks sums in index order: of chunks, then of the chosen chunk's pieces.
//
// Weights are whole multiples of 2^-43, so their sums are exact in any order and
// the result does not depend on timing.  A row's sum is at most 2^63 (2^20 equal logits), which takes
// the 64 bits without a sign.
//
// Bounds and times (fp16 logits, out of the caches; 61 x 50021 and 512 x 131072, whose one read takes 2.6 and 21 us in
// a kernel that only reads).  Lists: the chain of a first pass, 20 barriers and a short sort: top-k 50, top-p
// and min-p 14 and 42 us (1 x 32000 9.5), min-p alone 13 and 48; greedy, a first pass and a search, 8 and 45.
// Passes over all weights: vector instructions, some 20 a token (a weight alone is 16 in 64 bits) on the row's compute
// unit: unfiltered 20 and 92 us, top-p 0.9 45 and 181, of which histogram and border pass take 17 us each at
// 50021 tokens; top-k 3000 and top-p 70 and 273.
#include "awq_internal.h"
#include "row_common.h"

namespace awq {

constexpr double kWeightOne = 8796093022208.0;  // 2^43
constexpr double kHalfUnit = 4503599627370496.0;  // 2^52, from where on a double's spacing is 1
constexpr int kExpTable = 512, kSlots = 16;
constexpr double kExpRate = 738.6598609351493;  // kExpTable log2(e)

// 2^(43 + j / kExpTable), 0 <= j < kExpTable: the series of the exponential about 0 to the 12th power, whose next
// term is below 2^-52 for the nearer whole power of 2.
__device__ __forceinline__ double exp_entry(int j) {
  const bool upper = j >= kExpTable / 2;
  const double x = (upper ? j - kExpTable : j) * (0.69314718055994530942 / kExpTable);
  double sum = 1.0 / 479001600.0;  // 1 / 12!
  sum = fma(sum, x, 1.0 / 39916800.0);
  sum = fma(sum, x, 1.0 / 3628800.0);
  sum = fma(sum, x, 1.0 / 362880.0);
  sum = fma(sum, x, 1.0 / 40320.0);
  sum = fma(sum, x, 1.0 / 5040.0);
  sum = fma(sum, x, 1.0 / 720.0);
  sum = fma(sum, x, 1.0 / 120.0);
  sum = fma(sum, x, 1.0 / 24.0);
  sum = fma(sum, x, 1.0 / 6.0);
  sum = fma(sum, x, 0.5);
  sum = fma(sum, x, 1.0);
  sum = fma(sum, x, 1.0);
  return sum * (upper ? 2.0 * kWeightOne : kWeightOne);
}

// Order-preserving image of a logit (never 0 for one that can be chosen: not -inf, not NaN).
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 becomes +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t shifted64(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t scan64(uint64_t v) {  // inclusive, over the wave
  v += shifted64<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8, then the rows' sums to the rows above
  v += shifted64<0x112, 0xF>(v);
  v += shifted64<0x114, 0xF>(v);
  v += shifted64<0x118, 0xF>(v);
  v += shifted64<0x142, 0xA>(v);
  v += shifted64<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ uint64_t lane64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32;
}

// A wave's largest (smallest) value, in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float shifted(float v, float none) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, shifted<0x111, 0xF>(v, -INFINITY));
  v = fmaxf(v, shifted<0x112, 0xF>(v, -INFINITY));
  v = fmaxf(v, shifted<0x114, 0xF>(v, -INFINITY));
  v = fmaxf(v, shifted<0x118, 0xF>(v, -INFINITY));
  v = fmaxf(v, shifted<0x142, 0xA>(v, -INFINITY));
  v = fmaxf(v, shifted<0x143, 0xC>(v, -INFINITY));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_min(float v) { return -wave_max(-v); }

template <int THREADS>
struct SampleShared {
  static constexpr int kList = 5 * THREADS, kSort = 2 * THREADS, kBins = 2 * THREADS, kFound = 5 * THREADS;
  uint64_t list[kList];  // up to kSort entries, the bins' weights, or tokens that wait to be weighed
  union {
    uint32_t counts[kBins];         // the bins' counts
    uint32_t slots[kFound];         // slots with tokens for the list
    uint64_t chunks[kFound / 2];    // sums of what is kept, for each 64 pieces
  };
  double table[kExpTable];  // exp_entry
  uint64_t part[2][THREADS / 64];
  uint64_t found[4];
  float most[THREADS / 64], least[THREADS / 64];
  int n;
};

// What is kept: tokens above value, and of those equal to it the indices up to last.
struct Border {
  float value;
  int last;
  __device__ __forceinline__ bool keeps(float x, int i) const {
    return (x > value) | ((x == value) & (i <= last));  // without branches
  }
};

template <typename T, int THREADS>
struct SampleRow {
  static constexpr int E = 16 / sizeof(T), WAVES = THREADS / 64;
  typedef SampleShared<THREADS> Shared;
  static constexpr int kList = Shared::kList, kSort = Shared::kSort, kBins = Shared::kBins, kFound = Shared::kFound;
  typedef T vec __attribute__((ext_vector_type(E)));
  SampleShared<THREADS>& sh;
  __amdgpu_buffer_rsrc_t resource;  // from the 16-byte piece with the row's first element to the row's end
  int lead, V, cw;   // cw: chunks (64 pieces) of a wave; wave w has chunks w cw .. w cw + cw - 1
  bool infinite;     // some logit is +inf: those weigh 1 and all others nothing
  double top, rate;  // largest logit, kExpTable log2(e) / temperature

  // Piece j: elements j E - lead .. + E - 1.  Read with the hardware's bound at the row's end (a half's word there
  // may hold the next half too); before the row's start there are only other rows.
  __device__ __forceinline__ vec read(int j) const {
    return __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b128(resource, j * 16, 0, 0));
  }
  __device__ __forceinline__ bool whole(int j) const { return j * E >= lead && (j + 1) * E - lead <= V; }
  // The elements outside the row become NaN.
  __device__ __forceinline__ vec trim(vec x, int j) const {
    if (!whole(j)) {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = j * E + e >= lead && j * E + e - lead < V ? x[e] : (T)__builtin_nanf("");
    }
    if (infinite)
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = (float)x[e] == INFINITY ? (T)0.f : (T)-INFINITY;
    return x;
  }
  __device__ __forceinline__ vec load(int j) const { return trim(read(j), j); }
  __device__ __forceinline__ int piece(int u) const { return ((int)(threadIdx.x >> 6) * cw + u) * 64 + (threadIdx.x & 63); }
  static __device__ __forceinline__ float largest(vec x) {
    if constexpr (E == 8) {
      const auto a = __builtin_elementwise_max(x.lo, x.hi);
      const auto b = __builtin_elementwise_max(a.lo, a.hi);
      return fmaxf((float)b.x, (float)b.y);
    } else {
      // A signalling NaN would take its neighbour along in the three-way maximum that this becomes.
      auto quiet = [](float v) { return __builtin_canonicalizef(v); };
      return fmaxf(fmaxf(quiet(x[0]), quiet(x[1])), fmaxf(quiet(x[2]), quiet(x[3])));
    }
  }
  // f(piece, its number) for this thread's pieces, two under way.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    vec next = read(piece(0)), after = read(piece(1));
#pragma unroll 1
    for (int u = 0; u < cw; ++u) {
      const vec x = next;
      next = after;
      after = read(piece(u + 2));
      f(trim(x, piece(u)), piece(u));
    }
  }

  // The weight times 2^43, rounded to a whole number: with y = z 512 / ln 2 = i + f, i whole,
  //   exp(z) = 2^(i / 512) (1 + g),  g = exp(f ln2 / 512) - 1 to the third power of f, |f| <= 1/2
  // (the fourth is below 2^-46).  Below z = -31 it is none, and for a NaN.  Whole parts are split off
  // by adding and subtracting 1.5 2^52 and 2^52.
  __device__ __forceinline__ double unrounded(float x) const {
    constexpr double c1 = 0.0013538030870311431, c2 = 9.163913992275265e-07, c3 = 4.1353783506767136e-10;  // (ln2/512)^n / n!
    constexpr double kWhole = 6755399441055744.0;
    const double y = fmax(((double)x - top) * rate, -31.0 * kExpRate);
    const double shifted = y + kWhole, f = y - (shifted - kWhole);
    const int i = (int)(uint32_t)__double_as_longlong(shifted);
    const uint64_t t = (uint64_t)__double_as_longlong(sh.table[i & (kExpTable - 1)]);
    const double two = __longlong_as_double((int64_t)(t + ((uint64_t)(uint32_t)((i & -kExpTable) << (20 - 9)) << 32)));
    return fma(two, f * fma(f, fma(f, c3, c2), c1), two);
  }
  __device__ __forceinline__ double weight(float x) const {
    return (unrounded(x) + kHalfUnit) - kHalfUnit;
  }

  // The same as a whole number: adding 2^52 leaves it in the double's low bits.
  static __device__ __forceinline__ uint64_t whole(double unrounded) {
    return (uint64_t)__double_as_longlong(unrounded + kHalfUnit) - (uint64_t)__double_as_longlong(kHalfUnit);
  }
  // Those of a piece, with ALL of every token, otherwise of what b keeps from low on (0 for others); side
  // by side, so that the table's latency is paid once.
  template <bool ALL>
  __device__ __forceinline__ void weights(vec x, int j, const Border& b, double low, uint64_t (&w)[E]) const {
    double v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = unrounded((float)x[e]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (!ALL) v[e] = (b.keeps((float)x[e], j * E - lead + e) & (v[e] >= low)) ? v[e] : 0.0;
      w[e] = whole(v[e]);
    }
  }

  __device__ __forceinline__ uint64_t target_of(float share, uint64_t total) const {
    const double at = (share > 0.f ? (double)share : 0.0) * (double)total;
    const uint64_t target = at < (double)total ? (uint64_t)at : total - 1;
    return target < total ? target : total - 1;
  }

  // Sum over the block; inclusive sums up to this thread in *upto where asked for.
  __device__ __forceinline__ uint64_t block_sum(uint64_t mine, int which, uint64_t* upto = nullptr) const {
    const uint64_t s = scan64(mine);
    if ((threadIdx.x & 63) == 63) sh.part[which][threadIdx.x >> 6] = s;
    lds_barrier();
    // the waves' sums, one a lane: a single access instead of one for each wave
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t waves = scan64(lane < WAVES ? sh.part[which][lane] : 0);
    if (upto) *upto = (wave > 0 ? lane64(waves, wave - 1) : 0) + s;
    return lane64(waves, WAVES - 1);
  }

  static __device__ __forceinline__ uint64_t entry(float x, int i) { return (uint64_t)logit_key(x) << 32 | (uint32_t)~i; }
  static __device__ __forceinline__ float entry_logit(uint64_t e) { return key_logit((uint32_t)(e >> 32)); }

  // Sorts list[0 .. n) descending (n <= kSort); its entries differ.  Each wave ranks runs of 64 by comparing every pair,
  // then every entry looks its place up in the other runs.
  __device__ __forceinline__ void sort(int n) const {
    constexpr int Q = kSort / THREADS;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, runs = (n + 63) / 64;
    uint64_t e[Q];
    int rank[Q];
    lds_barrier();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int run = q * WAVES + wave;
      e[q] = 0;
      rank[q] = 0;
      if (run < runs) {
        e[q] = run * 64 + lane < n ? sh.list[run * 64 + lane] : 0;
#pragma unroll 4
        for (int j = 0; j < 64; ++j) rank[q] += lane64(e[q], j) > e[q] ? 1 : 0;
        rank[q] = e[q] == 0 ? lane : rank[q];  // behind the last run's entries
        sh.list[run * 64 + rank[q]] = e[q];
      }
    }
    lds_barrier();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int run = q * WAVES + wave;
      if (run < runs)
#pragma unroll 1
        for (int other = 0; other < runs; ++other) {
          if (other == run) continue;
          int above = 0;  // of the other run
#pragma unroll
          for (int step = 32; step > 0; step /= 2) above += sh.list[other * 64 + above + step - 1] > e[q] ? step : 0;
          rank[q] += above + (sh.list[other * 64 + above] > e[q] ? 1 : 0);
        }
    }
    lds_barrier();
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (e[q] != 0) sh.list[rank[q]] = e[q];
    lds_barrier();
  }

  // A piece's elements with bits in `in` to the list's end (sh.n, which counts on beyond kSort); by whole waves, with
  // one access to it for each.
  __device__ __forceinline__ void append(vec x, int j, uint32_t in) const {
    const int count = __popc(in), upto = wave_scan(count);
    int at = 0;
    if ((threadIdx.x & 63) == 0) at = atomicAdd(&sh.n, __builtin_amdgcn_readlane(upto, 63));
    at = __builtin_amdgcn_readfirstlane(at) + upto - count;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if ((in >> e & 1) && at < kSort) sh.list[at] = entry((float)x[e], j * E - lead + e);
      at += in >> e & 1;
    }
  }

  // list = the tokens that reach `least` with weights from low on, in any order, and returns their number (more than
  // kSort: only some are in the list).  most: the largest logits of this thread's slots (slot q: pieces q, q + kSlots,
  // .. of it).
  __device__ __forceinline__ int gather(const float (&most)[kSlots], float least, double low) const {
    uint32_t slots = 0;
    const float finite = fmaxf(least, -3.4028235e38f);  // not -inf, a slot without a logit
#pragma unroll
    for (int q = 0; q < kSlots; ++q) slots |= most[q] >= finite ? 1u << q : 0u;
    if (threadIdx.x == 0) {
      sh.n = 0;
      sh.found[0] = 0;
    }
    lds_barrier();
    const int mine = __popc(slots), upto = wave_scan(mine), all = __builtin_amdgcn_readlane(upto, 63);
    int place = 0;  // one access a wave: thousands to one address take their time
    if ((threadIdx.x & 63) == 0 && all > 0) place = atomicAdd(reinterpret_cast<int*>(&sh.found[0]), all);
    place = __builtin_amdgcn_readfirstlane(place) + upto - mine;
#pragma unroll 1
    for (; slots != 0; slots &= slots - 1, ++place)
      if (place < kFound) sh.slots[place] = (uint32_t)piece(__builtin_ctz(slots));
    lds_barrier();
    const int slots_found = __builtin_amdgcn_readfirstlane((int)(uint32_t)sh.found[0]);
    if (slots_found <= kFound) {
#pragma unroll 1
      for (int s0 = threadIdx.x & ~63; s0 < slots_found; s0 += THREADS) {  // whole waves
        const int s = s0 + (threadIdx.x & 63), j0 = s < slots_found ? (int)sh.slots[s] : 0;
        const int end = s < slots_found ? ((j0 / 64) / cw + 1) * cw * 64 : 0;  // of its wave's chunks
#pragma unroll 1
        for (int j = j0; __any(j < end); j += kSlots * 64) {
          const vec x = load(j < end ? j : 0);
          uint32_t in = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) in |= ((j < end) & ((float)x[e] >= finite)) ? 1u << e : 0u;
          if (low > 0.0)
#pragma unroll
            for (int e = 0; e < E; ++e) in &= unrounded((float)x[e]) >= low ? ~0u : ~(1u << e);
          if (__any(in != 0)) append(x, j, in);
        }
      }
    }
    lds_barrier();
    const int n = slots_found <= kFound ? __builtin_amdgcn_readfirstlane(sh.n) : kSort + 1;
    lds_barrier();
    return n;
  }

  // A logit that at least k tokens reach (-inf: all of them): the threads' largest logits counted over
  // equal steps from hi down by `range`, the smallest of them in the steps that hold the first k.
  __device__ __forceinline__ float reached_by(int k, float mine, float hi, float range) const {
    constexpr int STEPS = 256;
    const float step = fminf((float)STEPS / range, 1e30f);
    const int bin = (int)fminf((hi - mine) * step, (float)(STEPS - 1));
    if (threadIdx.x < STEPS) sh.counts[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.found[0] = STEPS;
    lds_barrier();
    if (mine > -INFINITY) atomicAdd(&sh.counts[bin], 1u);
    lds_barrier();
    if (threadIdx.x < 64) {
      int count[4], sum = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += count[q] = (int)sh.counts[4 * threadIdx.x + q];
      int before = wave_scan(sum) - sum;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (before < k && before + count[q] >= k) sh.found[0] = 4 * threadIdx.x + q;
        before += count[q];
      }
    }
    lds_barrier();
    const int last = __builtin_amdgcn_readfirstlane((int)sh.found[0]);
    float least = mine > -INFINITY && bin <= last ? mine : INFINITY;
    least = wave_min(least);
    if ((threadIdx.x & 63) == 0) sh.least[threadIdx.x >> 6] = least;
    lds_barrier();
    least = wave_min((threadIdx.x & 63) < WAVES ? sh.least[threadIdx.x & 63] : INFINITY);
    return last == STEPS ? -INFINITY : least;
  }

  // The token at `share` of those of the first n <= 64 entries of the sorted list with weights from low on, by the
  // first wave: lane i has entry i (0 from n on).
  __device__ __forceinline__ void choose_in_wave(uint64_t e, int n, double low, float share) const {
    const double exact = unrounded(entry_logit(e));
    const uint64_t w = (((int)threadIdx.x < n) & (exact >= low)) ? whole(exact) : 0, total = lane64(scan64(w), 63);
    const uint64_t target = target_of(share, total);
    uint64_t sum = 0;  // of the tokens up to this one, by index
#pragma unroll 2
    for (int j = 0; j < n; ++j) {
      const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)e, j);
      sum += other >= (uint32_t)e ? lane64(w, j) : 0;  // complements of the indices
    }
    if ((int)threadIdx.x < n && sum > target && sum - w <= target) {
      sh.found[0] = (uint32_t)e;
      sh.found[1] = (uint64_t)__double_as_longlong(exact / (double)total);
    }
  }
  __device__ __forceinline__ int chosen_in_wave(float* prob) const {
    lds_barrier();
    *prob = (float)__longlong_as_double((int64_t)sh.found[1]);
    return (int)~(uint32_t)sh.found[0];
  }
  // The token at `share` of the up to 64 entries of the list.
  __device__ __forceinline__ int choose_of_few(int n, int k, float p, double low, float share, float* prob) const {
    if (threadIdx.x < 64) {
      const int lane = threadIdx.x;
      uint64_t e = lane < n ? sh.list[lane] : 0;
      int rank = 0;
#pragma unroll 2
      for (int j = 0; j < n; ++j) rank += lane64(e, j) > e ? 1 : 0;
      if (lane < n) sh.list[rank] = e;  // a wave's accesses are done in order
      __asm__ volatile("" ::: "memory");
      e = lane < n ? sh.list[lane] : 0;
      if (k >= 1 && k < n) n = k;
      const uint64_t w = lane < n ? (uint64_t)weight(entry_logit(e)) : 0;
      const uint64_t upto = scan64(w);
      const double least = (double)p * (double)lane64(upto, 63);
      const bool in = lane < n && (lane == 0 || p >= 1.f || (double)(upto - w) < least);
      choose_in_wave(e, __popcll(__ballot(in)), low, share);
    }
    return chosen_in_wave(prob);
  }

  // The border with the list's entry i the last one kept.
  __device__ __forceinline__ Border border_of(int i) const {
    const uint64_t e = lane64(sh.list[i], 0);
    return {entry_logit(e), (int)~(uint32_t)e};
  }
  // Whether sh.chunks holds a sum for each chunk of the row.
  __device__ __forceinline__ int chunks() const { return ((lead + V + E - 1) / E + 63) / 64; }
  __device__ __forceinline__ bool chunks_fit() const { return chunks() <= kFound / 2; }

  // Of the sorted list's first n entries, how many top-k and top-p keep.  (min-p is asked of each token's unrounded
  // weight wherever tokens are weighed for the choice, so that it does not depend on the way they were found.)
  __device__ __forceinline__ int kept_of_list(int n, int k, float p) const {
    constexpr int Q = kSort / THREADS;
    if (k >= 1 && k < n) n = k;
    double w[Q];
    uint64_t upto[Q], carry = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = q * THREADS + threadIdx.x;
      w[q] = 0.0;
      upto[q] = 0;
      if (q * THREADS < n) {
        w[q] = i < n ? weight(entry_logit(sh.list[i])) : 0.0;
        const uint64_t all = block_sum((uint64_t)w[q], q & 1, &upto[q]);
        upto[q] += carry;
        carry += all;
      }
    }
    const double least = (double)p * (double)carry;
    uint64_t kept = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = q * THREADS + threadIdx.x;
      const bool in = i < n && (p >= 1.f || (double)(upto[q] - (uint64_t)w[q]) < least);
      kept += i == 0 || in ? 1 : 0;
    }
    lds_barrier();
    return __builtin_amdgcn_readfirstlane((int)block_sum(kept, 0));
  }

  // The token at `target` of what b keeps in the 64 pieces of a chunk, with weights from low on; by every thread.
  __device__ __forceinline__ int choose_of_chunk(int chunk, uint64_t target, uint64_t total, const Border& b, double low,
                                                 float* prob) const {
    if (threadIdx.x < 64) {
      const int j = chunk * 64 + (int)threadIdx.x;
      const vec x = load(j);
      uint64_t we[E], own = 0;
      weights<false>(x, j, b, low, we);
#pragma unroll
      for (int e = 0; e < E; ++e) own += we[e];
      const uint64_t upto = scan64(own), over = __ballot(upto > target);
      if ((int)threadIdx.x == __builtin_ctzll(over)) {
        uint64_t sum = upto - own;
        bool done = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          sum += we[e];
          if (!done && sum > target) {
            done = true;
            sh.found[0] = entry((float)x[e], j * E - lead + e);
          }
        }
      }
    }
    lds_barrier();
    const uint64_t e = sh.found[0];
    *prob = (float)(unrounded(entry_logit(e)) / (double)total);
    return (int)~(uint32_t)e;
  }

  // The token at `share` of the first n entries of the list (in any order), which are what b keeps, with weights
  // from low on: their weights summed by chunk, in index order.
  __device__ __forceinline__ int choose_of_list(int n, const Border& b, double low, float share, float* prob) const {
    lds_barrier();
#pragma unroll 1
    for (int i = threadIdx.x; i < chunks(); i += THREADS) sh.chunks[i] = 0;
    lds_barrier();
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += THREADS) {
      const uint64_t e = sh.list[i];
      const double v = unrounded(entry_logit(e));
      const uint64_t w = whole(v >= low ? v : 0.0);
      atomicAdd(reinterpret_cast<unsigned long long*>(&sh.chunks[((int)~(uint32_t)e + lead) / (64 * E)]), (unsigned long long)w);
    }
    return choose_of_chunks(b, low, share, prob);
  }
  // The same with the weights' sums by chunk in sh.chunks.
  __device__ __forceinline__ int choose_of_chunks(const Border& b, double low, float share, float* prob) const {
    const int per = (chunks() + THREADS - 1) / THREADS;
    lds_barrier();
    uint64_t mine = 0, upto;
#pragma unroll 1
    for (int i = threadIdx.x * per; i < (int)(threadIdx.x + 1) * per && i < chunks(); ++i) mine += sh.chunks[i];
    const uint64_t total = block_sum(mine, 0, &upto), target = target_of(share, total);
    if (upto > target && upto - mine <= target) {
      uint64_t left = target - (upto - mine);
      int i = threadIdx.x * per;
#pragma unroll 1
      while (sh.chunks[i] <= left) left -= sh.chunks[i++];
      sh.found[2] = i;
      sh.found[3] = left;
    }
    lds_barrier();
    return choose_of_chunk(__builtin_amdgcn_readfirstlane((int)sh.found[2]), lane64(sh.found[3], 0), total, b, low, prob);
  }

  // The token at `share` of all that b keeps with weights from low on.
  __device__ __forceinline__ int choose_of_row(const Border& b, double low, float share, float* prob) const {
    auto amount = [&](vec x, int j) {
      uint64_t w[E], s = 0;
      weights<false>(x, j, b, low, w);
#pragma unroll
      for (int e = 0; e < E; ++e) s += w[e];
      return s;
    };
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t mine = 0;
    if (b.value == -INFINITY && low == 0.0) {  // everything: without the comparisons
      each([&](vec x, int j) {
        uint64_t w[E];
        weights<true>(x, j, b, low, w);
#pragma unroll
        for (int e = 0; e < E; ++e) mine += w[e];
      });
    } else {
      // Only what b keeps is weighed: each wave lines its tokens up in LDS and takes 64 at a time.
      float* queue = reinterpret_cast<float*>(sh.list) + wave * (kList * 2 / WAVES);
      static_assert(64 * E + 63 <= kList * 2 / WAVES, "a wave's queue");
      int waiting = 0;
      lds_barrier();
      auto take = [&](int n) {  // the last n
        __asm__ volatile("" ::: "memory");  // a wave's LDS accesses are done in order
        waiting -= n;
        const double v = unrounded(queue[waiting + (lane < n ? lane : 0)]);
        mine += whole(((lane < n) & (v >= low)) ? v : 0.0);
        __asm__ volatile("" ::: "memory");
      };
      each([&](vec x, int j) {
        uint32_t in = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) in |= b.keeps((float)x[e], j * E - lead + e) ? 1u << e : 0u;
        const int count = __popc(in), upto = wave_scan(count);
        int at = waiting + upto - count;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (in >> e & 1) queue[at] = (float)x[e];
          at += in >> e & 1;
        }
        waiting += __builtin_amdgcn_readlane(upto, 63);
#pragma unroll 1
        while (waiting >= 64) take(64);
      });
      if (waiting > 0) take(waiting);
    }
    lds_barrier();
    const uint64_t total = block_sum(mine, 0);
    uint64_t target = target_of(share, total);
    // the wave, then its chunk, then the lane and its element
    const uint64_t waves = scan64(lane < WAVES ? sh.part[0][lane] : 0);
    const int w = __builtin_ctzll(__ballot(waves > target));
    target -= w > 0 ? lane64(waves, w - 1) : 0;
#pragma unroll 1
    for (int u = wave; u < cw; u += WAVES) {
      const int j = (w * cw + u) * 64 + lane;
      const uint64_t s = scan64(amount(load(j), j));
      if (lane == 63) sh.list[u] = s;
    }
    lds_barrier();
    int u = 0;
#pragma unroll 1
    for (;; u += 64) {
      const uint64_t sums = scan64(u + lane < cw ? sh.list[u + lane] : 0), over = __ballot(sums > target);
      if (over != 0) {
        const int first = __builtin_ctzll(over);
        u += first;
        target -= first > 0 ? lane64(sums, first - 1) : 0;
        break;
      }
      target -= lane64(sums, 63);
      if (u + 64 >= cw) break;  // not reached: the target is below the wave's sum
    }
    return choose_of_chunk(w * cw + u, target, total, b, low, prob);
  }

  // cut() digit by digit over the logits' images, for many tokens of nearly one logit.
  __device__ __noinline__ Border digits(const Border old, uint64_t rank_at, double least) const {
    Border b = old;
    const bool by_count = rank_at > 0;
    uint32_t prefix = 0;
    uint64_t above = 0, equal = 0;  // counts or weights above the digits fixed so far; tokens with the key found
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += THREADS) {
        sh.counts[i] = 0;
        sh.list[i] = 0;
      }
      lds_barrier();
      for (int u = 0; u < cw; ++u) {
        const vec x = load(piece(u));
        const int j = piece(u);
#pragma unroll 1
        for (int e = 0; e < E; ++e) {
          const float l = (float)x[e];
          const uint32_t key = logit_key(l);
          if (!old.keeps(l, j * E - lead + e) || (shift < 24 && (key >> (shift + 8)) != prefix)) continue;
          const uint64_t w = (uint64_t)weight(l);
          if (w == 0) continue;
          const uint32_t d = (key >> shift) & 255u;
          atomicAdd(&sh.counts[d], 1u);
          if (!by_count) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.list[d]), (unsigned long long)w);
        }
      }
      lds_barrier();
      if (threadIdx.x == 0) {
        sh.found[0] = 256;
        uint64_t sum = above;
        for (int d = 255; d >= 0; --d) {
          if (sh.counts[d] == 0) continue;
          const uint64_t next = sum + (by_count ? sh.counts[d] : sh.list[d]);
          if (by_count ? next >= rank_at : (double)next >= least) {
            sh.found[0] = d;
            sh.found[1] = sum;
            sh.found[2] = sh.counts[d];
            break;
          }
          sum = next;
        }
      }
      lds_barrier();
      const uint32_t d = (uint32_t)sh.found[0];
      above = sh.found[1];
      equal = sh.found[2];
      lds_barrier();
      if (d == 256) return old;
      prefix = prefix << 8 | d;
    }
    const float value = key_logit(prefix);
    // of the `equal` tokens with that logit the first `stay`
    uint64_t stay = 1;
    if (by_count) {
      stay = rank_at - above;
    } else {
      const double one = weight(value);  // above 0
      while (stay < equal && (double)above + (double)stay * one < least) {
        const double more = floor((least - ((double)above + (double)stay * one)) / one);
        stay += more < 1.0 ? 1 : more < (double)(equal - stay) ? (uint64_t)more : equal - stay;
      }
    }
    b.last = value > old.value ? 0x7FFFFFFF : old.last;
    b.value = value;
    if (stay >= equal) return b;
    // the stay-th of them in index order: its wave, its chunk, its lane, its element
    auto count = [&](vec x, int j) {
      uint64_t c = 0;
      for (int e = 0; e < E; ++e) c += (float)x[e] == value && old.keeps((float)x[e], j * E - lead + e) ? 1 : 0;
      return c;
    };
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t mine = 0;
    for (int u = 0; u < cw; ++u) mine += count(load(piece(u)), piece(u));
    block_sum(mine, 0);
    int w = 0;
    while (w < WAVES - 1 && sh.part[0][w] < stay) stay -= sh.part[0][w++];
    for (int u = wave; u < cw; u += WAVES) {
      const int j = (w * cw + u) * 64 + lane;
      const uint64_t s = scan64(count(load(j), j));
      if (lane == 63) sh.list[u] = s;
    }
    lds_barrier();
    if (wave == 0) {
      int u = 0;
      while (u < cw - 1 && sh.list[u] < stay) stay -= sh.list[u++];
      const int j = (w * cw + u) * 64 + lane;
      const vec x = load(j);
      const uint64_t own = count(x, j), upto = scan64(own);
      if (own > 0 && upto >= stay && upto - own < stay) {
        uint64_t left = stay - (upto - own);
        for (int e = 0; e < E; ++e)
          if ((float)x[e] == value && old.keeps((float)x[e], j * E - lead + e) && --left == 0) sh.found[0] = (uint64_t)(j * E - lead + e);
      }
    }
    lds_barrier();
    b.last = (int)sh.found[0];
    lds_barrier();
    return b;
  }

  // Narrows b to the tokens up to the rank_at-th in order (rank_at > 0), or up to the first at which the
  // weights reach the share p of all of b's; everything stays where that is not reached.  With `sums` (chunks_fit)
  // the weights from low on of what stays are left in sh.chunks where the result is true.
  __device__ __forceinline__ bool cut(Border* b, uint64_t rank_at, float p, float range, bool sums, double low) const {
    constexpr int PER = kBins / THREADS;
    const bool by_count = rank_at > 0;
    const float step = fminf((float)kBins / range, 1e30f);
    // NaN, behind the row's ends: the last bin, without weight
    auto bin_of = [&](float x) { return (int)fminf(((float)top - x) * step, (float)(kBins - 1)); };
    for (int i = threadIdx.x; i < kBins; i += THREADS) {
      sh.list[i] = 0;
      sh.counts[i] = 0;
    }
    lds_barrier();
    auto count = [&](vec x, const uint64_t (&w)[E]) {
      int bin[E];
#pragma unroll
      for (int e = 0; e < E; ++e) bin[e] = bin_of((float)x[e]);
#pragma unroll
      for (int e = 0; e < E; ++e) {  // one of no weight cannot be chosen, kept or not
        if (by_count) atomicAdd(&sh.counts[bin[e]], w[e] != 0 ? 1u : 0u);
        else atomicAdd(reinterpret_cast<unsigned long long*>(&sh.list[bin[e]]), (unsigned long long)w[e]);
      }
    };
    if (b->value == -INFINITY) {
      each([&](vec x, int j) {
        uint64_t w[E];
        weights<true>(x, j, *b, 0.0, w);
        count(x, w);
      });
    } else {
      each([&](vec x, int j) {
        uint64_t w[E];
        weights<false>(x, j, *b, 0.0, w);
        count(x, w);
      });
    }
    lds_barrier();
    uint64_t mine = 0, amount[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int i = threadIdx.x * PER + q;
      amount[q] = by_count ? sh.counts[i] : sh.list[i];
      mine += amount[q];
    }
    uint64_t upto;
    if (threadIdx.x == 0) sh.found[0] = kBins;
    const uint64_t all_bins = block_sum(mine, 0, &upto);
    uint64_t before = upto - mine;
    const double least = (double)p * (double)all_bins;
    auto reached = [&](uint64_t sum) { return by_count ? sum >= rank_at : (double)sum >= least; };
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (amount[q] > 0 && reached(before + amount[q]) && (before == 0 || !reached(before))) {
        sh.found[0] = threadIdx.x * PER + q;
        sh.found[1] = before;
      }
      before += amount[q];
    }
    lds_barrier();
    const int bin = __builtin_amdgcn_readfirstlane((int)sh.found[0]);
    const uint64_t above = lane64(sh.found[1], 0);
    lds_barrier();
    if (bin == kBins) return false;
    const Border old = *b;
    // the bin's logits and, for its roundings, a little more
    const float slack = 1e-5f * (fabsf((float)top) + range);
    const float to = step > 0.f ? (float)top - (float)bin / step + slack : INFINITY;  // 0: an infinite range, one bin
    const float from = step > 0.f ? (float)top - (float)(bin + 1) / step - slack : -INFINITY;  // below range: no weight
    if (threadIdx.x == 0) sh.n = 0;
    lds_barrier();
    // The list takes the bin's tokens and some beside it; the weights of those above, which stay for sure, are summed
    // by chunk.
    each([&](vec x, int j) {
      bool any = false;
#pragma unroll
      for (int e = 0; e < E; ++e) any |= ((float)x[e] >= from) & ((float)x[e] <= to);
      if (__any(any)) {
        uint32_t near = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float l = (float)x[e];
          near |= ((l >= from) & (l <= to) & old.keeps(l, j * E - lead + e)) ? 1u << e : 0u;
        }
        append(x, j, near);
      }
      if (!sums) return;
      double v[E];
      uint64_t sum = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = unrounded((float)x[e]);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += whole((((float)x[e] > to) & (v[e] >= low)) ? v[e] : 0.0);
      sum = scan64(sum);
      if ((threadIdx.x & 63) == 63 && j / 64 < chunks()) sh.chunks[j / 64] = sum;
    });
    lds_barrier();
    const int n = __builtin_amdgcn_readfirstlane(sh.n);
    if (n > kSort) {
      lds_barrier();
      *b = digits(old, rank_at, least);
      return false;
    }
    sort(n);
    // the entry at which it is reached, among those of the bin; one of no weight cannot be chosen, kept or not
    auto weight_of = [&](uint64_t e) { return bin_of(entry_logit(e)) == bin ? weight(entry_logit(e)) : 0.0; };
    uint64_t carry = above;
    for (int i0 = 0; i0 < n; i0 += THREADS) {
      const int i = i0 + threadIdx.x;
      const double w = i < n ? weight_of(sh.list[i]) : 0.0;
      const uint64_t own = !by_count ? (uint64_t)w : w > 0.0 ? 1 : 0;
      uint64_t to;
      const uint64_t all = block_sum(own, (i0 / THREADS) & 1, &to);
      to += carry;
      if (own > 0 && reached(to) && (to == own || !reached(to - own))) {
        sh.found[0] = sh.list[i];
        sh.found[1] = i;
      }
      carry += all;
    }
    lds_barrier();
    const uint64_t e = lane64(sh.found[0], 0);
    const int last = __builtin_amdgcn_readfirstlane((int)sh.found[1]);
    lds_barrier();
    b->value = entry_logit(e);
    b->last = (int)~(uint32_t)e;
    if (!sums) return false;
    for (int i = threadIdx.x; i <= last; i += THREADS) {
      const uint64_t at = sh.list[i];
      const double w = weight(entry_logit(at));
      if (unrounded(entry_logit(at)) >= low)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.chunks[((int)~(uint32_t)at + lead) / (64 * E)]), (unsigned long long)w);
    }
    return true;
  }
};

// top-k up to which a list is tried at once: of 1024 threads' maxima the k-th leaves about
// -1024 ln(1 - k / 1024) tokens, 904 at 600
template <int THREADS>
constexpr int kListK = THREADS * 600 / 1024;

template <typename T, int THREADS, int NV>
__global__ __launch_bounds__(THREADS, 4) void sample_kernel(SampleArgs a) {
  typedef SampleRow<T, THREADS> Row;
  typedef typename Row::vec vec;
  constexpr int E = Row::E, WAVES = THREADS / 64;
  static_assert(kSlots % NV == 0, "slots");
  __shared__ SampleShared<THREADS> sh;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, wave = tid >> 6;
  const T* start = reinterpret_cast<const T*>(a.logits) + r * a.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(start) & 15) / sizeof(T));
  const int pieces = (lead + (int)a.V + E - 1) / E, cw = (pieces + THREADS - 1) / THREADS;
  const int bytes = ((lead + (int)a.V) * (int)sizeof(T) + 3) & ~3;
  // a register of its own: as one of the arguments' sixteen it would bring all of them back in each step of a loop
  int V;
  __asm__("s_mov_b32 %0, %1" : "=s"(V) : "s"((int)a.V));
  Row s{sh, __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(start - lead), 0, bytes, 0x00020000), lead, V, cw, false, 0.0, 0.0};

  const float t = a.temperature ? a.temperature[r] : a.temperature_value;
  const int32_t k = a.top_k ? a.top_k[r] : a.top_k_value;
  const float p_given = a.top_p ? a.top_p[r] : a.top_p_value, p = p_given < 1.f ? p_given : 1.f;  // 1 for a NaN
  const float m = a.min_p ? a.min_p[r] : a.min_p_value, share = a.u[r];

  // the largest logit of each slot, and the smallest of all (NaN aside); NV pieces under way
  float slot[kSlots], lo = INFINITY;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) slot[q] = -INFINITY;
#pragma unroll 1
  for (int u0 = 0; u0 < cw; u0 += kSlots) {
#pragma unroll
    for (int h = 0; h < kSlots; h += NV) {
      if (u0 + h >= cw) break;
      vec x[NV];
#pragma unroll
      for (int q = 0; q < NV; ++q) x[q] = s.read(s.piece(u0 + h + q));
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int u = u0 + h + q;
        const bool in = u < cw && s.whole(s.piece(u));
        const float most = Row::largest(x[q]), least = -Row::largest(-x[q]);
        slot[h + q] = fmaxf(slot[h + q], in ? most : -INFINITY);
        lo = fminf(lo, in ? least : INFINITY);
      }
    }
  }
  // the two pieces that may reach out of the row
#pragma unroll 1
  for (int j = 0;; j = pieces - 1) {
    const int chunk = j / 64;
    if (!s.whole(j) && wave == chunk / cw && (tid & 63) == j % 64) {
      const vec x = s.load(j);
      const float most = Row::largest(x);
      lo = fminf(lo, -Row::largest(-x));
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (q == (chunk % cw) % kSlots) slot[q] = fmaxf(slot[q], most);
    }
    if (j == pieces - 1) break;
  }
  float mine = slot[0];
#pragma unroll
  for (int q = 1; q < kSlots; ++q) mine = fmaxf(mine, slot[q]);
  float hi = wave_max(mine);
  lo = wave_min(lo);
  if ((tid & 63) == 0) {
    sh.most[wave] = hi;
    sh.least[wave] = lo;
  }
  for (int i = tid; i < kExpTable; i += THREADS) sh.table[i] = exp_entry(i);
  if (tid == 0) sh.n = 0x7FFFFFFF;
  lds_barrier();
  hi = wave_max((tid & 63) < WAVES ? sh.most[tid & 63] : -INFINITY);
  lo = wave_min((tid & 63) < WAVES ? sh.least[tid & 63] : INFINITY);

  int token = -1;
  float prob = 0.f;
  if (hi == -INFINITY) {
    // nothing to choose
  } else if (!(t > 0.f) || k == 1 || p <= 0.f || m > 1.f) {  // the first in order alone
    if (mine == hi) {
      int first = 0x7FFFFFFF;
#pragma unroll 1
      for (int u = 0; u < cw; ++u) {
        const int j = s.piece(u);
        const vec x = s.load(j);
#pragma unroll
        for (int e = E - 1; e >= 0; --e)
          if ((float)x[e] == hi) first = j * E - lead + e < first ? j * E - lead + e : first;
      }
      atomicMin(&sh.n, first);
    }
    lds_barrier();
    token = sh.n;
    prob = 1.f;
  } else {
    const bool ranked = k >= 1 && k < V, cut_by_share = p < 1.f;
    s.infinite = hi == INFINITY;
    s.top = s.infinite ? 0.0 : (double)hi;
    s.rate = fmin(kExpRate / (double)t, 1e300);
    const double low = m > 0.f ? (double)m * kWeightOne : 0.0;
    // logits whose weights are not 0: from hi down to -31 t, or to the smallest there is
    const float range = s.infinite ? 31.f * t : fminf(31.f * t, hi - lo);
    // first a list of all that can be kept, where that is likely to be short
    Border b{-INFINITY, 0x7FFFFFFF};
    int n = Row::kSort + 1;
    if (s.infinite) {
      // ties: no list
    } else if (ranked && k <= kListK<THREADS>) {
      n = s.gather(slot, s.reached_by(k, mine, hi, range), 0.0);
    } else if (!cut_by_share && low > 0.0) {  // w >= m is l >= hi + t ln m, here a little less
      n = s.gather(slot, fmaxf(hi + t * logf(m) - 1e-4f * (fabsf(hi) + t), -INFINITY), low);
    }
    n = __builtin_amdgcn_readfirstlane(n);
    if (n <= 64) {
      token = s.choose_of_few(n, k, p, low, share, &prob);
    } else if (n <= Row::kSort) {
      s.sort(n);
      n = s.kept_of_list(n, k, p);
      b = s.border_of(n - 1);
      token = s.chunks_fit() ? s.choose_of_list(n, b, low, share, &prob) : s.choose_of_row(b, low, share, &prob);
    } else {
      bool summed = false;
#pragma unroll 1
      for (int by_weight = ranked ? 0 : 1; by_weight <= (cut_by_share ? 1 : 0); ++by_weight)
        summed = s.cut(&b, by_weight ? 0 : (uint64_t)k, p, range, by_weight == (cut_by_share ? 1 : 0) && s.chunks_fit(), low);
      token = summed ? s.choose_of_chunks(b, low, share, &prob) : s.choose_of_row(b, low, share, &prob);
    }
  }
  if (tid == 0) {
    a.tokens[r] = token;
    if (a.probs) a.probs[r] = prob;
  }
}

template <typename T>
static void sample_launch(const SampleArgs& a, int64_t B, hipStream_t st) {
  const int64_t pieces = (a.V + 2 * (16 / sizeof(T)) - 2) / (16 / sizeof(T));  // with any lead
  const dim3 grid((unsigned)B);
  // Rows of few pieces need few threads.  Where every row is cut to a short list, 512 threads: two rows share a
  // compute unit, and fewer waves meet at the barriers (top-k 50, top-p, min-p, before later steps: 512 x 131072
  // 42.7 us, 47.4 with 1024; 1 x 32000 10.2 and 12.3).  Where rows may need passes over all weights, 1024 (mixed
  // settings, likewise: 512 x 131072 139 us, 173 with 512).
  const bool lists = a.top_k == nullptr && a.top_k_value >= 1 && a.top_k_value <= kListK<512>;
  if (pieces <= 1024) sample_kernel<T, 256, 4><<<grid, dim3(256), 0, st>>>(a);
  else if (lists) sample_kernel<T, 512, 8><<<grid, dim3(512), 0, st>>>(a);
  else sample_kernel<T, 1024, 8><<<grid, dim3(1024), 0, st>>>(a);
}

hipError_t launch_sample(const SampleArgs& a, int logit_bytes, int64_t B, hipStream_t st) {
  if (logit_bytes == 2) sample_launch<f16>(a, B, st);
  else sample_launch<float>(a, B, st);
  return hipGetLastError();
}

}  // namespace awq
