// Routing of tokens to experts, the plan of the ragged groups it makes, and
// the weighted sum that ends an expert layer.
//
// Route: the top_k largest logits of a token (first of equal ones) and their
// softmax weights, 16 lanes per token (a wave above 256 experts or 16 choices)
// with the logits in registers.
// Plan: a stable counting sort of the pairs p = t * top_k + j by expert.  The
// pairs are cut into runs; each run's pairs are counted by expert, the counts
// become first rows (in the order expert, then run), and each run places its
// pairs, a lane's rank among the 64 pairs of its wave coming from ballots on the
// bits of the expert.  No order depends on timing.
// All of it is bound by launches and latency: up to kSmallPairs pairs one block
// does everything in one launch (32 tokens x 6 of 64 experts: 5.5 us, where a
// launch for each step took 10.4); beyond, three launches (16384 tokens x 8 of
// 128: 16 us).  The sum is bound by memory.
#include "awq_common.h"
#include "awq_internal.h"

namespace awq {

constexpr int kMoeThreads = 1024, kMoeWaves = kMoeThreads / 64;
constexpr int kSmallPairs = 1024;  // in one block
constexpr int kRunPairs = 512;     // of a run, at most (a route's run is whole tokens)

// Order-preserving image of a float: larger floats have larger images, equal
// ones (+0 and -0, which adding 0 makes +0) the same.  No float's image is 0.
__device__ inline uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// v joined by `op` over each run of L = 16 or 64 lanes, in every lane of it: by
// rotations within 16 lanes, then across.
template <int L, typename Op>
__device__ __forceinline__ uint32_t lanes_join(uint32_t v, Op op) {
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));  // row_ror 8, 4, 2, 1
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));
  if (L == 64) {
    v = op(v, (uint32_t)__shfl_xor((int)v, 16, kWave));
    v = op(v, (uint32_t)__shfl_xor((int)v, 32, kWave));
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return lanes_join<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  return lanes_join<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_join<L>(
      __float_as_uint(v), [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); }));
}

struct RouteArgs {
  const void* logits;
  float* weights;
  int half, top_k, renorm;
};

// Tokens t0 .. t0 + count - 1, one for each run of L lanes in turn (V logits per
// lane, E <= L V); lane j of the run writes the j-th choice and its weight, and
// the expert to copy [count * top_k] too.  Four tokens a wave (L = 16) share every
// instruction of the choice; one token a wave was bound by the vector ALU (choosing
// and counting 16384 tokens x 8 of 128: 13.8 us against 8.6).
template <int V, int L>
__device__ inline void route_tokens(const RouteArgs& a, int64_t t0, int count, int E, int32_t* __restrict__ experts,
                                    int* copy) {
  const int r = threadIdx.x % L;
  for (int i = threadIdx.x / L; i - (int)(threadIdx.x % 64) / L < count; i += kMoeThreads / L) {  // whole waves
    const int64_t t = t0 + (i < count ? i : count - 1);  // lanes past the last token repeat it
    uint32_t key[V];  // 0: not to be chosen (no such expert, -inf, NaN, or chosen already)
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int e = u * L + r;
      float v = -INFINITY;
      if (e < E)
        v = a.half ? (float)reinterpret_cast<const f16*>(a.logits)[t * E + e]
                   : reinterpret_cast<const float*>(a.logits)[t * E + e];
      key[u] = v > -INFINITY ? order_key(v) : 0u;
    }
    uint32_t best = 0;
#pragma unroll
    for (int u = 0; u < V; ++u) best = key[u] > best ? key[u] : best;
    const float top = key_value(lanes_max<L>(best));
    float sum = 0.f;
    if (!a.renorm) {
#pragma unroll
      for (int u = 0; u < V; ++u) sum += key[u] ? expf(key_value(key[u]) - top) : 0.f;
    }
    int mine = -1;
    uint32_t chosen = 0;
    for (int j = 0; j < a.top_k; ++j) {
      best = 0;
#pragma unroll
      for (int u = 0; u < V; ++u) best = key[u] > best ? key[u] : best;
      const uint32_t most = lanes_max<L>(best);
      uint32_t e = ~0u;  // the first expert that has it
#pragma unroll
      for (int u = V - 1; u >= 0; --u) e = key[u] == most ? u * L + r : e;
      e = lanes_min<L>(e);
#pragma unroll
      for (int u = 0; u < V; ++u) key[u] = e == (uint32_t)(u * L + r) ? 0u : key[u];
      if (r == j && most != 0) {  // 0: nothing was left to choose
        mine = (int)e;
        chosen = most;
      }
    }
    const float w = mine >= 0 ? expf(key_value(chosen) - top) : 0.f;
    sum = lanes_sum<L>(a.renorm ? w : sum);
    if (r < a.top_k && i < count) {
      experts[t * a.top_k + r] = mine;
      a.weights[t * a.top_k + r] = mine >= 0 ? w / sum : 0.f;
      copy[i * a.top_k + r] = mine;
    }
  }
}

// A pair's group in the plan: its expert, or E for a dropped pair (an id outside [0, E)).
__device__ inline int group_of(int expert, int E) { return expert >= 0 && expert < E ? expert : E; }

// Lanes of the wave whose group equals this lane's.
__device__ inline uint64_t same_group(int g, int bits) {
  uint64_t same = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((g >> b) & 1);
    same &= (g >> b) & 1 ? set : ~set;
  }
  return same;
}

// Exclusive sums of v over the block's threads (of whole waves), by way of `part` [16].
__device__ inline int block_scan(int v, int* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int upto = wave_scan(v);
  if (lane == 63) part[wave] = upto;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += part[w];
  __syncthreads();
  return before + upto - v;
}

// Places the block's pairs, one per thread: hist [16][E + 1] is scratch, start(g)
// the first row of the block's pairs of group g (called once per group by the
// thread g % kMoeThreads, the counts of the block's waves being in hist).
template <typename Start>
__device__ inline void place(int64_t p, bool valid, int g, int E, int bits, int* hist, Start start,
                             int32_t* __restrict__ rows, int32_t* __restrict__ pos) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t same = same_group(valid ? g : E + 1, bits);
  const int rank = __popcll(same & ((1ull << lane) - 1));
  if (rank == 0 && valid) hist[wave * (E + 1) + g] = __popcll(same);
  __syncthreads();
  start();
  __syncthreads();
  if (valid) {
    const int32_t row = hist[wave * (E + 1) + g] + rank;
    rows[row] = (int32_t)p;
    pos[p] = g < E ? row : -1;
  }
}

// Turns the waves' counts of a group into the first rows of each wave's pairs.
__device__ inline void spread(int* hist, int g, int E, int row) {
  for (int w = 0; w < kMoeWaves; ++w) {
    const int c = hist[w * (E + 1) + g];
    hist[w * (E + 1) + g] = row;
    row += c;
  }
}

// Everything in one block: V = 0 plans given experts, otherwise they are chosen first.
template <int V, int L>
__global__ __launch_bounds__(kMoeThreads) void plan_small_kernel(RouteArgs a, int64_t tokens, int pairs, int E,
                                                                 int bits, int32_t* __restrict__ experts,
                                                                 int32_t* __restrict__ offsets,
                                                                 int32_t* __restrict__ rows, int32_t* __restrict__ pos) {
  extern __shared__ int hist[];  // [16][E + 1]
  __shared__ int part[kMoeWaves], mine[kSmallPairs];
  const int tid = threadIdx.x;
  for (int i = tid; i < kMoeWaves * (E + 1); i += kMoeThreads) hist[i] = 0;
  if constexpr (V > 0) {
    route_tokens<V, L>(a, 0, (int)tokens, E, experts, mine);
  } else if (tid < pairs) {
    mine[tid] = experts[tid];
  }
  __syncthreads();
  const bool valid = tid < pairs;
  const int g = valid ? group_of(mine[tid], E) : 0;
  place(tid, valid, g, E, bits, hist,
        [&] {  // E + 1 <= 1025 groups: thread i takes group i, the dropped pairs (last) start where the others end
          int count = 0;
          if (tid < E)
            for (int w = 0; w < kMoeWaves; ++w) count += hist[w * (E + 1) + tid];
          const int first = block_scan(count, part);
          if (tid < E) {
            offsets[tid] = first;
            spread(hist, tid, E, first);
          }
          if (tid == E - 1) {
            offsets[E] = first + count;
            spread(hist, E, E, first + count);
          }
        },
        rows, pos);
}

// counts[g][run] of each run's pairs (V > 0: after choosing them; a run is `run` pairs, whole tokens).
template <int V, int L>
__global__ __launch_bounds__(kMoeThreads) void plan_count_kernel(RouteArgs a, int64_t tokens, int64_t pairs, int run,
                                                                 int E, int32_t* __restrict__ experts,
                                                                 int32_t* __restrict__ counts, int64_t runs) {
  extern __shared__ int hist[];  // [E + 1]
  __shared__ int mine[kRunPairs];
  const int tid = threadIdx.x;
  const int64_t p0 = (int64_t)blockIdx.x * run;
  const int n = pairs - p0 < run ? (int)(pairs - p0) : run;
  for (int g = tid; g <= E; g += kMoeThreads) hist[g] = 0;
  if constexpr (V > 0) {
    route_tokens<V, L>(a, p0 / a.top_k, n / a.top_k, E, experts, mine);
  } else if (tid < n) {
    mine[tid] = experts[p0 + tid];
  }
  __syncthreads();
  if (tid < n) atomicAdd(&hist[group_of(mine[tid], E)], 1);  // whole numbers: the order does not matter
  __syncthreads();
  for (int g = tid; g <= E; g += kMoeThreads) counts[(int64_t)g * runs + blockIdx.x] = hist[g];
}

// counts[g][run]: exclusive sums over the runs of group g = blockIdx.x; total[g].
__global__ __launch_bounds__(kMoeThreads) void plan_scan_kernel(int32_t* __restrict__ counts, int64_t runs,
                                                                int32_t* __restrict__ total) {
  __shared__ int part[kMoeWaves];
  int32_t* c = counts + (int64_t)blockIdx.x * runs;
  int before = 0;
  for (int64_t r0 = 0; r0 < runs; r0 += blockDim.x) {
    const int64_t r = r0 + threadIdx.x;
    const int v = r < runs ? c[r] : 0;
    const int first = block_scan(v, part);
    if (r < runs) c[r] = before + first;
    if (threadIdx.x == blockDim.x - 1) part[0] = first + v;
    __syncthreads();
    before += part[0];
    __syncthreads();
  }
  if (threadIdx.x == 0) total[blockIdx.x] = before;
}

__global__ __launch_bounds__(kMoeThreads) void plan_place_kernel(const int32_t* __restrict__ experts, int64_t pairs,
                                                                 int run, int E, int bits,
                                                                 const int32_t* __restrict__ counts, int64_t runs,
                                                                 const int32_t* __restrict__ total,
                                                                 int32_t* __restrict__ offsets,
                                                                 int32_t* __restrict__ rows, int32_t* __restrict__ pos) {
  extern __shared__ int hist[];  // [16][E + 1]
  __shared__ int part[kMoeWaves];
  const int tid = threadIdx.x;
  for (int i = tid; i < kMoeWaves * (E + 1); i += kMoeThreads) hist[i] = 0;
  __syncthreads();
  const int64_t p = (int64_t)blockIdx.x * run + tid;
  const bool valid = tid < run && p < pairs;
  const int g = valid ? group_of(experts[p], E) : 0;
  place(p, valid, g, E, bits, hist,
        [&] {
          const int count = tid < E ? total[tid] : 0;
          const int first = block_scan(count, part);  // of the group, over all runs
          if (tid < E) spread(hist, tid, E, first + counts[(int64_t)tid * runs + blockIdx.x]);
          if (tid == E - 1) spread(hist, E, E, first + count + counts[(int64_t)E * runs + blockIdx.x]);
          if (blockIdx.x == 0) {
            if (tid < E) offsets[tid] = first;
            if (tid == E - 1) offsets[E] = first + count;
          }
        },
        rows, pos);
}

// out[t][n] = sum_j weights[t][j] y[pos[t * k + j]][n], 8 channels per thread.  Every
// byte is moved once: 8192 tokens x 4 rows of 4096, 336 MB in 58 us (5.8 TB/s; 67
// us with one row's load under way at a time, kept in the caches).
__global__ __launch_bounds__(256) void combine_kernel(const f16* __restrict__ y, int64_t R,
                                                      const int32_t* __restrict__ pos,
                                                      const float* __restrict__ weights, int64_t T, int top_k,
                                                      int64_t N, f16* __restrict__ out) {
  const uint32_t per = (uint32_t)(N / 8), i = blockIdx.x * 256u + threadIdx.x;  // T N / 8 < 2^32 - 256
  if (i >= (uint64_t)T * per) return;
  const int64_t t = i / per, c = (int64_t)(i % per) * 8;
  float acc[8] = {};
  // four rows' loads under way before the first is used
  for (int j0 = 0; j0 < top_k; j0 += 4) {
    f16x8 v[4];
    float w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t p = t * top_k + (j0 + k < top_k ? j0 + k : top_k - 1);
      const int32_t row = pos[p];
      const bool live = j0 + k < top_k && row >= 0 && row < R;
      w[k] = live ? weights[p] : 0.f;
      v[k] = f16x8{};
      if (live) v[k] = __builtin_nontemporal_load(reinterpret_cast<const f16x8*>(y + row * N + c));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int u = 0; u < 8; ++u) acc[u] = fmaf(w[k], (float)v[k][u], acc[u]);
  }
  f16x8 o;
#pragma unroll
  for (int u = 0; u < 8; ++u) o[u] = (f16)acc[u];
  *reinterpret_cast<f16x8*>(out + t * N + c) = o;
}

// A run: whole tokens where the experts are chosen along (top_k > 1), at most kRunPairs pairs.
static int run_pairs(int top_k) { return kRunPairs / top_k * top_k; }

size_t moe_plan_workspace(int64_t pairs, int E, int top_k) {
  const int run = run_pairs(top_k);
  return (size_t)((pairs + run - 1) / run + 1) * (size_t)(E + 1) * sizeof(int32_t);
}

template <int V, int L>
static hipError_t plan_launch(const RouteArgs& a, int64_t T, int E, int32_t* experts, int32_t* offsets, int32_t* rows,
                              int32_t* pos, int32_t* ws, hipStream_t st) {
  const int64_t pairs = T * a.top_k;
  int bits = 0;
  while ((1 << bits) < E + 2) ++bits;
  const size_t hist = (size_t)(E + 1) * sizeof(int);
  if (pairs <= kSmallPairs) {
    plan_small_kernel<V, L><<<dim3(1), dim3(kMoeThreads), hist * kMoeWaves, st>>>(a, T, (int)pairs, E, bits, experts,
                                                                               offsets, rows, pos);
    return hipGetLastError();
  }
  const int run = run_pairs(a.top_k);
  const int64_t runs = (pairs + run - 1) / run;
  int32_t* total = ws + runs * (E + 1);
  plan_count_kernel<V, L><<<dim3((unsigned)runs), dim3(kMoeThreads), hist, st>>>(a, T, pairs, run, E, experts, ws, runs);
  plan_scan_kernel<<<dim3((unsigned)(E + 1)), dim3(runs > 256 ? kMoeThreads : 256), 0, st>>>(ws, runs, total);
  plan_place_kernel<<<dim3((unsigned)runs), dim3(kMoeThreads), hist * kMoeWaves, st>>>(experts, pairs, run, E, bits, ws,
                                                                                      runs, total, offsets, rows, pos);
  return hipGetLastError();
}

hipError_t launch_moe_route(const void* logits, int bytes, int64_t T, int E, int top_k, int renorm, int32_t* experts,
                            float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, int32_t* ws,
                            hipStream_t st) {
  const RouteArgs a{logits, weights, bytes == 2, top_k, renorm};
  if (top_k <= 16 && E <= 64) return plan_launch<4, 16>(a, T, E, experts, offsets, rows, pos, ws, st);
  if (top_k <= 16 && E <= 128) return plan_launch<8, 16>(a, T, E, experts, offsets, rows, pos, ws, st);
  if (top_k <= 16 && E <= 256) return plan_launch<16, 16>(a, T, E, experts, offsets, rows, pos, ws, st);
  return plan_launch<16, 64>(a, T, E, experts, offsets, rows, pos, ws, st);  // a choice for each lane, 1024 experts
}

hipError_t launch_moe_plan(const int32_t* experts, int64_t T, int E, int top_k, int32_t* offsets, int32_t* rows,
                           int32_t* pos, int32_t* ws, hipStream_t st) {
  return plan_launch<0, 16>(RouteArgs{nullptr, nullptr, 0, top_k, 0}, T, E, const_cast<int32_t*>(experts), offsets, rows,
                        pos, ws, st);
}

hipError_t launch_moe_combine(const void* y, int64_t R, const int32_t* pos, const float* weights, int64_t T, int top_k,
                              int64_t N, void* out, hipStream_t st) {
  const int64_t threads = T * (N / 8);
  combine_kernel<<<dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st>>>(
      reinterpret_cast<const f16*>(y), R, pos, weights, T, top_k, N, reinterpret_cast<f16*>(out));
  return hipGetLastError();
}

}  // namespace awq
