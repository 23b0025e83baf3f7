// Routing of tokens to experts, the plan of the ragged groups it makes, and
// the weighted sum that ends an expert layer.
//
// Route: the top_k largest logits of a token (first of equal ones) and their
// softmax weights, one wave per token with the logits in registers.
// Plan: a stable counting sort of the pairs p = t * top_k + j by expert.  A
// block counts the pairs of its run of kPlanPairs by expert; one block turns
// the counts into offsets (in the order expert, then run); each block then
// places its pairs, a lane's rank among the 64 pairs of its wave coming from
// ballots on the bits of the expert.  No atomics on memory: the order never
// depends on timing.
// All of it is small and bound by launches and latency; the sum is bound by
// memory.
#include "awq_common.h"
#include "awq_internal.h"

namespace awq {

constexpr int kPlanThreads = 1024;  // pairs of one run: one per thread

// Order-preserving image of a float: larger floats have larger images, equal
// ones (+0 and -0, which adding 0 makes +0) the same.
__device__ inline uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// V logits per lane (E <= 64 V); lane i holds experts V i .. V i + V - 1, so
// the first of equal logits is in the first lane that has one.
template <int V, typename T>
__global__ __launch_bounds__(256) void route_kernel(const T* __restrict__ logits, int64_t tokens, int E, int top_k,
                                                    int renorm, int32_t* __restrict__ experts,
                                                    float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= tokens) return;
  float v[V];
  uint32_t key[V];  // 0: not to be chosen (no such expert, -inf, NaN, or chosen already)
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    v[i] = e < E ? (float)logits[t * E + e] : -INFINITY;
    key[i] = v[i] > -INFINITY ? order_key(v[i]) : 0u;
    if (key[i]) top = fmaxf(top, v[i]);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += key[i] ? expf(v[i] - top) : 0.f;
  sum = wave_sum(sum);
  int mine = -1;      // lane j keeps choice j
  float w = 0.f, chosen = 0.f;
  for (int j = 0; j < top_k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = key[i] > best ? key[i] : best;
    uint32_t all = best;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)all, off, kWave);
      all = o > all ? o : all;
    }
    if (all == 0) break;  // nothing left to choose
    const int owner = __ffsll((unsigned long long)__ballot(best == all)) - 1;
    int slot = -1;
    float val = 0.f;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == all) {
        slot = i;
        val = v[i];
      }
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == slot) key[i] = 0u;
    }
    const int e = __shfl(lane * V + slot, owner, kWave);
    const float p = expf(__shfl(val, owner, kWave) - top);
    chosen += p;
    if (lane == j) {
      mine = e;
      w = p;
    }
  }
  if (lane < top_k) {
    experts[t * top_k + lane] = mine;
    weights[t * top_k + lane] = mine >= 0 ? w / (renorm ? chosen : sum) : 0.f;
  }
}

// Expert of pair p as a group of the plan: E for a dropped pair (an id outside
// [0, E)) and E + 1 past the last pair.
__device__ inline int group_of(const int32_t* experts, int64_t p, int64_t pairs, int E) {
  if (p >= pairs) return E + 1;
  const int e = experts[p];
  return e >= 0 && e < E ? e : E;
}

// Lanes of the wave whose group equals this lane's.
__device__ inline uint64_t same_group(int g, int bits) {
  uint64_t same = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((g >> b) & 1);
    same &= (g >> b) & 1 ? set : ~set;
  }
  return same;
}

constexpr int kPlanWaves = kPlanThreads / 64;

// counts[run][g] for the E + 1 groups.
__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const int32_t* __restrict__ experts, int64_t pairs,
                                                                  int E, int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];
  for (int g = threadIdx.x; g <= E; g += kPlanThreads) hist[g] = 0;
  __syncthreads();
  const int g = group_of(experts, (int64_t)blockIdx.x * kPlanThreads + threadIdx.x, pairs, E);
  if (g <= E) atomicAdd(&hist[g], 1);  // whole numbers: the order of the sum does not matter
  __syncthreads();
  for (int i = threadIdx.x; i <= E; i += kPlanThreads) counts[(int64_t)blockIdx.x * (E + 1) + i] = hist[i];
}

// counts[run][g] becomes the first row of run's pairs in group g; offsets too.
__global__ __launch_bounds__(kPlanThreads) void plan_scan_kernel(int32_t* __restrict__ counts, int64_t runs, int E,
                                                                 int32_t* __restrict__ offsets) {
  extern __shared__ int32_t total[];  // [E + 1]
  for (int g = threadIdx.x; g <= E; g += kPlanThreads) {
    int32_t s = 0;
    for (int64_t r = 0; r < runs; ++r) s += counts[r * (E + 1) + g];
    total[g] = s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int32_t s = 0;
    for (int g = 0; g <= E; ++g) {
      const int32_t c = total[g];
      total[g] = s;
      offsets[g] = s;
      s += c;
    }
  }
  __syncthreads();
  for (int g = threadIdx.x; g <= E; g += kPlanThreads) {
    int32_t s = total[g];
    for (int64_t r = 0; r < runs; ++r) {
      const int32_t c = counts[r * (E + 1) + g];
      counts[r * (E + 1) + g] = s;
      s += c;
    }
  }
}

__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(const int32_t* __restrict__ experts, int64_t pairs,
                                                                  int E, int bits, const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ rows,
                                                                  int32_t* __restrict__ pos) {
  extern __shared__ int32_t hist[];  // [waves][E + 1]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kPlanWaves * (E + 1); i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const int64_t p = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x;
  const int g = group_of(experts, p, pairs, E);
  const uint64_t same = same_group(g, bits);
  const int rank = __popcll(same & ((1ull << lane) - 1));
  if (rank == 0 && g <= E) hist[wave * (E + 1) + g] = __popcll(same);
  __syncthreads();
  for (int i = threadIdx.x; i <= E; i += kPlanThreads) {
    int32_t s = counts[(int64_t)blockIdx.x * (E + 1) + i];
    for (int w = 0; w < kPlanWaves; ++w) {
      const int32_t c = hist[w * (E + 1) + i];
      hist[w * (E + 1) + i] = s;
      s += c;
    }
  }
  __syncthreads();
  if (p < pairs) {
    const int32_t row = hist[wave * (E + 1) + g] + rank;
    rows[row] = (int32_t)p;
    pos[p] = g < E ? row : -1;
  }
}

// out[t][n] = sum_j weights[t][j] y[pos[t * k + j]][n], 8 channels per thread.
__global__ __launch_bounds__(256) void combine_kernel(const f16* __restrict__ y, int64_t R,
                                                      const int32_t* __restrict__ pos,
                                                      const float* __restrict__ weights, int64_t T, int top_k,
                                                      int64_t N, f16* __restrict__ out) {
  const int64_t per = N / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * per) return;
  const int64_t t = i / per, c = (i - t * per) * 8;
  float acc[8] = {};
  for (int j = 0; j < top_k; ++j) {
    const int32_t row = pos[t * top_k + j];
    if (row < 0 || row >= R) continue;
    const float w = weights[t * top_k + j];
    const f16x8 v = *reinterpret_cast<const f16x8*>(y + row * N + c);
#pragma unroll
    for (int u = 0; u < 8; ++u) acc[u] = fmaf(w, (float)v[u], acc[u]);
  }
  f16x8 o;
#pragma unroll
  for (int u = 0; u < 8; ++u) o[u] = (f16)acc[u];
  *reinterpret_cast<f16x8*>(out + t * N + c) = o;
}

size_t moe_plan_workspace(int64_t pairs, int E) {
  return (size_t)((pairs + kPlanThreads - 1) / kPlanThreads) * (size_t)(E + 1) * sizeof(int32_t);
}

template <int V>
static hipError_t route_launch(const void* logits, int bytes, int64_t T, int E, int top_k, int renorm,
                               int32_t* experts, float* weights, hipStream_t st) {
  const dim3 grid((unsigned)((T + 3) / 4)), block(256);
  if (bytes == 2)
    route_kernel<V, f16><<<grid, block, 0, st>>>(reinterpret_cast<const f16*>(logits), T, E, top_k, renorm, experts,
                                                 weights);
  else
    route_kernel<V, float><<<grid, block, 0, st>>>(reinterpret_cast<const float*>(logits), T, E, top_k, renorm,
                                                   experts, weights);
  return hipGetLastError();
}

hipError_t launch_moe_route(const void* logits, int bytes, int64_t T, int E, int top_k, int renorm, int32_t* experts,
                            float* weights, hipStream_t st) {
  if (E <= 64) return route_launch<1>(logits, bytes, T, E, top_k, renorm, experts, weights, st);
  if (E <= 128) return route_launch<2>(logits, bytes, T, E, top_k, renorm, experts, weights, st);
  if (E <= 256) return route_launch<4>(logits, bytes, T, E, top_k, renorm, experts, weights, st);
  return route_launch<16>(logits, bytes, T, E, top_k, renorm, experts, weights, st);
}

hipError_t launch_moe_plan(const int32_t* experts, int64_t pairs, int E, int32_t* offsets, int32_t* rows, int32_t* pos,
                           int32_t* counts, hipStream_t st) {
  const int64_t runs = (pairs + kPlanThreads - 1) / kPlanThreads;
  int bits = 0;
  while ((1 << bits) < E + 2) ++bits;
  const size_t hist = (size_t)(E + 1) * sizeof(int32_t);
  plan_count_kernel<<<dim3((unsigned)runs), dim3(kPlanThreads), hist, st>>>(experts, pairs, E, counts);
  plan_scan_kernel<<<dim3(1), dim3(kPlanThreads), hist, st>>>(counts, runs, E, offsets);
  plan_place_kernel<<<dim3((unsigned)runs), dim3(kPlanThreads), hist * kPlanWaves, st>>>(experts, pairs, E, bits,
                                                                                         counts, rows, pos);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* y, int64_t R, const int32_t* pos, const float* weights, int64_t T, int top_k,
                              int64_t N, void* out, hipStream_t st) {
  const int64_t threads = T * (N / 8);
  combine_kernel<<<dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st>>>(
      reinterpret_cast<const f16*>(y), R, pos, weights, T, top_k, N, reinterpret_cast<f16*>(out));
  return hipGetLastError();
}

}  // namespace awq
