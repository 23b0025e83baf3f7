// Host-side launchers of the libawq kernels (internal; the public interface is
// include/awq.h).  Each enqueues its kernels on `st` and returns the launch
// status; shapes have been validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "awq_common.h"
#include "kv_common.h"

namespace awq {

constexpr int kMaxAlphas = 64;

struct AlphaGrid {
  float v[kMaxAlphas];
};

// stats.hip
hipError_t launch_channel_mean_abs(const void* X, int64_t M, int64_t K, double* a, hipStream_t st);
hipError_t launch_transpose(const void* X, int64_t M, int64_t K, int64_t Mp, void* Xt, hipStream_t st);

// gram.hip: G = Xt Xt^T (fp32 [K][K], fp64 accumulation) from Xt fp16 [K][Mp], Mp % 64 == 0, K % 64 == 0.
// partial: gram_partial_bytes(K, Mp) bytes of device scratch (may be null when that is 0)
hipError_t launch_gram(const void* Xt, int64_t Mp, int64_t K, float* G, double* partial, hipStream_t st);
size_t gram_partial_bytes(int64_t K, int64_t Mp);

// quant.hip
// s_all fp32 [n_alpha][K] and inv_all = 1 / s_all in fp64
hipError_t launch_scales(const double* a, const AlphaGrid& al, int n_alpha, int64_t K, float* s_all,
                         double* inv_all, hipStream_t st);
// bits: 4 (16 levels) or 3 (8 levels); s and inv (its fp64 reciprocal) both NULL or both given
// keep: NULL, or uint8 [K] marking channels whose error is 0 (kept exact)
hipError_t launch_quant_error(const void* W, const float* s, const double* inv, const int32_t* ex,
                              const uint8_t* keep, int64_t N, int64_t K, int bits, void* Ehi, void* Elo,
                              hipStream_t st);
hipError_t launch_quant_error32(const void* W, const float* s, const double* inv, const uint8_t* keep, int64_t N,
                                int64_t K, int bits, float* E, hipStream_t st);
hipError_t launch_top_channels(const double* v, int64_t K, int n_keep, int32_t* out, hipStream_t st);
hipError_t launch_keep_mask(const int32_t* keep, int n_keep, int64_t K, uint8_t* mask, hipStream_t st);
hipError_t launch_pack(const void* W, const float* s, int64_t N, int64_t K, int bits, void* packed, void* scales,
                       void* zeros, hipStream_t st);
hipError_t launch_select_scale(const float* s_all, const int32_t* best, int64_t K, float* s_out, hipStream_t st);
hipError_t launch_unpack(const void* packed, const void* zeros, int64_t N, int64_t K, int bits, uint8_t* codes,
                         uint8_t* zeros_u8, hipStream_t st);

// loss.hip: channel exponents and the fp16 split of the scaled Gram matrix;
// partials of sum_n E'_n G' E'_n^T; reduce + argmin.
hipError_t launch_gram_split(const float* G, int64_t K, int32_t* e, void* Ghi, void* Glo, hipStream_t st);
int64_t loss_partial_count(int64_t N, int64_t K);
hipError_t launch_loss_partials(const void* Ehi, const void* Elo, const void* Ghi, const void* Glo, int64_t N,
                                int64_t K, double* partial, hipStream_t st);
int64_t loss_direct_partial_count(int64_t M, int64_t N);
hipError_t launch_loss_direct(const void* X, const float* E, int64_t M, int64_t N, int64_t K, double* partial,
                              hipStream_t st);
hipError_t launch_loss_reduce(const double* partial, int64_t count, double mn, double* loss, hipStream_t st);
hipError_t launch_argmin(const double* loss, int n, int32_t* best, hipStream_t st);

// gemv.hip (vector-ALU GEMV, M <= 2), skinny.hip (matrix-core decode kernels: LDS-ring kernel for M <= 16, register-staged up to
// 64 where it beats the GEMM), gemm.hip / gemm_pipe.hip (matrix-core GEMM)
bool gemv_dot2_supported(int64_t M, int64_t K);
// The input side of the per-channel scaling: xs = fp16(x / s).
hipError_t launch_scale_input(const void* x, const float* s, int64_t M, int64_t K, void* xs, hipStream_t st);
hipError_t launch_gemv_dot2(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                            int64_t M, int64_t N, int64_t K, hipStream_t st);
bool ring3_supported(int64_t M, int64_t N, int64_t K);
bool ring_mid_supported(int64_t M, int64_t N, int64_t K, int bits);  // 17 <= M <= 64 on the ring kernel
hipError_t launch_ring_mid(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                           int64_t M, int64_t N, int64_t K, int bits, hipStream_t st);
hipError_t launch_ring3(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                        int64_t M, int64_t N, int64_t K, hipStream_t st);
bool gemv_wide_preferred(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemv_wide(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                            int64_t M, int64_t N, int64_t K, hipStream_t st);
hipError_t launch_gemv(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                       int64_t M, int64_t N, int64_t K, hipStream_t st);
bool gemm_pipe_supported(int64_t M, int64_t N, int64_t K);
bool gemm_pipe3_supported(int64_t M, int64_t N, int64_t K);  // 3-bit codes, M > 16
bool ring_mid_pipe_preferred(int64_t M, int64_t N, int64_t K);
// ws: null, or gemm_pipe_workspace_bytes(M, N) bytes whose counter part is zero (left zero): the
// pipelined GEMM then splits its work evenly over the compute units (stream-K)
size_t gemm_pipe_workspace_bytes(int64_t M, int64_t N);
// whether the pipelined GEMM splits its work (stream-K) when it is given a workspace
bool gemm_pipe_streamk(int64_t M, int64_t N, int64_t K, int bits);
hipError_t launch_gemm_pipe3(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                             int64_t M, int64_t N, int64_t K, void* ws, hipStream_t st);
hipError_t launch_gemm_pipe(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                            int64_t M, int64_t N, int64_t K, void* ws, hipStream_t st);
hipError_t launch_gemm(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                       int64_t M, int64_t N, int64_t K, void* ws, hipStream_t st);
// 3-bit format: GEMV for M = 1 and short-row M = 2 (gemv.hip), the ring kernel up to M = 16 (skinny.hip),
// the general-shape matrix-core kernel otherwise (gemm.hip)
bool gemv3_supported(int64_t M, int64_t K);
hipError_t launch_gemv3(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                        int64_t M, int64_t N, int64_t K, hipStream_t st);
hipError_t launch_gemm3(const void* x, const void* packed, const void* scales, const void* zeros, void* y,
                        int64_t M, int64_t N, int64_t K, void* ws, hipStream_t st);

// moe.hip: routing, the plan of the ragged groups (ws: moe_plan_workspace bytes of scratch), the weighted sum
size_t moe_plan_workspace(int64_t pairs, int E, int top_k);
hipError_t launch_moe_route(const void* logits, int bytes, int64_t T, int E, int top_k, int renorm, int32_t* experts,
                            float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, int32_t* ws,
                            hipStream_t st);
hipError_t launch_moe_plan(const int32_t* experts, int64_t T, int E, int top_k, int32_t* offsets, int32_t* rows,
                           int32_t* pos, int32_t* ws, hipStream_t st);
hipError_t launch_moe_combine(const void* y, int64_t R, const int32_t* pos, const float* weights, int64_t T, int top_k,
                              int64_t N, void* out, hipStream_t st);

// grouped.hip: products grouped by expert (ws: R x K halfs when s is given)
bool gemm_grouped_fits(int64_t R, int64_t E, int64_t N, int64_t K, int bits, bool scaled);
hipError_t launch_gemm_grouped(const void* x, int64_t x_rows, const int32_t* rows, int top_k, const int32_t* offsets,
                               const float* s, const void* packed, const void* scales, const void* zeros, void* y,
                               int64_t R, int E, int64_t N, int64_t K, int bits, void* ws, hipStream_t st);

// kv_cache.hip, kv_attention.hip: one half (keys or values) of the paged cache
struct KvHalf {
  uint32_t* codes;   // [pages][H][P][D * bits / 32]
  uint32_t* params;  // [pages][H][P]: fp16 scale in the low half, fp16 zero point in the high half
};
hipError_t launch_kv_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* slots,
                           KvHalf kc, KvHalf vc, int64_t T, int D, int bits, KvShape sh, hipStream_t st);
hipError_t launch_kv_read(KvHalf kc, KvHalf vc, const int32_t* slots, void* k, void* v, int64_t T, int D, int bits,
                          KvShape sh, hipStream_t st);
size_t kv_attention_workspace(int64_t B, int64_t Hkv, int ratio, int D, int bits, int64_t max_len);
hipError_t launch_kv_attention(const void* q, int64_t q_stride, KvHalf kc, KvHalf vc, const int32_t* table,
                               int64_t width, const int32_t* lengths, int64_t B, int ratio, int D, int bits,
                               float scale, int64_t max_len, KvShape sh, void* out, void* ws, hipStream_t st);

// norm.hip: the residual sum and the next block's norm (fields as awq_norm's arguments)
struct NormArgs {
  const void* h;
  int64_t h_stride;
  const f16* y;
  int64_t y_stride;
  const f16 *post_weight, *post_bias, *gate;
  const int32_t* gate_rows;
  int64_t gates;
  const f16 *weight, *bias;
  void *h_out, *x;
  float* x_scales;
  int64_t T, N;
  float scale, eps;
  int kind;
};
hipError_t launch_norm(const NormArgs& a, int h_bytes, hipStream_t st);

// rows_i8.hip: rows to 8 bits, of x / s (divide) or x * s; s may be null
hipError_t launch_rows_i8(const void* x, int64_t stride, const float* s, bool divide, int64_t M, int64_t K, void* codes,
                          float* scales, hipStream_t st);

// gemm_i8.hip: the product in 8-bit integers
size_t gemm_i8_workspace(int64_t M, int64_t N, int64_t K, bool quantized);
hipError_t launch_gemm_i8(const void* x, const float* x_scales, const float* s, const void* codes, const float* scales,
                          void* y, int y_bytes, int64_t M, int64_t N, int64_t K, void* ws, hipStream_t st);

// sample.hip: the token of each row of logits (fields as awq_sample's arguments)
struct SampleArgs {
  const void* logits;
  int64_t stride, V;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *u;
  int32_t* tokens;
  float* probs;
  float temperature_value, top_p_value, min_p_value;
  int32_t top_k_value;
};
hipError_t launch_sample(const SampleArgs& a, int logit_bytes, int64_t B, hipStream_t st);

// Dry runs of the product dispatch.  While a KernelPlan is installed on the
// calling thread, each product launcher writes the kernel it would launch (its
// template arguments, block and grid) into it and returns hipSuccess without
// launching anything; the dispatch above it is the ordinary one.
struct KernelPlan {
  char text[160];
};
KernelPlan* active_plan();  // the calling thread's installed plan, or null
void install_plan(KernelPlan* p);
hipError_t plan_record(KernelPlan* p, const char* fmt, ...);

}  // namespace awq
