// The extern "C" entry points around the layers declared in include/awq.h: the
// block norm, rows in 8 bits and their product, the token choice.  Argument checks
// and launches; as in awq_api.hip, no entry point allocates memory, synchronises
// the device or lets a C++ exception escape.
#include <cmath>
#include <cstdio>

#include "awq.h"
#include "awq_api_util.h"
#include "awq_internal.h"

namespace {

using awq::as_stream;
using awq::check_aligned;
using awq::device_status;

constexpr int64_t kMaxRowsK = 1 << 17;   // 127^2 * 2^17 < 2^31
constexpr int64_t kMaxRows = 1 << 24;

int check_rows_k(int64_t K) {
  AWQ_REQUIRE(K >= AWQ_GROUP && K % AWQ_GROUP == 0 && K <= kMaxRowsK, AWQ_ERROR_INVALID_VALUE,
              "K=%lld must be a multiple of %d in [%d, 2^17]", (long long)K, AWQ_GROUP, AWQ_GROUP);
  return AWQ_OK;
}

int check_stride(int64_t stride, int64_t N, const char* name) {
  AWQ_REQUIRE(stride >= N && stride % 8 == 0 && stride < (int64_t(1) << 31), AWQ_ERROR_INVALID_VALUE,
              "%s=%lld must be a multiple of 8, at least a row (%lld) and below 2^31", name, (long long)stride,
              (long long)N);
  return AWQ_OK;
}

int check_product(int64_t M, int64_t N, int64_t K) {
  AWQ_REQUIRE(M >= 1 && M <= (int64_t(1) << 22), AWQ_ERROR_INVALID_VALUE, "M=%lld outside [1, 2^22]", (long long)M);
  AWQ_REQUIRE(N >= 1 && N <= kMaxRows, AWQ_ERROR_INVALID_VALUE, "N=%lld outside [1, 2^24]", (long long)N);
  if (int st = check_rows_k(K)) return st;
  AWQ_REQUIRE(M * N <= (int64_t(1) << 36), AWQ_ERROR_INVALID_VALUE, "M=%lld rows of N=%lld exceed one launch",
              (long long)M, (long long)N);
  return AWQ_OK;
}

}  // namespace

extern "C" {

int awq_norm(const void* h, int32_t h_bytes, int64_t h_stride, const void* y, int64_t y_stride,
             const void* post_weight, const void* post_bias, const void* gate, const int32_t* gate_rows, int64_t gates,
             float scale, const void* weight, const void* bias, int32_t kind, float eps, void* h_out, void* x,
             float* x_scales, int64_t T, int64_t N, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(h, AWQ_ERROR_INVALID_VALUE, "h must not be NULL");
  AWQ_REQUIRE(y || weight, AWQ_ERROR_INVALID_VALUE, "y and weight must not both be NULL (nothing to compute)");
  AWQ_REQUIRE((y != nullptr) == (h_out != nullptr), AWQ_ERROR_INVALID_VALUE,
              "h_out must be given with y, and NULL without it");
  AWQ_REQUIRE((weight != nullptr) == (x != nullptr), AWQ_ERROR_INVALID_VALUE,
              "x must be given with weight, and NULL without it");
  AWQ_REQUIRE(y || (!post_weight && !gate), AWQ_ERROR_INVALID_VALUE, "post_weight and gate are for y, which is NULL");
  AWQ_REQUIRE(post_weight || !post_bias, AWQ_ERROR_INVALID_VALUE, "post_bias without post_weight");
  AWQ_REQUIRE(gate || !gate_rows, AWQ_ERROR_INVALID_VALUE, "gate_rows without gate");
  AWQ_REQUIRE(weight || (!bias && !x_scales), AWQ_ERROR_INVALID_VALUE, "bias or x_scales without weight");
  AWQ_REQUIRE(h_bytes == 2 || h_bytes == 4, AWQ_ERROR_INVALID_VALUE, "h_bytes must be 2 (fp16) or 4 (fp32), got %d",
              h_bytes);
  AWQ_REQUIRE(kind == AWQ_NORM_RMS || kind == AWQ_NORM_LAYER, AWQ_ERROR_INVALID_VALUE, "kind must be 0 or 1 (got %d)",
              kind);
  AWQ_REQUIRE(!x_scales || (kind == AWQ_NORM_RMS && !bias), AWQ_ERROR_INVALID_VALUE,
              "rows in 8 bits are of the rms kind, without bias");
  AWQ_REQUIRE(eps >= 0.f && std::isfinite(eps) && std::isfinite(scale), AWQ_ERROR_INVALID_VALUE,
              "eps must be finite and >= 0, scale finite");
  AWQ_REQUIRE(T >= 1 && T <= kMaxRows, AWQ_ERROR_INVALID_VALUE, "T=%lld outside [1, 2^24]", (long long)T);
  AWQ_REQUIRE(N >= 8 && N % 8 == 0 && N <= 65536, AWQ_ERROR_INVALID_VALUE, "N=%lld must be a multiple of 8 in [8, 65536]",
              (long long)N);
  if (int st = check_stride(h_stride, N, "h_stride")) return st;
  if (y)
    if (int st = check_stride(y_stride, N, "y_stride")) return st;
  AWQ_REQUIRE(h_out != h || !h_out || h_stride == N, AWQ_ERROR_INVALID_VALUE, "h_out may be h only with h_stride = N");
  if (gate) {
    AWQ_REQUIRE(gates >= 1 && gates <= kMaxRows, AWQ_ERROR_INVALID_VALUE, "gates=%lld outside [1, 2^24]",
                (long long)gates);
    AWQ_REQUIRE(gate_rows || gates == 1 || gates == T, AWQ_ERROR_INVALID_VALUE,
                "gates=%lld must be 1 or T without gate_rows", (long long)gates);
  }
  if (int st = check_aligned({{h, "h"}, {y, "y"}, {post_weight, "post_weight"}, {post_bias, "post_bias"}, {gate, "gate"},
                              {gate_rows, "gate_rows"}, {weight, "weight"}, {bias, "bias"}, {h_out, "h_out"}, {x, "x"},
                              {x_scales, "x_scales"}}))
    return st;
  const auto half = [](const void* p) { return reinterpret_cast<const awq::f16*>(p); };
  const awq::NormArgs a{h, h_stride, half(y), y_stride, half(post_weight), half(post_bias), half(gate), gate_rows, gates,
                        half(weight), half(bias), h_out, x, x_scales, T, N, scale, eps, kind};
  return device_status(awq::launch_norm(a, h_bytes, as_stream(stream)), "awq_norm");
  AWQ_GUARD_END
}

int awq_quantize_rows(const void* x, int64_t x_stride, const float* s, int64_t M, int64_t K, void* codes, float* scales,
                      void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(x && codes && scales, AWQ_ERROR_INVALID_VALUE, "x, codes and scales must not be NULL");
  AWQ_REQUIRE(M >= 1 && M <= kMaxRows, AWQ_ERROR_INVALID_VALUE, "M=%lld outside [1, 2^24]", (long long)M);
  if (int st = check_rows_k(K)) return st;
  if (int st = check_stride(x_stride, K, "x_stride")) return st;
  if (int st = check_aligned({{x, "x"}, {s, "s"}, {codes, "codes"}, {scales, "scales"}})) return st;
  return device_status(awq::launch_rows_i8(x, x_stride, s, true, M, K, codes, scales, as_stream(stream)),
                       "awq_quantize_rows");
  AWQ_GUARD_END
}

int awq_pack_i8(const void* W, const float* s, int64_t N, int64_t K, void* codes, float* scales, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(W && codes && scales, AWQ_ERROR_INVALID_VALUE, "W, codes and scales must not be NULL");
  AWQ_REQUIRE(N >= 1 && N <= kMaxRows, AWQ_ERROR_INVALID_VALUE, "N=%lld outside [1, 2^24]", (long long)N);
  if (int st = check_rows_k(K)) return st;
  if (int st = check_aligned({{W, "W"}, {s, "s"}, {codes, "codes"}, {scales, "scales"}})) return st;
  return device_status(awq::launch_rows_i8(W, K, s, false, N, K, codes, scales, as_stream(stream)), "awq_pack_i8");
  AWQ_GUARD_END
}

size_t awq_gemm_i8_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t quantized) {
  if (check_product(M, N, K) != AWQ_OK) return 0;
  return awq::gemm_i8_workspace(M, N, K, quantized != 0);
}

int awq_gemm_i8(const void* x, const float* x_scales, const float* s, const void* codes, const float* scales, void* y,
                int32_t y_bytes, int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(x && codes && scales && y, AWQ_ERROR_INVALID_VALUE, "x, codes, scales and y must not be NULL");
  AWQ_REQUIRE(!x_scales || !s, AWQ_ERROR_INVALID_VALUE, "s is for an fp16 x, and x is in 8 bits");
  AWQ_REQUIRE(y_bytes == 2 || y_bytes == 4, AWQ_ERROR_INVALID_VALUE, "y_bytes must be 2 (fp16) or 4 (fp32), got %d",
              y_bytes);
  if (int st = check_product(M, N, K)) return st;
  const size_t need = awq::gemm_i8_workspace(M, N, K, x_scales != nullptr);
  AWQ_REQUIRE(workspace || need == 0, AWQ_ERROR_INVALID_VALUE, "workspace must not be NULL (%zu bytes needed)", need);
  if (int st = check_aligned({{x, "x"}, {x_scales, "x_scales"}, {s, "s"}, {codes, "codes"}, {scales, "scales"}, {y, "y"},
                              {workspace, "workspace"}}))
    return st;
  AWQ_REQUIRE(workspace_bytes >= need, AWQ_ERROR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes,
              need);
  return device_status(awq::launch_gemm_i8(x, x_scales, s, codes, scales, y, y_bytes, M, N, K, workspace,
                                           as_stream(stream)),
                       "awq_gemm_i8");
  AWQ_GUARD_END
}

int awq_gemm_i8_kernel(int64_t M, int64_t N, int64_t K, int32_t quantized, char* out, size_t out_bytes) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(out && out_bytes > 0, AWQ_ERROR_INVALID_VALUE, "out must not be NULL or empty");
  out[0] = 0;
  if (int st = check_product(M, N, K)) return st;
  awq::KernelPlan plan{};
  awq::install_plan(&plan);
  const float dummy = 0.f;
  const hipError_t e = awq::launch_gemm_i8(nullptr, quantized ? &dummy : nullptr, nullptr, nullptr, nullptr, nullptr, 2, M,
                                           N, K, nullptr, nullptr);
  awq::install_plan(nullptr);
  snprintf(out, out_bytes, "%s", plan.text);
  return device_status(e, "awq_gemm_i8_kernel");
  AWQ_GUARD_END
}

int awq_sample(const void* logits, int32_t logit_bytes, int64_t stride, int64_t B, int64_t V, const float* temperature,
               float temperature_value, const int32_t* top_k, int32_t top_k_value, const float* top_p,
               float top_p_value, const float* min_p, float min_p_value, const float* u, int32_t* tokens, float* probs,
               void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(logits && u && tokens, AWQ_ERROR_INVALID_VALUE, "logits, u and tokens must not be NULL");
  AWQ_REQUIRE(logit_bytes == 2 || logit_bytes == 4, AWQ_ERROR_INVALID_VALUE,
              "logit_bytes must be 2 (fp16) or 4 (fp32), got %d", logit_bytes);
  AWQ_REQUIRE(B >= 1 && B <= (1 << 20), AWQ_ERROR_INVALID_VALUE, "B=%lld outside [1, 2^20]", (long long)B);
  AWQ_REQUIRE(V >= 1 && V <= (1 << 20), AWQ_ERROR_INVALID_VALUE, "V=%lld outside [1, 2^20]", (long long)V);
  AWQ_REQUIRE(stride >= V && stride < (int64_t(1) << 40) / B, AWQ_ERROR_INVALID_VALUE,
              "stride=%lld must be at least V, and B * stride below 2^40", (long long)stride);
  AWQ_REQUIRE(!std::isnan(temperature_value) && !std::isnan(top_p_value) && !std::isnan(min_p_value),
              AWQ_ERROR_INVALID_VALUE, "temperature, top_p and min_p must be numbers");
  if (int st = check_aligned({{logits, "logits"}, {temperature, "temperature"}, {top_k, "top_k"}, {top_p, "top_p"},
                              {min_p, "min_p"}, {u, "u"}, {tokens, "tokens"}, {probs, "probs"}}))
    return st;
  const awq::SampleArgs a{logits, stride, V, temperature, top_k, top_p, min_p, u, tokens, probs, temperature_value,
                          top_p_value, min_p_value, top_k_value};
  return device_status(awq::launch_sample(a, logit_bytes, B, as_stream(stream)), "awq_sample");
  AWQ_GUARD_END
}

}  // extern "C"
