// The extern "C" entry points of the expert and key-value cache operators
// declared in include/awq.h: argument checks and launches.  As in awq_api.hip,
// no entry point allocates memory, synchronises the device or lets a C++
// exception escape.
#include <cmath>
#include <cstdio>

#include "awq.h"
#include "awq_api_util.h"
#include "awq_internal.h"

namespace {

using awq::as_stream;
using awq::check_aligned;
using awq::check_bits;
using awq::check_layer;
using awq::device_status;

constexpr int64_t kMaxGroupedK = 1 << 17;  // a block holds its weight rows' scales and zeros in LDS

int check_pairs(int64_t T, int32_t E, int32_t top_k) {
  AWQ_REQUIRE(T >= 1 && T <= (int64_t(1) << 24), AWQ_ERROR_INVALID_VALUE, "T=%lld outside [1, 2^24]", (long long)T);
  AWQ_REQUIRE(E >= 1 && E <= AWQ_MAX_EXPERTS, AWQ_ERROR_INVALID_VALUE, "E=%d outside [1, %d]", E, AWQ_MAX_EXPERTS);
  AWQ_REQUIRE(top_k >= 1 && top_k <= 64, AWQ_ERROR_INVALID_VALUE, "top_k=%d outside [1, 64]", top_k);
  AWQ_REQUIRE(T * top_k <= AWQ_MAX_PAIRS, AWQ_ERROR_INVALID_VALUE, "T * top_k = %lld exceeds 2^24",
              (long long)(T * top_k));
  return AWQ_OK;
}

// One cache: sizes every cache entry point checks alike.
int check_cache(int64_t pages, int32_t H, int32_t page, int32_t D, int32_t bits, awq::KvShape* sh) {
  AWQ_REQUIRE(bits == 4 || bits == 8, AWQ_ERROR_INVALID_VALUE, "bits must be 4 or 8 (got %d)", bits);
  AWQ_REQUIRE(D == 64 || D == 128 || D == 256, AWQ_ERROR_INVALID_VALUE, "D must be 64, 128 or 256 (got %d)", D);
  AWQ_REQUIRE(page >= 16 && page <= 1024 && (page & (page - 1)) == 0, AWQ_ERROR_INVALID_VALUE,
              "page must be a power of two in [16, 1024] (got %d)", page);
  AWQ_REQUIRE(H >= 1 && H <= 1024, AWQ_ERROR_INVALID_VALUE, "H=%d outside [1, 1024]", H);
  AWQ_REQUIRE(pages >= 1 && pages * page < (int64_t(1) << 31) && pages < (int64_t(1) << 31), AWQ_ERROR_INVALID_VALUE,
              "pages=%lld: a cache has between one page and 2^31 - 1 slots", (long long)pages);
  int ps = 0;
  while ((1 << ps) < page) ++ps;
  *sh = awq::KvShape{pages, H, ps};
  return AWQ_OK;
}

awq::KvHalf half_of(const void* codes, const void* params) {
  return {reinterpret_cast<uint32_t*>(const_cast<void*>(codes)), reinterpret_cast<uint32_t*>(const_cast<void*>(params))};
}

}  // namespace

extern "C" {

size_t awq_moe_workspace_bytes(int64_t T, int32_t E, int32_t top_k) {
  if (T < 1 || E < 1 || E > AWQ_MAX_EXPERTS || top_k < 1 || top_k > 64 || T > AWQ_MAX_PAIRS || T * top_k > AWQ_MAX_PAIRS)
    return 0;
  return (awq::moe_plan_workspace(T * top_k, E, top_k) + 255) / 256 * 256;
}

int awq_moe_plan(const int32_t* experts, int64_t T, int32_t E, int32_t top_k, int32_t* offsets, int32_t* rows,
                 int32_t* pos, void* workspace, size_t workspace_bytes, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(experts && offsets && rows && pos && workspace, AWQ_ERROR_INVALID_VALUE,
              "experts, offsets, rows, pos and workspace must not be NULL");
  if (int st = check_pairs(T, E, top_k)) return st;
  if (int st = check_aligned({{experts, "experts"}, {offsets, "offsets"}, {rows, "rows"}, {pos, "pos"},
                              {workspace, "workspace"}}))
    return st;
  const size_t need = awq_moe_workspace_bytes(T, E, top_k);
  AWQ_REQUIRE(workspace_bytes >= need, AWQ_ERROR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes,
              need);
  return device_status(awq::launch_moe_plan(experts, T, E, top_k, offsets, rows, pos,
                                            reinterpret_cast<int32_t*>(workspace), as_stream(stream)),
                       "awq_moe_plan");
  AWQ_GUARD_END
}

int awq_moe_route(const void* logits, int32_t logit_bytes, int64_t T, int32_t E, int32_t top_k, int32_t renormalize,
                  int32_t* experts, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* workspace,
                  size_t workspace_bytes, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(logits && experts && weights && offsets && rows && pos && workspace, AWQ_ERROR_INVALID_VALUE,
              "logits, experts, weights, offsets, rows, pos and workspace must not be NULL");
  AWQ_REQUIRE(logit_bytes == 2 || logit_bytes == 4, AWQ_ERROR_INVALID_VALUE,
              "logit_bytes must be 2 (fp16) or 4 (fp32), got %d", logit_bytes);
  if (int st = check_pairs(T, E, top_k)) return st;
  AWQ_REQUIRE(top_k <= E, AWQ_ERROR_INVALID_VALUE, "top_k=%d exceeds the %d experts", top_k, E);
  AWQ_REQUIRE(renormalize == 0 || renormalize == 1, AWQ_ERROR_INVALID_VALUE, "renormalize must be 0 or 1 (got %d)",
              renormalize);
  if (int st = check_aligned({{logits, "logits"}, {experts, "experts"}, {weights, "weights"}, {offsets, "offsets"},
                              {rows, "rows"}, {pos, "pos"}, {workspace, "workspace"}}))
    return st;
  const size_t need = awq_moe_workspace_bytes(T, E, top_k);
  AWQ_REQUIRE(workspace_bytes >= need, AWQ_ERROR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes,
              need);
  return device_status(awq::launch_moe_route(logits, logit_bytes, T, E, top_k, renormalize, experts, weights, offsets,
                                             rows, pos, reinterpret_cast<int32_t*>(workspace), as_stream(stream)),
                       "awq_moe_route");
  AWQ_GUARD_END
}

size_t awq_gemm_grouped_workspace_bytes(int64_t R, int64_t K, int32_t scaled) {
  if (R < 1 || R > AWQ_MAX_PAIRS || K < 1 || K > kMaxGroupedK || K % AWQ_GROUP != 0 || scaled == 0) return 0;
  const size_t bytes = R <= 2 * AWQ_MAX_EXPERTS ? 4 : 2;  // x / s of few rows is two numbers
  return ((size_t)R * (size_t)K * bytes + 255) / 256 * 256;
}

int awq_gemm_grouped(const void* x, int64_t x_rows, const int32_t* rows, int32_t top_k, const int32_t* offsets,
                     const float* s, const void* packed, const void* scales, const void* zeros, void* y, int64_t R,
                     int32_t E, int64_t N, int64_t K, int32_t group, int32_t bits, void* workspace,
                     size_t workspace_bytes, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(x && offsets && packed && scales && zeros && y, AWQ_ERROR_INVALID_VALUE,
              "x, offsets, packed, scales, zeros and y must not be NULL");
  int st = check_layer(N, K, group);
  if (st == AWQ_OK) st = check_bits(bits);
  if (st != AWQ_OK) return st;
  AWQ_REQUIRE(K <= kMaxGroupedK, AWQ_ERROR_INVALID_VALUE, "K=%lld exceeds 2^17", (long long)K);
  AWQ_REQUIRE(R >= 1 && R <= AWQ_MAX_PAIRS, AWQ_ERROR_INVALID_VALUE, "R=%lld outside [1, 2^24]", (long long)R);
  AWQ_REQUIRE(E >= 1 && E <= AWQ_MAX_EXPERTS, AWQ_ERROR_INVALID_VALUE, "E=%d outside [1, %d]", E, AWQ_MAX_EXPERTS);
  AWQ_REQUIRE(top_k >= 1, AWQ_ERROR_INVALID_VALUE, "top_k must be >= 1 (got %d)", top_k);
  AWQ_REQUIRE(x_rows >= 1 && x_rows <= AWQ_MAX_PAIRS && (rows || x_rows >= R), AWQ_ERROR_INVALID_VALUE,
              "x_rows=%lld outside [1, 2^24], or fewer than R without rows", (long long)x_rows);
  AWQ_REQUIRE(awq::gemm_grouped_fits(R, E, N, K, bits, s != nullptr), AWQ_ERROR_INVALID_VALUE,
              "R=%lld rows of N=%lld exceed one launch", (long long)R, (long long)N);
  const size_t need = awq_gemm_grouped_workspace_bytes(R, K, s != nullptr);
  AWQ_REQUIRE(workspace || need == 0, AWQ_ERROR_INVALID_VALUE, "workspace must not be NULL (%zu bytes needed)", need);
  if (int st2 = check_aligned({{x, "x"}, {rows, "rows"}, {offsets, "offsets"}, {s, "s"}, {packed, "packed"},
                               {scales, "scales"}, {zeros, "zeros"}, {y, "y"}, {workspace, "workspace"}}))
    return st2;
  AWQ_REQUIRE(workspace_bytes >= need, AWQ_ERROR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes,
              need);
  return device_status(awq::launch_gemm_grouped(x, x_rows, rows, top_k, offsets, s, packed, scales, zeros, y, R, E, N, K,
                                                bits, workspace, as_stream(stream)),
                       "awq_gemm_grouped");
  AWQ_GUARD_END
}

int awq_gemm_grouped_kernel(int64_t R, int32_t E, int64_t N, int64_t K, int32_t group, int32_t bits, char* out,
                            size_t out_bytes) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(out && out_bytes > 0, AWQ_ERROR_INVALID_VALUE, "out must not be NULL or empty");
  out[0] = 0;
  int st = check_layer(N, K, group);
  if (st == AWQ_OK) st = check_bits(bits);
  if (st != AWQ_OK) return st;
  AWQ_REQUIRE(K <= kMaxGroupedK && R >= 1 && R <= AWQ_MAX_PAIRS && E >= 1 && E <= AWQ_MAX_EXPERTS &&
                  awq::gemm_grouped_fits(R, E, N, K, bits, false),
              AWQ_ERROR_INVALID_VALUE, "R=%lld E=%d N=%lld K=%lld: sizes awq_gemm_grouped refuses", (long long)R, E,
              (long long)N, (long long)K);
  awq::KernelPlan plan{};
  awq::install_plan(&plan);
  const hipError_t e = awq::launch_gemm_grouped(nullptr, R, nullptr, 1, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                R, E, N, K, bits, nullptr, nullptr);
  awq::install_plan(nullptr);
  snprintf(out, out_bytes, "%s", plan.text);
  return device_status(e, "awq_gemm_grouped_kernel");
  AWQ_GUARD_END
}

int awq_moe_combine(const void* y, int64_t R, const int32_t* pos, const float* weights, int64_t T, int32_t top_k,
                    int64_t N, void* out, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(y && pos && weights && out, AWQ_ERROR_INVALID_VALUE, "y, pos, weights and out must not be NULL");
  if (int st = check_pairs(T, 1, top_k)) return st;
  AWQ_REQUIRE(R >= 1 && R <= AWQ_MAX_PAIRS, AWQ_ERROR_INVALID_VALUE, "R=%lld outside [1, 2^24]", (long long)R);
  AWQ_REQUIRE(N >= 8 && N % 8 == 0 && N <= (int64_t(1) << 20), AWQ_ERROR_INVALID_VALUE,
              "N=%lld must be a multiple of 8 in [8, 2^20]", (long long)N);
  AWQ_REQUIRE(T * (N / 8) < (int64_t(1) << 32) - 256, AWQ_ERROR_INVALID_VALUE, "T=%lld rows of N=%lld exceed one launch",
              (long long)T, (long long)N);
  if (int st = check_aligned({{y, "y"}, {pos, "pos"}, {weights, "weights"}, {out, "out"}})) return st;
  return device_status(awq::launch_moe_combine(y, R, pos, weights, T, top_k, N, out, as_stream(stream)),
                       "awq_moe_combine");
  AWQ_GUARD_END
}

size_t awq_kv_codes_bytes(int64_t pages, int32_t H, int32_t page, int32_t D, int32_t bits) {
  awq::KvShape sh;
  if (check_cache(pages, H, page, D, bits, &sh) != AWQ_OK) return 0;
  return (size_t)(pages * page) * (size_t)H * (size_t)(D * bits / 8);
}

size_t awq_kv_params_bytes(int64_t pages, int32_t H, int32_t page) {
  awq::KvShape sh;
  if (check_cache(pages, H, page, 64, 4, &sh) != AWQ_OK) return 0;
  return (size_t)(pages * page) * (size_t)H * 4;
}

int awq_kv_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* slots, void* k_codes,
                 void* k_params, void* v_codes, void* v_params, int64_t T, int32_t H, int32_t D, int64_t pages,
                 int32_t page, int32_t bits, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(k && v && slots && k_codes && k_params && v_codes && v_params, AWQ_ERROR_INVALID_VALUE,
              "k, v, slots and the cache's four arrays must not be NULL");
  awq::KvShape sh;
  if (int st = check_cache(pages, H, page, D, bits, &sh)) return st;
  AWQ_REQUIRE(T >= 1 && T <= AWQ_MAX_KV_TOKENS && (T + 31) * H * (D / 8) < (int64_t(1) << 32), AWQ_ERROR_INVALID_VALUE,
              "T=%lld: between 1 and 2^22 tokens, (T + 31) * H * D below 2^35, are moved by one call", (long long)T);
  for (int64_t s : {k_stride, v_stride})
    AWQ_REQUIRE(s >= (int64_t)H * D && s % 8 == 0 && s < (int64_t(1) << 31), AWQ_ERROR_INVALID_VALUE,
                "a token stride of %lld elements: a multiple of 8, at least H * D and below 2^31, is needed",
                (long long)s);
  if (int st = check_aligned({{k, "k"}, {v, "v"}, {slots, "slots"}, {k_codes, "k_codes"}, {k_params, "k_params"},
                              {v_codes, "v_codes"}, {v_params, "v_params"}}))
    return st;
  return device_status(awq::launch_kv_write(k, v, k_stride, v_stride, slots, half_of(k_codes, k_params),
                                            half_of(v_codes, v_params), T, D, bits, sh, as_stream(stream)),
                       "awq_kv_write");
  AWQ_GUARD_END
}

int awq_kv_read(const void* k_codes, const void* k_params, const void* v_codes, const void* v_params,
                const int32_t* slots, void* k, void* v, int64_t T, int32_t H, int32_t D, int64_t pages, int32_t page,
                int32_t bits, void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(k && v && slots && k_codes && k_params && v_codes && v_params, AWQ_ERROR_INVALID_VALUE,
              "k, v, slots and the cache's four arrays must not be NULL");
  awq::KvShape sh;
  if (int st = check_cache(pages, H, page, D, bits, &sh)) return st;
  AWQ_REQUIRE(T >= 1 && T <= AWQ_MAX_KV_TOKENS && (T + 31) * H * (D / 8) < (int64_t(1) << 32), AWQ_ERROR_INVALID_VALUE,
              "T=%lld: between 1 and 2^22 tokens, (T + 31) * H * D below 2^35, are moved by one call", (long long)T);
  if (int st = check_aligned({{k_codes, "k_codes"}, {k_params, "k_params"}, {v_codes, "v_codes"},
                              {v_params, "v_params"}, {slots, "slots"}, {k, "k"}, {v, "v"}}))
    return st;
  return device_status(awq::launch_kv_read(half_of(k_codes, k_params), half_of(v_codes, v_params), slots, k, v, T, D,
                                           bits, sh, as_stream(stream)),
                       "awq_kv_read");
  AWQ_GUARD_END
}

size_t awq_kv_attention_workspace_bytes(int64_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t bits, int64_t max_len) {
  if (B < 1 || B > 65535 || Hkv < 1 || Hkv > 1024 || Hq < Hkv || Hq % Hkv != 0 || Hq > 65536 ||
      (D != 64 && D != 128 && D != 256) || (bits != 4 && bits != 8) || max_len < 1 || max_len > AWQ_MAX_KV_LENGTH)
    return 0;
  return (awq::kv_attention_workspace(B, Hkv, Hq / Hkv, D, bits, max_len) + 255) / 256 * 256;
}

int awq_kv_attention(const void* q, int64_t q_stride, const void* k_codes, const void* k_params, const void* v_codes,
                     const void* v_params, const int32_t* page_table, int64_t table_width, const int32_t* lengths,
                     void* out, int64_t B, int32_t Hq, int32_t Hkv, int32_t D, int64_t pages, int32_t page,
                     int32_t bits, float scale, int64_t max_len, void* workspace, size_t workspace_bytes,
                     void* stream) {
  AWQ_GUARD_BEGIN
  AWQ_REQUIRE(q && k_codes && k_params && v_codes && v_params && page_table && lengths && out, AWQ_ERROR_INVALID_VALUE,
              "q, the cache's four arrays, page_table, lengths and out must not be NULL");
  awq::KvShape sh;
  if (int st = check_cache(pages, Hkv, page, D, bits, &sh)) return st;
  AWQ_REQUIRE(B >= 1 && B <= 65535, AWQ_ERROR_INVALID_VALUE, "B=%lld outside [1, 65535]", (long long)B);
  AWQ_REQUIRE(Hq >= Hkv && Hq % Hkv == 0 && Hq <= 65536, AWQ_ERROR_INVALID_VALUE,
              "Hq=%d must be a multiple of Hkv=%d, at most 65536", Hq, Hkv);
  AWQ_REQUIRE(B * Hq * D < (int64_t(1) << 32), AWQ_ERROR_INVALID_VALUE, "B * Hq * D = %lld: below 2^32 is needed",
              (long long)(B * Hq * D));
  AWQ_REQUIRE(q_stride >= (int64_t)Hq * D && q_stride % 8 == 0 && q_stride < (int64_t(1) << 31),
              AWQ_ERROR_INVALID_VALUE,
              "a q stride of %lld elements: a multiple of 8, at least Hq * D and below 2^31, is needed",
              (long long)q_stride);
  AWQ_REQUIRE(table_width >= 1 && table_width * page < (int64_t(1) << 31) && table_width < (int64_t(1) << 31),
              AWQ_ERROR_INVALID_VALUE, "table_width=%lld: between one page and 2^31 - 1 slots", (long long)table_width);
  const int64_t room = table_width * page;
  const int64_t most = max_len == 0 || max_len > room ? room : max_len;
  AWQ_REQUIRE(max_len >= 0 && most <= AWQ_MAX_KV_LENGTH, AWQ_ERROR_INVALID_VALUE,
              "a longest length of %lld tokens: at most 2^25 are served (give max_len)", (long long)most);
  AWQ_REQUIRE(std::isfinite(scale) && std::fabs(scale) <= 0x1p64f, AWQ_ERROR_INVALID_VALUE,
              "scale must be finite and at most 2^64 in magnitude");
  const size_t need = awq_kv_attention_workspace_bytes(B, Hq, Hkv, D, bits, most);
  AWQ_REQUIRE(workspace || need == 0, AWQ_ERROR_INVALID_VALUE, "workspace must not be NULL (%zu bytes needed)", need);
  if (int st = check_aligned({{q, "q"}, {k_codes, "k_codes"}, {k_params, "k_params"}, {v_codes, "v_codes"},
                              {v_params, "v_params"}, {page_table, "page_table"}, {lengths, "lengths"}, {out, "out"},
                              {workspace, "workspace"}}))
    return st;
  AWQ_REQUIRE(workspace_bytes >= need, AWQ_ERROR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes,
              need);
  return device_status(awq::launch_kv_attention(q, q_stride, half_of(k_codes, k_params), half_of(v_codes, v_params),
                                                page_table, table_width, lengths, B, Hq / Hkv, D, bits, scale, most, sh,
                                                out, need ? workspace : nullptr, as_stream(stream)),
                       "awq_kv_attention");
  AWQ_GUARD_END
}

}  // extern "C"
