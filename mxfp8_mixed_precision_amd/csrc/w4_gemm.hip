// Entry points of the GEMMs with 4-bit weights (kernels in w4_core.h).
#include "w4_core.h"

namespace temx {
namespace {

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

te_status run(const W4Params& p, te_dtype dtype, te_w4_format fmt, te_dtype d_dtype, bool gated, hipStream_t stream) {
  TE_REQUIRE(fmt == TE_W4_INT4 || fmt == TE_W4_E2M1, TE_ERR_VALUE);
  TE_REQUIRE(!gated || p.act == TE_ACT_SILU || p.act == TE_ACT_GELU, TE_ERR_VALUE);
  TE_REQUIRE(dtype == TE_BF16 || dtype == TE_FP16, TE_ERR_DTYPE);
  TE_REQUIRE(p.scale_dtype == dtype || p.scale_dtype == TE_FP32 || p.scale_dtype == TE_E8M0, TE_ERR_DTYPE);
  TE_REQUIRE(d_dtype == dtype || d_dtype == TE_FP32, TE_ERR_DTYPE);
  constexpr int64_t kMostSize = ((int64_t)1 << 31) - 65536;
  // N: a launch has fewer than 2^32 threads side by side; K: the kernels' offsets into 64 rows of x and 16 of W are of
  // 32 bits
  TE_REQUIRE(p.M >= 0 && p.M <= kMostSize && p.N >= 0 && p.N <= (int64_t)1 << 26, TE_ERR_SHAPE);
  TE_REQUIRE(p.K >= 0 && p.K <= (int64_t)1 << 23, TE_ERR_SHAPE);
  TE_REQUIRE(p.group >= 32 && p.group % 32 == 0 && p.K % p.group == 0, TE_ERR_SHAPE);
  TE_REQUIRE(p.groups >= 1 && p.groups <= kW4MaxGroups, TE_ERR_SHAPE);
  TE_REQUIRE(fmt == TE_W4_INT4 || p.zero == nullptr, TE_ERR_NULL);
  if (p.M == 0 || p.N == 0) return TE_OK;
  TE_REQUIRE(p.d != nullptr && (p.K == 0 || (p.x && p.w && p.scale)), TE_ERR_NULL);
  TE_REQUIRE(aligned16(p.x) && aligned16(p.w) && aligned16(p.d) && aligned_to(p.bias, 2), TE_ERR_ALIGN);
  TE_REQUIRE(aligned_to(p.scale, p.scale_dtype == TE_FP32 ? 4 : p.scale_dtype == TE_E8M0 ? 1 : 2), TE_ERR_ALIGN);
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  if (dtype == TE_BF16) return fmt == TE_W4_INT4 ? launch_w4_bf16_int4(p, stream) : launch_w4_bf16_e2m1(p, stream);
  return fmt == TE_W4_INT4 ? launch_w4_fp16_int4(p, stream) : launch_w4_fp16_e2m1(p, stream);
}

te_status run_grouped(const W4Params& p, te_dtype dtype, te_w4_format fmt, te_dtype d_dtype, bool gated,
                      hipStream_t stream) {
  TE_REQUIRE(p.groups >= 1 && p.groups <= kW4MaxGroups, TE_ERR_SHAPE);
  TE_REQUIRE(p.N > 0 && p.K > 0, TE_ERR_SHAPE);
  TE_REQUIRE(p.m_splits != nullptr, TE_ERR_NULL);
  TE_REQUIRE(aligned_to(p.m_splits, 4), TE_ERR_ALIGN);
  return run(p, dtype, fmt, d_dtype, gated, stream);
}

}  // namespace
}  // namespace temx

using namespace temx;

extern "C" te_status te_w4_gemm(const void* x, te_dtype dtype, const uint8_t* w, te_w4_format w_fmt,
                                const void* w_scale, te_dtype scale_dtype, const uint8_t* w_zero, int32_t group_size,
                                int64_t M, int64_t N, int64_t K, void* d, te_dtype d_dtype, const void* bias,
                                hipStream_t stream) {
  return run(W4Params{x, w, w_scale, w_zero, bias, d, nullptr, M, N, K, group_size, 1, -1, scale_dtype, d_dtype == TE_FP32, 0, 0, 0, 0},
             dtype, w_fmt, d_dtype, false, stream);
}

extern "C" te_status te_w4_gated_gemm(const void* x, te_dtype dtype, const uint8_t* w, te_w4_format w_fmt,
                                      const void* w_scale, te_dtype scale_dtype, const uint8_t* w_zero,
                                      int32_t group_size, int64_t M, int64_t N, int64_t K, te_activation act, void* d,
                                      te_dtype d_dtype, const void* bias, hipStream_t stream) {
  return run(W4Params{x, w, w_scale, w_zero, bias, d, nullptr, M, N, K, group_size, 1, (int)act, scale_dtype,
                      d_dtype == TE_FP32, 0, 0, 0, 0},
             dtype, w_fmt, d_dtype, true, stream);
}

extern "C" te_status te_w4_grouped_gemm(int32_t num_groups, const int32_t* m_splits, int64_t total_m, const void* x,
                                        te_dtype dtype, const uint8_t* w, te_w4_format w_fmt, const void* w_scale,
                                        te_dtype scale_dtype, const uint8_t* w_zero, int32_t group_size, int64_t N,
                                        int64_t K, void* d, te_dtype d_dtype, const void* bias, hipStream_t stream) {
  return run_grouped(W4Params{x, w, w_scale, w_zero, bias, d, m_splits, total_m, N, K, group_size, num_groups, -1,
                              scale_dtype, d_dtype == TE_FP32, 0, 0, 0, 0},
                     dtype, w_fmt, d_dtype, false, stream);
}

extern "C" te_status te_w4_grouped_gated_gemm(int32_t num_groups, const int32_t* m_splits, int64_t total_m,
                                              const void* x, te_dtype dtype, const uint8_t* w, te_w4_format w_fmt,
                                              const void* w_scale, te_dtype scale_dtype, const uint8_t* w_zero,
                                              int32_t group_size, int64_t N, int64_t K, te_activation act, void* d,
                                              te_dtype d_dtype, const void* bias, hipStream_t stream) {
  return run_grouped(W4Params{x, w, w_scale, w_zero, bias, d, m_splits, total_m, N, K, group_size, num_groups,
                              (int)act, scale_dtype, d_dtype == TE_FP32, 0, 0, 0, 0},
                     dtype, w_fmt, d_dtype, true, stream);
}
