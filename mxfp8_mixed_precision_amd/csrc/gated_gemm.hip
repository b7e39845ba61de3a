// Entry points of the gated feed-forward GEMMs (kernels in gated_core.h).
#include "gated_core.h"

namespace temx {
namespace {

template <class C, bool BWD>
te_status launch_gated(const GatedParams& p, te_dtype fa, te_dtype fb, hipStream_t stream) {
  constexpr int BN = tile_cols<C, BWD>();
  const dim3 grid((unsigned)(((p.M + C::BM - 1) / C::BM) * ((p.N + BN - 1) / BN)));
  if (fa == TE_E4M3 && fb == TE_E4M3)
    hipLaunchKernelGGL((gated_gemm_kernel<C, TE_E4M3, TE_E4M3, BWD>), grid, dim3(C::kThreads), 0, stream, p);
  else if (fa == TE_E5M2)
    hipLaunchKernelGGL((gated_gemm_kernel<C, TE_E5M2, TE_E4M3, BWD>), grid, dim3(C::kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((gated_gemm_kernel<C, TE_E4M3, TE_E5M2, BWD>), grid, dim3(C::kThreads), 0, stream, p);
  return launch_status();
}

template <class C, bool BWD>
te_status launch_grouped_gated(const GatedParams& p, te_dtype fa, te_dtype fb, unsigned grid, hipStream_t stream) {
  if (fa == TE_E4M3 && fb == TE_E4M3)
    hipLaunchKernelGGL((grouped_gated_gemm_kernel<C, TE_E4M3, TE_E4M3, BWD>), dim3(grid), dim3(C::kThreads), 0, stream,
                       p);
  else if (fa == TE_E5M2)
    hipLaunchKernelGGL((grouped_gated_gemm_kernel<C, TE_E5M2, TE_E4M3, BWD>), dim3(grid), dim3(C::kThreads), 0, stream,
                       p);
  else
    hipLaunchKernelGGL((grouped_gated_gemm_kernel<C, TE_E4M3, TE_E5M2, BWD>), dim3(grid), dim3(C::kThreads), 0, stream,
                       p);
  return launch_status();
}

// Shape limits: those of the dense GEMMs with the 2N rows of the forward's weights, whose scales are addressed
// with 32-bit offsets, as are 128 rows of 2N bf16 pre-activations.
bool gated_shape_ok(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || K % 128 != 0 || N % 16 != 0) return false;
  if (N > ((int64_t)1 << 22) || !dense_shape_ok(M, 2 * N, K)) return false;
  return 2 * N * (K / 32) < ((int64_t)1 << 31) - 4096;
}

// Workspace of the 4-wave tile: the rearranged scales of A and of B's `cols` rows; 0 where it does not serve.
size_t gated_workspace(int64_t M, int64_t cols, int64_t K, int64_t N) {
  if (M <= 0 || N <= 0 || K <= 0 || !gated_shape_ok(M, N, K)) return 0;
  return four_wave_mx(M, cols, K) ? scale_blocks_bytes(M, cols, K) : 0;
}

// The few-row kernel instead of a tile: up to 64 rows; from 33 only where 128-row tiles would leave a quarter of the
// CUs idle (N = 14336, K = 4096, 64 rows: 54 us against 37 with tiles; N = 8192, K = 8192: 56 against 57; N = 4096,
// K = 4096: 17 against 29).  Forward only: a backward of few rows takes the tiles, (N + 127) / 128 workgroups that each
// walk all of K, a third of the CUs or less at these sizes (one and 128 rows, us, and one row's weights at a copy's
// rate: N = 14336, K = 4096 28, 36 and 12; N = K = 8192 47, 61 and 14; N = K = 4096 27, 34 and 3; N = 2048, K = 8192
// 46, 59 and 3).  Gradients are taken of batches, so it has no kernel of its own.
bool few_rows(int64_t M, int64_t N) {
  return M <= 32 || (M <= kFewRows && 4 * ((2 * N + 127) / 128) < 3 * (int64_t)device_cu_count());
}

template <bool BWD>
te_status dense_gated(const GatedParams& p, te_dtype fa, te_dtype fb, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
  const int64_t cols = BWD ? p.N : 2 * p.N;
  if (!BWD && few_rows(p.M, p.N)) return launch_gated_rows(p, fa, fb, stream);
  const size_t want = gated_workspace(p.M, cols, p.K, p.N);
  if (want > 0 && workspace != nullptr && workspace_bytes >= want && ((uintptr_t)workspace & 255u) == 0 &&
      aligned16(p.a_scale) && aligned16(p.b_scale))
    return launch_gated4(p, BWD, fa, fb, workspace, stream);
  const Tile t = pick_tile(p.M, cols, p.K);
  if (t == Tile::SmallDeep) return launch_gated<SmallDeep, BWD>(p, fa, fb, stream);
  if (t == Tile::Small) return launch_gated<Small, BWD>(p, fa, fb, stream);
  return launch_gated<Big, BWD>(p, fa, fb, stream);
}

te_status check_operands(const uint8_t* a, const uint8_t* a_scale, const uint8_t* b, const uint8_t* b_scale) {
  TE_REQUIRE(a && a_scale && b && b_scale, TE_ERR_NULL);
  TE_REQUIRE(aligned16(a) && aligned16(b), TE_ERR_ALIGN);
  TE_REQUIRE(((uintptr_t)a_scale & 3u) == 0 && ((uintptr_t)b_scale & 3u) == 0, TE_ERR_ALIGN);
  return TE_OK;
}

te_status check_formats(te_dtype a_fmt, te_dtype b_fmt, te_activation act) {
  TE_REQUIRE(act == TE_ACT_SILU || act == TE_ACT_GELU, TE_ERR_VALUE);
  TE_REQUIRE(is_fp8(a_fmt) && is_fp8(b_fmt) && !(a_fmt == TE_E5M2 && b_fmt == TE_E5M2), TE_ERR_DTYPE);
  return TE_OK;
}

}  // namespace
}  // namespace temx

using namespace temx;

extern "C" size_t te_mxfp8_gated_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  return gated_workspace(M, 2 * N, K, N);
}

extern "C" te_status te_mxfp8_gated_gemm(const uint8_t* a, const uint8_t* a_scale, te_dtype a_fmt, const uint8_t* b,
                                         const uint8_t* b_scale, te_dtype b_fmt, int64_t M, int64_t N, int64_t K,
                                         te_activation act, void* d, uint8_t* d_scale, te_dtype d_dtype,
                                         const uint16_t* bias, uint16_t* aux, void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
  te_status st = check_formats(a_fmt, b_fmt, act);
  if (st != TE_OK) return st;
  TE_REQUIRE(d_dtype == TE_BF16 || is_fp8(d_dtype), TE_ERR_DTYPE);
  TE_REQUIRE(gated_shape_ok(M, N, K), TE_ERR_SHAPE);
  TE_REQUIRE(d_dtype == TE_BF16 || N % 32 == 0, TE_ERR_SHAPE);
  TE_REQUIRE(d_dtype != TE_BF16 || d_scale == nullptr, TE_ERR_NULL);
  if (M == 0 || N == 0) return TE_OK;
  TE_REQUIRE(d != nullptr && (d_dtype == TE_BF16 || d_scale != nullptr), TE_ERR_NULL);
  TE_REQUIRE(aligned16(d) && aligned16(aux) && ((uintptr_t)bias & 7u) == 0, TE_ERR_ALIGN);
  if (K > 0 && (st = check_operands(a, a_scale, b, b_scale)) != TE_OK) return st;
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const GatedParams p{a, a_scale, b, b_scale, d, d_scale, bias, aux, M, N, K, act, d_dtype, nullptr, 0};
  return dense_gated<false>(p, a_fmt, b_fmt, workspace, workspace_bytes, stream);
}

extern "C" size_t te_mxfp8_dgated_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  return gated_workspace(M, N, K, N);
}

extern "C" te_status te_mxfp8_dgated_gemm(const uint8_t* a, const uint8_t* a_scale, te_dtype a_fmt, const uint8_t* b,
                                          const uint8_t* b_scale, te_dtype b_fmt, int64_t M, int64_t N, int64_t K,
                                          te_activation act, const uint16_t* aux, uint16_t* d, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream) {
  te_status st = check_formats(a_fmt, b_fmt, act);
  if (st != TE_OK) return st;
  TE_REQUIRE(gated_shape_ok(M, N, K), TE_ERR_SHAPE);
  if (M == 0 || N == 0) return TE_OK;
  TE_REQUIRE(d != nullptr && aux != nullptr, TE_ERR_NULL);
  TE_REQUIRE(aligned16(d) && aligned16(aux), TE_ERR_ALIGN);
  if (K > 0 && (st = check_operands(a, a_scale, b, b_scale)) != TE_OK) return st;
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const GatedParams p{a, a_scale, b,  b_scale, d,   nullptr, nullptr, const_cast<uint16_t*>(aux),
                      M, N,       K,  act,     TE_BF16, nullptr, 0};
  return dense_gated<true>(p, a_fmt, b_fmt, workspace, workspace_bytes, stream);
}

namespace temx {
namespace {

// The grouped GEMMs' common part: checks beyond the operands' own, and the launch.
template <bool BWD>
te_status grouped_gated(GatedParams p, te_dtype a_fmt, te_dtype b_fmt, hipStream_t stream) {
  te_status st = check_formats(a_fmt, b_fmt, p.act);
  if (st != TE_OK) return st;
  TE_REQUIRE(p.groups >= 1 && p.groups <= kMaxGroups, TE_ERR_SHAPE);
  TE_REQUIRE(p.N > 0 && p.K > 0 && gated_shape_ok(p.M, p.N, p.K), TE_ERR_SHAPE);
  const int64_t cols = BWD ? p.N : 2 * p.N;
  TE_REQUIRE((p.M / 128 + p.groups) * ((cols + 127) / 128) < ((int64_t)1 << 31), TE_ERR_SHAPE);
  TE_REQUIRE(p.m_splits != nullptr, TE_ERR_NULL);
  TE_REQUIRE(((uintptr_t)p.m_splits & 3u) == 0, TE_ERR_ALIGN);
  if (p.M == 0) return TE_OK;
  TE_REQUIRE(p.d != nullptr && (!BWD || p.aux != nullptr), TE_ERR_NULL);
  TE_REQUIRE(aligned16(p.d) && aligned16(p.aux) && ((uintptr_t)p.bias & 7u) == 0, TE_ERR_ALIGN);
  if ((st = check_operands(p.a, p.a_scale, p.b, p.b_scale)) != TE_OK) return st;
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const int cus = device_cu_count();
  const unsigned grid = cus < 8 ? 8u : (unsigned)(cus / 8 * 8);
  // The splits stay on the device.  Groups of at most a small tile's rows on average take that tile: the weights bound
  // them, and its grid is 4 times as fine (big and small tile, us, forward / backward: N = K = 2048, 8 rows over 64
  // groups 26 / 29 and 20 / 22, 16 groups of 40 rows 35 / 25 and 33 / 20, 16 of 200 rows 43 / 46 and 55 / 38; 32 groups
  // of 64 rows, N = 1536, K = 4096, 123 / 70 and 113 / 71).  One rule for both directions: it is the forward's, and the
  // backward of 16 groups of 200 rows takes the tile that is 8 us slower there.  Else by the big-tile count, estimated
  // from the total rows and one ragged tail per group.
  if (p.M <= 128 * (int64_t)p.groups || use_small_tile((p.M / 256 + p.groups) * ((cols + 255) / 256)))
    return launch_grouped_gated<Small, BWD>(p, a_fmt, b_fmt, 2 * grid, stream);
  return launch_grouped_gated<Big, BWD>(p, a_fmt, b_fmt, grid, stream);
}

}  // namespace
}  // namespace temx

extern "C" te_status te_mxfp8_grouped_gated_gemm(int32_t num_groups, const int32_t* m_splits, int64_t total_m,
                                                 const uint8_t* a, const uint8_t* a_scale, te_dtype a_fmt,
                                                 const uint8_t* b, const uint8_t* b_scale, te_dtype b_fmt, int64_t N,
                                                 int64_t K, te_activation act, uint16_t* d, const uint16_t* bias,
                                                 uint16_t* aux, hipStream_t stream) {
  return grouped_gated<false>(GatedParams{a, a_scale, b, b_scale, d, nullptr, bias, aux, total_m, N, K, act, TE_BF16,
                                          m_splits, num_groups},
                              a_fmt, b_fmt, stream);
}

extern "C" te_status te_mxfp8_grouped_dgated_gemm(int32_t num_groups, const int32_t* m_splits, int64_t total_m,
                                                  const uint8_t* a, const uint8_t* a_scale, te_dtype a_fmt,
                                                  const uint8_t* b, const uint8_t* b_scale, te_dtype b_fmt, int64_t N,
                                                  int64_t K, te_activation act, const uint16_t* aux, uint16_t* d,
                                                  hipStream_t stream) {
  return grouped_gated<true>(GatedParams{a, a_scale, b, b_scale, d, nullptr, nullptr, const_cast<uint16_t*>(aux),
                                         total_m, N, K, act, TE_BF16, m_splits, num_groups},
                             a_fmt, b_fmt, stream);
}
