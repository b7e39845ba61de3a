// GEMMs of few rows with 4-bit weights and group scales, for gfx950.
//
//   P[m, n] = sum_g s[n, g] sum_{k in group g} x[m, k] (q[n, k] - z[n, g])   (+ bias[n])
//   D = P, or act(P[:, :N]) * P[:, N:]
// q are the codes of INT4 (0 .. 15, z the zero point, 8 without one) or E2M1 (z = 0).
//
// A workgroup takes 16 NF rows of W (16 output columns, or their gate and up rows); its waves deal the K steps of 128
// among themselves and their partial sums meet in LDS, in wave order.  Lane 16 q + r loads 16 bytes of row r, the codes
// of the step's 32-block q; a 4 x 4 transpose across the lanes gives MFMA i (16 x 16 x 32) block i: lane 16 q + r holds
// codes 8 q .. 8 q + 7 of row r, turned into bf16 / fp16 by exact conversions (a code 0 .. 15 is the E4M3 code of
// 2^-9 times itself).  Products and sums are fp32; a group's sum is scaled in fp32, after its zero point times the sum
// of x, which another MFMA gives with ones for weights.
#include "row_chunks.h"

namespace temx {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;        // K of a wave's step: 4 blocks of 32
constexpr int kMaxGroups = 1024;  // experts

struct W4Params {
  const void* x;
  const uint8_t* w;
  const void* scale;
  const uint8_t* zero;
  const void* bias;
  void* d;
  const int32_t* m_splits;  // grouped only
  int64_t M, N, K;
  int group, groups;
  int act;  // te_activation, or -1: not gated
  te_dtype scale_dtype;
  bool d_fp32;
};

template <class T> struct Half;  // the activations' type in the MFMA
template <> struct Half<bf16_t> {
  typedef v8bf v8;
  static __device__ __forceinline__ v4f mfma(v8 a, v8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t v) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, HI));
  }
  template <int BYTE>
  static __device__ __forceinline__ uint32_t from_e2m1(uint32_t v) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, BYTE));
  }
  static constexpr uint32_t ones = 0x3F803F80u;
};
template <> struct Half<f16_t> {
  typedef v8h v8;
  static __device__ __forceinline__ v4f mfma(v8 a, v8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t v) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.f, HI));
  }
  template <int BYTE>
  static __device__ __forceinline__ uint32_t from_e2m1(uint32_t v) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.f, BYTE));
  }
  static constexpr uint32_t ones = 0x3C003C00u;
};

// 8 codes (low half-byte first) as the MFMA's operand.
template <class T, te_w4_format FMT>
__device__ __forceinline__ typename Half<T>::v8 weights(uint32_t v) {
  u32x4 r;
  if constexpr (FMT == TE_W4_INT4) {
    const uint32_t h = v >> 4;
    const uint32_t lo = __builtin_amdgcn_perm(h, v, 0x05010400u) & 0x0F0F0F0Fu;  // v0 h0 v1 h1
    const uint32_t hi = __builtin_amdgcn_perm(h, v, 0x07030602u) & 0x0F0F0F0Fu;  // v2 h2 v3 h3
    r = u32x4{Half<T>::template from_e4m3<false>(lo), Half<T>::template from_e4m3<true>(lo),
              Half<T>::template from_e4m3<false>(hi), Half<T>::template from_e4m3<true>(hi)};
  } else {
    r = u32x4{Half<T>::template from_e2m1<0>(v), Half<T>::template from_e2m1<1>(v),
              Half<T>::template from_e2m1<2>(v), Half<T>::template from_e2m1<3>(v)};
  }
  return __builtin_bit_cast(typename Half<T>::v8, r);
}

// Lane 16 q + r: dwords 0 .. 3 of block q of row r -> dword q of blocks 0 .. 3.
__device__ __forceinline__ u32x4 transpose_blocks(u32x4 v) {
  const u32x2 a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const u32x2 b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const u32x2 c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const u32x2 d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float load_scale(const void* p, int64_t i, te_dtype dtype) {
  if (dtype == TE_E8M0) {
    const uint32_t code = static_cast<const uint8_t*>(p)[i];
    return code == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_float(code);
  }
  if (dtype == TE_FP32) return static_cast<const float*>(p)[i];
  if (dtype == TE_BF16) return to_float(static_cast<const bf16_t*>(p)[i]);
  return to_float(static_cast<const f16_t*>(p)[i]);
}

__device__ __forceinline__ float silu(float x) { return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f)); }

// W waves, NF fragments of 16 weight rows (a gated pair counts two), MF fragments of 16 rows of x, scaling every SB
// blocks of 32 (the group is a multiple of them).
template <class T, te_w4_format FMT, bool GATED, int W, int NF, int MF, int SB>
__global__ __launch_bounds__(64 * W) void w4_kernel(W4Params p) {
  constexpr int kCols = GATED ? 8 * NF : 16 * NF;  // output columns of the workgroup
  constexpr bool kZero = FMT == TE_W4_INT4;
  __shared__ float part[W][NF * MF][256];
  typedef typename Half<T>::v8 v8;
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * kCols, K = p.K, ng = K / p.group;
  int64_t t0 = 0, t_end = p.M, t_step = 16 * MF, w_row = 0, b_row = 0;
  if (p.m_splits != nullptr) {  // this expert's rows and weights
    const int g = blockIdx.y;
    for (int e = 0; e < g; ++e) t0 += max(p.m_splits[e], 0);
    t_end = min(t0 + max(p.m_splits[g], 0), p.M);
    w_row = (int64_t)g * (GATED ? 2 * p.N : p.N);
    b_row = w_row;
  } else {
    t0 = blockIdx.y * t_step;
    t_step *= gridDim.y;
  }
  // the lane's weight rows: row r of each fragment, the last row where there is none (its column is not stored)
  const uint8_t* wp[NF];
  int64_t row_of[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int64_t n = min(n0 + (GATED ? 16 * (f >> 1) : 16 * f) + r, p.N - 1);
    row_of[f] = w_row + n + (GATED && (f & 1) ? p.N : 0);
    wp[f] = p.w + row_of[f] * (K / 2);
  }

  for (; t0 < t_end; t0 += t_step) {
    v4f total[NF][MF];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j) total[f][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int64_t k0 = wave * kStep; k0 < K; k0 += W * kStep) {
      u32x4 codes[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        codes[f] = u32x4{0, 0, 0, 0};
        if (k0 + 32 * q < K) codes[f] = *reinterpret_cast<const u32x4*>(wp[f] + k0 / 2 + 16 * q);
        codes[f] = transpose_blocks(codes[f]);
      }
      v4f acc[NF][MF], xsum[MF];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i % SB == 0) {
#pragma unroll
          for (int j = 0; j < MF; ++j) {
            xsum[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[f][j] = v4f{0.f, 0.f, 0.f, 0.f};
          }
        }
        if (k0 + 32 * i >= K) break;
        v8 xf[MF];
#pragma unroll
        for (int j = 0; j < MF; ++j) {
          u32x4 v = {0, 0, 0, 0};
          const int64_t t = t0 + 16 * j + r;
          if (t < t_end) v = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.x) + t * K + k0 + 32 * i + 8 * q);
          xf[j] = __builtin_bit_cast(v8, v);
          if constexpr (kZero)
            xsum[j] = Half<T>::mfma(xf[j], __builtin_bit_cast(v8, u32x4{Half<T>::ones, Half<T>::ones, Half<T>::ones, Half<T>::ones}), xsum[j]);
        }
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const v8 wf = weights<T, FMT>(codes[f][i]);
#pragma unroll
          for (int j = 0; j < MF; ++j) acc[f][j] = Half<T>::mfma(xf[j], wf, acc[f][j]);
        }
        if (i % SB == SB - 1 || k0 + 32 * (i + 1) >= K) {
          const int64_t g = (k0 + 32 * i) / p.group;
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const float s = load_scale(p.scale, row_of[f] * ng + g, p.scale_dtype);
            const float z = !kZero ? 0.f : p.zero != nullptr ? (float)p.zero[row_of[f] * ng + g] : 8.f;
#pragma unroll
            for (int j = 0; j < MF; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = kZero ? __builtin_fmaf(-z, xsum[j][e], acc[f][j][e]) : acc[f][j][e];
                total[f][j][e] = __builtin_fmaf(s, a, total[f][j][e]);
              }
          }
        }
      }
    }
    // lane (q, r), element e: row 4 q + e of x, weight row r of the fragment
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][f * MF + j][16 * (4 * q + e) + r] = total[f][j][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * MF * kCols; o += 64 * W) {
      const int m = o / kCols, c = o % kCols;
      const int64_t t = t0 + m, n = n0 + c;
      if (t >= t_end || n >= p.N) continue;
      const int f = GATED ? 2 * (c >> 4) : c >> 4, at = 16 * (m & 15) + (c & 15);
      float v = 0.f, up = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        v += part[w][f * MF + (m >> 4)][at];
        if constexpr (GATED) up += part[w][(f + 1) * MF + (m >> 4)][at];
      }
      if (p.bias != nullptr) {
        v += to_float(static_cast<const T*>(p.bias)[b_row + n]);
        if constexpr (GATED) up += to_float(static_cast<const T*>(p.bias)[b_row + p.N + n]);
      }
      if constexpr (GATED) v = (p.act == TE_ACT_SILU ? silu(v) : gelu_tanh(v)) * up;
      if (p.d_fp32) static_cast<float*>(p.d)[t * p.N + n] = v;
      else static_cast<T*>(p.d)[t * p.N + n] = from_float<T>(v);
    }
    __syncthreads();
  }
}

template <class T, te_w4_format FMT, bool GATED, int MF, int SB>
te_status launch(const W4Params& p, hipStream_t stream) {
  constexpr int W = 8, NF = GATED ? 2 : 1, kCols = GATED ? 8 * NF : 16 * NF;
  const dim3 grid((unsigned)((p.N + kCols - 1) / kCols),
                  p.m_splits != nullptr ? (unsigned)p.groups : (unsigned)std::min<int64_t>((p.M + 16 * MF - 1) / (16 * MF), 65535));
  hipLaunchKernelGGL((w4_kernel<T, FMT, GATED, W, NF, MF, SB>), grid, dim3(64 * W), 0, stream, p);
  return launch_status();
}

template <class T, te_w4_format FMT, bool GATED, int MF>
te_status by_group(const W4Params& p, hipStream_t stream) {
  if (p.group % 128 == 0) return launch<T, FMT, GATED, MF, 4>(p, stream);
  if (p.group % 64 == 0) return launch<T, FMT, GATED, MF, 2>(p, stream);
  return launch<T, FMT, GATED, MF, 1>(p, stream);
}

template <class T, te_w4_format FMT, bool GATED>
te_status by_rows(const W4Params& p, hipStream_t stream) {
  const int64_t rows = p.m_splits != nullptr ? (p.M + p.groups - 1) / p.groups : p.M;
  if (rows <= 16) return by_group<T, FMT, GATED, 1>(p, stream);
  if (rows <= 32) return by_group<T, FMT, GATED, 2>(p, stream);
  return by_group<T, FMT, GATED, 4>(p, stream);
}

template <class T, te_w4_format FMT>
te_status by_act(const W4Params& p, hipStream_t stream) {
  return p.act >= 0 ? by_rows<T, FMT, true>(p, stream) : by_rows<T, FMT, false>(p, stream);
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

te_status run(const W4Params& p, te_dtype dtype, te_w4_format fmt, te_dtype d_dtype, bool gated, hipStream_t stream) {
  TE_REQUIRE(fmt == TE_W4_INT4 || fmt == TE_W4_E2M1, TE_ERR_VALUE);
  TE_REQUIRE(!gated || p.act == TE_ACT_SILU || p.act == TE_ACT_GELU, TE_ERR_VALUE);
  TE_REQUIRE(dtype == TE_BF16 || dtype == TE_FP16, TE_ERR_DTYPE);
  TE_REQUIRE(p.scale_dtype == dtype || p.scale_dtype == TE_FP32 || p.scale_dtype == TE_E8M0, TE_ERR_DTYPE);
  TE_REQUIRE(d_dtype == dtype || d_dtype == TE_FP32, TE_ERR_DTYPE);
  constexpr int64_t kMostSize = ((int64_t)1 << 31) - 65536;
  TE_REQUIRE(p.M >= 0 && p.M <= kMostSize && p.N >= 0 && p.N <= kMostSize / 2 && p.K >= 0 && p.K <= kMostSize, TE_ERR_SHAPE);
  TE_REQUIRE(p.group >= 32 && p.group % 32 == 0 && p.K % p.group == 0, TE_ERR_SHAPE);
  TE_REQUIRE(p.groups >= 1 && p.groups <= kMaxGroups, TE_ERR_SHAPE);
  TE_REQUIRE(fmt == TE_W4_INT4 || p.zero == nullptr, TE_ERR_NULL);
  if (p.M == 0 || p.N == 0) return TE_OK;
  TE_REQUIRE(p.d != nullptr && (p.K == 0 || (p.x && p.w && p.scale)), TE_ERR_NULL);
  TE_REQUIRE(aligned16(p.x) && aligned16(p.w) && aligned16(p.d) && aligned_to(p.bias, 2), TE_ERR_ALIGN);
  TE_REQUIRE(aligned_to(p.scale, p.scale_dtype == TE_FP32 ? 4 : p.scale_dtype == TE_E8M0 ? 1 : 2), TE_ERR_ALIGN);
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  if (dtype == TE_BF16)
    return fmt == TE_W4_INT4 ? by_act<bf16_t, TE_W4_INT4>(p, stream) : by_act<bf16_t, TE_W4_E2M1>(p, stream);
  return fmt == TE_W4_INT4 ? by_act<f16_t, TE_W4_INT4>(p, stream) : by_act<f16_t, TE_W4_E2M1>(p, stream);
}

te_status run_grouped(const W4Params& p, te_dtype dtype, te_w4_format fmt, te_dtype d_dtype, bool gated, hipStream_t stream) {
  TE_REQUIRE(p.groups >= 1 && p.groups <= kMaxGroups, TE_ERR_SHAPE);
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
  return run(W4Params{x, w, w_scale, w_zero, bias, d, nullptr, M, N, K, group_size, 1, -1, scale_dtype, d_dtype == TE_FP32},
             dtype, w_fmt, d_dtype, false, stream);
}

extern "C" te_status te_w4_gated_gemm(const void* x, te_dtype dtype, const uint8_t* w, te_w4_format w_fmt,
                                      const void* w_scale, te_dtype scale_dtype, const uint8_t* w_zero,
                                      int32_t group_size, int64_t M, int64_t N, int64_t K, te_activation act, void* d,
                                      te_dtype d_dtype, const void* bias, hipStream_t stream) {
  return run(W4Params{x, w, w_scale, w_zero, bias, d, nullptr, M, N, K, group_size, 1, (int)act, scale_dtype,
                      d_dtype == TE_FP32},
             dtype, w_fmt, d_dtype, true, stream);
}

extern "C" te_status te_w4_grouped_gemm(int32_t num_groups, const int32_t* m_splits, int64_t total_m, const void* x,
                                        te_dtype dtype, const uint8_t* w, te_w4_format w_fmt, const void* w_scale,
                                        te_dtype scale_dtype, const uint8_t* w_zero, int32_t group_size, int64_t N,
                                        int64_t K, void* d, te_dtype d_dtype, const void* bias, hipStream_t stream) {
  return run_grouped(W4Params{x, w, w_scale, w_zero, bias, d, m_splits, total_m, N, K, group_size, num_groups, -1,
                              scale_dtype, d_dtype == TE_FP32},
                     dtype, w_fmt, d_dtype, false, stream);
}

extern "C" te_status te_w4_grouped_gated_gemm(int32_t num_groups, const int32_t* m_splits, int64_t total_m,
                                              const void* x, te_dtype dtype, const uint8_t* w, te_w4_format w_fmt,
                                              const void* w_scale, te_dtype scale_dtype, const uint8_t* w_zero,
                                              int32_t group_size, int64_t N, int64_t K, te_activation act, void* d,
                                              te_dtype d_dtype, const void* bias, hipStream_t stream) {
  return run_grouped(W4Params{x, w, w_scale, w_zero, bias, d, m_splits, total_m, N, K, group_size, num_groups,
                              (int)act, scale_dtype, d_dtype == TE_FP32},
                     dtype, w_fmt, d_dtype, true, stream);
}
