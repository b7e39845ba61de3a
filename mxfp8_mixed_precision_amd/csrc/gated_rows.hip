// The gated feed-forward GEMM for few rows (decoding steps): M <= 64.
//
// The weights are read once and the products are few: the time is the
// weights' bytes over the HBM bandwidth, so the kernel keeps many of their
// lines in flight and needs no LDS for them.  A workgroup takes 16 NG output
// columns (their gate and up rows of B); its waves deal the K steps of 128
// among themselves in runs of 4, a run's operands held in registers in the
// MFMA's own layout (lane 16 g + r: bytes 16 g .. and 64 + 16 g .. of row r)
// and its scales (a row's 16 bytes) one load.  The waves' partial sums meet in
// LDS and are added in wave order (deterministic); bias, activation, product
// and the MXFP8 encode follow.  All reads go through buffer resources: rows
// past M and K steps past the end read zeros.
// Measured on MI355X, one row, N = 14336, K = 4096: 25.5 us, 121 MB of weights
// and scales at 4.8 TB/s (a large copy: 5.1).  Every workgroup reads all of A,
// twice its weights' bytes at 64 rows: 64 rows of N = K = 4096 take 17 us, of
// N = K = 8192 56 us, where the weights alone take 7 and 27.
#include "gated_core.h"

namespace temx {
namespace {

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, kRsrcWord3);
}

__device__ __forceinline__ v8i load_frag(__amdgpu_buffer_rsrc_t rsrc, int voff, int soff) {
  const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff, soff, 0);
  const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff + 64, soff, 0);
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

constexpr int kRun = 4;  // consecutive K steps of a wave, in flight together

// The scales of 4 steps of a lane's row (byte 4 u + g: step u, block g) for the MFMA, which takes the low byte.  A step
// past the end has zero operands; its scale must not be the NaN code.
__device__ __forceinline__ int run_scale(const u32x4& s, int u, int g, bool ok) { return ok ? (int)(s[u] >> (8 * g)) : 127; }

// W waves, NG groups of 16 output columns, MF groups of 16 rows.
template <int W, int NG, int MF, int FA, int FB>
__global__ __launch_bounds__(64 * W) void gated_rows_kernel(GatedParams p) {
  constexpr int NF = 2 * NG * MF;  // accumulator fragments: [NG][gate, up][MF]
  __shared__ float part[W][NF][256];
  __shared__ __attribute__((aligned(16))) uint16_t out[16 * MF][16 * NG];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t K = p.K, N = p.N, ks = K / 32;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NG);
  const int ng = (int)min((int64_t)NG, (N - n0) / 16);  // column groups of the last workgroup
  const int kt_n = (int)(K / BK);

  const __amdgpu_buffer_rsrc_t ra = buffer_of(p.a, p.M * K), rsa = buffer_of(p.a_scale, p.M * ks);
  __amdgpu_buffer_rsrc_t rb[2], rsb[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    rb[h] = buffer_of(p.b + (h * N + n0) * K, 16 * ng * K);
    rsb[h] = buffer_of(p.b_scale + (h * N + n0) * ks, 16 * ng * ks);
  }
  const int vo = (int)(r * K) + 16 * g, vs = (int)(r * ks);
  v4f acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int k0 = kRun * wave; k0 < kt_n; k0 += kRun * W) {
    v8i b[kRun][2 * NG], a[kRun][MF];
    u32x4 sb[2 * NG], sa[MF];
#pragma unroll
    for (int f = 0; f < 2 * NG; ++f)
      sb[f] = __builtin_amdgcn_raw_buffer_load_b128(rsb[f & 1], vs + (int)(16 * (f >> 1) * ks), 4 * k0, 0);
#pragma unroll
    for (int j = 0; j < MF; ++j) sa[j] = __builtin_amdgcn_raw_buffer_load_b128(rsa, vs + (int)(16 * j * ks), 4 * k0, 0);
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      // a step past the end: an offset beyond every resource (their sizes are below 2^30), zeros are read
      const int so = k0 + u < kt_n ? (k0 + u) * BK : 0x40000000;
#pragma unroll
      for (int f = 0; f < 2 * NG; ++f) b[u][f] = load_frag(rb[f & 1], vo + (int)(16 * (f >> 1) * K), so);
#pragma unroll
      for (int j = 0; j < MF; ++j) a[u][j] = load_frag(ra, vo + (int)(16 * j * K), so);
    }
#pragma unroll
    for (int u = 0; u < kRun; ++u)
#pragma unroll
      for (int f = 0; f < 2 * NG; ++f)
#pragma unroll
        for (int j = 0; j < MF; ++j)
          acc[f * MF + j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              b[u][f], a[u][j], acc[f * MF + j], MfmaFmt<FB>::v, MfmaFmt<FA>::v, 0,
              run_scale(sb[f], u, g, k0 + u < kt_n), 0, run_scale(sa[j], u, g, k0 + u < kt_n));
  }
  // lane (g, r), element e: row r of the fragment, column 4 g + e
#pragma unroll
  for (int f = 0; f < NF; ++f)
    *reinterpret_cast<float4*>(&part[wave][f][4 * lane]) = make_float4(acc[f][0], acc[f][1], acc[f][2], acc[f][3]);
  __syncthreads();

  const bool mx = p.out != TE_BF16;
  for (int o = threadIdx.x; o < 16 * MF * 16 * NG; o += 64 * W) {
    const int m = o / (16 * NG), c = o % (16 * NG);
    const int64_t n = n0 + c;
    if (m >= p.M || n >= N) continue;  // their codes below are not stored either
    const int f = 2 * (c >> 4) * MF + (m >> 4), at = 64 * ((c >> 2) & 3) + 4 * (m & 15) + (c & 3);
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      gate += part[w][f][at];
      up += part[w][f + MF][at];
    }
    if (p.bias != nullptr) {
      gate += bf16_bits_to_float(p.bias[n]);
      up += bf16_bits_to_float(p.bias[N + n]);
    }
    if (p.aux != nullptr) {
      const uint32_t both = pack_bf16x2(gate, up);
      p.aux[m * 2 * N + n] = (uint16_t)both;
      p.aux[m * 2 * N + N + n] = (uint16_t)(both >> 16);
    }
    const float d = (p.act == TE_ACT_SILU ? silu(gate) : gelu_tanh(gate)) * up;
    const uint16_t bits = (uint16_t)pack_bf16x2(d, 0.f);
    if (mx) out[m][c] = bits;
    else static_cast<uint16_t*>(p.d)[m * N + n] = bits;
  }
  if constexpr (NG % 2 == 0) {
    if (!mx) return;
    __syncthreads();
    // N % 32 == 0: NG / 2 32-blocks of each row, 4 lanes (a DPP quad) a block
    for (int o = threadIdx.x; o < 16 * MF * 2 * NG; o += 64 * W) {
      const int m = o / (2 * NG), q = o % (2 * NG);
      const uint4 v = *reinterpret_cast<const uint4*>(&out[m][8 * q]);
      const uint32_t amax = quad_max(absmax_bits8(v));
      const bool e4m3 = p.out == TE_E4M3;
      const uint32_t code = e4m3 ? e8m0_code_from_amax_bits<TE_E4M3>(amax) : e8m0_code_from_amax_bits<TE_E5M2>(amax);
      const float s = e8m0_to_float(code);
      const uint2 x = e4m3 ? cvt8_scaled<TE_E4M3>(v, s) : cvt8_scaled<TE_E5M2>(v, s);
      const int64_t n = n0 + 8 * q;
      if (m < p.M && n < N) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.d) + m * N + n) = x;
        if ((q & 3) == 0) p.d_scale[m * (N / 32) + n / 32] = (uint8_t)code;
      }
    }
  }
}

template <int W, int NG, int MF>
te_status launch(const GatedParams& p, te_dtype fa, te_dtype fb, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 16 * NG - 1) / (16 * NG))), block(64 * W);
  if (fa == TE_E4M3 && fb == TE_E4M3)
    hipLaunchKernelGGL((gated_rows_kernel<W, NG, MF, TE_E4M3, TE_E4M3>), grid, block, 0, stream, p);
  else if (fa == TE_E5M2)
    hipLaunchKernelGGL((gated_rows_kernel<W, NG, MF, TE_E5M2, TE_E4M3>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((gated_rows_kernel<W, NG, MF, TE_E4M3, TE_E5M2>), grid, block, 0, stream, p);
  return launch_status();
}

}  // namespace

// 8 waves and 16 columns a workgroup: as many CUs as possible read weights (one CU takes in ~26 bytes a ns whatever
// its waves; K = 8192, N = 2048, one row: 12 us with 16 columns, 21.8 with 32).  32 columns where MXFP8 output needs
// its 32-blocks (64 workgroups for that row to MXFP8, 21.8 us), and for 17 to 32 rows of wide layers, which read the
// rows' operands half as often (N = 14336, K = 4096, 32 rows: 40 -> 35 us; N = 8192, K = 8192: 42 -> 41, N = 4096,
// K = 4096: 13 -> 18).
te_status launch_gated_rows(const GatedParams& p, te_dtype fa, te_dtype fb, hipStream_t stream) {
  if (p.out == TE_BF16) {
    if (p.M <= 16) return launch<8, 1, 1>(p, fa, fb, stream);
    if (p.M <= 32 && p.N / 16 < 2 * (int64_t)device_cu_count()) return launch<8, 1, 2>(p, fa, fb, stream);
    if (p.M <= 32) return launch<8, 2, 2>(p, fa, fb, stream);
    return launch<8, 1, 4>(p, fa, fb, stream);
  }
  if (p.M <= 16) return launch<8, 2, 1>(p, fa, fb, stream);
  if (p.M <= 32) return launch<8, 2, 2>(p, fa, fb, stream);
  return launch<4, 2, 4>(p, fa, fb, stream);
}

}  // namespace temx
