// The gated feed-forward GEMM for few rows (decoding steps): M <= 64.
//
// The weights are read once and the products are few: the time is the
// weights' bytes over the HBM bandwidth, so the kernel keeps many of their
// lines in flight and needs no LDS for them.  A workgroup takes 16 NG output
// columns (their gate and up rows of B) and its waves deal the K steps of 128
// among themselves, so a workgroup reads runs of consecutive lines of each
// row; a wave holds kUnroll steps of operands in registers in the MFMA's own
// layout (lane 16 g + r: bytes 16 g .. and 64 + 16 g .. of row r, the scale
// byte of block g).  The waves' partial sums meet in LDS and are added in wave
// order (deterministic); bias, activation, product and the MXFP8 encode follow.
// All reads go through buffer resources: rows past M and K steps past the end
// read zeros.
#include "gated_core.h"

namespace temx {
namespace {

constexpr int kUnroll = 4;  // K steps of a wave in flight

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, kRsrcWord3);
}

template <int POLICY>
__device__ __forceinline__ v8i load_frag(__amdgpu_buffer_rsrc_t rsrc, int voff, int soff) {
  const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff, soff, POLICY);
  const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff + 64, soff, POLICY);
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// W waves, NG groups of 16 output columns, MF groups of 16 rows.
template <int W, int NG, int MF, int FA, int FB>
__global__ __launch_bounds__(64 * W) void gated_rows_kernel(GatedParams p) {
  constexpr int NF = 2 * NG * MF;  // accumulator fragments: [gate, up][NG][MF]
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
  const int vo = (int)(r * K) + 16 * g, vs = (int)(r * ks) + g;
  v4f acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int k0 = wave; k0 < kt_n; k0 += W * kUnroll) {
    v8i b[kUnroll][2 * NG], a[kUnroll][MF];
    int sb[kUnroll][2 * NG], sa[kUnroll][MF];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int kt = k0 + W * u;
      // a step past the end: an offset beyond every resource (their sizes are below 2^30), zeros are read
      const int so = kt < kt_n ? kt * BK : 0x40000000, ss = kt < kt_n ? kt * 4 : 0x40000000;
#pragma unroll
      for (int f = 0; f < 2 * NG; ++f) {
        const int row = (int)(16 * (f >> 1));
        b[u][f] = load_frag<kNonTemporal>(rb[f & 1], vo + (int)(row * K), so);
        sb[u][f] = __builtin_amdgcn_raw_buffer_load_b8(rsb[f & 1], vs + (int)(row * ks), ss, 0);
      }
#pragma unroll
      for (int j = 0; j < MF; ++j) {
        a[u][j] = load_frag<0>(ra, vo + (int)(16 * j * K), so);
        sa[u][j] = __builtin_amdgcn_raw_buffer_load_b8(rsa, vs + (int)(16 * j * ks), ss, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int f = 0; f < 2 * NG; ++f)
#pragma unroll
        for (int j = 0; j < MF; ++j)
          acc[f * MF + j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              b[u][f], a[u][j], acc[f * MF + j], MfmaFmt<FB>::v, MfmaFmt<FA>::v, 0, sb[u][f], 0, sa[u][j]);
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
  if constexpr (NG == 2) {
    if (!mx) return;
    __syncthreads();
    // N % 32 == 0: the workgroup's columns are one 32-block of each row; 4 lanes (a DPP quad) a row
    for (int o = threadIdx.x; o < 16 * MF * 4; o += 64 * W) {
      const int m = o >> 2, q = o & 3;
      const uint4 v = *reinterpret_cast<const uint4*>(&out[m][8 * q]);
      const uint32_t amax = quad_max(absmax_bits8(v));
      const bool e4m3 = p.out == TE_E4M3;
      const uint32_t code = e4m3 ? e8m0_code_from_amax_bits<TE_E4M3>(amax) : e8m0_code_from_amax_bits<TE_E5M2>(amax);
      const float s = e8m0_to_float(code);
      const uint2 x = e4m3 ? cvt8_scaled<TE_E4M3>(v, s) : cvt8_scaled<TE_E5M2>(v, s);
      if (m < p.M) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.d) + m * N + n0 + 8 * q) = x;
        if (q == 0) p.d_scale[m * (N / 32) + n0 / 32] = (uint8_t)code;
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

te_status launch_gated_rows(const GatedParams& p, te_dtype fa, te_dtype fb, hipStream_t stream) {
  if (p.out == TE_BF16) {
    if (p.M <= 16) return launch<8, 1, 1>(p, fa, fb, stream);
    if (p.M <= 32) return launch<8, 1, 2>(p, fa, fb, stream);
    return launch<8, 1, 4>(p, fa, fb, stream);
  }
  if (p.M <= 16) return launch<8, 2, 1>(p, fa, fb, stream);
  if (p.M <= 32) return launch<8, 2, 2>(p, fa, fb, stream);
  return launch<4, 2, 4>(p, fa, fb, stream);
}

}  // namespace temx
