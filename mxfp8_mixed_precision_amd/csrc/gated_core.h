// The gated feed-forward GEMMs on MXFP8 operands for gfx950, built on the
// tiles and main loops of gemm_core.h.
//
// Forward, with W = [gate rows 0 .. N-1; up rows N .. 2N-1] ([2N, K]):
//   P = A . W^T + bias,  D[m, n] = act(P[m, n]) * P[m, N + n]
// in one kernel: both projections share the A tile, and the accumulators of
// P[m, n] and P[m, N + n] sit in the same lane, so the activation and the
// product need no exchange.  A B tile of BN rows is BN / 2 gate rows and the
// BN / 2 up rows of the same columns, in alternating 16-row groups (tile row
// r: group r / 16, even groups gate, odd groups up); column fragment 2 p of a
// wave is then 16 gate columns and fragment 2 p + 1 the same columns' up.
//
// Backward: acc = dY . W2 (the output gradient through the down projection,
// [M, N]), and from the saved pre-activations aux = [gate | up] ([M, 2N])
//   D[m, n] = acc up act'(gate),  D[m, N + n] = acc act(gate).
#pragma once

#include "gemm_core.h"

namespace temx {
namespace {

struct GatedParams {
  const uint8_t* a;
  const uint8_t* a_scale;
  const uint8_t* b;
  const uint8_t* b_scale;
  void* d;
  uint8_t* d_scale;      // MXFP8 D only
  const uint16_t* bias;  // [2N] ([groups, 2N]), or NULL
  uint16_t* aux;         // forward: written, or NULL; backward: read
  int64_t M, N, K;       // N: columns of the gated product
  te_activation act;
  te_dtype out;          // forward: TE_BF16, TE_E4M3, TE_E5M2
  const int32_t* m_splits;  // grouped only
  int32_t groups;
};

// ---- activations ------------------------------------------------------------

// silu(x) = x / (1 + e) with e = 2^(-x log2 e)
__device__ __forceinline__ float silu(float x) {
  return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}

// silu and its derivative s + x s (1 - s), s = 1 / (1 + e); s (1 - s) = 1 / (2 + e + 1 / e) keeps its relative
// accuracy in both tails, and the product is 0 once that factor is (x may be infinite there)
__device__ __forceinline__ void silu_and_grad(float x, float& v, float& dv) {
  const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * x);
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  const float sd = __builtin_amdgcn_rcpf(2.0f + e + __builtin_amdgcn_rcpf(e));
  v = x * s;
  dv = s + (sd == 0.0f ? 0.0f : x * sd);
}

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == TE_ACT_SILU) return silu(x);
  else return gelu_tanh(x);
}

template <int ACT>
__device__ __forceinline__ void act_and_grad(float x, float& v, float& dv) {
  if constexpr (ACT == TE_ACT_SILU) {
    silu_and_grad(x, v, dv);
  } else {
    v = gelu_tanh(x);
    dv = dgelu_tanh(x);
  }
}

// ---- the two-part B operand -------------------------------------------------

// B tile of the forward GEMM, BN / 2 output columns from n0.  A copier wave's
// data slices (8 tile rows, q = c + 4 i) all lie in groups of one kind, gate
// for copiers 0 and 1 and up for 2 and 3, since q / 2 has c / 2's parity; so
// each copier needs one of the two resources.  Slice q is rows 16 i + 8 (c & 1)
// of that part where the plain tile has 32 i + 8 c: the copy loops' offsets
// hold 8 c rows, so the up part's resource starts 16 rows early (no lane's
// offset falls below those 16 rows).
// The scale resource covers both parts: a lane's row of a 64-row scale slice
// is gate or up by its tile row.  Gate rows past N (ragged N) read up scales;
// their data rows read as zeros and their columns are never stored.
struct GatedOperand {
  i32x4 data;
  i32x4 scale;
  int voff_scale;  // lane l's row of a 64-row scale slice, in bytes
};

template <class C>
__device__ __forceinline__ GatedOperand make_gated_operand(const uint8_t* b, const uint8_t* b_scale, int64_t n0,
                                                           int64_t N, int64_t K, int wave, int lane) {
  static_assert(C::NCOPY == 4, "slice q of copier c is gate or up by c / 2");
  const int64_t rows = min((int64_t)C::BN / 2, N - n0);
  const bool up = ((wave - (C::NW - C::NCOPY)) & 2) != 0;
  GatedOperand o;
  o.data = up ? make_rsrc(b + (N + n0 - 16) * K, (rows + 16) * K) : make_rsrc(b + n0 * K, rows * K);
  o.scale = make_rsrc(b_scale + n0 * (K / 32), (2 * N - n0) * (K / 32));
  o.voff_scale = (int)(((lane >> 5) * 16 + (lane & 15) + (int64_t)((lane >> 4) & 1) * N) * (K / 32));
  return o;
}

template <class C, int SM>
__device__ __forceinline__ void load_stage(uint32_t stage, const Operand& A, const GatedOperand& B,
                                           const CopyOffsets& off, int64_t K, int kt, int c) {
  constexpr int kA = C::BM / 8 / C::NCOPY, kB = C::BN / 8 / C::NCOPY;  // slices per copier
#pragma unroll
  for (int i = 0; i < (kA > kB ? kA : kB); ++i) {
    const int q = c + C::NCOPY * i;
    if (i < kA) lds_dma16(A.data, stage + q * 1024, off.data, (int)(8 * C::NCOPY * i * K) + kt * BK);
    if (i < kB) lds_dma16(B.data, stage + C::kOffBData + q * 1024, off.data, (int)(16 * i * K) + kt * BK);
  }
  if constexpr (C::SB == 1) {
#pragma unroll
    for (int i = 0; i < C::kScaleSlicesPerCopier; ++i) {
      const int q = c + C::NCOPY * i, s64 = q >> 1;
      if (q & 1)
        lds_dma4(B.scale, stage + C::kOffBScale + s64 * 256, B.voff_scale, (int)(32 * s64 * (K / 32)) + kt * 4);
      else
        lds_dma4(A.scale, stage + C::kOffAScale + s64 * 256, off.scale, (int)(64 * s64 * (K / 32)) + kt * 4);
    }
  }
}

template <class C, int SM>
__device__ __forceinline__ void load_scale_block(uint32_t sbuf, const Operand& A, const GatedOperand& B,
                                                 const CopyOffsets& off, int64_t K, int blk, int c) {
  constexpr int kSa = C::BM / 64, kSb = C::BN / 64;
#pragma unroll
  for (int i = 0; i < (kSa + kSb + C::NCOPY - 1) / C::NCOPY; ++i) {
    const int q = c + C::NCOPY * i;
    if (q >= kSa + kSb) break;
    const int s64 = q < kSa ? q : q - kSa;
    if (q < kSa)
      lds_dma16(A.scale, sbuf + s64 * 1024, off.scale, (int)(64 * s64 * (K / 32)) + 16 * blk);
    else
      lds_dma16(B.scale, sbuf + C::BM * 16 + s64 * 1024, B.voff_scale, (int)(32 * s64 * (K / 32)) + 16 * blk);
  }
}

// ---- epilogues --------------------------------------------------------------

__device__ __forceinline__ void bf16x4(uint2 v, float (&f)[4]) {
  f[0] = bf16_bits_to_float(v.x & 0xFFFFu);
  f[1] = bf16_bits_to_float(v.x >> 16);
  f[2] = bf16_bits_to_float(v.y & 0xFFFFu);
  f[3] = bf16_bits_to_float(v.y >> 16);
}

__device__ __forceinline__ uint2 pack4(const float (&f)[4]) {
  return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// Forward: fragments 2 p (gate) and 2 p + 1 (up) hold columns n0 + (WTN / 2) wn + 16 p + 4 g + e.
template <class LY, int ACT, int OUT>
__device__ __forceinline__ void epilogue_gated(v4f (&acc)[LY::FRN][LY::FRM], const GatedParams& p,
                                               const uint16_t* bias, int64_t m0, int64_t m_end, int64_t n0, int wave,
                                               int lane) {
  constexpr int NP = LY::FRN / 2;
  const int wm = wave / LY::NWN, wn = wave % LY::NWN;
  const int g = lane >> 4, r = lane & 15;
  const int64_t N = p.N, nw = n0 + wn * (LY::WTN / 2) + 4 * g;
  if (bias != nullptr) {
#pragma unroll
    for (int i = 0; i < LY::FRN; ++i) {
      const int64_t n = nw + 16 * (i >> 1);
      float b[4];
      bf16x4(*reinterpret_cast<const uint2*>(bias + (n < N ? n : 0) + (i & 1) * N), b);
#pragma unroll
      for (int j = 0; j < LY::FRM; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] += b[e];
    }
  }
#pragma unroll
  for (int j = 0; j < LY::FRM; ++j) {
    const int64_t m = m0 + wm * LY::WTM + 16 * j + r;
    const bool row_ok = m < m_end;
    uint2 bits[NP];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int64_t n = nw + 16 * q;
      float ga[4], up[4], v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ga[e] = acc[2 * q][j][e];
        up[e] = acc[2 * q + 1][j][e];
        v[e] = act_value<ACT>(ga[e]) * up[e];
      }
      bits[q] = pack4(v);
      if (row_ok && n < N) {
        if (p.aux != nullptr) {
          *reinterpret_cast<uint2*>(p.aux + m * 2 * N + n) = pack4(ga);
          *reinterpret_cast<uint2*>(p.aux + m * 2 * N + N + n) = pack4(up);
        }
        if constexpr (OUT == TE_BF16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.d) + m * N + n) = bits[q];
      }
    }
    if constexpr (OUT != TE_BF16) {
      // MXFP8: the bf16 values in 32-column blocks, two fragment pairs each; lanes g = 0..3 of a row hold
      // a block's columns 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3
      static_assert(NP % 2 == 0, "a 32-column block is two fragment pairs of one wave");
#pragma unroll
      for (int b = 0; b < NP / 2; ++b) {
        const int64_t nb = n0 + wn * (LY::WTN / 2) + 32 * b;
        const uint4 v = make_uint4(bits[2 * b].x, bits[2 * b].y, bits[2 * b + 1].x, bits[2 * b + 1].y);
        uint32_t amax = absmax_bits8(v);
        amax = max(amax, (uint32_t)__builtin_amdgcn_ds_swizzle((int)amax, 0x401F));           // lane ^ 16
        amax = max(amax, (uint32_t)__builtin_amdgcn_ds_bpermute((lane ^ 32) << 2, (int)amax));  // lane ^ 32
        const uint32_t code = e8m0_code_from_amax_bits<OUT>(amax);
        const uint2 c = cvt8_scaled<OUT>(v, e8m0_to_float(code));
        if (row_ok && nb < p.N) {
          uint8_t* d = static_cast<uint8_t*>(p.d) + m * N + nb + 4 * g;
          *reinterpret_cast<uint32_t*>(d) = c.x;
          *reinterpret_cast<uint32_t*>(d + 16) = c.y;
          if (g == 0) p.d_scale[m * (N / 32) + nb / 32] = (uint8_t)code;
        }
      }
    }
  }
}

template <class LY, int ACT>
__device__ __forceinline__ void epilogue_dgated(v4f (&acc)[LY::FRN][LY::FRM], const GatedParams& p, int64_t m0,
                                                int64_t m_end, int64_t n0, int wave, int lane) {
  const int wm = wave / LY::NWN, wn = wave % LY::NWN;
  const int g = lane >> 4, r = lane & 15;
  const int64_t N = p.N;
#pragma unroll
  for (int j = 0; j < LY::FRM; ++j) {
    const int64_t m = m0 + wm * LY::WTM + 16 * j + r;
    if (m >= m_end) continue;
#pragma unroll
    for (int i = 0; i < LY::FRN; ++i) {
      const int64_t n = n0 + wn * LY::WTN + 16 * i + 4 * g;
      if (n >= N) continue;
      float ga[4], up[4];
      bf16x4(*reinterpret_cast<const uint2*>(p.aux + m * 2 * N + n), ga);
      bf16x4(*reinterpret_cast<const uint2*>(p.aux + m * 2 * N + N + n), up);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v, dv;
        act_and_grad<ACT>(ga[e], v, dv);
        ga[e] = acc[i][j][e] * up[e] * dv;
        up[e] = acc[i][j][e] * v;
      }
      uint16_t* d = static_cast<uint16_t*>(p.d) + m * 2 * N + n;
      *reinterpret_cast<uint2*>(d) = pack4(ga);
      *reinterpret_cast<uint2*>(d + N) = pack4(up);
    }
  }
}

// A tile's accumulators to D (and aux / MXFP8 scales).
template <class LY, bool BWD>
__device__ __forceinline__ void finish_gated(v4f (&acc)[LY::FRN][LY::FRM], const GatedParams& p,
                                             const uint16_t* bias, int64_t m0, int64_t m_end, int64_t n0, int wave,
                                             int lane) {
  auto with_act = [&](auto act) __attribute__((always_inline)) {
    constexpr int ACT = decltype(act)::value;
    if constexpr (BWD) {
      epilogue_dgated<LY, ACT>(acc, p, m0, m_end, n0, wave, lane);
    } else {
      if (p.out == TE_BF16) epilogue_gated<LY, ACT, TE_BF16>(acc, p, bias, m0, m_end, n0, wave, lane);
      else if (p.out == TE_E4M3) epilogue_gated<LY, ACT, TE_E4M3>(acc, p, bias, m0, m_end, n0, wave, lane);
      else epilogue_gated<LY, ACT, TE_E5M2>(acc, p, bias, m0, m_end, n0, wave, lane);
    }
  };
  if (p.act == TE_ACT_SILU) with_act(std::integral_constant<int, TE_ACT_SILU>{});
  else with_act(std::integral_constant<int, TE_ACT_GELU>{});
}

// Output columns of a tile: a forward tile's B rows are gate and up rows of BN / 2 columns.
template <class LY, bool BWD>
constexpr int tile_cols() { return BWD ? LY::BN : LY::BN / 2; }

// One tile: main loop and epilogue.  b / b_scale: this tile's expert's weights.
template <class LY, int FA, int FB, bool BWD>
__device__ __forceinline__ void gated_tile(uint8_t* lds, const GatedParams& p, const uint8_t* b,
                                           const uint8_t* b_scale, const uint16_t* bias, int64_t m0, int64_t m_end,
                                           int64_t n0, int wave, int lane) {
  const Operand A = make_operand(p.a, p.a_scale, m0, m_end - m0, p.K, LY::BM);
  v4f acc[LY::FRN][LY::FRM];
  if constexpr (BWD) {
    const Operand B = make_operand(b, b_scale, n0, p.N - n0, p.K, LY::BN);
    mainloop<LY, FA, FB>(lds, acc, A, B, p.K, wave, lane);
  } else {
    const GatedOperand B = make_gated_operand<LY>(b, b_scale, n0, p.N, p.K, wave, lane);
    mainloop<LY, FA, FB>(lds, acc, A, B, p.K, wave, lane);
  }
  finish_gated<LY, BWD>(acc, p, bias, m0, m_end, n0, wave, lane);
}

template <class LY, int FA, int FB, bool BWD>
__global__ __launch_bounds__(LY::kThreads) void gated_gemm_kernel(GatedParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LY::kLds];
  constexpr int BN = tile_cols<LY, BWD>();
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  raster_tile(blockIdx.x, (int)((p.M + LY::BM - 1) / LY::BM), (int)((p.N + BN - 1) / BN), tm, tn);
  gated_tile<LY, FA, FB, BWD>(lds, p, p.b, p.b_scale, p.bias, (int64_t)tm * LY::BM, p.M, (int64_t)tn * BN, wave, lane);
}

// Grouped: a persistent grid walks the flat list of (expert row-tile, n-tile)
// pairs, built in LDS from the device-resident splits.  Rows behind the last
// group belong to no tile and stay as they were.
template <class LY, int FA, int FB, bool BWD>
__global__ __launch_bounds__(LY::kThreads) void grouped_gated_gemm_kernel(GatedParams p) {
  constexpr int BM = LY::BM, BN = tile_cols<LY, BWD>();
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LY::kLds];
  __shared__ int tile_prefix[kMaxGroups + 1];
  __shared__ int row_off[kMaxGroups + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = p.groups;
  for (int e = threadIdx.x; e < G; e += LY::kThreads) row_off[e + 1] = p.m_splits[e];
  __syncthreads();
  if (threadIdx.x == 0) {
    int tiles = 0, off = 0;
    tile_prefix[0] = 0;
    row_off[0] = 0;
    for (int e = 0; e < G; ++e) {
      const int me = max(row_off[e + 1], 0);
      const int end = (int)min((int64_t)off + me, p.M);  // bad splits stay inside the tensors
      tiles += (end - off + BM - 1) / BM;
      off = end;
      tile_prefix[e + 1] = tiles;
      row_off[e + 1] = off;
    }
  }
  __syncthreads();
  const int ntn = (int)((p.N + BN - 1) / BN);
  const int total = tile_prefix[G] * ntn;
  const int xcd = blockIdx.x % 8, slot = blockIdx.x / 8, nslots = gridDim.x / 8;
  const int chunk = (total + 7) / 8;
  const int t_end = min((xcd + 1) * chunk, total);
  for (int t = xcd * chunk + slot; t < t_end; t += nslots) {
    const int rt = t / ntn, tn = t % ntn;
    int lo = 0, hi = G;  // the expert e with tile_prefix[e] <= rt < tile_prefix[e + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_prefix[mid] <= rt) lo = mid; else hi = mid;
    }
    const int e = __builtin_amdgcn_readfirstlane(lo);
    const int64_t m0 = __builtin_amdgcn_readfirstlane(row_off[e]) +
                       (int64_t)(rt - __builtin_amdgcn_readfirstlane(tile_prefix[e])) * BM;
    const int64_t m_end = __builtin_amdgcn_readfirstlane(row_off[e + 1]);
    const int64_t rows_b = (int64_t)e * p.N * (BWD ? 1 : 2);
    __syncthreads();  // the previous tile's reads of the LDS are done
    gated_tile<LY, FA, FB, BWD>(lds, p, p.b + rows_b * p.K, p.b_scale + rows_b * (p.K / 32),
                                p.bias ? p.bias + rows_b : nullptr, m0, m_end, (int64_t)tn * BN, wave, lane);
  }
}

}  // namespace
}  // namespace temx
