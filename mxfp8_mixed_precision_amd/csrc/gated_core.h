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
//
// Bounds and times on MI355X (M x N x K), us a call with its scale
// rearrangement, in a stream of calls whose inputs are not in the caches (a
// profiler's trace, which keeps dispatches apart, gives up to 9% more):
//   forward 8192 x 14336 x 4096 to MXFP8: the main loop's MFMA rate; 753,
//     2.55 PFLOP/s (a plain GEMM of both projections to bf16: 739)
//   forward 4096 x 4096 x 1024 with bias and aux: two rounds of tiles of 8 K
//     steps, and the 100 MB they write; 53 (48 with inputs in the last-level
//     cache; without bias and aux 42, a plain GEMM, 67 MB, 43)
//   backward 4096 x 4096 x 1024: 143 MB of aux, gradients and operands; 41 (35
//     with inputs in the last-level cache)
//   backward 4096 x 14336 x 4096: 248, of them 175 the main loop (1.94 PFLOP/s
//     over all): every CU's tile ends at the same time, so the 470 MB of aux
//     and gradients move in bursts that no MFMA covers
#pragma once

#include "gemm_core.h"

namespace temx {

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

// The 4-wave tile's launch (gated_gemm4.hip), with the scales rearranged into the workspace.
te_status launch_gated4(GatedParams p, bool backward, te_dtype fa, te_dtype fb, void* workspace, hipStream_t stream);

// The launch for at most kFewRows rows (gated_rows.hip): forward, dense.
constexpr int kFewRows = 64;
te_status launch_gated_rows(const GatedParams& p, te_dtype fa, te_dtype fb, hipStream_t stream);

namespace {

// ---- activations ------------------------------------------------------------

// silu(x) = x / (1 + e) with e = 2^(-x log2 e)
__device__ __forceinline__ float silu(float x) {
  return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == TE_ACT_SILU) return silu(x);
  else return gelu_tanh(x);
}

// act(x) = x s and its derivative s + x s (1 - s) w with s = 1 / (1 + e): silu has e = 2^(-x log2 e) and w = 1; GELU
// e = 2^(-2 u log2 e) (u as in gelu_tanh) and w = 2 du/dx.  The product s (1 - s) x w takes x within +-128, where s
// has long been 0 or 1: far gates then give 0 or 1 and never 0 times infinity.  1 - s is rounded to 2^-25 at worst,
// which s (>= 1/2 there) dwarfs.  Two transcendentals in all: one wave per SIMD computes the 4-wave tile's epilogue,
// which took 29 us a tile with the four of dgelu_tanh and takes about 18 with these.
template <int ACT>
__device__ __forceinline__ void act_and_grad(float x, float& v, float& dv) {
  const float c = __builtin_amdgcn_fmed3f(x, -128.0f, 128.0f);
  if constexpr (ACT == TE_ACT_SILU) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
    v = x * s;
    dv = __builtin_fmaf(c * s, 1.0f - s, s);
  } else {
    constexpr float kK = 0.7978845608028654f;                       // sqrt(2/pi)
    constexpr float kC = -2.0f * kK * 1.4426950408889634f;          // -2 sqrt(2/pi) log2(e)
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * (kC + (kC * 0.044715f) * (x * x))));
    v = x * s;
    dv = __builtin_fmaf(c * s * (1.0f - s), 2.0f * kK + (6.0f * kK * 0.044715f) * (c * c), s);
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

template <class C, int SM, bool WAIT>
__device__ __forceinline__ void load_stage(uint32_t stage, const Operand& A, const GatedOperand& B,
                                           const CopyOffsets& off, int64_t K, int kt, int c) {
  constexpr int kA = C::BM / 8 / C::NCOPY, kB = C::BN / 8 / C::NCOPY;  // slices per copier
#pragma unroll
  for (int i = 0; i < (kA > kB ? kA : kB); ++i) {
    const int q = c + C::NCOPY * i;
    if (i < kA) lds_dma16<WAIT>(A.data, stage + q * 1024, off.data, (int)(8 * C::NCOPY * i * K) + kt * BK);
    if (i < kB) lds_dma16<WAIT>(B.data, stage + C::kOffBData + q * 1024, off.data, (int)(16 * i * K) + kt * BK);
  }
  if constexpr (C::SB == 1) {
#pragma unroll
    for (int i = 0; i < C::kScaleSlicesPerCopier; ++i) {
      const int q = c + C::NCOPY * i, s64 = q >> 1;
      if (q & 1)
        lds_dma4<WAIT>(B.scale, stage + C::kOffBScale + s64 * 256, B.voff_scale, (int)(32 * s64 * (K / 32)) + kt * 4);
      else
        lds_dma4<WAIT>(A.scale, stage + C::kOffAScale + s64 * 256, off.scale, (int)(64 * s64 * (K / 32)) + kt * 4);
    }
  }
}

template <class C, int SM, bool WAIT>
__device__ __forceinline__ void load_scale_block(uint32_t sbuf, const Operand& A, const GatedOperand& B,
                                                 const CopyOffsets& off, int64_t K, int blk, int c) {
  constexpr int kSa = C::BM / 64, kSb = C::BN / 64;
#pragma unroll
  for (int i = 0; i < (kSa + kSb + C::NCOPY - 1) / C::NCOPY; ++i) {
    const int q = c + C::NCOPY * i;
    if (q >= kSa + kSb) break;
    const int s64 = q < kSa ? q : q - kSa;
    if (q < kSa)
      lds_dma16<WAIT>(A.scale, sbuf + s64 * 1024, off.scale, (int)(64 * s64 * (K / 32)) + 16 * blk);
    else
      lds_dma16<WAIT>(B.scale, sbuf + C::BM * 16 + s64 * 1024, B.voff_scale, (int)(32 * s64 * (K / 32)) + 16 * blk);
  }
}

// The 4-wave tile's: copy t of wave w is B slice 8 w + t of the tile, rows
// 32 w + 16 (t / 4) + 8 (t & 1) of the gate (t / 2 even) or up part.  The
// lane offsets hold 64 w rows (A's rows), so both resources start 32 w rows
// early; copies 2, 3, 6 and 7, all up, have 2 KB of their LDS slot in the
// immediate, which moves the global address too: that resource starts 2 KB
// earlier still, and the offset takes only the odd copies' 1 KB back.
// No lane's offset falls below what was taken off the base.
struct GatedOperand4 {
  i32x4 data;
  i32x4 up;
  i32x4 scale;  // both parts' rows in tile order (gated_scale_blocks_kernel)
};

__device__ __forceinline__ const i32x4& copy4_b_rsrc(const GatedOperand4& B, int t) { return (t & 2) ? B.up : B.data; }
__device__ __forceinline__ int copy4_b_soff(const GatedOperand4&, int t, int K) {
  return (16 * (t >> 2) + 8 * (t & 1)) * K - (t & 1) * 1024;
}

__device__ __forceinline__ GatedOperand4 make_gated_operand4(const uint8_t* b, const uint8_t* b_scale, int64_t n0,
                                                             int64_t N, int64_t K, int wave) {
  const int64_t bytes = min((int64_t)Big4::BN / 2, N - n0) * K, early = 32 * wave * K, nblk = K / 512;
  GatedOperand4 o;
  o.data = make_rsrc(b + n0 * K - early, bytes + early);
  o.up = make_rsrc(b + (N + n0) * K - early - 2048, bytes + early + 2048);
  o.scale = make_rsrc(b_scale + 2 * n0 * 16, (nblk * 2 * N - 2 * n0) * 16);
  return o;
}

// ---- epilogues --------------------------------------------------------------
//
// Results leave through LDS: a wave writes blocks of 16-row fragments to a
// region of its own in rows of 16-byte chunks (chunk c of row q at
// c ^ (q % chunks), which keeps the 8-byte fragment accesses and the 16-byte
// row accesses free of bank conflicts), reads them back row-major and stores
// whole lines.  Stored straight from the MFMA layout an instruction writes 32
// bytes of each of 16 rows.  A region is 16 KB; LDS accesses of one wave
// complete in order, so a region needs no barrier of its own.
constexpr int kRegion = 16 * 1024;
constexpr int kNonTemporal = 2;  // cache policy of a buffer access
constexpr int kOutOfRange = (int)0x80000000u;  // a buffer offset past every tile's rows (at most 2^31 bytes)

__device__ __forceinline__ void bf16x4(uint2 v, float (&f)[4]) {
  f[0] = bf16_bits_to_float(v.x & 0xFFFFu);
  f[1] = bf16_bits_to_float(v.x >> 16);
  f[2] = bf16_bits_to_float(v.y & 0xFFFFu);
  f[3] = bf16_bits_to_float(v.y >> 16);
}

__device__ __forceinline__ uint2 pack4(const float (&f)[4]) {
  return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// Lane (g, r)'s 8 bytes of fragment column chunk pair `pair` (16 columns = chunks 2 pair, 2 pair + 1) in row
// 16 jj + r of a region with CH chunks per row.
template <int CH>
__device__ __forceinline__ int frag_off(int jj, int pair, int g, int r) {
  const int q = 16 * jj + r, chunk = 2 * pair + (g >> 1);
  return q * CH * 16 + ((chunk ^ (q & (CH - 1))) << 4) + ((g & 1) << 3);
}

// Rows mb .. mb + rows - 1 (below m_end) of a row-major tensor as a buffer resource: accesses past them are
// dropped or read zeros.  `off` is a lane's offset: row lane / CH and 16-byte chunk lane % CH of a region's rows
// (UNIT bytes of the tensor per chunk; in TWO-part rows the second CH / 2 chunks lie `half` bytes further on), out
// of range where its columns are not below N.
struct RowBuffer {
  __amdgpu_buffer_rsrc_t rsrc;
  int off;
  int stride;  // bytes
};

template <int CH, int UNIT, bool TWO>
__device__ __forceinline__ RowBuffer row_buffer(const void* t, int64_t stride, int64_t half, int64_t mb, int64_t m_end,
                                                int rows, int64_t nb, int64_t N, int lane) {
  constexpr int CC = TWO ? CH / 2 : CH;
  const int64_t valid = m_end - mb < 0 ? 0 : (m_end - mb < rows ? m_end - mb : rows);
  const uint64_t base = reinterpret_cast<uint64_t>(t) + mb * stride;
  const uint64_t uniform = (uint64_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)base) & 0xFFFFFFFFu;
  const uint64_t upper = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(base >> 32)) << 32;
  RowBuffer r;
  r.rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(upper | uniform), 0,
                                             __builtin_amdgcn_readfirstlane((int)(valid * stride)), kRsrcWord3);
  const int c = lane % CH;
  const int64_t n = nb + 8 * (c % CC);  // N % 16 == 0: a chunk's 8 columns are all in or all out
  r.off = n < N ? (int)((lane / CH) * stride + (n / 8) * UNIT + (TWO && c >= CC ? half : 0)) : kOutOfRange;
  r.stride = (int)stride;
  return r;
}

// 16 bytes to row `row` of a buffer.  The row goes into the lane's offset and not into the scalar one: with a scalar
// offset the compiler takes a wide store's data registers as free for the next VALU instruction, and on gfx950 such a
// write has reached the stored data (first dword, every other 8 lanes).
template <int POLICY>
__device__ __forceinline__ void store16(const RowBuffer& to, u32x4 v, int row) {
  __builtin_amdgcn_raw_buffer_store_b128(v, to.rsrc, to.off + row * to.stride, 0, POLICY);
}

template <int CH>
__device__ __forceinline__ int region_off(int t, int lane) {
  const int q = (64 * t + lane) / CH, c = lane % CH;
  return q * CH * 16 + ((c ^ (q & (CH - 1))) << 4);
}

// ROWS rows x CH chunks of a region to the buffer's rows row0 ..
template <int CH, int ROWS, int POLICY = 0>
__device__ __forceinline__ void store_rows(const uint8_t* region, const RowBuffer& to, int row0, int lane) {
#pragma unroll
  for (int t = 0; t < ROWS * CH / 64; ++t) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(region + region_off<CH>(t, lane));
    store16<POLICY>(to, v, row0 + t * (64 / CH));
  }
}

// The same region of bf16 values as MXFP8 codes and scales (the buffers' chunks are 8 codes; scales: one byte for
// every 4 chunks): the four lanes of a DPP quad read a row's 32-block.
template <int CH, int ROWS, int FMT>
__device__ __forceinline__ void store_rows_mx(const uint8_t* region, const RowBuffer& to, const RowBuffer& scales,
                                              int row0, int lane) {
#pragma unroll
  for (int t = 0; t < ROWS * CH / 64; ++t) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(region + region_off<CH>(t, lane));
    const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
    const uint32_t code = e8m0_code_from_amax_bits<FMT>(quad_max(absmax_bits8(v)));
    const uint2 x = cvt8_scaled<FMT>(v, e8m0_to_float(code));
    const int row = row0 + t * (64 / CH);
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{x.x, x.y}, to.rsrc, to.off, row * to.stride, 0);
    if ((lane & 3) == 0)
      __builtin_amdgcn_raw_buffer_store_b8((uint8_t)code, scales.rsrc, scales.off, row * scales.stride, 0);
  }
}

// AGPR accumulators (the 4-wave tile) are read fragment by fragment: the empty asm statement keeps the compiler
// from pulling all 256 into VGPRs at once.
template <class LY>
constexpr bool in_agprs() { return LY::FRN * LY::FRM > 32; }

// Forward: fragments 2 p (gate) and 2 p + 1 (up) hold columns n0 + (WTN / 2) wn + 16 p + 4 g + e.
template <class LY>
__device__ __forceinline__ void epilogue_gated(v4f (&acc)[LY::FRN][LY::FRM], uint8_t* lds, const GatedParams& p,
                                               const uint16_t* bias, int64_t m0, int64_t m_end, int64_t n0, int wave,
                                               int lane) {
  constexpr int NP = LY::FRN / 2, CW = LY::WTN / 2, CHD = CW / 8, FRH = 4, ROWS = 16 * FRH;
  static_assert(ROWS * CHD * 2 * 16 <= kRegion && LY::FRM % FRH == 0 && (CHD & (CHD - 1)) == 0, "staging layout");
  const int wm = wave / LY::NWN, wn = wave % LY::NWN;
  const int g = lane >> 4, r = lane & 15;
  const int64_t N = p.N, mw = m0 + wm * LY::WTM, nw = n0 + wn * CW;
  uint8_t* region = lds + wave * (ROWS * CHD * 2 * 16);
  // the bias goes in place where the accumulators are VGPRs; AGPR ones take it as they are read
  float bv[in_agprs<LY>() ? LY::FRN : 1][4];
#pragma unroll
  for (int i = 0; i < LY::FRN; ++i) {
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (bias != nullptr) {
      const int64_t n = nw + 16 * (i >> 1) + 4 * g;  // columns past N (never stored) read column 0's
      bf16x4(*reinterpret_cast<const uint2*>(bias + (n < N ? n : 0) + (i & 1) * N), b);
    }
    if constexpr (in_agprs<LY>()) {
#pragma unroll
      for (int e = 0; e < 4; ++e) bv[i][e] = b[e];
    } else if (bias != nullptr) {
#pragma unroll
      for (int j = 0; j < LY::FRM; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] += b[e];
    }
  }
  auto read = [&](int i, int j, float (&f)[4]) __attribute__((always_inline)) {
    if constexpr (in_agprs<LY>()) asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = acc[i][j][e];
      if constexpr (in_agprs<LY>()) f[e] += bv[i][e];
    }
  };
  const bool mx = p.out != TE_BF16;
  const RowBuffer to_d = mx ? row_buffer<CHD, 8, false>(p.d, N, 0, mw, m_end, LY::WTM, nw, N, lane)
                            : row_buffer<CHD, 16, false>(p.d, 2 * N, 0, mw, m_end, LY::WTM, nw, N, lane);
  __syncthreads();  // every wave's reads of the last stage are done: the LDS is free
#pragma unroll
  for (int h = 0; h < LY::FRM / FRH; ++h) {
    if (p.aux != nullptr) {
#pragma unroll
      for (int jj = 0; jj < FRH; ++jj)
#pragma unroll
        for (int i = 0; i < LY::FRN; ++i) {
          float f[4];
          read(i, FRH * h + jj, f);
          *reinterpret_cast<uint2*>(region + frag_off<2 * CHD>(jj, (i >> 1) + (i & 1) * NP, g, r)) = pack4(f);
        }
      asm volatile("" ::: "memory");
      store_rows<2 * CHD, ROWS>(
          region, row_buffer<2 * CHD, 16, true>(p.aux, 4 * N, 2 * N, mw, m_end, LY::WTM, nw, N, lane), ROWS * h, lane);
      asm volatile("" ::: "memory");
    }
    auto product = [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int jj = 0; jj < FRH; ++jj)
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          float ga[4], up[4];
          read(2 * q, FRH * h + jj, ga);
          read(2 * q + 1, FRH * h + jj, up);
#pragma unroll
          for (int e = 0; e < 4; ++e) ga[e] = act_value<decltype(act)::value>(ga[e]) * up[e];
          *reinterpret_cast<uint2*>(region + frag_off<CHD>(jj, q, g, r)) = pack4(ga);
        }
    };
    if (p.act == TE_ACT_SILU) product(std::integral_constant<int, TE_ACT_SILU>{});
    else product(std::integral_constant<int, TE_ACT_GELU>{});
    asm volatile("" ::: "memory");
    if (!mx) {
      store_rows<CHD, ROWS>(region, to_d, ROWS * h, lane);
    } else {
      // a chunk's scale byte: (n / 32) bytes into its row, so n / 8 chunks of 1 / 4 byte
      RowBuffer scales = row_buffer<CHD, 4, false>(p.d_scale, N / 32, 0, mw, m_end, LY::WTM, nw, N, lane);
      if (scales.off != kOutOfRange)
        scales.off = (lane / CHD) * scales.stride + (int)((nw + 8 * (lane % CHD)) / 32);
      if (p.out == TE_E4M3) store_rows_mx<CHD, ROWS, TE_E4M3>(region, to_d, scales, ROWS * h, lane);
      else store_rows_mx<CHD, ROWS, TE_E5M2>(region, to_d, scales, ROWS * h, lane);
    }
    asm volatile("" ::: "memory");
  }
}

// Backward: fragment i holds columns n0 + WTN wn + 16 i + 4 g + e of acc.  Blocks of 16 rows of aux come through
// the wave's region the same way the gradients leave (row = gate chunks, then up chunks), a block's loads in flight
// while the one before is computed, the first's from before the epilogue (begin).
template <class LY>
struct DgatedAux {
  static constexpr int CH = LY::WTN / 4, ROWS = 16, kT = ROWS * CH / 64;  // 16-byte accesses per lane and block
  static constexpr int kPolicy = in_agprs<LY>() ? kNonTemporal : 0;
  static_assert((CH & (CH - 1)) == 0, "staging layout");
  RowBuffer from;
  u32x4 v[kT];

  __device__ __forceinline__ void load(int h) {
#pragma unroll
    for (int t = 0; t < kT; ++t)
      v[t] = __builtin_amdgcn_raw_buffer_load_b128(from.rsrc, from.off, (ROWS * h + t * (64 / CH)) * from.stride,
                                                   kPolicy);
  }
  __device__ __forceinline__ void begin(const GatedParams& p, int64_t m0, int64_t m_end, int64_t n0, int wave,
                                        int lane) {
    const int64_t mw = m0 + wave / LY::NWN * LY::WTM, nw = n0 + wave % LY::NWN * LY::WTN;
    from = row_buffer<CH, 16, true>(p.aux, 4 * p.N, 2 * p.N, mw, m_end, LY::WTM, nw, p.N, lane);
    load(0);
  }
};

template <class LY>
__device__ __forceinline__ void epilogue_dgated(v4f (&acc)[LY::FRN][LY::FRM], uint8_t* lds, const GatedParams& p,
                                                DgatedAux<LY>& aux, int64_t m0, int64_t m_end, int64_t n0, int wave,
                                                int lane) {
  using X = DgatedAux<LY>;
  constexpr int CH = X::CH;
  const int g = lane >> 4, r = lane & 15;
  const int64_t N = p.N, mw = m0 + wave / LY::NWN * LY::WTM, nw = n0 + wave % LY::NWN * LY::WTN;
  uint8_t* region = lds + wave * (X::ROWS * CH * 16);
  const RowBuffer to = row_buffer<CH, 16, true>(p.d, 4 * N, 2 * N, mw, m_end, LY::WTM, nw, N, lane);
  __syncthreads();  // every wave's reads of the last stage are done: the LDS is free
#pragma unroll
  for (int h = 0; h < LY::FRM; ++h) {
#pragma unroll
    for (int t = 0; t < X::kT; ++t) *reinterpret_cast<u32x4*>(region + region_off<CH>(t, lane)) = aux.v[t];
    if (h + 1 < LY::FRM) aux.load(h + 1);
    asm volatile("" ::: "memory");
    auto gradients = [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < LY::FRN; ++i) {
        if constexpr (in_agprs<LY>()) asm volatile("" : "+a"(acc[i][h]));
        uint2* pg = reinterpret_cast<uint2*>(region + frag_off<CH>(0, i, g, r));
        uint2* pu = reinterpret_cast<uint2*>(region + frag_off<CH>(0, LY::FRN + i, g, r));
        float ga[4], up[4];
        bf16x4(*pg, ga);
        bf16x4(*pu, up);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = acc[i][h][e];
          float f, df;
          act_and_grad<decltype(act)::value>(ga[e], f, df);
          ga[e] = a * up[e] * df;
          up[e] = a * f;
        }
        *pg = pack4(ga);
        *pu = pack4(up);
      }
    };
    if (p.act == TE_ACT_SILU) gradients(std::integral_constant<int, TE_ACT_SILU>{});
    else gradients(std::integral_constant<int, TE_ACT_GELU>{});
    asm volatile("" ::: "memory");
    store_rows<CH, X::ROWS, kNonTemporal>(region, to, X::ROWS * h, lane);
    asm volatile("" ::: "memory");
  }
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
    mainloop<LY, FA, FB, SM_MX, true>(lds, acc, A, B, p.K, wave, lane);
  } else {
    const GatedOperand B = make_gated_operand<LY>(b, b_scale, n0, p.N, p.K, wave, lane);
    mainloop<LY, FA, FB, SM_MX, true>(lds, acc, A, B, p.K, wave, lane);
  }
  if constexpr (BWD) {
    DgatedAux<LY> aux;
    aux.begin(p, m0, m_end, n0, wave, lane);
    epilogue_dgated<LY>(acc, lds, p, aux, m0, m_end, n0, wave, lane);
  } else {
    epilogue_gated<LY>(acc, lds, p, bias, m0, m_end, n0, wave, lane);
  }
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

// Grouped: a persistent grid walks the flat list of (expert row-tile, n-tile) pairs, built in LDS from the
// device-resident splits.  Rows behind the last group belong to no tile and stay as they were.
// A tail tile (TailTile) holds an expert's last rows where at most half of a big tile's are left: half the MFMAs
// and three quarters of the copies.  Where all experts' weights fit the 256 MB MALL, an XCD's whole tiles come first
// and its tails last, which evens the last round out; larger weights would be fetched from HBM for each, so there a
// tail follows its expert's whole tiles and runs beside them.  Measured, us, forward / backward (without tail tiles;
// tails last; tails next to their expert's):
//   16 ragged experts, 8192 rows, N = K = 2048      105 / 88   100 / 78   107 / 89   (weights 134 / 67 MB)
//   8 experts of 600 rows, N = 4096, K = 1024        62 / 65    61 / 58    61 / 58   (67 / 34 MB)
//   32 experts of 290 rows, N = 1536, K = 4096      187 / 141  201 / 132  174 / 142  (403 / 201 MB)
//   16 experts of 40..800 rows, N = K = 4096        354 / 203  355 / 213  343 / 190  (537 / 268 MB)
template <class LY>
struct TailTile {
  static constexpr bool kHas = false;
  using type = LY;
};
template <>
struct TailTile<Big> {
  static constexpr bool kHas = true;
  using type = Cfg<128, 256, 2, 4, 4, 2, 4>;
};

// a + b, at most `most`, of values in [0, most]: associative, so a scan of it is the clamped sum.
__device__ __forceinline__ int capped_sum(int a, int b, int most) {
  return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)most);
}

// Lane l: the capped sum of lanes 0 .. l.  (One thread adding the experts up took 73 ns for each.)
__device__ __forceinline__ int lanes_scan(int v, int most, int l) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __builtin_amdgcn_ds_bpermute((l - d) << 2, v);
    if (l >= d) v = capped_sum(u, v, most);
  }
  return v;
}

template <class LY, int FA, int FB, bool BWD>
__global__ __launch_bounds__(LY::kThreads) void grouped_gated_gemm_kernel(GatedParams p) {
  using Tail = typename TailTile<LY>::type;
  constexpr bool kTails = TailTile<LY>::kHas;
  constexpr int BM = LY::BM, BN = tile_cols<LY, BWD>();
  static_assert(Tail::kLds <= LY::kLds && Tail::kThreads == LY::kThreads && tile_cols<Tail, BWD>() == BN, "tail tile");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LY::kLds];
  __shared__ int prefix[kTails ? 2 : 1][kMaxGroups + 1];  // whole tiles, tail tiles of the experts before e
  __shared__ int row_off[kMaxGroups + 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = p.groups;
  if (wave == 0) {  // 64 experts at a time, the sums before them in every lane
    const int l = threadIdx.x, most = (int)p.M;
    int rows_before = 0, whole_before = 0, tails_before = 0;
    if (l == 0) {
      row_off[0] = prefix[0][0] = 0;
      if constexpr (kTails) prefix[1][0] = 0;
    }
    for (int e0 = 0; e0 < G; e0 += 64) {
      const int e = e0 + l;
      const int split = e < G ? min(max(p.m_splits[e], 0), most) : 0;
      const int end = capped_sum(rows_before, lanes_scan(split, most, l), most);  // bad splits stay inside the tensors
      const int lower = __builtin_amdgcn_ds_bpermute((l - 1) << 2, end), rows = end - (l == 0 ? rows_before : lower);
      const int left = rows % BM;
      const bool tail = kTails && left > 0 && left <= Tail::BM;
      const int whole = whole_before + lanes_scan(rows / BM + (left > 0 && !tail ? 1 : 0), most, l);
      const int tails = kTails ? tails_before + lanes_scan(tail ? 1 : 0, most, l) : 0;
      if (e < G) {
        row_off[e + 1] = end;
        prefix[0][e + 1] = whole;
        if constexpr (kTails) prefix[1][e + 1] = tails;
      }
      rows_before = __builtin_amdgcn_readlane(end, 63);
      whole_before = __builtin_amdgcn_readlane(whole, 63);
      tails_before = __builtin_amdgcn_readlane(tails, 63);
    }
  }
  __syncthreads();
  const int ntn = (int)((p.N + BN - 1) / BN);
  const int xcd = blockIdx.x % 8, nslots = gridDim.x / 8;
  // the XCD's share of `tiles` row tiles: items [from, from + n)
  struct Share {
    int from, n;
  };
  auto share = [&](int tiles) __attribute__((always_inline)) {
    const int total = __builtin_amdgcn_readfirstlane(tiles) * ntn, chunk = (total + 7) / 8;
    return Share{xcd * chunk, max(min(chunk, total - xcd * chunk), 0)};
  };
  const bool apart = kTails && (BWD ? 1 : 2) * (int64_t)G * p.N * p.K < (int64_t)256 << 20;
  const int tails = kTails ? prefix[1][G] : 0;
  const Share first = share(prefix[0][G] + (apart ? 0 : tails)), second = apart ? share(tails) : Share{0, 0};
  for (int i = blockIdx.x / 8; i < first.n + second.n; i += nslots) {
    const bool behind = i >= first.n;
    const int item = behind ? second.from + i - first.n : first.from + i;
    const int rt = item / ntn, tn = item % ntn;
    auto before = [&](int e) __attribute__((always_inline)) {  // the list's row tiles of the experts before e
      if constexpr (!kTails) return prefix[0][e];
      else return apart ? prefix[behind][e] : prefix[0][e] + prefix[1][e];
    };
    int lo = 0, hi = G;  // the expert e with before(e) <= rt < before(e + 1)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before(mid) <= rt) lo = mid; else hi = mid;
    }
    const int e = __builtin_amdgcn_readfirstlane(lo);
    const int whole = __builtin_amdgcn_readfirstlane(prefix[0][e + 1] - prefix[0][e]);
    const int at = behind ? whole : __builtin_amdgcn_readfirstlane(rt - before(e));  // a tail follows the whole tiles
    const int64_t m0 = __builtin_amdgcn_readfirstlane(row_off[e]) + (int64_t)at * BM;
    const int64_t m_end = __builtin_amdgcn_readfirstlane(row_off[e + 1]);
    const int64_t n0 = (int64_t)tn * BN, rows_b = (int64_t)e * p.N * (BWD ? 1 : 2);
    const uint8_t* b = p.b + rows_b * p.K;
    const uint8_t* b_scale = p.b_scale + rows_b * (p.K / 32);
    const uint16_t* bias = p.bias ? p.bias + rows_b : nullptr;
    const int lane = lane_id_fresh();  // so that no tile's lane offsets are kept live through the other's
    __syncthreads();  // the previous tile's reads of the LDS are done
    if (kTails && at == whole) gated_tile<Tail, FA, FB, BWD>(lds, p, b, b_scale, bias, m0, m_end, n0, wave, lane);
    else gated_tile<LY, FA, FB, BWD>(lds, p, b, b_scale, bias, m0, m_end, n0, wave, lane);
  }
}

}  // namespace
}  // namespace temx
