// The gated feed-forward GEMMs on the 4-wave tile (gated_core.h, and mainloop4 in gemm_core.h).
#include "gated_core.h"

namespace temx {
namespace {

// The E8M0 scales rearranged for the 4-wave tile as scale_blocks_kernel does (blocks of 4 K steps, a row's 16
// bytes [32-block][step]), B's rows in the order of its tiles: gate row n at 32 (n / 16) + n % 16, up row n 16
// further on.  Threads [0, rows_a nblk) take A's (row, block) pairs, the rest B's.
__global__ __launch_bounds__(256) void gated_scale_blocks_kernel(const uint8_t* __restrict__ a_in, int64_t rows_a,
                                                                 uint8_t* __restrict__ a_out,
                                                                 const uint8_t* __restrict__ b_in, int64_t n,
                                                                 uint8_t* __restrict__ b_out, int64_t ks) {
  const int64_t nblk = ks / 16;
  int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool is_a = idx < rows_a * nblk;
  if (!is_a) idx -= rows_a * nblk;
  const int64_t rows = is_a ? rows_a : 2 * n;
  if (idx >= rows * nblk) return;
  const int64_t row = idx / nblk, blk = idx - row * nblk;
  const uint4 v = *reinterpret_cast<const uint4*>((is_a ? a_in : b_in) + row * ks + blk * 16);
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};  // d[s]: blocks 0..3 of step s
  uint32_t o[4];
#pragma unroll
  for (int gb = 0; gb < 4; ++gb) {
    o[gb] = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) o[gb] |= ((d[t] >> (8 * gb)) & 0xFFu) << (8 * t);
  }
  const int64_t col = row < n ? row : row - n;
  const int64_t to = is_a ? row : 32 * (col >> 4) + (col & 15) + (row < n ? 0 : 16);
  *reinterpret_cast<uint4*>((is_a ? a_out : b_out) + (blk * rows + to) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
}

// The 4-wave big tile, persistent over its tiles as mx_gemm4_kernel is: the next tile's first copies are issued
// before a tile's epilogue, which stages in stage 1.  p.a_scale / p.b_scale are the rearranged copies.
// Taken where four_wave_mx takes it for a plain GEMM of as many tiles, which loses 4-6% on two of these.  4-wave and
// 8-wave, us, in turn, the best of four rounds on inputs that are not in the caches: forward to MXFP8 8192 x 14336 x
// 4096 731 and 788; forward with aux 4096 x 4096 x 4096 127 and 130, 1024 x 8192 x 4096 69 and 65; backward 4096 x
// 14336 x 4096 247 and 284, 4096 x 4096 x 4096 70 and 80, 8192 x 8192 x 2048 219 and 210.
template <int FA, int FB, bool BWD>
__global__ __launch_bounds__(Big4::kThreads, 1) void gated_gemm4_kernel(GatedParams p) {
  using LY = Big4;
  static_assert(LY::NW * kRegion <= LY::kStage, "the staged epilogue fits in stage 1");
  using OB = std::conditional_t<BWD, Operand, GatedOperand4>;
  constexpr int BN = tile_cols<LY, BWD>();
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LY::kLds];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ntm = (int)((p.M + LY::BM - 1) / LY::BM), ntn = (int)((p.N + BN - 1) / BN);
  const int ntiles = ntm * ntn;
  const int a_blk = (int)(p.M * 16), b_blk = (int)(p.N * (BWD ? 16 : 32));
  auto tile = [&](int v, int64_t& m0, int64_t& n0, Operand& A, OB& B) __attribute__((always_inline)) {
    int tm, tn;
    raster_tile(v, ntm, ntn, tm, tn);
    m0 = (int64_t)tm * LY::BM;
    n0 = (int64_t)tn * BN;
    const int64_t nblk = p.K / 512;
    A = make_operand(p.a, p.a_scale, m0, p.M - m0, p.K, LY::BM);
    A.scale = make_rsrc(p.a_scale + m0 * 16, (nblk * p.M - m0) * 16);
    if constexpr (BWD) {
      B = make_operand(p.b, p.b_scale, n0, p.N - n0, p.K, LY::BN);
      B.scale = make_rsrc(p.b_scale + n0 * 16, (nblk * p.N - n0) * 16);
    } else {
      B = make_gated_operand4(p.b, p.b_scale, n0, p.N, p.K, wave);
    }
  };
  int v = blockIdx.x;
  int64_t m0, n0;
  Operand A;
  OB B;
  tile(v, m0, n0, A, B);
  prologue4<SM_MX>(lds, A, B, p.K, wave, a_blk, b_blk);
  for (;;) {
    v4f acc[LY::FRN][LY::FRM];
    mainloop4<FA, FB, SM_MX, true>(lds, acc, A, B, p.K, wave, a_blk, b_blk);
    DgatedAux<LY> aux;
    if constexpr (BWD) aux.begin(p, m0, p.M, n0, wave, lane_id_fresh());
    const int vn = v + (int)gridDim.x;
    int64_t m0n = 0, n0n = 0;
    Operand An = A;
    OB Bn = B;
    if (vn < ntiles) {
      tile(vn, m0n, n0n, An, Bn);
      prologue4<SM_MX>(lds, An, Bn, p.K, wave, a_blk, b_blk);
    }
    if constexpr (BWD) epilogue_dgated<LY>(acc, lds + LY::kStage, p, aux, m0, p.M, n0, wave, lane_id_fresh());
    else epilogue_gated<LY>(acc, lds + LY::kStage, p, p.bias, m0, p.M, n0, wave, lane_id_fresh());
    if (vn >= ntiles) break;
    v = vn;
    m0 = m0n;
    n0 = n0n;
    A = An;
    B = Bn;
  }
}

template <bool BWD>
te_status launch(const GatedParams& p, te_dtype fa, te_dtype fb, hipStream_t stream) {
  constexpr int BN = tile_cols<Big4, BWD>();
  const int64_t tiles = ((p.M + Big4::BM - 1) / Big4::BM) * ((p.N + BN - 1) / BN);
  // one workgroup per CU (a multiple of 8, so each stays on the XCD its tiles are rastered for)
  const int64_t cap = device_cu_count() / 8 * 8;
  const dim3 grid((unsigned)(cap >= 8 && tiles > cap ? cap : tiles));
  if (fa == TE_E4M3 && fb == TE_E4M3)
    hipLaunchKernelGGL((gated_gemm4_kernel<TE_E4M3, TE_E4M3, BWD>), grid, dim3(Big4::kThreads), 0, stream, p);
  else if (fa == TE_E5M2)
    hipLaunchKernelGGL((gated_gemm4_kernel<TE_E5M2, TE_E4M3, BWD>), grid, dim3(Big4::kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((gated_gemm4_kernel<TE_E4M3, TE_E5M2, BWD>), grid, dim3(Big4::kThreads), 0, stream, p);
  return launch_status();
}

}  // namespace

te_status launch_gated4(GatedParams p, bool backward, te_dtype fa, te_dtype fb, void* workspace, hipStream_t stream) {
  uint8_t* as = static_cast<uint8_t*>(workspace);
  uint8_t* bs = as + scale_blocks_b_offset(p.M, p.K);
  if (backward) {
    const te_status st = launch_scale_blocks(p.a_scale, p.M, as, p.b_scale, p.N, bs, p.K, stream);
    if (st != TE_OK) return st;
  } else {
    const int64_t threads = (p.M + 2 * p.N) * (p.K / 512);
    hipLaunchKernelGGL(gated_scale_blocks_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream,
                       p.a_scale, p.M, as, p.b_scale, p.N, bs, p.K / 32);
    const te_status st = launch_status();
    if (st != TE_OK) return st;
  }
  p.a_scale = as;
  p.b_scale = bs;
  return backward ? launch<true>(p, fa, fb, stream) : launch<false>(p, fa, fb, stream);
}

}  // namespace temx
