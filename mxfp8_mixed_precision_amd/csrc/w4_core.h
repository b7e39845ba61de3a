// GEMMs of few rows with 4-bit weights and group scales, for gfx950.
//
//   P[m, n] = sum_g s[n, g] sum_{k in group g} x[m, k] (q[n, k] - z[n, g])   (+ bias[n])
//   D = P, or act(P[:, :N]) * P[:, N:]
// q are the codes of INT4 (0 .. 15, z the zero point, 8 without one) or E2M1 (z = 0).
//
// A workgroup takes 16 NF rows of W (output columns, or 16 columns' gate and up rows); its waves deal the K steps of
// 128 among themselves and their partial sums meet in LDS, in wave order (deterministic).  Lane 16 q + r loads 16
// bytes of row r, the codes of the step's 32-block q; a 4 x 4 transpose across the lanes gives MFMA i (16 x 16 x 32)
// block i: lane 16 q + r holds codes 8 q .. 8 q + 7 of row r, turned into bf16 / fp16 by exact conversions (a code 0
// .. 15 is the E4M3 code of 2^-9 times itself).  The weights are the MFMA's second operand, so that a lane's results
// are of one weight row, whose scale the lane holds.  Products and sums are fp32; a group's sum is scaled in fp32,
// after its zero point times the sum of x, which another MFMA gives with ones for weights.
//
// The weights' bytes bound one to four rows (w4_few_kernel), with 149 vector instructions for the 2 KB of a step that
// take half of the time themselves; with more rows (w4_ring_kernel) every workgroup's reading of all of x does, the more
// the more rows: a CU takes in ~75 bytes a ns from L2, 917 KB of 32 x 14336 in 12 us.  Loading x and the scales where
// they are used, straight into the MFMA's layout, took 1.5 to 2 times as long: such a load takes 64 bytes of each of 16
// rows, and loads return in order, so that each waits for the weights' ones before it.
// Measured on MI355X, us a kernel, weights from HBM (calls in turn of more than 700 MB, from a graph) and of three calls
// in turn, which the last-level cache holds: one row, N = 14336 gated, K = 4096, groups of 128: 16.1 and 15.6 (61 MB, 3.8
// TB/s; a large copy 5.0); 64 rows over 32 experts, N = 1536, K = 4096: 27.3 and 26.8 (91 MB); 32 rows, N = 4096, K =
// 14336, E2M1 in groups of 32: 23.2 and 18.5 (39 MB of weights and x); 5 rows, N = 1001, K = 2080: 6.1, latencies.
#pragma once

#include "gemm_core.h"
#include "row_chunks.h"

namespace temx {

constexpr int kW4MaxGroups = 1024;  // experts

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
  // set at the launch
  int per_row;            // scales of a weight row
  int blocks_of_group;    // blocks of 32
  uint64_t group_magic;   // ceil(2^40 / blocks_of_group): the quotient of both below 2^19 by a product
  int span;               // steps whose scales a workgroup keeps at a time
};

// One source file each.
te_status launch_w4_bf16_int4(const W4Params& p, hipStream_t stream);
te_status launch_w4_bf16_e2m1(const W4Params& p, hipStream_t stream);
te_status launch_w4_fp16_int4(const W4Params& p, hipStream_t stream);
te_status launch_w4_fp16_e2m1(const W4Params& p, hipStream_t stream);

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// A group is whole steps, one block, or anything else.
enum class W4Groups { Steps, Block, Any };

constexpr int kStep = 128;              // K of a wave's step: 4 blocks of 32
constexpr int kBeyond = 0x60000000;     // an offset past the end of every buffer below (2^30 bytes at most): zeros

template <class T> struct Half;  // the activations' type in the MFMA
// Weights enter in units of 1 / kUnit, and the sums are multiplied by it once, at the end: 128 products of a bf16 value
// and a code or zero point (up to 255 < 2^15 / 128) then stay in range where the values themselves do, and a group's
// sum before its scale and before its zero point's part is taken off cannot overflow.  The price are the last 15 of the
// 149 binary places below 1, sums below 2^-111 that lose some of theirs.  fp16 values are at most 2^16.
template <> struct Half<bf16_t> {
  typedef v8bf v8;
  static constexpr float kUnit = 32768.f;
  static __device__ __forceinline__ v4f mfma(v8 a, v8 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t v) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f / kUnit, HI));
  }
  template <int BYTE>
  static __device__ __forceinline__ uint32_t from_e2m1(uint32_t v) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f / kUnit, BYTE));
  }
  static constexpr uint32_t ones = 0x38003800u;  // 1 / kUnit
};
template <> struct Half<f16_t> {
  typedef v8h v8;
  static constexpr float kUnit = 1.f;
  static __device__ __forceinline__ v4f mfma(v8 a, v8 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
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

__device__ __forceinline__ float e8m0_value(uint32_t code) {
  return code == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_float(code);
}

// Scale i (E8M0, fp32 or T) as a float.
template <class T>
__device__ __forceinline__ float load_scale(const void* p, int64_t i, te_dtype dtype) {
  if (dtype == TE_E8M0) return e8m0_value(static_cast<const uint8_t*>(p)[i]);
  if (dtype == TE_FP32) return static_cast<const float*>(p)[i];
  return to_float(static_cast<const T*>(p)[i]);
}

// x / (1 + e^-x)
__device__ __forceinline__ float silu(float x) {
  return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

// Sum over the wave's lanes of values from 0 to 2^31 - 1: its halves' sums in 32 bits.
__device__ __forceinline__ int64_t wave_sum(int v) {
  const auto add = [](int a, int b) { return a + b; };
  return ((int64_t)lanes_all<64>(v >> 16, add) << 16) + lanes_all<64>(v & 0xFFFF, add);
}

// Every wave's LDS accesses so far have ended, and the barrier: copies and loads stay on their way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// What a workgroup computes: rows t0, t0 + t_step, .. below t_end of x, weight rows from w_row on.
struct W4Job {
  int64_t t0, t_end, t_step, w_row, n0, first0, first1, N;
  bool gated;
  int cols;  // output columns

  __device__ __forceinline__ W4Job(const W4Params& p, int kRows, int RX)
      : t0(0), t_end(p.M), t_step(RX), w_row(0), N(p.N), gated(kRows == 32 && p.act >= 0), cols(gated ? 16 : kRows) {
    n0 = (int64_t)blockIdx.x * cols;
    first0 = min(n0, N - 1);
    first1 = gated ? n0 : min(n0 + 16, N - 1);
    if (p.m_splits != nullptr) {  // this expert's rows and weights
      const int g = blockIdx.y, lane = threadIdx.x & 63;
      for (int e0 = 0; e0 < g; e0 += 64) t0 += wave_sum(e0 + lane < g ? max(p.m_splits[e0 + lane], 0) : 0);
      t_end = min(t0 + max(p.m_splits[g], 0), p.M);
      w_row = (int64_t)g * (gated ? 2 * N : N);
    } else {
      t0 = blockIdx.y * t_step;
      t_step *= gridDim.y;
    }
  }
  __device__ __forceinline__ int64_t first(int f) const { return f == 0 ? first0 : first1; }
  // Weight row i of fragment f, or the last where there is none (its column is not stored).
  __device__ __forceinline__ int64_t weight_row(int f, int i) const {
    return w_row + min(first(f) + i, N - 1) + (gated && f == 1 ? N : 0);
  }
};

__device__ __forceinline__ int w4_group(const W4Params& p, int block) { return (int)((block * p.group_magic) >> 40); }

// COUNT values from p, which has the alignment of its type only.
template <class V, int COUNT>
struct Unaligned {
  V v[COUNT];
};
template <int COUNT, class V>
__device__ __forceinline__ Unaligned<V, COUNT> load_unaligned(const void* p) {
  Unaligned<V, COUNT> r;
  __builtin_memcpy(&r, __builtin_assume_aligned(p, alignof(V)), sizeof(r));
  return r;
}

// The scales and zero points of groups g0 .. g1 - 1 of the workgroup's weight rows to LDS, [group][weight row].
template <class T, bool ZERO, int THREADS, int ROWS>
__device__ __forceinline__ void fill_tables(const W4Params& p, const W4Job& job, int g0, int g1, float* scales,
                                            uint8_t* zeros) {
  constexpr int kShare = THREADS / ROWS, kAtOnce = 8;  // threads of a row; groups of a thread
  const int row = threadIdx.x / kShare;
  const int64_t from = job.weight_row(row >> 4, row & 15) * p.per_row;
  float* out = scales + row - g0 * (ROWS + 1);
#pragma unroll 2
  for (int g = g0 + kAtOnce * (threadIdx.x % kShare); g < g1; g += kAtOnce * kShare) {
    if (g + kAtOnce <= g1) {
      float s[kAtOnce];
      if (p.scale_dtype == TE_E8M0) {
        const auto v = load_unaligned<kAtOnce, uint8_t>(static_cast<const uint8_t*>(p.scale) + from + g);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) s[i] = e8m0_value(v.v[i]);
      } else if (p.scale_dtype == TE_FP32) {
        const auto v = load_unaligned<kAtOnce, float>(static_cast<const float*>(p.scale) + from + g);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) s[i] = v.v[i];
      } else {
        const auto v = load_unaligned<kAtOnce, T>(static_cast<const T*>(p.scale) + from + g);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) s[i] = to_float(v.v[i]);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) out[(g + i) * (ROWS + 1)] = s[i];
      if constexpr (ZERO) {
        Unaligned<uint8_t, kAtOnce> z = {{8, 8, 8, 8, 8, 8, 8, 8}};
        if (p.zero != nullptr) z = load_unaligned<kAtOnce, uint8_t>(p.zero + from + g);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) zeros[(g + i - g0) * ROWS + row] = z.v[i];
      }
    } else {
      for (int i = g; i < g1; ++i) {
        out[i * (ROWS + 1)] = load_scale<T>(p.scale, from + i, p.scale_dtype);
        if constexpr (ZERO) zeros[(i - g0) * ROWS + row] = p.zero != nullptr ? p.zero[from + i] : 8;
      }
    }
  }
}

// A wave's sums: of NF fragments of 16 weight rows and MF fragments of 16 rows of x.  Lane (q, r), element e: row 4 q
// + e of x, weight row r.
template <class T, te_w4_format FMT, int NF, int MF>
struct W4Sums {
  static constexpr bool kInt = FMT == TE_W4_INT4;
  static constexpr int kRows = 16 * NF, kPitch = kRows + 1;  // a group's neighbour lies on other banks: a row's writes
  typedef typename Half<T>::v8 v8;
  v4f total[NF][MF], acc[NF][MF], xsum[MF];

  __device__ __forceinline__ void clear_total() {
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j) total[f][j] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      xsum[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[f][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
  }
  // A block's products, onto acc.
  __device__ __forceinline__ void multiply(const u32x4 (&x)[MF], const uint32_t (&codes)[NF]) {
    constexpr uint32_t one = Half<T>::ones;
#pragma unroll
    for (int j = 0; j < MF; ++j)
      if constexpr (kInt)
        xsum[j] = Half<T>::mfma(__builtin_bit_cast(v8, x[j]), __builtin_bit_cast(v8, u32x4{one, one, one, one}),
                                xsum[j]);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const v8 wf = weights<T, FMT>(codes[f]);
#pragma unroll
      for (int j = 0; j < MF; ++j) acc[f][j] = Half<T>::mfma(__builtin_bit_cast(v8, x[j]), wf, acc[f][j]);
    }
  }
  // acc, scaled by its group's scales (entry `at` of the tables), onto total.
  __device__ __forceinline__ void scale(const float* scales, const uint8_t* zeros, int at) {
    const int r = threadIdx.x & 15;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const float s = scales[at * kPitch + 16 * f + r];
      const float z = kInt ? (float)zeros[at * kRows + 16 * f + r] : 0.f;
#pragma unroll
      for (int j = 0; j < MF; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = kInt ? __builtin_fmaf(-z, xsum[j][e], acc[f][j][e]) : acc[f][j][e];
          total[f][j][e] = __builtin_fmaf(s, a, total[f][j][e]);
        }
    }
  }
  // A step (4 blocks from `block` on): its codes, transposed, and x in LDS, in rows of 256 bytes whose piece c of 16
  // bytes lies at place c ^ (row % 16).
  template <int RX, W4Groups GROUPS>
  __device__ __forceinline__ void step(const W4Params& p, const u32x4 (&codes)[NF], const uint8_t* x_at, int block,
                                       int g0, const float* scales, const uint8_t* zeros) {
    const int q = (threadIdx.x & 63) >> 4, r = threadIdx.x & 15;
    u32x4 x[4][MF];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < MF; ++j) {
        const int m = RX < 16 ? r & (RX - 1) : 16 * j + r;
        x[i][j] = *reinterpret_cast<const u32x4*>(x_at + m * 256 + 16 * ((4 * i + q) ^ (m & 15)));
      }
    int group = GROUPS == W4Groups::Block ? block : w4_group(p, block), left = (group + 1) * p.blocks_of_group - block;
    clear();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) w[f] = codes[f][i];
      multiply(x[i], w);
      if (i == 3 || GROUPS == W4Groups::Block || (GROUPS == W4Groups::Any && --left == 0)) {
        scale(scales, zeros, group - g0);
        if (i < 3) clear();
        ++group;
        left = p.blocks_of_group;
      }
    }
  }
  // The last blocks of a K that is no multiple of a step, one at a time, from memory.
  __device__ __forceinline__ void tail(const W4Params& p, const W4Job& job, int64_t t0, int rows, int g0,
                                       const float* scales, const uint8_t* zeros) {
    const int q = (threadIdx.x & 63) >> 4, r = threadIdx.x & 15;
    for (int block = (int)(p.K / 32) / 4 * 4; block < p.K / 32; ++block) {
      u32x4 x[MF];
      uint32_t w[NF];
#pragma unroll
      for (int j = 0; j < MF; ++j) {
        const int m = min(16 * j + r, rows - 1);
        x[j] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.x) + (t0 + m) * p.K + 32 * block + 8 * q);
      }
#pragma unroll
      for (int f = 0; f < NF; ++f)
        w[f] = *reinterpret_cast<const uint32_t*>(p.w + job.weight_row(f, r) * (p.K / 2) + 16 * block + 4 * q);
      clear();
      multiply(x, w);
      scale(scales, zeros, w4_group(p, block) - g0);
    }
  }
  // The W waves' sums met in LDS (part: [W][NF * MF][256]), the epilogue and the output.  By all waves.
  template <int W>
  __device__ __forceinline__ void finish(const W4Params& p, const W4Job& job, int64_t t0, int rows, float* part) {
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15, wave = threadIdx.x >> 6;
    __syncthreads();
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[(wave * NF * MF + f * MF + j) * 256 + 16 * (4 * q + e) + r] = total[f][j][e];
    __syncthreads();
    for (int o = threadIdx.x; o < rows * job.cols; o += 64 * W) {
      const int c = o & (job.cols - 1), m = o / job.cols;
      const int64_t t = t0 + m, n = job.n0 + c;
      if (n >= p.N) continue;
      const int f = job.gated ? 0 : c >> 4, at = 16 * (m & 15) + (c & 15);
      float v = 0.f, up = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        v += part[(w * NF * MF + f * MF + (m >> 4)) * 256 + at];
        if (job.gated) up += part[(w * NF * MF + (NF - 1) * MF + (m >> 4)) * 256 + at];
      }
      v *= Half<T>::kUnit;
      up *= Half<T>::kUnit;
      if (p.bias != nullptr) {
        v += to_float(static_cast<const T*>(p.bias)[job.w_row + n]);
        if (job.gated) up += to_float(static_cast<const T*>(p.bias)[job.w_row + p.N + n]);
      }
      if (job.gated) v = (p.act == TE_ACT_SILU ? silu(v) : gelu_tanh(v)) * up;
      if (p.d_fp32) static_cast<float*>(p.d)[t * p.N + n] = v;
      else static_cast<T*>(p.d)[t * p.N + n] = from_float<T>(v);
    }
  }
};

// Up to RX = 4 rows at a time: the weights bound them.  x and the scales of a chunk of K lie in LDS, copied by all
// waves; the codes of U steps of a wave are on their way in registers.
template <int W_, int NF_, int RX_, int U_, int CHUNK_ = 32>
struct W4Few {
  static constexpr int W = W_, NF = NF_, RX = RX_, U = U_, kRows = 16 * NF, MF = 1;
  static constexpr bool kFew = true;
  static constexpr int kChunk = CHUNK_;  // steps
  static constexpr int kX = kChunk * RX * 256, kPart = W * NF * 1024, kArena = kX > kPart ? kX : kPart;
  static constexpr int kGroups(W4Groups groups) {  // of a chunk, and the tail's
    return groups == W4Groups::Steps ? kChunk + 1 : 4 * kChunk + 4;
  }
  static_assert(kChunk % (W * U) == 0 && U % 2 == 0 && kChunk * RX % (4 * W) == 0);
};

template <class T, te_w4_format FMT, class C, W4Groups GROUPS>
__global__ __launch_bounds__(64 * C::W) void w4_few_kernel(W4Params p) {
  constexpr bool kInt = FMT == TE_W4_INT4;
  constexpr int W = C::W, NF = C::NF, RX = C::RX, U = C::U;
  __shared__ __attribute__((aligned(16))) uint8_t arena[C::kArena];
  __shared__ float scales[C::kGroups(GROUPS) * (C::kRows + 1)];
  __shared__ uint8_t zeros[kInt ? C::kGroups(GROUPS) * C::kRows : 1];
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const W4Job job(p, C::kRows, RX);
  const int steps = (int)(p.K / kStep), row_bytes = (int)(p.K / 2);
  const uint32_t x_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)arena;

  for (int64_t t0 = job.t0; t0 < job.t_end; t0 += job.t_step) {
    const int rows = (int)min(job.t_end - t0, (int64_t)RX);
    __amdgpu_buffer_rsrc_t rw[NF];
    int vw[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      rw[f] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.w) + job.weight_row(f, 0) * row_bytes, 0,
                                                (int)(min((int64_t)16, p.N - job.first(f)) * row_bytes), kRsrcWord3);
      vw[f] = (int)(job.weight_row(f, r) - job.weight_row(f, 0)) * row_bytes + 16 * q;
    }
    // the wave's step n: pairs (a row's whole 128 bytes), dealt to the waves in turn
    const auto step_of = [&](int n) { return n / 2 * (2 * W) + 2 * wave + n % 2; };
    u32x4 codes[U][NF];
    const auto load = [&](int u, int n) {
      const int step = step_of(n);
#pragma unroll
      for (int f = 0; f < NF; ++f)
        codes[u][f] =
            __builtin_amdgcn_raw_buffer_load_b128(rw[f], vw[f], step < steps ? step * (kStep / 2) : kBeyond, 0);
      __builtin_amdgcn_sched_barrier(0);
    };
    const i32x4 rx = make_rsrc(static_cast<const T*>(p.x) + t0 * p.K, rows * p.K * 2);
    // a chunk's x: a copy moves 1 KB, 4 / RX steps of RX rows
    const auto copy = [&](int s0) {
      constexpr int kPer = 4 / RX;  // steps
#pragma unroll
      for (int i = 0; i < C::kChunk / kPer / W; ++i) {
        const int at = wave + W * i, step = s0 + at * kPer, m = RX == 1 ? 0 : q, s = RX == 1 ? q : 0;
        const int from = m < rows && step + s < steps ? (int)(m * p.K * 2) + s * 256 + 16 * (r ^ m) : kBeyond;
        lds_dma16(rx, x_lds + at * 1024, from, step < steps ? step * (kStep * 2) : kBeyond);
      }
    };

    W4Sums<T, FMT, NF, 1> sums;
    sums.clear_total();
    copy(0);
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, u);
    int g0 = 0;
    for (int s0 = 0; s0 == 0 || s0 < steps; s0 += C::kChunk) {
      const int s1 = min(s0 + C::kChunk, steps);
      g0 = w4_group(p, 4 * s0);
      if (s0 > 0) {
        lds_barrier();
        copy(s0);
      }
      const int g1 = s1 == steps ? p.per_row : w4_group(p, 4 * s1 - 1) + 1;
      fill_tables<T, kInt, 64 * W, C::kRows>(p, job, g0, g1, scales, zeros);
      wait_vmcnt<0>();
      lds_barrier();
#pragma unroll 1
      for (int n0 = 0; n0 < C::kChunk / W; n0 += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int n = s0 / W + n0 + u, step = step_of(n);
          u32x4 now[NF];
#pragma unroll
          for (int f = 0; f < NF; ++f) now[f] = transpose_blocks(codes[u][f]);
          load(u, n + U);
          if (step < s1)
            sums.template step<RX, GROUPS>(p, now, arena + (step - s0) * (RX * 256), 4 * step, g0, scales, zeros);
        }
      }
    }
    if (p.K % kStep != 0 && wave == W - 1) sums.tail(p, job, t0, rows, g0, scales, zeros);
    sums.template finish<W>(p, job, t0, rows, reinterpret_cast<float*>(arena));
    if (t0 + job.t_step < job.t_end) __syncthreads();
  }
}

// Tiles of RX = 16 or 32 rows: what a workgroup reads of x bounds them.  Each wave keeps D steps, x and codes, in LDS
// of its own, D - 1 of them on their way, and waits for nobody.
template <int W_, int NF_, int RX_, int D_>
struct W4Ring {
  static constexpr int W = W_, NF = NF_, RX = RX_, D = D_, kRows = 16 * NF, MF = RX / 16;
  static constexpr bool kFew = false;
  static constexpr int kSlot = RX * 256 + NF * 1024;  // a step's x and codes
  static constexpr int kCopies = kSlot / 1024;        // of 1 KB each, to fill it
  static constexpr int kRing = W * D * kSlot, kPart = W * NF * MF * 1024, kArena = kRing > kPart ? kRing : kPart;
  // The rest of a CU's LDS (of half of it, for two workgroups) holds the scales and zero points of a span of K.
  static constexpr int kGroups(bool zeros) {
    return ((kArena <= 72 * 1024 ? 80 : 160) * 1024 - kArena - 64) / (4 * (kRows + 1) + (zeros ? kRows : 0));
  }
};

template <class T, te_w4_format FMT, class C, W4Groups GROUPS>
__global__ __launch_bounds__(64 * C::W) void w4_ring_kernel(W4Params p) {
  constexpr bool kInt = FMT == TE_W4_INT4;
  constexpr int W = C::W, NF = C::NF, RX = C::RX, D = C::D;
  __shared__ __attribute__((aligned(16))) uint8_t arena[C::kArena];
  __shared__ float scales[C::kGroups(kInt) * (C::kRows + 1)];
  __shared__ uint8_t zeros[kInt ? C::kGroups(kInt) * C::kRows : 1];
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const W4Job job(p, C::kRows, RX);
  const int steps = (int)(p.K / kStep), row_bytes = (int)(p.K / 2);
  const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)arena + wave * (D * C::kSlot);
  const uint8_t* slots = arena + wave * (D * C::kSlot);

  for (int64_t t0 = job.t0; t0 < job.t_end; t0 += job.t_step) {
    const int rows = (int)min(job.t_end - t0, (int64_t)RX);
    i32x4 rw[NF];
    int vw[NF], vx[RX / 4];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      rw[f] = make_rsrc(p.w + job.weight_row(f, 0) * row_bytes, min((int64_t)16, p.N - job.first(f)) * row_bytes);
      vw[f] = (int)(job.weight_row(f, r) - job.weight_row(f, 0)) * row_bytes + 16 * q;
    }
    const i32x4 rx = make_rsrc(static_cast<const T*>(p.x) + t0 * p.K, rows * p.K * 2);
#pragma unroll
    for (int j = 0; j < RX / 4; ++j) {  // copy j: rows 4 j + q of x; zeros past the end
      const int m = 4 * j + q;
      vx[j] = m < rows ? (int)(m * p.K * 2) + 16 * (r ^ (m & 15)) : kBeyond;
    }
    const auto issue = [&](int slot, int step, bool there) {
      const uint32_t to = ring + slot * C::kSlot;
#pragma unroll
      for (int f = 0; f < NF; ++f)
        lds_dma16(rw[f], to + RX * 256 + f * 1024, vw[f], there ? step * (kStep / 2) : kBeyond);
#pragma unroll
      for (int j = 0; j < RX / 4; ++j) lds_dma16(rx, to + j * 1024, vx[j], there ? step * (kStep * 2) : kBeyond);
    };

    W4Sums<T, FMT, NF, C::MF> sums;
    sums.clear_total();
    int g0 = 0;
    for (int s0 = 0; s0 == 0 || s0 < steps; s0 += p.span) {
      const int s1 = min(s0 + p.span, steps);
      // the wave's step n of the span: pairs (a row's whole 128 bytes), dealt to the waves in turn
      const auto step_of = [&](int n) { return s0 + n / 2 * (2 * W) + 2 * wave + n % 2; };
#pragma unroll
      for (int n = 0; n < D - 1; ++n) issue(n, step_of(n), step_of(n) < s1);
      g0 = w4_group(p, 4 * s0);
      if (s0 > 0) lds_barrier();
      const int g1 = s1 == steps ? p.per_row : w4_group(p, 4 * s1 - 1) + 1;
      fill_tables<T, kInt, 64 * W, C::kRows>(p, job, g0, g1, scales, zeros);
      lds_barrier();
      for (int n = 0; step_of(n) < s1; ++n) {
        wait_vmcnt<(D - 2) * C::kCopies>();  // this step's copies; the reads of the slot filled next have ended
        const int ahead = n + D - 1;
        issue(ahead % D, step_of(ahead), step_of(ahead) < s1);
        const uint8_t* slot = slots + n % D * C::kSlot;
        u32x4 codes[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f)
          codes[f] = transpose_blocks(*reinterpret_cast<const u32x4*>(slot + RX * 256 + f * 1024 + lane * 16));
        sums.template step<RX, GROUPS>(p, codes, slot, 4 * step_of(n), g0, scales, zeros);
      }
      wait_vmcnt<0>();
    }
    if (p.K % kStep != 0 && wave == W - 1) sums.tail(p, job, t0, rows, g0, scales, zeros);
    sums.template finish<W>(p, job, t0, rows, reinterpret_cast<float*>(arena));
    if (t0 + job.t_step < job.t_end) __syncthreads();
  }
}

template <class T, te_w4_format FMT, class C>
dim3 w4_grid(const W4Params& p) {
  const int cols = C::NF == 2 && p.act >= 0 ? 16 : C::kRows;
  const int64_t y = p.m_splits != nullptr ? p.groups : std::min<int64_t>((p.M + C::RX - 1) / C::RX, 65535);
  return dim3((unsigned)((p.N + cols - 1) / cols), (unsigned)y);
}

template <class T, te_w4_format FMT, class C, W4Groups GROUPS>
te_status launch_w4(W4Params p, hipStream_t stream) {
  const dim3 grid = w4_grid<T, FMT, C>(p), block(64 * C::W);
  if constexpr (C::kFew) {
    hipLaunchKernelGGL((w4_few_kernel<T, FMT, C, GROUPS>), grid, block, 0, stream, p);
  } else {
    // a span's first and last group may be parts of groups, and the tail's (3 at most) follow the last span's
    const int64_t groups = C::kGroups(FMT == TE_W4_INT4) - 5;
    p.span = (int)std::max<int64_t>(1, std::min<int64_t>(groups * p.blocks_of_group / 4, 1 << 20));
    hipLaunchKernelGGL((w4_ring_kernel<T, FMT, C, GROUPS>), grid, block, 0, stream, p);
  }
  return launch_status();
}

template <class T, te_w4_format FMT, class C>
te_status w4_by_group(const W4Params& p, hipStream_t stream) {
  if (p.group % kStep == 0) return launch_w4<T, FMT, C, W4Groups::Steps>(p, stream);
  if (p.group == 32) return launch_w4<T, FMT, C, W4Groups::Block>(p, stream);
  return launch_w4<T, FMT, C, W4Groups::Any>(p, stream);
}

// Kernels by the rows of a tile and by the tiles of 16 NF weight rows.  Many tiles (3 a CU): small workgroups,
// several on a CU, whose starts and ends overlap; few: as many waves as there are on one tile.  us with the one and
// the other:
//   1 row:  N = 14336 gated, K = 4096 (896 tiles) 2 waves 15.8, 8 waves 23.7;  N = 4096, K = 14336 (256) 22.5 and 12.6
//   3 rows: N = 28672, K = 4096 4 waves 18.3, 8 waves 29.4;  N = 4096, K = 14336 15.4 and 13.9;  N = 8192, K = 4096 (512)
//           8.6 and 9.3, so that 8 waves need a long K;  N = 28672, K = 1024 2 waves 9.3, 4 waves 12.2: a short K
//   16 rows: N = 14336 gated, K = 4096 4 waves and 2 slots 21.4, 8 and 3 32.1;  N = K = 4096 (256) 8.2 and 7.9
//   32 rows: the same N 3 waves 32.0, 7 waves 38.0;  N = 4096, K = 14336 27.9 and 19.5;  64 rows of N = K = 4096 (512 tiles
//           with their two tiles of rows) 13.6 and 17.0
// The chunk of K that x and the scales are copied for: 64 steps where 32 are not all of it, if the joints, where every
// load ends, cost more than the later start.  With 64 and 32 (many tiles: 4 and 2 waves), weights from HBM:
//   1 row, many tiles: N = 28672 gated, K = 8192 58.3 (4.2 TB/s) and 70.5;  N = 16384, K = 16384, E2M1 in groups of 32
//           34.8 and 42.4;  N = 16384, K = 6144 16.0 and 17.6, but K = 4608 14.1 and 13.9, K = 5120 in groups of 32 23.0
//           and 20.7;  N = 14336 gated, K = 4096 21.2 and 17.5
//   1 row, few: N = 4096, K = 14336 11.7 and 13.1, K = 4608 6.4 and 6.9, but K = 4096 5.6 and 5.1
//   3 and 4 rows, few: N = 4096, K = 14336 13.7 and 14.7, N = K = 8192 13.3 and 13.5;  many: N = 28672 gated, K = 8192
//           66.8 and 61.9
// Two fragments a wave where many tiles are left of them (64 rows over 32 experts, N = 1536: 28.0, one fragment
// 28.4).
template <class T, te_w4_format FMT, int NF>
te_status w4_by_rows(const W4Params& p, int64_t rows, int64_t tiles, hipStream_t stream) {
  const int64_t cus = device_cu_count();
  const bool many = tiles >= 3 * cus;
  // a workgroup of the ring kernels has a CU's LDS for itself, or shares it: with tiles of rows beside each other
  const bool ring_many = 2 * tiles * (p.m_splits != nullptr ? 1 : (p.M + 31) / 32) > 3 * cus;
  if (rows <= 1) {
    if (many && p.K >= 6144) return w4_by_group<T, FMT, W4Few<4, NF, 1, 4, 64>>(p, stream);
    if (many) return w4_by_group<T, FMT, W4Few<2, NF, 1, 2>>(p, stream);
    if (p.K > 4096) return w4_by_group<T, FMT, W4Few<8, NF, 1, 2, 64>>(p, stream);
    return w4_by_group<T, FMT, W4Few<8, NF, 1, 2>>(p, stream);
  }
  if (rows <= 4) {
    if (many && p.K <= 2048) return w4_by_group<T, FMT, W4Few<2, NF, 4, 2, 16>>(p, stream);
    if (!many && p.K >= 8192) return w4_by_group<T, FMT, W4Few<8, NF, 4, 2, 64>>(p, stream);
    return w4_by_group<T, FMT, W4Few<4, NF, 4, 2>>(p, stream);
  }
  if (rows <= 16) {
    if (ring_many) return w4_by_group<T, FMT, W4Ring<4, NF, 16, 2>>(p, stream);
    return w4_by_group<T, FMT, W4Ring<8, NF, 16, 3>>(p, stream);
  }
  if (ring_many) return w4_by_group<T, FMT, W4Ring<3, NF, 32, 2>>(p, stream);
  return w4_by_group<T, FMT, W4Ring<7, NF, 32, 2>>(p, stream);
}

template <class T, te_w4_format FMT>
te_status w4_run(W4Params p, hipStream_t stream) {
  p.per_row = (int)(p.K / p.group);
  p.blocks_of_group = p.group / 32;
  p.group_magic = (((uint64_t)1 << 40) + p.blocks_of_group - 1) / p.blocks_of_group;
  const bool grouped = p.m_splits != nullptr;
  // Rows of a tile: all, or those of an expert on average and one more, since the host does not know the splits.  An
  // expert with more is walked in several tiles, and the launch waits for it.  us of an even batch, with a quarter and
  // with half of its rows on one expert, by this rule (tiles of 1 or 4 rows) and in tiles of 16: 64 rows over 64 experts,
  // N = 1536, K = 4096 34.7, 34.9, 51.7 and 44.3, 40.5, 33.9;  N = 512 gated, K = 1024 11.0, 19.6, 32.3 and 15.5, 14.7,
  // 12.7;  64 over 32, N = 1536, K = 4096 28.5, 34.1, 52.1 and 31.0, 30.5, 29.1
  const int64_t rows = grouped ? p.M / p.groups + 1 : p.M, experts = grouped ? std::min<int64_t>(p.groups, p.M) : 1;
  const int64_t tiles = (p.N + 15) / 16 * experts;
  if (p.act >= 0) return w4_by_rows<T, FMT, 2>(p, rows, tiles, stream);
  if (tiles >= 6 * (int64_t)device_cu_count()) return w4_by_rows<T, FMT, 2>(p, rows, tiles / 2, stream);
  return w4_by_rows<T, FMT, 1>(p, rows, tiles, stream);
}

}  // namespace
}  // namespace temx
