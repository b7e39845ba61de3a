// Layer norm and RMS norm, forward and backward, for gfx950.
//
//   s    = x + residual (rounded to the tensors' type), or x
//   mean = sum s / n (RMS norm: 0), var = sum (s - mean)^2 / n, rstd = 1 / sqrt(var + eps)
//   y    = (s - mean) rstd gamma + beta
// and, with xh = (x - mean) rstd and g = dy gamma,
//   dx     = rstd (g - sum g / n [layer norm] - xh sum(g xh) / n) + dskip
//   dgamma = sum over rows of dy xh,   dbeta = sum over rows of dy.
//
// All statistics, products and sums are fp32; each output is rounded once.
// The passes do ~10 operations per element: HBM bandwidth bounds them.
#include "temx_device.h"

namespace temx {
namespace {

// ---- element types ----------------------------------------------------------

struct bf16_t {
  uint16_t bits;
};
typedef _Float16 f16_t;

__device__ __forceinline__ float to_float(bf16_t v) { return bf16_bits_to_float(v.bits); }
__device__ __forceinline__ float to_float(f16_t v) { return (float)v; }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ bf16_t from_float<bf16_t>(float v) {
  return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)v)};
}
template <>
__device__ __forceinline__ f16_t from_float<f16_t>(float v) { return (f16_t)v; }
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }

// Rows are cut into chunks of 8 elements from their own start, so a row of any
// length is whole chunks and one tail.  A whole chunk moves as 16-byte
// accesses whose address has the element's alignment only (an odd row length
// leaves rows unaligned; the hardware takes such addresses).
constexpr int kChunk = 8;

template <class T>
struct Raw {
  uint32_t w[sizeof(T) * kChunk / 4];
};

template <int ALIGN>
struct Vec16;
template <>
struct Vec16<2> {
  typedef u32x4 type __attribute__((aligned(2)));
};
template <>
struct Vec16<4> {
  typedef u32x4 type __attribute__((aligned(4)));
};

// n: the chunk's valid elements (>= kChunk: all); elements past them read as 0
template <class T>
__device__ __forceinline__ Raw<T> load_chunk(const T* p, int n) {
  Raw<T> r;
  constexpr int kV = sizeof(T) * kChunk / 16;
  if (n >= kChunk) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const u32x4 v = reinterpret_cast<const typename Vec16<sizeof(T)>::type*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) r.w[4 * i + e] = v[e];
    }
  } else {
    T t[kChunk];
#pragma unroll
    for (int e = 0; e < kChunk; ++e) t[e] = e < n ? p[e] : from_float<T>(0.f);
    r = __builtin_bit_cast(Raw<T>, t);
  }
  return r;
}

template <class T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&f)[kChunk]) {
#pragma unroll
  for (int e = 0; e < kChunk; ++e) {
    if constexpr (sizeof(T) == 4) {
      f[e] = __uint_as_float(r.w[e]);
    } else {
      const uint16_t h = (uint16_t)(r.w[e / 2] >> (16 * (e & 1)));
      f[e] = to_float(__builtin_bit_cast(T, h));
    }
  }
}

template <class T>
__device__ __forceinline__ Raw<T> pack(const float (&f)[kChunk]) {
  Raw<T> r;
#pragma unroll
  for (int e = 0; e < kChunk; ++e) {
    if constexpr (sizeof(T) == 4) {
      r.w[e] = __float_as_uint(f[e]);
    } else if (e & 1) {
      if constexpr (__is_same(T, bf16_t)) r.w[e / 2] = pack_bf16x2(f[e - 1], f[e]);
      else r.w[e / 2] = pack_f16x2(f[e - 1], f[e]);
    }
  }
  return r;
}

template <class T>
__device__ __forceinline__ void store_chunk(T* p, const Raw<T>& r, int n) {
  constexpr int kV = sizeof(T) * kChunk / 16;
  if (n >= kChunk) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      reinterpret_cast<typename Vec16<sizeof(T)>::type*>(p)[i] = u32x4{r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
  } else {
    float f[kChunk];
    unpack<T>(r, f);
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (e < n) p[e] = from_float<T>(f[e]);
  }
}

template <class T>
__device__ __forceinline__ void load_floats(const T* p, int n, float (&f)[kChunk]) {
  unpack<T>(load_chunk(p, n), f);
}

// ---- block sums -------------------------------------------------------------

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Sum over the workgroup, the same bits in every thread; `slots` holds one float per wave and is free
// again once every thread has returned from the next call or barrier.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* slots) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) s += slots[w];
  return s;
}

// ---- forward ----------------------------------------------------------------

struct NormFwd {
  const void* x;
  const void* residual;
  const void* gamma;
  const void* beta;
  void* sum;
  void* y;
  uint8_t* q;
  uint8_t* q_scale;
  float* mean;
  float* rstd;
  int64_t rows;
  int cols;
  float eps;
  bool layer;
  bool q_e5m2;
};

// The MXFP8 codes of a chunk (8 of a 32-block's elements, the 4 lanes of a DPP quad holding the block):
// the values rounded to bf16, quantized as the rowwise quantize kernel does.
__device__ __forceinline__ void store_mx(const Raw<bf16_t>& r, uint8_t* q, uint8_t* q_scale, int64_t at, bool ok,
                                         bool e5m2) {
  const uint4 bits = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  const uint32_t amax = quad_max(ok ? absmax_bits8(bits) : 0u);
  const uint32_t code = e5m2 ? e8m0_code_from_amax_bits<TE_E5M2>(amax) : e8m0_code_from_amax_bits<TE_E4M3>(amax);
  const float scale = e8m0_to_float(code);
  const uint2 c = e5m2 ? cvt8_scaled<TE_E5M2>(bits, scale) : cvt8_scaled<TE_E4M3>(bits, scale);
  if (ok) {
    *reinterpret_cast<uint2*>(q + at) = c;
    if ((at & 31) == 0) q_scale[at >> 5] = (uint8_t)code;
  }
}

constexpr int kWideThreads = 1024;

// One workgroup per row, the row read again for each of mean, variance and output: rows of any length.
template <class T, class W>
__global__ __launch_bounds__(kWideThreads) void norm_fwd_wide_kernel(NormFwd p) {
  __shared__ float slots[kWideThreads / 64];
  const int n = p.cols, nch = (n + kChunk - 1) / kChunk;
  const int64_t row = blockIdx.x, at = row * n;
  const T* x = static_cast<const T*>(p.x) + at;
  float mean = 0.f;
  if (p.layer || p.residual) {
    float s = 0.f;
    for (int c = threadIdx.x; c < nch; c += kWideThreads) {
      float f[kChunk];
      load_floats(x + c * kChunk, n - c * kChunk, f);
      if (p.residual) {
        float r[kChunk];
        load_floats(static_cast<const T*>(p.residual) + at + c * kChunk, n - c * kChunk, r);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) f[e] += r[e];
        const Raw<T> raw = pack<T>(f);
        store_chunk(static_cast<T*>(p.sum) + at + c * kChunk, raw, n - c * kChunk);
        unpack<T>(raw, f);
      }
#pragma unroll
      for (int e = 0; e < kChunk; ++e) s += f[e];
    }
    if (p.layer) mean = block_sum<kWideThreads>(s, slots) / (float)n;
  }
  if (p.residual) x = static_cast<const T*>(p.sum) + at;  // each thread reads back what it wrote
  float v = 0.f;
  for (int c = threadIdx.x; c < nch; c += kWideThreads) {
    float f[kChunk];
    load_floats(x + c * kChunk, n - c * kChunk, f);
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (c * kChunk + e < n) v += (f[e] - mean) * (f[e] - mean);
  }
  const float rstd = 1.0f / sqrtf(block_sum<kWideThreads>(v, slots) / (float)n + p.eps);
  // every lane of a wave takes part in the MXFP8 block maxima: the loop runs whole waves
  for (int c0 = 0; c0 < nch; c0 += kWideThreads) {
    const int c = c0 + threadIdx.x, left = n - c * kChunk;
    const bool ok = c < nch;
    float f[kChunk], g[kChunk], b[kChunk];
    if (ok) {
      load_floats(x + c * kChunk, left, f);
      load_floats(static_cast<const W*>(p.gamma) + c * kChunk, left, g);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[e] = (f[e] - mean) * rstd * g[e];
      if (p.beta) {
        load_floats(static_cast<const W*>(p.beta) + c * kChunk, left, b);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) f[e] += b[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[e] = 0.f;
    }
    const Raw<T> raw = pack<T>(f);
    if (p.y && ok) store_chunk(static_cast<T*>(p.y) + at + c * kChunk, raw, left);
    if constexpr (__is_same(T, bf16_t))
      if (p.q) store_mx(raw, p.q, p.q_scale, at + c * kChunk, ok, p.q_e5m2);
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// ---- backward ---------------------------------------------------------------

struct NormBwd {
  const void* dy;
  const void* x;
  const void* dskip;
  const void* gamma;
  const float* mean;  // NULL: RMS norm
  const float* rstd;
  void* dx;
  void* dgamma;
  void* dbeta;        // NULL: not wanted
  float* part;        // [tiles][cols] of dgamma, then of dbeta
  int64_t rows;
  int cols;
  int tiles;
};

// dx, one workgroup per row, the row read twice: rows of any length.
template <class T, class W>
__global__ __launch_bounds__(kWideThreads) void norm_bwd_wide_kernel(NormBwd p) {
  __shared__ float slots[2][kWideThreads / 64];
  const int n = p.cols, nch = (n + kChunk - 1) / kChunk;
  const int64_t row = blockIdx.x, at = row * n;
  const float mean = p.mean ? p.mean[row] : 0.f, rstd = p.rstd[row];
  const T* x = static_cast<const T*>(p.x) + at;
  const T* dy = static_cast<const T*>(p.dy) + at;
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < nch; c += kWideThreads) {
    float fx[kChunk], fd[kChunk], g[kChunk];
    const int left = n - c * kChunk;
    load_floats(x + c * kChunk, left, fx);
    load_floats(dy + c * kChunk, left, fd);
    load_floats(static_cast<const W*>(p.gamma) + c * kChunk, left, g);
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (e < left) {
        const float gd = fd[e] * g[e];
        s1 += gd;
        s2 += gd * ((fx[e] - mean) * rstd);
      }
  }
  s1 = p.mean ? block_sum<kWideThreads>(s1, slots[0]) / (float)n : 0.f;
  s2 = block_sum<kWideThreads>(s2, slots[1]) / (float)n;
  for (int c = threadIdx.x; c < nch; c += kWideThreads) {
    float fx[kChunk], fd[kChunk], g[kChunk];
    const int left = n - c * kChunk;
    load_floats(x + c * kChunk, left, fx);
    load_floats(dy + c * kChunk, left, fd);
    load_floats(static_cast<const W*>(p.gamma) + c * kChunk, left, g);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) fx[e] = rstd * (fd[e] * g[e] - s1 - (fx[e] - mean) * rstd * s2);
    if (p.dskip) {
      load_floats(static_cast<const T*>(p.dskip) + at + c * kChunk, left, g);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) fx[e] += g[e];
    }
    store_chunk(static_cast<T*>(p.dx) + at + c * kChunk, pack<T>(fx), left);
  }
}

// Column sums of dy xh and dy over a tile of rows: 32 chunks of columns x 8 row lanes per workgroup.
constexpr int kColThreads = 256, kColChunks = 32, kColLanes = kColThreads / kColChunks;

template <class T>
__global__ __launch_bounds__(kColThreads) void norm_bwd_columns_kernel(NormBwd p) {
  __shared__ float red[kColLanes][kColChunks * kChunk + 1];
  const int n = p.cols, cx = threadIdx.x % kColChunks, ry = threadIdx.x / kColChunks;
  const int c = blockIdx.x * kColChunks + cx, left = n - c * kChunk;
  const int64_t per = (p.rows + p.tiles - 1) / p.tiles;
  const int64_t r0 = blockIdx.y * per, r1 = min(r0 + per, p.rows);
  float dg[kChunk], db[kChunk];
#pragma unroll
  for (int e = 0; e < kChunk; ++e) dg[e] = db[e] = 0.f;
  if (left > 0) {
    for (int64_t r = r0 + ry; r < r1; r += kColLanes) {
      const float mean = p.mean ? p.mean[r] : 0.f, rstd = p.rstd[r];
      float fx[kChunk], fd[kChunk];
      load_floats(static_cast<const T*>(p.x) + r * n + c * kChunk, left, fx);
      load_floats(static_cast<const T*>(p.dy) + r * n + c * kChunk, left, fd);
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (e < left) {
          dg[e] += fd[e] * ((fx[e] - mean) * rstd);
          db[e] += fd[e];
        }
    }
  }
  for (int pass = 0; pass < (p.dbeta ? 2 : 1); ++pass) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kChunk; ++e) red[ry][cx * kChunk + e] = pass ? db[e] : dg[e];
    __syncthreads();
    const int col = blockIdx.x * kColChunks * kChunk + threadIdx.x;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kColLanes; ++w) s += red[w][threadIdx.x];
    if (col < n) p.part[((int64_t)pass * p.tiles + blockIdx.y) * n + col] = s;
  }
}

// dgamma / dbeta: the tiles' sums added in order, 32 columns x 32 tile lanes per workgroup.
constexpr int kFinCols = 32, kFinLanes = 32;

template <class W>
__global__ __launch_bounds__(kFinCols* kFinLanes) void norm_bwd_final_kernel(NormBwd p) {
  __shared__ float red[kFinLanes][kFinCols + 1];
  const int cx = threadIdx.x % kFinCols, ty = threadIdx.x / kFinCols;
  const int col = blockIdx.x * kFinCols + cx;
  const float* part = p.part + (int64_t)blockIdx.y * p.tiles * p.cols;
  float s = 0.f;
  if (col < p.cols)
    for (int t = ty; t < p.tiles; t += kFinLanes) s += part[(int64_t)t * p.cols + col];
  red[ty][cx] = s;
  __syncthreads();
  if (ty == 0 && col < p.cols) {
    float v = 0.f;
#pragma unroll
    for (int t = 0; t < kFinLanes; ++t) v += red[t][cx];
    (static_cast<W*>(blockIdx.y ? p.dbeta : p.dgamma))[col] = from_float<W>(v);
  }
}

// Row tiles whose column sums are kept apart (one workspace row each per gradient).
inline int norm_tiles(int64_t rows, int64_t cols) {
  (void)cols;
  const int64_t t = (rows + 31) / 32;
  return (int)(t < 256 ? t : 256);
}

bool float_dtype(te_dtype t) { return t == TE_BF16 || t == TE_FP16 || t == TE_FP32; }

template <class T, class W>
te_status run_fwd(const NormFwd& p, hipStream_t stream) {
  hipLaunchKernelGGL((norm_fwd_wide_kernel<T, W>), dim3((unsigned)p.rows), dim3(kWideThreads), 0, stream, p);
  return launch_status();
}

template <class T, class W>
te_status run_bwd(const NormBwd& p, hipStream_t stream) {
  if (p.rows > 0) {
    hipLaunchKernelGGL((norm_bwd_wide_kernel<T, W>), dim3((unsigned)p.rows), dim3(kWideThreads), 0, stream, p);
    hipLaunchKernelGGL((norm_bwd_columns_kernel<T>),
                       dim3((unsigned)((p.cols + kColChunks * kChunk - 1) / (kColChunks * kChunk)), (unsigned)p.tiles),
                       dim3(kColThreads), 0, stream, p);
  }
  hipLaunchKernelGGL((norm_bwd_final_kernel<W>),
                     dim3((unsigned)((p.cols + kFinCols - 1) / kFinCols), p.dbeta ? 2u : 1u),
                     dim3(kFinCols * kFinLanes), 0, stream, p);
  return launch_status();
}

// f<T, W> of the tensors' and the weights' types
#define TEMX_NORM_TYPES(CALL)                                               \
  switch (dtype) {                                                          \
    case TE_BF16: return w_dtype == TE_BF16 ? CALL<bf16_t, bf16_t>(p, stream) : CALL<bf16_t, float>(p, stream); \
    case TE_FP16: return w_dtype == TE_FP16 ? CALL<f16_t, f16_t>(p, stream) : CALL<f16_t, float>(p, stream);    \
    default: return CALL<float, float>(p, stream);                          \
  }

te_status check_sizes(te_norm_kind kind, te_dtype dtype, int64_t rows, int64_t cols, te_dtype w_dtype) {
  constexpr int64_t kMost = ((int64_t)1 << 31) - 65536;
  TE_REQUIRE(kind == TE_NORM_LAYER || kind == TE_NORM_RMS, TE_ERR_VALUE);
  TE_REQUIRE(float_dtype(dtype) && (w_dtype == dtype || w_dtype == TE_FP32), TE_ERR_DTYPE);
  TE_REQUIRE(rows >= 0 && cols >= 0 && rows <= kMost && cols <= kMost, TE_ERR_SHAPE);
  return TE_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace temx

using namespace temx;

extern "C" te_status te_norm_forward(te_norm_kind kind, const void* x, te_dtype dtype, int64_t rows, int64_t cols,
                                     const void* residual, const void* gamma, const void* beta, te_dtype w_dtype,
                                     float eps, void* sum_out, void* y, uint8_t* q, uint8_t* q_scale, te_dtype q_fmt,
                                     float* mean, float* rstd, hipStream_t stream) {
  const te_status st = check_sizes(kind, dtype, rows, cols, w_dtype);
  if (st != TE_OK) return st;
  TE_REQUIRE(eps >= 0.f && eps <= 3.0e38f, TE_ERR_VALUE);
  TE_REQUIRE((residual != nullptr) == (sum_out != nullptr), TE_ERR_NULL);
  TE_REQUIRE((q != nullptr) == (q_scale != nullptr), TE_ERR_NULL);
  if (kind == TE_NORM_RMS) {
    TE_REQUIRE(beta == nullptr && mean == nullptr, TE_ERR_NULL);
  } else {
    TE_REQUIRE((mean != nullptr) == (rstd != nullptr), TE_ERR_NULL);
  }
  if (q != nullptr) {
    TE_REQUIRE(dtype == TE_BF16 && is_fp8(q_fmt), TE_ERR_DTYPE);
    TE_REQUIRE(cols % 32 == 0, TE_ERR_SHAPE);
  }
  if (rows == 0 || cols == 0) return TE_OK;
  TE_REQUIRE(x != nullptr && gamma != nullptr && (y != nullptr || q != nullptr), TE_ERR_NULL);
  TE_REQUIRE(aligned16(x) && aligned16(residual) && aligned16(sum_out) && aligned16(gamma) && aligned16(beta) &&
                 aligned16(y) && aligned16(q) && aligned4(mean) && aligned4(rstd),
             TE_ERR_ALIGN);
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const NormFwd p{x,    residual, gamma, beta, sum_out,   y,   q, q_scale, mean, rstd,
                  rows, (int)cols, eps,  kind == TE_NORM_LAYER, q_fmt == TE_E5M2};
  TEMX_NORM_TYPES(run_fwd)
}

extern "C" size_t te_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  constexpr int64_t kMost = ((int64_t)1 << 31) - 65536;
  if (rows <= 0 || cols <= 0 || rows > kMost || cols > kMost) return 0;
  return (size_t)2 * norm_tiles(rows, cols) * (size_t)cols * sizeof(float);
}

extern "C" te_status te_norm_backward(te_norm_kind kind, const void* dy, const void* x, const void* dskip,
                                      te_dtype dtype, int64_t rows, int64_t cols, const void* gamma, te_dtype w_dtype,
                                      const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const te_status st = check_sizes(kind, dtype, rows, cols, w_dtype);
  if (st != TE_OK) return st;
  if (kind == TE_NORM_RMS) TE_REQUIRE(mean == nullptr && dbeta == nullptr, TE_ERR_NULL);
  if (cols == 0) return TE_OK;
  TE_REQUIRE(dgamma != nullptr, TE_ERR_NULL);
  TE_REQUIRE(aligned16(dgamma) && aligned16(dbeta), TE_ERR_ALIGN);
  if (rows > 0) {
    TE_REQUIRE(dy && x && gamma && rstd && dx && workspace && (kind == TE_NORM_RMS || mean), TE_ERR_NULL);
    TE_REQUIRE(aligned16(dy) && aligned16(x) && aligned16(dskip) && aligned16(gamma) && aligned16(dx) &&
                   aligned16(workspace) && aligned4(mean) && aligned4(rstd),
               TE_ERR_ALIGN);
    TE_REQUIRE(workspace_bytes >= te_norm_backward_workspace_size(rows, cols), TE_ERR_WORKSPACE);
  }
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const NormBwd p{dy, x, dskip, gamma, mean, rstd, dx, dgamma, dbeta, static_cast<float*>(workspace), rows, (int)cols,
                  rows > 0 ? norm_tiles(rows, cols) : 0};
  TEMX_NORM_TYPES(run_bwd)
}
