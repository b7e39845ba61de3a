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
// The passes do ~10 operations per element: HBM bandwidth bounds them, so a
// row is read once and held in registers between its statistics and its
// outputs, and the weights' gradients come from the same reads.  Only longer
// rows than the registers take (forward past 32768 columns; backward past
// 16384 16-bit or 8192 fp32 ones) are read again, by the wide kernels.
// Measured on MI355X (a 1 GiB copy moves 5.1 TB/s), us a call with the inputs
// of each call not in the caches: 16384 x 8192 bf16, RMS norm with residual to
// MXFP8, 163 (944 MB, 5.8 TB/s); its backward with dskip 200 (1074 MB, 5.4
// TB/s); 3001 x 5003 fp32 30 (120 MB, 4.0 TB/s); 4096 x 1024 bf16 backward
// 12.5, two launches of 9 and 3 us (25 MB at that rate: 4.9 us).
#include <type_traits>

#include "row_chunks.h"

namespace temx {
namespace {

// Rows that a workgroup of about `threads` threads holds, NT threads each.
constexpr int rows_at_a_time(int nt, int threads) { return nt < threads ? threads / nt : 1; }

// The thread's row among a workgroup's, NT threads each; the same for a whole wave (and known to be) from 64 up.
template <int NT>
__device__ __forceinline__ int row_lane() {
  return NT >= 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / NT) : threadIdx.x / NT;
}

// ---- sums and roots ----------------------------------------------------------

// Sum over the workgroup, the same bits in every thread; `slots` holds one float per wave and is free
// again once every thread has returned from the next call or barrier.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* slots) {
  v = lanes_sum<64>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) s += slots[w];
  return s;
}

// 1 / sqrt(v) to within one unit in the last place: the hardware's estimate and one Newton step, which is
// left out where it has no value (v = 0 or infinite).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float e = __builtin_fmaf(-(v * r), r, 1.0f);
  return __builtin_fabsf(e) < 0.5f ? __builtin_fmaf(0.5f * r, e, r) : r;
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
  int64_t row0;  // of the launch
  int64_t rows;
  int cols;
  float eps;
  bool layer;
  bool q_e5m2;
};

// A row held in registers: NT threads per row, NC chunks per thread (thread t: chunks t, t + NT, ..), rows read
// once.  The statistics of each wave's part are joined in one exchange: with n_w, m_w and M_w the count, mean and
// centred sum of squares of wave w, mean = sum n_w m_w / n and M = sum M_w + n_w (m_w - mean)^2.
template <class T, class W, int NT, int NC>
__global__ __launch_bounds__(NT* rows_at_a_time(NT, 256)) void norm_fwd_kernel(NormFwd p) {
  constexpr int kRows = rows_at_a_time(NT, 256), kWaves = NT > 64 ? NT / 64 : 1;
  constexpr int kLanes = NT < 64 ? NT : 64;
  __shared__ float2 all_slots[kRows][kWaves];
  float2(&slots)[kWaves] = all_slots[row_lane<NT>()];
  const int n = p.cols, t = threadIdx.x % NT;
  const int64_t row = p.row0 + (int64_t)blockIdx.x * kRows + row_lane<NT>(), at = row * n;
  const bool row_ok = kRows == 1 || row < p.rows;  // every lane takes part in the exchanges below
  // A row past the end computes on the first and stores nothing.  sum_out may be one of the inputs: what a tail's or
  // such a row's load may see changed is not used.
  const int64_t from = row_ok ? at : 0;
  float f[NC][kChunk];
  Raw<T> raw[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) raw[j] = load_ahead(static_cast<const T*>(p.x) + from, (t + j * NT) * kChunk, n);
  if (p.residual != nullptr) {
    Raw<T> res[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j)
      res[j] = load_ahead(static_cast<const T*>(p.residual) + from, (t + j * NT) * kChunk, n);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (t + j * NT) * kChunk;
      float r[kChunk];
      settle<T>(raw[j], c, n);
      settle<T>(res[j], c, n);
      unpack<T>(raw[j], f[j]);
      unpack<T>(res[j], r);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[j][e] += r[e];
      raw[j] = pack<T>(f[j]);
      store_chunk(static_cast<T*>(p.sum) + at + c, raw[j], row_ok ? n - c : 0);
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if (p.residual == nullptr) settle<T>(raw[j], (t + j * NT) * kChunk, n);
    unpack<T>(raw[j], f[j]);
  }

  // elements of the wave's lanes (of the row group's, NT < 64)
  const int wave = NT > 64 ? __builtin_amdgcn_readfirstlane(t >> 6) : 0, w0 = wave * 64 * kChunk;
  auto held = [&](int first) {
    int held = 0;
#pragma unroll
    for (int j = 0; j < NC; ++j) held += min(max(n - first - j * NT * kChunk, 0), kLanes * kChunk);
    return (float)held;
  };
  float mean = 0.f, m2 = 0.f;
  if (p.layer) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int e = 0; e < kChunk; ++e) s += f[j][e];
    s = lanes_sum<kLanes>(s);
    const float cnt = held(w0);
    mean = cnt > 0.f ? s / cnt : 0.f;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int left = n - (t + j * NT) * kChunk;
    if (left >= kChunk) {
#pragma unroll
      for (int e = 0; e < kChunk; ++e) m2 = __builtin_fmaf(f[j][e] - mean, f[j][e] - mean, m2);
    } else {
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (e < left) m2 = __builtin_fmaf(f[j][e] - mean, f[j][e] - mean, m2);
    }
  }
  m2 = lanes_sum<kLanes>(m2);
  if constexpr (NT > 64) {
    if ((t & 63) == 0) slots[wave] = make_float2(mean, m2);
    __syncthreads();
    m2 = 0.f;
    if (p.layer) {
      mean = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mean += slots[w].x * held(w * 64 * kChunk);
      mean /= (float)n;
    }
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float d = slots[w].x - mean;
      m2 += slots[w].y;
      if (p.layer) m2 = __builtin_fmaf(d * d, held(w * 64 * kChunk), m2);
    }
  }
  const float rstd = inv_sqrt(m2 / (float)n + p.eps);

#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = (t + j * NT) * kChunk, left = row_ok ? n - c : 0;
    float g[kChunk];
    load_floats(static_cast<const W*>(p.gamma), c, n, g);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) f[j][e] = ((f[j][e] - mean) * g[e]) * rstd;
    if (p.beta != nullptr) {
      load_floats(static_cast<const W*>(p.beta), c, n, g);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[j][e] += g[e];
    }
    raw[j] = pack<T>(f[j]);
    if (p.y != nullptr) store_chunk(static_cast<T*>(p.y) + at + c, raw[j], left);
    if constexpr (__is_same(T, bf16_t))
      if (p.q != nullptr) store_mx(raw[j], p.q, p.q_scale, at + c, left > 0, p.q_e5m2);
  }
  if (t == 0 && row_ok) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
}

constexpr int kWideThreads = 1024;

// One workgroup per row, the row read again for each of mean (layer norm), variance and output: rows of any length.
// The passes wait for one another (bf16: layer norm 2048 x 40000 98 us, 64 for one read at a copy's rate; RMS norm,
// two reads, 4096 x 65536 243 us, 210).
template <class T, class W>
__global__ __launch_bounds__(kWideThreads) void norm_fwd_wide_kernel(NormFwd p) {
  __shared__ float slots[kWideThreads / 64];
  const int n = p.cols, nch = (n + kChunk - 1) / kChunk;
  const int64_t row = p.row0 + blockIdx.x, at = row * n;
  const T* x = static_cast<const T*>(p.x) + at;
  float mean = 0.f;
  if (p.layer || p.residual) {
    float s = 0.f;
    for (int c = threadIdx.x; c < nch; c += kWideThreads) {
      float f[kChunk];
      load_floats(x, c * kChunk, n, f);
      if (p.residual) {
        float r[kChunk];
        load_floats(static_cast<const T*>(p.residual) + at, c * kChunk, n, r);
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
    load_floats(x, c * kChunk, n, f);
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (c * kChunk + e < n) v += (f[e] - mean) * (f[e] - mean);
  }
  const float rstd = inv_sqrt(block_sum<kWideThreads>(v, slots) / (float)n + p.eps);
  // every lane of a wave takes part in the MXFP8 block maxima: the loop runs whole waves
  for (int c0 = 0; c0 < nch; c0 += kWideThreads) {
    const int c = c0 + threadIdx.x, left = n - c * kChunk;
    const bool ok = c < nch;
    float f[kChunk], g[kChunk], b[kChunk];
    if (ok) {
      load_floats(x, c * kChunk, n, f);
      load_floats(static_cast<const W*>(p.gamma), c * kChunk, n, g);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[e] = (f[e] - mean) * rstd * g[e];
      if (p.beta) {
        load_floats(static_cast<const W*>(p.beta), c * kChunk, n, b);
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
  int64_t row0;       // of the launch (wide kernel)
  int64_t rows;
  int cols;
  int tiles;
  int col0;           // of the launch (final kernel)
};

// Rows held in registers as in norm_fwd_kernel; each workgroup walks rows and keeps its columns' sums of dy xh and
// dy in registers, so dy and x are read once for dx and for the weights' gradients.  The next rows' loads are in
// flight while a row is computed.  At the end a workgroup's row lanes join in LDS and leave one row of partial sums.
template <class T, class W, int THREADS, int NT, int NC = 1>
__global__ __launch_bounds__(NT* rows_at_a_time(NT, THREADS)) void norm_bwd_kernel(NormBwd p) {
  constexpr int kRows = rows_at_a_time(NT, THREADS), kWaves = NT > 64 ? NT / 64 : 1, kLanes = NT < 64 ? NT : 64;
  constexpr bool kAhead = NC == 1;  // the next rows' loads in flight (more chunks leave no registers for them)
  __shared__ float2 slots[2][kRows * kWaves];
  __shared__ float joined[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? NT * kChunk : 1];
  const int n = p.cols, t = threadIdx.x % NT, sub = row_lane<NT>();
  const bool layer = p.mean != nullptr, skip = p.dskip != nullptr;
  auto col = [&](int j) { return (t + j * NT) * kChunk; };
  Raw<W> gamma[NC];
  float dg[NC][kChunk], db[NC][kChunk];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    gamma[j] = load_chunk(static_cast<const W*>(p.gamma), col(j), n);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) dg[j][e] = db[j][e] = 0.f;
  }
  struct Row {
    Raw<T> x[NC], dy[NC], skip[NC];
    float mean, rstd;
  };
  auto load = [&](Row& v, int64_t row) __attribute__((always_inline)) {
    row = min(row, p.rows - 1);  // a row past the end: the last one again, used for nothing
    const int64_t at = row * n;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      v.x[j] = load_ahead(static_cast<const T*>(p.x) + at, col(j), n);
      v.dy[j] = load_ahead(static_cast<const T*>(p.dy) + at, col(j), n);
      if (skip) v.skip[j] = load_ahead(static_cast<const T*>(p.dskip) + at, col(j), n);
    }
    v.mean = layer ? p.mean[row] : 0.f;
    v.rstd = p.rstd[row];
  };
  const float inv_n = 1.0f / (float)n;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t base = (int64_t)blockIdx.x * kRows;
  Row now, next;
  load(now, base + sub);
  int buf = 0;
  for (; base < p.rows; base += step, buf ^= 1) {
    if constexpr (kAhead)
      if (base + step < p.rows) load(next, base + step + sub);
    float s1 = 0.f, s2 = 0.f;
    const bool row_ok = base + sub < p.rows;
    float xh[kChunk], d[kChunk], g[kChunk];
    auto terms = [&](int j) __attribute__((always_inline)) {  // xh, dy and g of chunk j
      unpack<T>(now.x[j], xh);
      unpack<T>(now.dy[j], d);
      unpack<W>(gamma[j], g);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        xh[e] = (xh[e] - now.mean) * now.rstd;
        g[e] *= d[e];
      }
    };
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      settle<T>(now.x[j], col(j), n);
      settle<T>(now.dy[j], col(j), n);
      terms(j);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        s1 += g[e];
        s2 = __builtin_fmaf(g[e], xh[e], s2);
      }
      if (row_ok) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          dg[j][e] = __builtin_fmaf(d[e], xh[e], dg[j][e]);
          db[j][e] += d[e];
        }
      }
    }
    s1 = lanes_sum<kLanes>(s1);
    s2 = lanes_sum<kLanes>(s2);
    if constexpr (NT > 64) {
      // two buffers: a wave may be one row ahead of another, and the barrier of that row keeps it from two
      if ((threadIdx.x & 63) == 0) slots[buf][threadIdx.x >> 6] = make_float2(s1, s2);  // NT % 64 == 0
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        s1 += slots[buf][sub * kWaves + w].x;
        s2 += slots[buf][sub * kWaves + w].y;
      }
    }
    s1 = layer ? s1 * inv_n : 0.f;
    s2 *= inv_n;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if constexpr (NC > 1) {  // formed again: kept, the chunks' terms do not fit the registers
        opaque(now.x[j]);
        opaque(now.dy[j]);
        terms(j);
      }
#pragma unroll
      for (int e = 0; e < kChunk; ++e) g[e] = now.rstd * (g[e] - s1 - xh[e] * s2);
      if (skip) {
        settle<T>(now.skip[j], col(j), n);
        unpack<T>(now.skip[j], d);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) g[e] += d[e];
      }
      if (row_ok) store_chunk(static_cast<T*>(p.dx) + (base + sub) * n + col(j), pack<T>(g), n - col(j));
    }
    if constexpr (kAhead) now = next;
    else if (base + step < p.rows) load(now, base + step + sub);
  }
  // the row lanes' sums in order, one 8-column chunk per thread at a time
  float* part = p.part + (int64_t)blockIdx.x * n;
  for (int pass = 0; pass < (p.dbeta != nullptr ? 2 : 1); ++pass) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float v[kChunk];
#pragma unroll
      for (int e = 0; e < kChunk; ++e) v[e] = pass ? db[j][e] : dg[j][e];
      if constexpr (kRows > 1) {
        __syncthreads();
        if (sub > 0)
#pragma unroll
          for (int e = 0; e < kChunk; ++e) joined[sub - 1][e * NT + t] = v[e];
        __syncthreads();
        if (sub == 0)
          for (int w = 0; w < kRows - 1; ++w)
#pragma unroll
            for (int e = 0; e < kChunk; ++e) v[e] += joined[w][e * NT + t];
      }
      if (sub == 0) store_chunk(part + (int64_t)pass * p.tiles * n + col(j), pack<float>(v), n - col(j));
    }
  }
}

// dx, one workgroup per row, the row read twice: rows of any length.  norm_bwd_columns_kernel reads x and dy a third
// time: 2048 x 40000 bf16 202 us in all (96 for one read at a copy's rate), 4096 x 12288 fp32 236 us (118).
template <class T, class W>
__global__ __launch_bounds__(kWideThreads) void norm_bwd_wide_kernel(NormBwd p) {
  __shared__ float slots[2][kWideThreads / 64];
  const int n = p.cols, nch = (n + kChunk - 1) / kChunk;
  const int64_t row = p.row0 + blockIdx.x, at = row * n;
  const float mean = p.mean ? p.mean[row] : 0.f, rstd = p.rstd[row];
  const T* x = static_cast<const T*>(p.x) + at;
  const T* dy = static_cast<const T*>(p.dy) + at;
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < nch; c += kWideThreads) {
    float fx[kChunk], fd[kChunk], g[kChunk];
    const int left = n - c * kChunk;
    load_floats(x, c * kChunk, n, fx);
    load_floats(dy, c * kChunk, n, fd);
    load_floats(static_cast<const W*>(p.gamma), c * kChunk, n, g);
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
    load_floats(x, c * kChunk, n, fx);
    load_floats(dy, c * kChunk, n, fd);
    load_floats(static_cast<const W*>(p.gamma), c * kChunk, n, g);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) fx[e] = rstd * (fd[e] * g[e] - s1 - (fx[e] - mean) * rstd * s2);
    if (p.dskip) {
      load_floats(static_cast<const T*>(p.dskip) + at, c * kChunk, n, g);
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
      load_floats(static_cast<const T*>(p.x) + r * n, c * kChunk, n, fx);
      load_floats(static_cast<const T*>(p.dy) + r * n, c * kChunk, n, fd);
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
  const int col = p.col0 + blockIdx.x * kFinCols + cx;
  const float* part = p.part + (int64_t)blockIdx.y * p.tiles * p.cols;
  float s = 0.f;
  if (col < p.cols) {
    constexpr int kAhead = 8;  // loads in flight
    for (int t0 = ty; t0 < p.tiles; t0 += kFinLanes * kAhead) {
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int t = t0 + i * kFinLanes;
        v[i] = t < p.tiles ? part[(int64_t)t * p.cols + col] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s += v[i];
    }
  }
  red[ty][cx] = s;
  __syncthreads();
  if (ty == 0 && col < p.cols) {
    float v = 0.f;
#pragma unroll
    for (int t = 0; t < kFinLanes; ++t) v += red[t][cx];
    (static_cast<W*>(blockIdx.y ? p.dbeta : p.dgamma))[col] = from_float<W>(v);
  }
}

// Backward: threads per row (NT), one chunk per thread, rounded up to one of these; 0: the wide kernels.
inline int bwd_threads_per_row(int64_t cols) {
  const int64_t ch = (cols + kChunk - 1) / kChunk;
  for (int nt : {16, 32, 64, 128, 192, 256, 384, 512, 640, 768, 1024})
    if (ch <= nt) return nt;
  return 0;
}

// Threads of a backward workgroup: 1024 where that leaves a workgroup for every CU, else 256 (or the row's).  Bf16, us,
// 1024 and 256 threads: 16384 x 2048 41.2 and 45.1, 16384 x 1024 25.2 and 26.8, 131072 x 512 77.7 and 80.3; with few
// rows, 2048 x 512, 13.4 and 11.6.
inline int bwd_threads(int nt, int64_t rows) {
  return rows * nt >= (int64_t)device_cu_count() * 1024 ? 1024 : 256;
}

// Rows of partial sums of each weight gradient: the register kernel's workgroups, or the wide kernels' row tiles.
// One workgroup of more than 640 threads per CU, two smaller ones (two of 1024 leave twice the partial sums: 16384 x
// 2048 44.0 us and not 41.3, 8192 x 8192 85.4 and 78.5).
inline int norm_tiles(int64_t rows, int64_t cols) {
  const int nt = bwd_threads_per_row(cols);
  const int64_t cus = device_cu_count();
  const int64_t per = nt == 0 ? (cols <= 2048 * kChunk ? 1 : 32) : rows_at_a_time(nt, bwd_threads(nt, rows));  // rows at a time
  const int64_t most = nt == 0 || nt * per > 640 ? cus : 2 * cus;
  const int64_t t = (rows + per - 1) / per;
  return (int)(t < most ? t : most);
}

// Bytes of both gradients' partial sums, from bounds of norm_tiles that grow with the rows and the columns (it does
// not itself: 512 rows of sums for 2047 rows of 1024 columns, 256 for 4096): the workspace of the longest and widest
// call serves every smaller one.  Up to 2048 chunks norm_tiles is at most min(rows, two a CU), past them
// min(ceil(rows / 32), one a CU), taken as no fewer bytes than 2048 chunks have.
inline size_t norm_workspace(int64_t rows, int64_t cols) {
  constexpr int64_t kHeld = 2048 * kChunk;
  const int64_t cus = device_cu_count();
  const int64_t held = (cols < kHeld ? cols : kHeld) * (rows < 2 * cus ? rows : 2 * cus);
  const int64_t tiles = (rows + 31) / 32, wide = cols > kHeld ? cols * (tiles < cus ? tiles : cus) : 0;
  return (size_t)2 * sizeof(float) * (size_t)(held > wide ? held : wide);
}

// f(NT) for a row's threads, false where no register kernel takes the row
template <class F>
bool with_threads(int nt, F f) {
  switch (nt) {
    case 16: f(std::integral_constant<int, 16>{}); return true;
    case 32: f(std::integral_constant<int, 32>{}); return true;
    case 64: f(std::integral_constant<int, 64>{}); return true;
    case 128: f(std::integral_constant<int, 128>{}); return true;
    case 192: f(std::integral_constant<int, 192>{}); return true;
    case 256: f(std::integral_constant<int, 256>{}); return true;
    case 384: f(std::integral_constant<int, 384>{}); return true;
    case 512: f(std::integral_constant<int, 512>{}); return true;
    case 640: f(std::integral_constant<int, 640>{}); return true;
    case 768: f(std::integral_constant<int, 768>{}); return true;
    case 1024: f(std::integral_constant<int, 1024>{}); return true;
    default: return false;
  }
}

bool float_dtype(te_dtype t) { return t == TE_BF16 || t == TE_FP16 || t == TE_FP32; }

// f(workgroups) for launches of `each` rows per workgroup, p.row0 their first row: a launch holds fewer than 2^32
// threads.
template <class P, class F>
void for_launches(P& p, int each, F f) {
  constexpr int64_t kMost = (int64_t)1 << 21;  // workgroups of up to 1024 threads
  const int64_t blocks = (p.rows + each - 1) / each;
  for (int64_t b = 0; b < blocks; b += kMost) {
    p.row0 = b * each;
    f((unsigned)(blocks - b < kMost ? blocks - b : kMost));
  }
}

// Forward: a wave (or less) per row up to 256 chunks and 256 threads up to 1024, up to 4 chunks per thread: several
// rows' loads are in flight per CU and few waves have to meet (8192 x 8192 bf16: 52 us with 256 x 4, 76 with
// 1024 x 1; 8192 x 4096: 29 and 35).  At most a row per CU takes a thread per chunk instead (1 x 8192: 3.8 us).
template <class T, class W>
te_status run_fwd(NormFwd p, hipStream_t stream) {
  auto go = [&](auto nt, auto nc) {
    constexpr int NT = decltype(nt)::value, NC = decltype(nc)::value, kRows = rows_at_a_time(NT, 256);
    for_launches(p, kRows, [&](unsigned blocks) {
      hipLaunchKernelGGL((norm_fwd_kernel<T, W, NT, NC>), dim3(blocks), dim3(NT * kRows), 0, stream, p);
    });
  };
  using std::integral_constant;
  const int ch = (int)(((int64_t)p.cols + kChunk - 1) / kChunk);
  const bool few = p.rows <= device_cu_count();
  if (ch <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (ch <= 32) go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (ch <= 64) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (ch <= 256 && few) go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (ch <= 128) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (ch <= 192) go(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  else if (ch <= 256) go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (ch <= 1024 && few) go(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
  else if (ch <= 512) go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (ch <= 768) go(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  else if (ch <= 1024) go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else if (ch <= 2048) go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else if (ch <= 4096) go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  else
    for_launches(p, 1, [&](unsigned blocks) {
      hipLaunchKernelGGL((norm_fwd_wide_kernel<T, W>), dim3(blocks), dim3(kWideThreads), 0, stream, p);
    });
  return launch_status();
}

template <class T, class W>
te_status run_bwd(NormBwd p, hipStream_t stream) {
  const dim3 tiles((unsigned)p.tiles);
  if (p.rows > 0) {
    const int nt = bwd_threads_per_row(p.cols);
    bool held = with_threads(nt, [&](auto n) {
      constexpr int NT = decltype(n)::value;
      if constexpr (rows_at_a_time(NT, 1024) > 1)
        if (bwd_threads(nt, p.rows) == 1024) {
          hipLaunchKernelGGL((norm_bwd_kernel<T, W, 1024, NT>), tiles, dim3(NT * rows_at_a_time(NT, 1024)), 0, stream,
                             p);
          return;
        }
      hipLaunchKernelGGL((norm_bwd_kernel<T, W, 256, NT>), tiles, dim3(NT * rows_at_a_time(NT, 256)), 0, stream, p);
    });
    // up to 2048 chunks of 2-byte elements: four per thread (4096 x 16384 bf16: 96 us, 151 with the wide kernels)
    if constexpr (sizeof(T) == 2) {
      if (!held && p.cols <= 2048 * kChunk) {
        hipLaunchKernelGGL((norm_bwd_kernel<T, W, 512, 512, 4>), tiles, dim3(512), 0, stream, p);
        held = true;
      }
    }
    if (!held) {
      for_launches(p, 1, [&](unsigned blocks) {
        hipLaunchKernelGGL((norm_bwd_wide_kernel<T, W>), dim3(blocks), dim3(kWideThreads), 0, stream, p);
      });
      hipLaunchKernelGGL((norm_bwd_columns_kernel<T>),
                         dim3((unsigned)((p.cols + kColChunks * kChunk - 1) / (kColChunks * kChunk)),
                              (unsigned)p.tiles),
                         dim3(kColThreads), 0, stream, p);
    }
  }
  constexpr int64_t kMost = (int64_t)1 << 21;  // workgroups per launch, as in for_launches
  const int64_t blocks = ((int64_t)p.cols + kFinCols - 1) / kFinCols;
  for (int64_t b = 0; b < blocks; b += kMost) {
    p.col0 = (int)(b * kFinCols);
    hipLaunchKernelGGL((norm_bwd_final_kernel<W>),
                       dim3((unsigned)(blocks - b < kMost ? blocks - b : kMost), p.dbeta ? 2u : 1u),
                       dim3(kFinCols * kFinLanes), 0, stream, p);
  }
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
  const NormFwd p{x, residual, gamma, beta, sum_out,   y,   q,  q_scale, mean,
                  rstd, 0,     rows,  (int)cols, eps, kind == TE_NORM_LAYER, q_fmt == TE_E5M2};
  TEMX_NORM_TYPES(run_fwd)
}

extern "C" size_t te_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  constexpr int64_t kMost = ((int64_t)1 << 31) - 65536;
  if (rows <= 0 || cols <= 0 || rows > kMost || cols > kMost) return 0;
  return norm_workspace(rows, cols);
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
  const NormBwd p{dy, x, dskip, gamma, mean, rstd, dx, dgamma, dbeta, static_cast<float*>(workspace), 0, rows, (int)cols,
                  rows > 0 ? norm_tiles(rows, cols) : 0};
  TEMX_NORM_TYPES(run_bwd)
}
