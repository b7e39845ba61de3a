// The rows of a mixture-of-experts block: tokens to their experts' rows and back, and the gradients, for gfx950.
//
//   dispatch:  y[row_of[t, k]] = x[t]                        (also as MXFP8 codes and block scales)
//   combine:   y[t] = sum_k w[t, k] rows[row_of[t, k]]        (w = 1: the dispatch's gradient)
//   combine backward:  drows[row_of[t, k]] = w[t, k] dy[t],   dw[t, k] = sum_c dy[t, c] rows[row_of[t, k], c]
//
// A few operations per element: HBM bandwidth bounds all of them, so a token's row is read once whatever its number of
// experts (its codes are made once, too), an expert's row once, and the sums stay in registers.  Rows start anywhere
// (odd lengths): chunks of 8 elements from each row's own start, tails in the same loads (row_chunks.h).
// Measured on MI355X (a 1 GiB copy moves 5.0 TB/s), us a kernel, inputs of three calls in turn: 16384 tokens x 8 of 256
// experts, 4096 bf16 to MXFP8, 127 (689 MB, 5.4 TB/s); the gradient of 16384 rows of 4096 bf16, two a token, 34.9 (201
// MB, 5.8 TB/s); combine of 3001 x 6 rows of 2311 fp16 18.9 (97 MB, 5.1 TB/s); combine backward of 65536 rows of 4096
// bf16 216 (1142 MB, 5.3 TB/s).
#include "row_chunks.h"

namespace temx {
namespace {

constexpr int kThreads = 256;

struct RowsParams {
  const void* x;          // [tokens, cols]: dispatch x, combine backward dy
  const void* rows;       // [total_rows, cols]: combine, combine backward
  const int32_t* row_of;  // [tokens, topk]
  const float* weights;   // [tokens, topk] or NULL
  void* y;                // [total_rows, cols] or [tokens, cols]
  uint8_t* q;
  uint8_t* q_scale;
  float* dweights;
  int64_t tokens, total_rows, block0;
  int topk, cols;
  bool q_e5m2;
};

// The rows of kSlots slots of a token from slot k on, -1 where there is none (or one outside the tensor): loaded
// together, ahead of the accesses that need them.
constexpr int kSlots = 4;
__device__ __forceinline__ void rows_at(const RowsParams& p, int64_t token, int k, int64_t (&rows)[kSlots]) {
  int r[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) r[j] = p.row_of[token * p.topk + min(k + j, p.topk - 1)];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) rows[j] = k + j < p.topk && r[j] >= 0 && r[j] < p.total_rows ? r[j] : -1;
}

// Whole chunks past the caches where STREAM (see streams()).
template <class T, bool STREAM>
__device__ __forceinline__ void put_chunk(T* p, const Raw<T>& r, int n) {
  if (!STREAM || n < kChunk) return store_chunk(p, r, n);
#pragma unroll
  for (unsigned i = 0; i < sizeof(r.w) / 16; ++i)
    __builtin_nontemporal_store(u32x4{r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]},
                                reinterpret_cast<typename Vec16<sizeof(T)>::type*>(p) + i);
}

// load_ahead, past the caches where STREAM.  (With load_ahead's own load of a whole chunk beside it the compiler
// makes one load of both, without the hint.)
template <class T, bool STREAM>
__device__ __forceinline__ Raw<T> get_ahead(const T* row, int c, int n) {
  if constexpr (!STREAM) return load_ahead(row, c, n);
  Raw<T> r;
#pragma unroll
  for (unsigned i = 0; i < sizeof(r.w) / 4; ++i) r.w[i] = 0;
  if (n >= kChunk) {
    if (c < n) {
#pragma unroll
      for (unsigned i = 0; i < sizeof(r.w) / 16; ++i) {
        const u32x4 v = __builtin_nontemporal_load(
            reinterpret_cast<const typename Vec16<sizeof(T)>::type*>(row + min(c, n - kChunk)) + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.w[4 * i + e] = v[e];
      }
    }
  } else {
    r = load_ahead(row, c, n);
  }
  return r;
}

// A thread takes one chunk of a token: read once, written to each of its rows.
template <class T, bool STREAM>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(RowsParams p, int chunks) {
  const int64_t i = (p.block0 + blockIdx.x) * kThreads + threadIdx.x;
  const int64_t token = i / chunks;
  if (token >= p.tokens) return;  // whole quads: MXFP8 rows are whole 32-blocks
  const int c = (int)(i - token * chunks) * kChunk;
  const Raw<T> v = load_chunk(static_cast<const T*>(p.x) + token * p.cols, c, p.cols);
  uint32_t code = 0;
  uint2 codes = make_uint2(0, 0);
  if constexpr (std::is_same_v<T, bf16_t>) {
    if (p.q != nullptr) {
      const uint4 bits = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
      const uint32_t amax = quad_max(absmax_bits8(bits));
      code = p.q_e5m2 ? e8m0_code_from_amax_bits<TE_E5M2>(amax) : e8m0_code_from_amax_bits<TE_E4M3>(amax);
      const float scale = e8m0_to_float(code);
      codes = p.q_e5m2 ? cvt8_scaled<TE_E5M2>(bits, scale) : cvt8_scaled<TE_E4M3>(bits, scale);
    }
  }
  for (int k = 0; k < p.topk; k += kSlots) {
    int64_t rows[kSlots];
    rows_at(p, token, k, rows);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (rows[j] < 0) continue;
      const int64_t at = rows[j] * p.cols + c;
      if (p.y != nullptr) put_chunk<T, STREAM>(static_cast<T*>(p.y) + at, v, p.cols - c);
      if constexpr (std::is_same_v<T, bf16_t>) {
        if (p.q != nullptr) {
          if (STREAM) store_nt8(p.q + at, codes);
          else *reinterpret_cast<uint2*>(p.q + at) = codes;
          if ((c & 31) == 0) p.q_scale[at >> 5] = (uint8_t)code;
        }
      }
    }
  }
}

// A thread takes one chunk of a token: its rows' chunks added up in fp32 in the order of the slots, rounded once.
template <class T, bool STREAM>
__global__ __launch_bounds__(kThreads) void combine_kernel(RowsParams p, int chunks) {
  const int64_t i = (p.block0 + blockIdx.x) * kThreads + threadIdx.x;
  const int64_t token = i / chunks;
  if (token >= p.tokens) return;
  const int c = (int)(i - token * chunks) * kChunk;
  float sum[kChunk];
#pragma unroll
  for (int e = 0; e < kChunk; ++e) sum[e] = 0.f;
  for (int k = 0; k < p.topk; k += kSlots) {
    int64_t rows[kSlots];
    rows_at(p, token, k, rows);
    float w[kSlots];
    Raw<T> raw[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      w[j] = p.weights != nullptr && rows[j] >= 0 ? p.weights[token * p.topk + k + j] : 1.f;
      if (rows[j] >= 0) raw[j] = get_ahead<T, STREAM>(static_cast<const T*>(p.rows) + rows[j] * p.cols, c, p.cols);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (rows[j] < 0) continue;
      float f[kChunk];
      settle<T>(raw[j], c, p.cols);
      unpack<T>(raw[j], f);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) sum[e] = __builtin_fmaf(w[j], f[e], sum[e]);
    }
  }
  store_chunk(static_cast<T*>(p.y) + token * p.cols + c, pack<T>(sum), p.cols - c);
}

// LANES lanes take one slot: w dy to its row and the dot product of dy with the experts' output there, with no
// exchange but the lanes' own; dy comes from the caches for all but a token's first slot.  16 lanes for rows of at
// most 256 elements, whose waves would mostly idle.  (More chunks of a lane in flight made it slower: 65536 rows of
// 4096 bf16 216 us, with 4 chunks ahead 225.)
template <class T, bool STREAM, int LANES>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(RowsParams p) {
  const int lane = threadIdx.x % LANES;
  int64_t slot = (p.block0 + blockIdx.x) * (kThreads / LANES);
  slot += LANES == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / LANES) : threadIdx.x / LANES;
  const bool ok = slot < p.tokens * p.topk;
  const int row = ok ? p.row_of[slot] : -1;
  const bool there = row >= 0 && row < p.total_rows;
  float dot = 0.f;
  if (there) {
    const float w = p.weights[slot];
    const T* dy = static_cast<const T*>(p.x) + slot / p.topk * p.cols;
    const T* out = static_cast<const T*>(p.rows) + (int64_t)row * p.cols;
    for (int c0 = 0; c0 < p.cols; c0 += LANES * kChunk) {  // every lane takes part in the quads' exchanges
      const int c = c0 + lane * kChunk;
      float g[kChunk], f[kChunk];
      load_floats(dy, c, p.cols, g);
      Raw<T> raw = get_ahead<T, STREAM>(out, c, p.cols);
      settle<T>(raw, c, p.cols);
      unpack<T>(raw, f);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        dot = __builtin_fmaf(g[e], f[e], dot);
        g[e] *= w;
      }
      const Raw<T> v = pack<T>(g);
      const int64_t at = (int64_t)row * p.cols + c;
      if (p.y != nullptr) put_chunk<T, STREAM>(static_cast<T*>(p.y) + at, v, p.cols - c);
      if constexpr (std::is_same_v<T, bf16_t>) {
        if (p.q != nullptr) store_mx(v, p.q, p.q_scale, at, c < p.cols, p.q_e5m2);
      }
    }
  }
  dot = lanes_sum<LANES>(dot);
  if (ok && lane == 0) p.dweights[slot] = dot;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMost = ((int64_t)1 << 31) - 65536;
constexpr int64_t kMostBlocks = (int64_t)1 << 23;  // of one launch: 2^31 threads and fewer

// `blocks` workgroups in launches of at most kMostBlocks.
template <class Launch>
te_status in_parts(RowsParams p, int64_t blocks, Launch launch) {
  for (p.block0 = 0; p.block0 < blocks; p.block0 += kMostBlocks) {
    launch(p, dim3((unsigned)std::min(blocks - p.block0, kMostBlocks)));
    const te_status st = launch_status();
    if (st != TE_OK) return st;
  }
  return TE_OK;
}

// Whether the experts' rows pass the caches: above 96 MB.  Within them they may wait there for whoever takes them next,
// and came from there (us a combine, calls in a stream on inputs in turn: 83 MB of rows 18.4 and 21.7 past the caches,
// 134 MB 39.2 and 34.4; both read from cold caches 35 and 22, 62 and 37).
template <class T>
bool streams(const RowsParams& p) {
  return p.tokens * p.topk * (int64_t)p.cols * (int64_t)sizeof(T) > (int64_t)96 << 20;
}

template <class T>
te_status run_dispatch(const RowsParams& p, hipStream_t stream) {
  const int chunks = (p.cols + kChunk - 1) / kChunk;
  return in_parts(p, (p.tokens * chunks + kThreads - 1) / kThreads, [&](const RowsParams& q, dim3 grid) {
    if (streams<T>(q)) hipLaunchKernelGGL((dispatch_kernel<T, true>), grid, dim3(kThreads), 0, stream, q, chunks);
    else hipLaunchKernelGGL((dispatch_kernel<T, false>), grid, dim3(kThreads), 0, stream, q, chunks);
  });
}

template <class T>
te_status run_combine(const RowsParams& p, hipStream_t stream) {
  const int chunks = (p.cols + kChunk - 1) / kChunk;
  return in_parts(p, (p.tokens * chunks + kThreads - 1) / kThreads, [&](const RowsParams& q, dim3 grid) {
    if (streams<T>(q)) hipLaunchKernelGGL((combine_kernel<T, true>), grid, dim3(kThreads), 0, stream, q, chunks);
    else hipLaunchKernelGGL((combine_kernel<T, false>), grid, dim3(kThreads), 0, stream, q, chunks);
  });
}

template <class T, int LANES>
te_status run_combine_backward(const RowsParams& p, hipStream_t stream) {
  const int64_t per = kThreads / LANES;
  return in_parts(p, (p.tokens * p.topk + per - 1) / per, [&](const RowsParams& q, dim3 grid) {
    const dim3 block(kThreads);
    if (streams<T>(q)) hipLaunchKernelGGL((combine_backward_kernel<T, true, LANES>), grid, block, 0, stream, q);
    else hipLaunchKernelGGL((combine_backward_kernel<T, false, LANES>), grid, block, 0, stream, q);
  });
}

template <class T>
te_status run_combine_backward(const RowsParams& p, hipStream_t stream) {
  return p.cols <= 256 ? run_combine_backward<T, 16>(p, stream) : run_combine_backward<T, 64>(p, stream);
}

te_status check_rows(te_dtype dtype, int64_t tokens, int64_t cols, int topk, int64_t total_rows, const uint8_t* q,
                     const uint8_t* q_scale, te_dtype q_fmt) {
  TE_REQUIRE(dtype == TE_BF16 || dtype == TE_FP16 || dtype == TE_FP32, TE_ERR_DTYPE);
  TE_REQUIRE(topk >= 1 && topk <= 64, TE_ERR_SHAPE);
  TE_REQUIRE(cols >= 0 && cols <= kMost && tokens >= 0 && tokens <= kMost / topk, TE_ERR_SHAPE);
  TE_REQUIRE(total_rows >= 0 && total_rows <= kMost, TE_ERR_SHAPE);
  TE_REQUIRE((q != nullptr) == (q_scale != nullptr), TE_ERR_NULL);
  if (q != nullptr) {
    TE_REQUIRE(dtype == TE_BF16 && is_fp8(q_fmt), TE_ERR_DTYPE);
    TE_REQUIRE(cols % 32 == 0, TE_ERR_SHAPE);
  }
  return TE_OK;
}

}  // namespace
}  // namespace temx

using namespace temx;

#define TEMX_ROW_TYPES(run)                          \
  if (dtype == TE_BF16) return run<bf16_t>(p, stream); \
  if (dtype == TE_FP16) return run<f16_t>(p, stream);  \
  return run<float>(p, stream);

extern "C" te_status te_moe_dispatch(const void* x, te_dtype dtype, int64_t tokens, int64_t cols,
                                     const int32_t* row_of, int32_t topk, int64_t total_rows, void* y, uint8_t* q,
                                     uint8_t* q_scale, te_dtype q_fmt, hipStream_t stream) {
  const te_status st = check_rows(dtype, tokens, cols, topk, total_rows, q, q_scale, q_fmt);
  if (st != TE_OK) return st;
  if (tokens == 0 || cols == 0 || total_rows == 0) return TE_OK;
  TE_REQUIRE(x && row_of && (y || q), TE_ERR_NULL);
  TE_REQUIRE(aligned16(x) && aligned4(row_of) && aligned16(y) && aligned16(q), TE_ERR_ALIGN);
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const RowsParams p{x, nullptr, row_of, nullptr, y, q, q_scale, nullptr, tokens, total_rows, 0, topk, (int)cols,
                     q_fmt == TE_E5M2};
  TEMX_ROW_TYPES(run_dispatch)
}

extern "C" te_status te_moe_combine(const void* rows, te_dtype dtype, int64_t total_rows, int64_t cols,
                                    const int32_t* row_of, const float* weights, int64_t tokens, int32_t topk, void* y,
                                    hipStream_t stream) {
  const te_status st = check_rows(dtype, tokens, cols, topk, total_rows, nullptr, nullptr, TE_E4M3);
  if (st != TE_OK) return st;
  if (tokens == 0 || cols == 0) return TE_OK;
  TE_REQUIRE((rows || total_rows == 0) && row_of && y, TE_ERR_NULL);
  TE_REQUIRE(aligned16(rows) && aligned4(row_of) && aligned4(weights) && aligned16(y), TE_ERR_ALIGN);
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const RowsParams p{nullptr, rows, row_of, weights, y, nullptr, nullptr, nullptr, tokens, total_rows, 0, topk,
                     (int)cols, false};
  TEMX_ROW_TYPES(run_combine)
}

extern "C" te_status te_moe_combine_backward(const void* dy, const void* rows, te_dtype dtype, int64_t tokens,
                                             int64_t cols, const int32_t* row_of, const float* weights, int32_t topk,
                                             int64_t total_rows, void* drows, uint8_t* q, uint8_t* q_scale,
                                             te_dtype q_fmt, float* dweights, hipStream_t stream) {
  const te_status st = check_rows(dtype, tokens, cols, topk, total_rows, q, q_scale, q_fmt);
  if (st != TE_OK) return st;
  if (tokens == 0) return TE_OK;
  TE_REQUIRE(dweights && row_of && weights, TE_ERR_NULL);
  TE_REQUIRE(cols == 0 || total_rows == 0 || (dy && rows && (drows || q)), TE_ERR_NULL);
  TE_REQUIRE(aligned16(dy) && aligned16(rows) && aligned4(row_of) && aligned4(weights) && aligned16(drows) &&
                 aligned16(q) && aligned4(dweights),
             TE_ERR_ALIGN);
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const RowsParams p{dy, rows, row_of, weights, drows, q, q_scale, dweights, tokens, total_rows, 0, topk, (int)cols,
                     q_fmt == TE_E5M2};
  TEMX_ROW_TYPES(run_combine_backward)
}
