// The rows of a mixture-of-experts block: tokens to their experts' rows and back, and the gradients, for gfx950.
//
//   dispatch:  y[row_of[t, k]] = x[t]                        (also as MXFP8 codes and block scales)
//   combine:   y[t] = sum_k w[t, k] rows[row_of[t, k]]        (w = 1: the dispatch's gradient)
//   combine backward:  drows[row_of[t, k]] = w[t, k] dy[t],   dw[t, k] = sum_c dy[t, c] rows[row_of[t, k], c]
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

// The row of a slot, -1 where it has none (or one outside the tensor).
__device__ __forceinline__ int64_t row_at(const RowsParams& p, int64_t slot) {
  const int r = p.row_of[slot];
  return r >= 0 && r < p.total_rows ? r : -1;
}

// A thread takes one chunk of a token: read once, written to each of its rows.
template <class T>
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
  for (int k = 0; k < p.topk; ++k) {
    const int64_t r = row_at(p, token * p.topk + k);
    if (r < 0) continue;
    const int64_t at = r * p.cols + c;
    if (p.y != nullptr) store_chunk(static_cast<T*>(p.y) + at, v, p.cols - c);
    if constexpr (std::is_same_v<T, bf16_t>) {
      if (p.q != nullptr) {
        *reinterpret_cast<uint2*>(p.q + at) = codes;
        if ((c & 31) == 0) p.q_scale[at >> 5] = (uint8_t)code;
      }
    }
  }
}

// A thread takes one chunk of a token: its rows' chunks added up in fp32 in the order of the slots, rounded once.
template <class T>
__global__ __launch_bounds__(kThreads) void combine_kernel(RowsParams p, int chunks) {
  const int64_t i = (p.block0 + blockIdx.x) * kThreads + threadIdx.x;
  const int64_t token = i / chunks;
  if (token >= p.tokens) return;
  const int c = (int)(i - token * chunks) * kChunk;
  float sum[kChunk];
#pragma unroll
  for (int e = 0; e < kChunk; ++e) sum[e] = 0.f;
  for (int k = 0; k < p.topk; ++k) {
    const int64_t slot = token * p.topk + k, r = row_at(p, slot);
    if (r < 0) continue;
    const float w = p.weights != nullptr ? p.weights[slot] : 1.f;
    float f[kChunk];
    load_floats(static_cast<const T*>(p.rows) + r * p.cols, c, p.cols, f);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) sum[e] = __builtin_fmaf(w, f[e], sum[e]);
  }
  store_chunk(static_cast<T*>(p.y) + token * p.cols + c, pack<T>(sum), p.cols - c);
}

// A wave takes one slot: w dy to its row and the dot product of dy with the experts' output there.
template <class T>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(RowsParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t slot = (p.block0 + blockIdx.x) * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (slot >= p.tokens * p.topk) return;
  const int64_t token = slot / p.topk, r = row_at(p, slot);
  float dot = 0.f;
  if (r >= 0) {
    const float w = p.weights[slot];
    const int cols_up = (p.cols + 64 * kChunk - 1) / (64 * kChunk) * (64 * kChunk);
    for (int c = lane * kChunk; c < cols_up; c += 64 * kChunk) {  // every lane takes part in the quads' exchanges
      float g[kChunk], f[kChunk];
      load_floats(static_cast<const T*>(p.x) + token * p.cols, c, p.cols, g);
      load_floats(static_cast<const T*>(p.rows) + r * p.cols, c, p.cols, f);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        dot = __builtin_fmaf(g[e], f[e], dot);
        g[e] *= w;
      }
      const Raw<T> v = pack<T>(g);
      const int64_t at = r * p.cols + c;
      if (p.y != nullptr) store_chunk(static_cast<T*>(p.y) + at, v, p.cols - c);
      if constexpr (std::is_same_v<T, bf16_t>) {
        if (p.q != nullptr) store_mx(v, p.q, p.q_scale, at, c < p.cols, p.q_e5m2);
      }
    }
  }
  dot = lanes_sum<64>(dot);
  if (lane == 0) p.dweights[slot] = dot;
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

template <class T>
te_status run_dispatch(const RowsParams& p, hipStream_t stream) {
  const int chunks = (p.cols + kChunk - 1) / kChunk;
  return in_parts(p, (p.tokens * chunks + kThreads - 1) / kThreads, [&](const RowsParams& q, dim3 grid) {
    hipLaunchKernelGGL((dispatch_kernel<T>), grid, dim3(kThreads), 0, stream, q, chunks);
  });
}

template <class T>
te_status run_combine(const RowsParams& p, hipStream_t stream) {
  const int chunks = (p.cols + kChunk - 1) / kChunk;
  return in_parts(p, (p.tokens * chunks + kThreads - 1) / kThreads, [&](const RowsParams& q, dim3 grid) {
    hipLaunchKernelGGL((combine_kernel<T>), grid, dim3(kThreads), 0, stream, q, chunks);
  });
}

template <class T>
te_status run_combine_backward(const RowsParams& p, hipStream_t stream) {
  const int64_t per = kThreads / 64;
  return in_parts(p, (p.tokens * p.topk + per - 1) / per, [&](const RowsParams& q, dim3 grid) {
    hipLaunchKernelGGL((combine_backward_kernel<T>), grid, dim3(kThreads), 0, stream, q);
  });
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
