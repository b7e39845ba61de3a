// Rows of a tensor in chunks of 8 elements, as the kernels that stream rows (norms, experts' rows) move them; sums and
// other operations across the lanes of a row; the MXFP8 codes of a chunk.
#pragma once

#include <type_traits>

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

template <class T>
__device__ __forceinline__ Raw<T> load_whole(const T* p) {
  Raw<T> r;
#pragma unroll
  for (unsigned i = 0; i < sizeof(r.w) / 16; ++i) {
    const u32x4 v = reinterpret_cast<const typename Vec16<sizeof(T)>::type*>(p)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) r.w[4 * i + e] = v[e];
  }
  return r;
}

// Element e becomes element e + k, and 0 past the chunk's end (0 <= k < kChunk).
template <class T>
__device__ __forceinline__ void shift_down(Raw<T>& r, int k) {
  constexpr int kN = sizeof(r.w) / 4, kPer = 4 / sizeof(T);  // registers, elements of one
#pragma unroll
  for (int bit = kChunk / 2; bit >= kPer; bit >>= 1) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t from = i + bit / kPer < kN ? r.w[i + bit / kPer] : 0u;
      r.w[i] = (k & bit) ? from : r.w[i];
    }
  }
  if constexpr (kPer == 2) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t above = i + 1 < kN ? r.w[i + 1] : 0u;
      r.w[i] = (k & 1) ? (r.w[i] >> 16 | above << 16) : r.w[i];
    }
  }
}

// Chunk at element c of a row of n elements, in two halves (zeros past the row).  load_ahead loads a tail lane's
// chunk as the row's last kChunk elements, in the same instruction as every other lane's; settle, where the values
// are first used, shifts a tail into place.  With the shift next to
// the load a wave with a tail waited for each of its loads in turn (16384 x 1023 bf16 backward: 35 us that way).
// Rows shorter than a chunk go element by element.
template <class T>
__device__ __forceinline__ Raw<T> load_ahead(const T* row, int c, int n) {
  Raw<T> r;
#pragma unroll
  for (unsigned i = 0; i < sizeof(r.w) / 4; ++i) r.w[i] = 0;
  if (n >= kChunk) {
    if (c < n) r = load_whole(row + min(c, n - kChunk));
  } else if (c == 0) {
#pragma unroll 1
    for (int e = n - 1; e >= 0; --e) {  // the elements so far one place up, and this one in front
#pragma unroll
      for (int i = sizeof(r.w) / 4 - 1; i >= 0; --i) {
        const uint32_t below = i > 0 ? r.w[i - 1] : 0u;
        r.w[i] = sizeof(T) == 4 ? below : (r.w[i] << 16 | below >> 16);
      }
      if constexpr (sizeof(T) == 4) r.w[0] = __builtin_bit_cast(uint32_t, row[e]);
      else r.w[0] |= __builtin_bit_cast(uint16_t, row[e]);
    }
  }
  return r;
}

template <class T>
__device__ __forceinline__ void settle(Raw<T>& r, int c, int n) {
  const int k = c + kChunk - n;
  if (n >= kChunk && k > 0 && k < kChunk) shift_down<T>(r, k);
}

template <class T>
__device__ __forceinline__ Raw<T> load_chunk(const T* row, int c, int n) {
  Raw<T> r = load_ahead(row, c, n);
  settle<T>(r, c, n);
  return r;
}

// The chunk's registers as values the compiler knows nothing about.
template <class T>
__device__ __forceinline__ void opaque(Raw<T>& r) {
#pragma unroll
  for (unsigned i = 0; i < sizeof(r.w) / 4; ++i) asm volatile("" : "+v"(r.w[i]));
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
__device__ __forceinline__ void load_floats(const T* row, int c, int n, float (&f)[kChunk]) {
  unpack<T>(load_chunk(row, c, n), f);
}

// ---- sums across lanes -------------------------------------------------------

// Sum over the LANES (16, 32 or 64) lanes of a row group, in a fixed butterfly order: every lane ends with the same bits.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  auto ror = [](float x, auto n) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x120 + decltype(n)::value, 0xF, 0xF, false));
  };
  v += ror(v, std::integral_constant<int, 8>{});  // row_ror within 16 lanes
  v += ror(v, std::integral_constant<int, 4>{});
  v += ror(v, std::integral_constant<int, 2>{});
  v += ror(v, std::integral_constant<int, 1>{});
  if constexpr (LANES >= 32)
    v += __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));  // lane ^ 16
  if constexpr (LANES == 64) {
    const int lane = threadIdx.x & 63;
    v += __int_as_float(__builtin_amdgcn_ds_bpermute((lane ^ 32) << 2, __float_as_int(v)));  // lane ^ 32
  }
  return v;
}

// op over the values of the lane's LANES (16, 32 or 64) lanes, in every lane.
template <int LANES, class V, class Op>
__device__ __forceinline__ V lanes_all(V v, Op op) {
  constexpr int kWords = sizeof(V) / 4;
  struct Words {
    int w[kWords];
  };
  const auto ror = [](V x, auto n) {  // row_ror within 16 lanes
    Words u = __builtin_bit_cast(Words, x);
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      u.w[i] = __builtin_amdgcn_mov_dpp(u.w[i], 0x120 + decltype(n)::value, 0xF, 0xF, false);
    return __builtin_bit_cast(V, u);
  };
  v = op(v, ror(v, std::integral_constant<int, 8>{}));
  v = op(v, ror(v, std::integral_constant<int, 4>{}));
  v = op(v, ror(v, std::integral_constant<int, 2>{}));
  v = op(v, ror(v, std::integral_constant<int, 1>{}));
  if constexpr (LANES >= 32) {  // the two rows of 16 of each half
    Words a = __builtin_bit_cast(Words, v), b;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const u32x2 both = __builtin_amdgcn_permlane16_swap((unsigned)a.w[i], (unsigned)a.w[i], false, false);
      a.w[i] = (int)both[0], b.w[i] = (int)both[1];
    }
    v = op(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b));
  }
  if constexpr (LANES == 64) {
    Words a = __builtin_bit_cast(Words, v), b;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const u32x2 both = __builtin_amdgcn_permlane32_swap((unsigned)a.w[i], (unsigned)a.w[i], false, false);
      a.w[i] = (int)both[0], b.w[i] = (int)both[1];
    }
    v = op(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b));
  }
  return v;
}

// ---- MXFP8 output ---------------------------------------------------------------

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

}  // namespace
}  // namespace temx
