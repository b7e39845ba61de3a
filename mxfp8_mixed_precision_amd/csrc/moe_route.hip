// The router of a mixture-of-experts block and the sort of its slots by expert, for gfx950.
//
// With l the logits of a token and s_e = softmax(l)_e over its experts that are not masked (l_e > -inf), or
// sigmoid(l_e), the chosen experts e_0, e_1, .. are the topk largest of s_e + bias_e (of l_e without a bias: the
// scores rise with the logits) in falling order, equal ones in rising order of e, and
//   w_k = scale s_{e_k} / S,   S = sum over the chosen of s, or 1 (normalize = 0).
// Backward, with g_k = scale dw_k and v_k = w_k / scale:
//   normalize:  d_k = v_k (g_k - sum_j g_j v_j);   softmax: dl = d of the chosen;  sigmoid: dl = d (1 - s) of the chosen
//   normalize = 0:  sigmoid: dl_e = g_e s_e (1 - s_e);  softmax: dl_e = s_e (g_e - sum_j g_j s_j)
// Shares do not change if all scores are divided by e^c: softmax takes c so that the largest is 1, sigmoid the largest
// chosen logit where that is below 0, so that scores that no float holds (logits below -104) have their shares.
//
// A token's experts lie in the registers of 16 lanes (more than 256 experts or 16 slots: 64); a slot is a maximum
// over them.  The forward is bound by its instructions: 16384 tokens of 256 experts, 8 chosen, sigmoid, take 12 us with
// a bias (6.9 us of vector instructions, then the waves that compare near sums exactly), 8.6 (bf16) and 10.2
// (fp32) without, where the logits alone take 1.7 and 3.3.  With 64-bit keys for all and a maximum and a minimum a slot the
// same took 20 us.  The backward reads and writes the logits' tensor at 2.8 TB/s (16384 x 256 fp32 softmax shares: 12.4
// us): accesses of 4 or 2 bytes a lane, and the slots' way through LDS between two barriers.
#include <algorithm>
#include <type_traits>

#include "row_chunks.h"

namespace temx {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 64;
constexpr int kNoExpert = 0x7FFFFFFF;

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* experts;        // written by the forward, read by the backward
  float* weights;          // forward
  const float* dweights;   // backward
  void* dlogits;           // backward
  int64_t token0, tokens;  // a launch's first token, the one behind its last
  int num_experts, topk;
  float scale;
  bool sigmoid, normalize;
};

template <class T>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) { return to_float(static_cast<const T*>(p)[i]); }
template <>
__device__ __forceinline__ float load_logit<float>(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }

constexpr float kInf = __builtin_huge_valf();

// e^-c / (1 + e^-x), c <= 0 and c >= x where it is not 0: in range for every x.
__device__ __forceinline__ float sigmoid_of(float x, float c) {
  return (x < 0.f ? expf(x - c) : 1.0f) / (1.0f + expf(-fabsf(x)));
}
// The derivative of 1 / (1 + e^-x), without cancellation on either side.
__device__ __forceinline__ float sigmoid_slope(float x) {
  const float e = expf(-fabsf(x));
  return e / ((1.0f + e) * (1.0f + e));
}

// e^x by the hardware's 2^x: to (|x| + 2) 2^-23 relative.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// The topk largest keys of a token's LANES lanes, V a lane (expert v LANES + lane), a round each: the largest key, then
// the lowest expert that has it, which lane k keeps.
template <int LANES, int V, class Key>
__device__ __forceinline__ int choose(Key (&key)[V], int topk) {
  constexpr Key kNone = -(Key)kInf;
  const int lane = threadIdx.x % LANES;
  int mine = -1;
  for (int k = 0; k < topk; ++k) {
    Key best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = best > key[v] ? best : key[v];  // keys are never NaN
    best = lanes_all<LANES>(best, [](Key a, Key b) { return a > b ? a : b; });
    int e = kNoExpert;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) e = key[v] == best ? v * LANES + lane : e;
    e = lanes_all<LANES>(e, [](int a, int b) { return a < b ? a : b; });
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = v * LANES + lane == e ? kNone : key[v];
    if (lane == k) mine = best > kNone ? e : -1;
  }
  return mine;
}

// The same of keys of 22 bits above 1023 - expert (0: none), so that one maximum finds key and expert (a round 44
// instructions where `choose` takes 130, at V = 16).  `close`: whether two neighbours among the topk and the next one
// are less than `near` apart in a token of the wave; the rounds then go on until the last chosen and the next one are
// not, so that the experts that the lanes keep hold all that may belong to the topk.  false: not within LANES rounds.
template <int LANES, int V>
__device__ __forceinline__ bool choose_packed(uint32_t (&key)[V], int topk, uint32_t near, int& mine, bool& close) {
  const int lane = threadIdx.x % LANES;
  uint32_t before = 0;
  mine = -1;
  for (int k = 0;; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    best = lanes_all<LANES>(best, [](uint32_t a, uint32_t b) { return max(a, b); });
    const bool next = k > 0 && best != 0 && (before >> 10) - (best >> 10) < near;
    if (k <= topk) close |= __ballot(next) != 0;
    if (k >= topk && __ballot(next) == 0) return true;
    if (k == LANES) return false;
    before = best;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] == best ? 0 : key[v];
    if (lane == k && best != 0) mine = 1023 - (int)(best & 1023);
  }
}

// The place of the lane's expert among its LANES lanes' by their exact keys, equal ones by number; lanes without one
// keep theirs (the last).
template <int LANES, class Key>
__device__ __forceinline__ int place_of(Key key, int e) {
  const int lane = threadIdx.x % LANES, base = (threadIdx.x & 63) - lane;
  int place = e < 0 ? lane : 0;
#pragma unroll 4
  for (int i = 0; i < LANES; ++i) {
    const Key other = __shfl(key, base + i);
    const int other_e = __shfl(e, base + i);
    place += e >= 0 && other_e >= 0 && (other > key || (other == key && other_e < e));
  }
  return place;
}

// A logit of 16 bits as 16 bits that rise with it (both zeros one value).
__device__ __forceinline__ uint32_t rising_bits(uint32_t h) {
  h = h == 0x8000u ? 0u : h;
  return (h & 0x8000u) ? 0xFFFFu - h : h | 0x8000u;
}

// The choice is made on keys of 22 bits.  Logits of 16 bits are whole in them, and equal keys are equal logits.  fp32
// logits are compared by their distance from the largest, in steps of 2^-18, and sums with a bias in steps of 2^-20
// (off by less than 2^-18: the score by at most 48 roundings of 2^-24, the sum by two, the step); where two that
// matter are not told apart by that (fp32: one step; sums: 9 steps), the candidates are put in order by the logits
// themselves or by sums in 64 bits (two sums may lie closer than 32 bits tell apart); too many candidates: all
// experts are, the slow way, whose waves a launch waits for.  us at 16384 x 256, 8 chosen, sigmoid, normal logits with
// a bias, with a bias of zeros (bf16 logits tie), and where all are the same: bf16 11.7, 13.1, 28.1 (softmax 13.5, 16.9,
// 31.4); fp32 12.4, 12.5, 28.8.  Without a bias bf16 takes 8.6 whatever the logits, fp32 10.2, 19.4 where all are equal.
template <class T, int LANES, int V, bool BIAS>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteParams p) {
  constexpr bool kWhole = !BIAS && sizeof(T) == 2;
  constexpr uint32_t kMostKey = (1u << 22) - 1;
  const int lane = threadIdx.x % LANES;
  const int64_t token = p.token0 + (int64_t)blockIdx.x * (kRouteThreads / LANES) + threadIdx.x / LANES;
  const bool ok = token < p.tokens;  // every lane takes part in the exchanges
  const int64_t at = (ok ? token : 0) * p.num_experts;
  const auto sum = [](auto a, auto b) { return a + b; };
  const auto most = [](float a, float b) { return fmaxf(a, b); };

  float l[V];
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = load_logit<T>(p.logits, at + min(v * LANES + lane, p.num_experts - 1));
  float bias[BIAS ? V : 1];
  if constexpr (BIAS) {
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = p.bias[min(v * LANES + lane, p.num_experts - 1)];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = v * LANES + lane < p.num_experts ? l[v] : -kInf;
  float top = 0.f, total = 1.f;  // the largest logit; softmax: sum of e^(l - top)
  if (!kWhole || !(p.sigmoid || p.normalize)) {
    float m = -kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);
    m = lanes_all<LANES>(m, most);
    top = m > -kInf ? m : 0.f;
  }
  if (!p.sigmoid && (BIAS || !p.normalize)) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += fast_exp(l[v] - top);
    total = lanes_all<LANES>(s, sum);
  }
  bool close = false;
  if constexpr (BIAS) {
    float k[V];
    if (p.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) k[v] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[v])) + bias[v];
    } else {
      const float inv = 1.0f / total;
#pragma unroll
      for (int v = 0; v < V; ++v) k[v] = __builtin_fmaf(fast_exp(l[v] - top), inv, bias[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {  // -2 .. 2, what lies outside at the ends; NaN and -inf: left out
      const float f = fminf(fmaxf(__builtin_fmaf(k[v], 0x1p20f, 0x1p21f), 1.f), (float)kMostKey);
      key[v] = l[v] > -kInf && k[v] > -kInf ? (uint32_t)f << 10 | (1023 - (v * LANES + lane)) : 0u;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint32_t u;
      if constexpr (kWhole) u = 1 + rising_bits(__builtin_bit_cast(uint16_t, from_float<T>(l[v])));
      else u = (uint32_t)fminf(fmaxf((16.f - (top - l[v])) * 0x1p18f, 1.f), (float)kMostKey);
      key[v] = l[v] > -kInf ? u << 10 | (1023 - (v * LANES + lane)) : 0u;
    }
    if constexpr (!kWhole) close = __ballot(top == kInf) != 0;  // no distances: all keys are the lowest
  }
  int mine, slot = lane;
  const bool listed = choose_packed<LANES, V>(key, p.topk, kWhole ? 0u : BIAS ? 9u : 1u, mine, close);
  if (!kWhole && close) {
    double sum64 = 1.0;
    if (BIAS && !p.sigmoid) {
      sum64 = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) sum64 += exp((double)l[v] - (double)top);
      sum64 = lanes_all<LANES>(sum64, sum);
    }
    const auto exact = [&](float x, float b) {
      if constexpr (!BIAS) return x;
      else return (p.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / sum64) + (double)b;
    };
    typedef std::conditional_t<BIAS, double, float> Key;
    if (listed) {
      const Key own = mine < 0 ? -(Key)kInf : exact(load_logit<T>(p.logits, at + mine), BIAS ? p.bias[mine] : 0.f);
      slot = place_of<LANES>(own, mine);
      if (slot >= p.topk) mine = -1;
    } else {
      Key all[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Key k = exact(l[v], BIAS ? bias[v] : 0.f);
        all[v] = l[v] > -kInf && k > -(Key)kInf ? k : -(Key)kInf;
      }
      mine = choose<LANES, V>(all, p.topk);
    }
  }

  const float mine_l = mine >= 0 ? load_logit<T>(p.logits, at + mine) : -kInf;
  if (p.normalize) {
    const float m = lanes_all<LANES>(mine_l, most);
    top = m > -kInf ? m : 0.f;
  }
  float w = 0.f;
  if (mine >= 0) w = p.sigmoid ? sigmoid_of(mine_l, p.normalize ? fminf(top, 0.f) : 0.f) : expf(mine_l - top);
  if (p.normalize) total = lanes_all<LANES>(w, sum);
  if (mine >= 0 && (p.normalize || !p.sigmoid)) w /= total;  // the total of a token with a NaN logit may be NaN
  if (ok && slot < p.topk) {
    p.experts[token * p.topk + slot] = mine;
    p.weights[token * p.topk + slot] = p.scale * w;
  }
}

// LANES lanes a token as in the forward.  The slots' gradients meet the experts' lanes in LDS (two slots that name one
// expert are added).
template <class T, int LANES, int V>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteParams p) {
  __shared__ float slots[kRouteThreads / LANES][V * LANES];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int64_t token = p.token0 + (int64_t)blockIdx.x * (kRouteThreads / LANES) + group;
  const bool ok = token < p.tokens;
  const int64_t at = (ok ? token : 0) * p.num_experts;
  const auto sum = [](float a, float b) { return a + b; };
  const auto most = [](float a, float b) { return fmaxf(a, b); };
#pragma unroll
  for (int v = 0; v < V; ++v) slots[group][v * LANES + lane] = 0.f;

  int e = -1;
  float g = 0.f, l = -kInf;
  if (ok && lane < p.topk) {
    e = p.experts[token * p.topk + lane];
    if ((unsigned)e >= (unsigned)p.num_experts) e = -1;
    if (e >= 0) {
      g = p.scale * p.dweights[token * p.topk + lane];
      l = load_logit<T>(p.logits, at + e);
    }
  }
  const bool all = !p.sigmoid && !p.normalize;  // every expert's logit has a gradient
  float x[V], top = 0.f, total = 1.f;
  if (all) {
    float m = -kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = v * LANES + lane < p.num_experts ? load_logit<T>(p.logits, at + v * LANES + lane) : -kInf;
      m = fmaxf(m, x[v]);
    }
    m = lanes_all<LANES>(m, most);
    top = m > -kInf ? m : 0.f;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = expf(x[v] - top);
      s += x[v];
    }
    total = lanes_all<LANES>(s, sum);
    total = total == 0.f ? 1.f : total;
  } else if (p.normalize) {
    const float m = lanes_all<LANES>(l, most);
    top = m > -kInf ? m : 0.f;
  }
  float c = 0.f;  // what every expert subtracts
  if (p.normalize) {
    // the slot's score, up to the factor that cancels, and its share
    float s = e < 0 ? 0.f : p.sigmoid ? sigmoid_of(l, fminf(top, 0.f)) : expf(l - top);
    const float S = lanes_all<LANES>(s, sum);
    s = S == 0.f ? 0.f : s / S;
    const float gw = lanes_all<LANES>(g * s, sum);
    g = e < 0 ? 0.f : (g - gw) * s;
    if (p.sigmoid && e >= 0) g *= sigmoid_of(-l, 0.f);
  } else if (p.sigmoid) {
    if (e >= 0) g *= sigmoid_slope(l);
  } else {
    c = lanes_all<LANES>(e < 0 ? 0.f : g * (expf(l - top) / total), sum);
  }
  __syncthreads();
  if (e >= 0) atomicAdd(&slots[group][e], g);
  __syncthreads();
  if (!ok) return;
  T* out = static_cast<T*>(p.dlogits) + at;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = v * LANES + lane;
    if (j >= p.num_experts) continue;
    const float d = slots[group][j];
    out[j] = from_float<T>(all ? x[v] / total * (d - c) : d);
  }
}

// ---- the sort ---------------------------------------------------------------

// A stable counting sort: the slots in runs, a workgroup each; a run's slots in parts, a wave each.  Up to 2048 slots
// one launch, else two: no atomics on memory, so the rows do not depend on the schedule.  131072 slots over 256
// experts: 5 + 9 us, latencies of a few dependent steps (1.6 MB move); with the counts added up by a thread an expert
// the second launch took 28.
constexpr int kSortWaves = 8;
constexpr int kSortThreads = 64 * kSortWaves;
constexpr int kSortRun = 2048;    // slots of a workgroup, more where kSortBlocks of them do not suffice
constexpr int kSortBlocks = 256;

int64_t sort_run(int64_t slots) {
  const int64_t run = (slots + kSortBlocks - 1) / kSortBlocks;
  return run <= kSortRun ? kSortRun : (run + kSortRun - 1) / kSortRun * kSortRun;
}
int64_t sort_blocks(int64_t slots) { return (slots + sort_run(slots) - 1) / sort_run(slots); }

struct SortParams {
  const int32_t* experts;
  int32_t* m_splits;
  int32_t* row_of;
  int32_t* slot_of;
  int32_t* counts;  // [blocks][num_experts], of the runs (more than one)
  int64_t slots, run;
  int num_experts, blocks;
};

// Each run's slots per expert.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams p) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < p.num_experts; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * p.run, end = min(begin + p.run, p.slots);
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const int e = p.experts[i];
    if ((unsigned)e < (unsigned)p.num_experts) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.num_experts; e += kSortThreads)
    p.counts[(int64_t)blockIdx.x * p.num_experts + e] = count[e];
}

// Lanes of the wave whose value equals the lane's own, in the low `bits` bits.
__device__ __forceinline__ uint64_t same_lanes(int v, int bits) {
  uint64_t same = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((v >> b) & 1);
    same &= (v >> b) & 1 ? set : ~set;
  }
  return same;
}

// The rows of a run's slots: the rows of smaller experts, of the expert's slots in earlier runs, in the run's earlier
// parts and in the part before the slot.  Every workgroup adds up the counts it needs by itself.  ONE: a run of
// kSortRun slots, whose experts stay in registers.
template <bool ONE>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortParams p) {
  constexpr int kMine = ONE ? kSortRun / kSortThreads : 1;  // slots of a lane
  __shared__ int part[kSortWaves][kMaxExperts];  // slots of a wave's part; then the next row of each expert in it
  __shared__ int totals[kMaxExperts], befores[kMaxExperts];  // slots of an expert: in all, in earlier runs
  __shared__ int wave_sum[kSortWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, E = p.num_experts;
  const int64_t begin = blockIdx.x * p.run, share = p.run / kSortWaves;
  const int64_t part_begin = begin + wave * share, part_end = min(part_begin + share, p.slots);
  int mine[kMine];
  if constexpr (ONE) {
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int64_t i = part_begin + 64 * j + lane;
      mine[j] = i < part_end ? p.experts[i] : -1;
    }
  }
  for (int e = threadIdx.x; e < kSortWaves * kMaxExperts; e += kSortThreads) {
    if (e % kMaxExperts < E) part[0][e] = 0;
  }
  for (int e = threadIdx.x; e < E; e += kSortThreads) totals[e] = befores[e] = 0;
  __syncthreads();
  if constexpr (ONE) {
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if ((unsigned)mine[j] < (unsigned)E) atomicAdd(&part[wave][mine[j]], 1);
  } else {
    for (int64_t i = part_begin + lane; i < part_end; i += 64) {
      const int e = p.experts[i];
      if ((unsigned)e < (unsigned)E) atomicAdd(&part[wave][e], 1);
    }
  }
  if (p.blocks > 1) {  // threads side by side take one run's experts, or a part of them
    const int side = min(E, kSortThreads), lines = kSortThreads / side, line = threadIdx.x / side;
    for (int e = threadIdx.x % side; line < lines && e < E; e += side) {
      int all = 0, before = 0;
#pragma unroll 8
      for (int b = line; b < p.blocks; b += lines) {
        const int c = p.counts[(int64_t)b * E + e];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
      atomicAdd(&totals[e], all);
      atomicAdd(&befores[e], before);
    }
  }
  __syncthreads();
  // two experts a thread: 2 t, 2 t + 1
  int total[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * threadIdx.x + j;
    if (e >= E) continue;
    if (p.blocks > 1) {
      total[j] = totals[e];
    } else {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) total[j] += part[w][e];
    }
  }
  // rows of the smaller experts: a scan over the threads
  int scan = total[0] + total[1];
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(scan, d);
    scan += lane >= d ? up : 0;
  }
  if (lane == 63) wave_sum[wave] = scan;
  __syncthreads();
  int rows = 0, first = scan - total[0] - total[1];
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    first += w < wave ? wave_sum[w] : 0;
    rows += wave_sum[w];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * threadIdx.x + j;
    if (e >= E) continue;
    if (blockIdx.x == 0) p.m_splits[e] = total[j];
    int row = first + (j == 1 ? total[0] : 0) + befores[e];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = part[w][e];
      part[w][e] = row;
      row += n;
    }
  }
  __syncthreads();
  int bits = 1;
  while ((1 << bits) <= E) ++bits;  // the experts and one more value
  const auto place = [&](int64_t i, int e) {
    const bool valid = (unsigned)e < (unsigned)E;
    e = valid ? e : E;
    const uint64_t same = same_lanes(e, bits);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = -1;
    if (valid) {
      row = part[wave][e] + rank;
      p.slot_of[row] = (int)i;
    }
    __builtin_amdgcn_wave_barrier();
    if (valid && rank == 0) part[wave][e] = row + __popcll(same);
    if (i < part_end) p.row_of[i] = row;
    __builtin_amdgcn_wave_barrier();
  };
  if constexpr (ONE) {
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (part_begin + 64 * j < part_end) place(part_begin + 64 * j + lane, mine[j]);
  } else {
    for (int64_t i = part_begin + lane; i - lane < part_end; i += 64) place(i, i < part_end ? p.experts[i] : -1);
  }
  for (int64_t r = begin + threadIdx.x; r < min(begin + p.run, p.slots); r += kSortThreads)
    if (r >= rows) p.slot_of[r] = -1;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMostTokens = (int64_t)1 << 25;  // of one launch: 2^31 threads and fewer

template <class T, int LANES, int V>
te_status launch_route(RouteParams p, bool backward, hipStream_t stream) {
  constexpr int kPer = kRouteThreads / LANES;
  const int64_t tokens = p.tokens;
  for (p.token0 = 0; p.token0 < tokens; p.token0 += kMostTokens) {
    p.tokens = std::min(tokens, p.token0 + kMostTokens);
    const dim3 grid((unsigned)((p.tokens - p.token0 + kPer - 1) / kPer)), block(kRouteThreads);
    if (backward) hipLaunchKernelGGL((route_backward_kernel<T, LANES, V>), grid, block, 0, stream, p);
    else if (p.bias != nullptr) hipLaunchKernelGGL((route_kernel<T, LANES, V, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_kernel<T, LANES, V, false>), grid, block, 0, stream, p);
    const te_status st = launch_status();
    if (st != TE_OK) return st;
  }
  return TE_OK;
}

template <class T>
te_status run_route(const RouteParams& p, bool backward, hipStream_t stream) {
  if (p.topk <= 16 && p.num_experts <= 256) {
    if (p.num_experts <= 32) return launch_route<T, 16, 2>(p, backward, stream);
    if (p.num_experts <= 64) return launch_route<T, 16, 4>(p, backward, stream);
    if (p.num_experts <= 128) return launch_route<T, 16, 8>(p, backward, stream);
    return launch_route<T, 16, 16>(p, backward, stream);
  }
  if (p.num_experts <= 256) return launch_route<T, 64, 4>(p, backward, stream);
  if (p.num_experts <= 512) return launch_route<T, 64, 8>(p, backward, stream);
  return launch_route<T, 64, 16>(p, backward, stream);
}

te_status run_route(const RouteParams& p, te_dtype dtype, bool backward, hipStream_t stream) {
  if (dtype == TE_BF16) return run_route<bf16_t>(p, backward, stream);
  if (dtype == TE_FP16) return run_route<f16_t>(p, backward, stream);
  return run_route<float>(p, backward, stream);
}

constexpr int64_t kMostSlots = ((int64_t)1 << 31) - 65536;

te_status check_route(te_score score, te_dtype dtype, int64_t tokens, int num_experts, int topk, int normalize,
                      float scale) {
  TE_REQUIRE(score == TE_SCORE_SOFTMAX || score == TE_SCORE_SIGMOID, TE_ERR_VALUE);
  TE_REQUIRE((normalize == 0 || normalize == 1) && fabsf(scale) <= 3.0e38f, TE_ERR_VALUE);
  TE_REQUIRE(dtype == TE_BF16 || dtype == TE_FP16 || dtype == TE_FP32, TE_ERR_DTYPE);
  TE_REQUIRE(num_experts >= 1 && num_experts <= kMaxExperts, TE_ERR_SHAPE);
  TE_REQUIRE(topk >= 1 && topk <= num_experts && topk <= kMaxTopk, TE_ERR_SHAPE);
  TE_REQUIRE(tokens >= 0 && tokens <= kMostSlots / topk, TE_ERR_SHAPE);
  return TE_OK;
}

}  // namespace
}  // namespace temx

using namespace temx;

extern "C" te_status te_moe_route(te_score score, const void* logits, te_dtype dtype, int64_t tokens,
                                  int32_t num_experts, int32_t topk, const float* bias, int normalize, float scale,
                                  int32_t* experts, float* weights, hipStream_t stream) {
  const te_status st = check_route(score, dtype, tokens, num_experts, topk, normalize, scale);
  if (st != TE_OK) return st;
  if (tokens == 0) return TE_OK;
  TE_REQUIRE(logits && experts && weights, TE_ERR_NULL);
  TE_REQUIRE(aligned16(logits) && aligned4(bias) && aligned4(experts) && aligned4(weights), TE_ERR_ALIGN);
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const RouteParams p{logits, bias, experts, weights, nullptr, nullptr, 0, tokens, num_experts, topk, scale,
                      score == TE_SCORE_SIGMOID, normalize != 0};
  return run_route(p, dtype, false, stream);
}

extern "C" te_status te_moe_route_backward(te_score score, const void* logits, te_dtype dtype, int64_t tokens,
                                           int32_t num_experts, int32_t topk, int normalize, float scale,
                                           const int32_t* experts, const float* dweights, void* dlogits,
                                           hipStream_t stream) {
  const te_status st = check_route(score, dtype, tokens, num_experts, topk, normalize, scale);
  if (st != TE_OK) return st;
  if (tokens == 0) return TE_OK;
  TE_REQUIRE(logits && experts && dweights && dlogits, TE_ERR_NULL);
  TE_REQUIRE(aligned16(logits) && aligned16(dlogits) && aligned4(experts) && aligned4(dweights), TE_ERR_ALIGN);
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const RouteParams p{logits, nullptr, const_cast<int32_t*>(experts), nullptr, dweights, dlogits, 0, tokens,
                      num_experts, topk, scale, score == TE_SCORE_SIGMOID, normalize != 0};
  return run_route(p, dtype, true, stream);
}

extern "C" size_t te_moe_sort_workspace_size(int64_t slots, int32_t num_experts) {
  if (slots <= 0 || slots > kMostSlots || num_experts < 1 || num_experts > kMaxExperts) return 0;
  // that of runs of kSortRun, which are more than the longer ones: a batch's workspace serves every smaller one
  const int64_t blocks = std::min<int64_t>((slots + kSortRun - 1) / kSortRun, kSortBlocks);
  return blocks == 1 ? 0 : (size_t)(blocks * num_experts) * sizeof(int32_t);
}

extern "C" te_status te_moe_sort(const int32_t* experts, int64_t slots, int32_t num_experts, int32_t* m_splits,
                                 int32_t* row_of, int32_t* slot_of, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  TE_REQUIRE(num_experts >= 1 && num_experts <= kMaxExperts, TE_ERR_SHAPE);
  TE_REQUIRE(slots >= 0 && slots <= kMostSlots, TE_ERR_SHAPE);
  TE_REQUIRE(m_splits != nullptr && (slots == 0 || (experts && row_of && slot_of)), TE_ERR_NULL);
  TE_REQUIRE(aligned4(experts) && aligned4(m_splits) && aligned4(row_of) && aligned4(slot_of), TE_ERR_ALIGN);
  const int blocks = slots == 0 ? 1 : (int)sort_blocks(slots);
  if (blocks > 1) {
    TE_REQUIRE(workspace != nullptr, TE_ERR_NULL);
    TE_REQUIRE(aligned4(workspace), TE_ERR_ALIGN);
    TE_REQUIRE(workspace_bytes >= te_moe_sort_workspace_size(slots, num_experts), TE_ERR_WORKSPACE);
  }
  TE_REQUIRE(device_is_gfx950(), TE_ERR_ARCH);
  const SortParams p{experts, m_splits, row_of, slot_of, static_cast<int32_t*>(workspace), slots, sort_run(slots),
                     num_experts, blocks};
  if (blocks > 1) {
    hipLaunchKernelGGL(sort_count_kernel, dim3(blocks), dim3(kSortThreads), 0, stream, p);
    const te_status st = launch_status();
    if (st != TE_OK) return st;
  }
  if (p.run == kSortRun) hipLaunchKernelGGL((sort_place_kernel<true>), dim3(blocks), dim3(kSortThreads), 0, stream, p);
  else hipLaunchKernelGGL((sort_place_kernel<false>), dim3(blocks), dim3(kSortThreads), 0, stream, p);
  return launch_status();
}
