// The choice of experts from the router's logits ("SGLang、NCCL 与 MoE EP",
// §2.3.1: topk_idx and topk_w, the dispatch's and the combine's inputs).
//
//   s = softmax(l) or 1 / (1 + exp(-l))      scores, fp32
//   c = s + bias                             what chooses; the bias never enters a weight
//   groups: experts in `groups` equal runs, each scored by its best c or by the
//           sum of its best two; the best `keep` runs stay
//   the K largest c of what stays, ties to the lowest id, in descending order
//   w = s[id], divided by max(sum, 1e-20) if renormalised, times scale
// A logit of -inf or NaN is masked: that expert is never chosen.  Where fewer
// than K can be chosen the rest of the row is id -1 (the dispatch's padding
// route) and weight 0, so a row with nothing left routes nowhere.
// Without a bias the scores rise strictly with the logits, so the logits
// choose: equal choices at any spread of the logits, and only the K chosen
// scores are computed.
//
// A warp takes a token: lane i holds the keys of experts [i*V, i*V + V) in
// registers, so the lowest lane with the largest key holds the lowest id.  The
// kernel is bound by instructions, not by its few bytes, so a choice is kept
// short: a warp maximum over the lanes' largest keys (redux on order-preserving
// integers) finds the lane; that lane's V keys are read from shared memory by V
// lanes at once, which find the expert, strike it out and give the lane its next
// largest by one more redux, where the lane alone would walk its registers.
// Scores are computed up front only where they choose (a bias, or sums of two);
// otherwise lane k computes the k-th chosen one at the end, from its logit.
// The two score functions are kernels of their own: the test for which, per
// expert, was a twelfth of the time.
//
// Measured: 16384 tokens x 256 experts (sigmoid, bias, the best 4 of 8 groups by
// sums of two, K = 8; 18 MB) take 17.3 us, 1 TB/s, at 3 instructions a clock: 990
// warp instructions a token, 264 of them the scores and the bias, 191 the groups,
// 35 each of the eight rounds, the rest loads, keys and outputs.  256 tokens x 64
// experts take 3.1 us, launch latency.  The lane with the maximum walking its own
// registers instead of shared memory: 23.5 us.
#include "common.cuh"
#include "kernels.h"

#include <algorithm>

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct TopkArgs {
  const void* logits;
  const float* bias;  // [E] or null
  int T, E, K;
  int sigmoid;
  int groups, keep, top;
  int renorm;
  float scale;
  void* idx;
  int idx64;
  float* w;
};

// Order-preserving key of c; 0 for what can never be chosen (-inf, NaN).
__device__ __forceinline__ uint32_t choice_key(float c) {
  const int u = __float_as_int(__fadd_rn(c, 0.f));   // -0 and +0 are one value
  return c > -INFINITY ? static_cast<uint32_t>(u ^ ((u >> 31) | static_cast<int>(0x80000000u))) : 0u;
}
template <typename LogitT>
__device__ __forceinline__ float logit_value(LogitT v) {
  if constexpr (sizeof(LogitT) == 2) return __uint_as_float(static_cast<uint32_t>(v) << 16);
  else return v;
}
// Words of a lane's V values in the warp's shared memory: 16-byte accesses of
// neighbouring lanes meet different banks.
__host__ __device__ constexpr int lane_words(int V) { return V >= 8 ? V + 4 : V; }
template <int V>
__device__ __forceinline__ int word_of(int e) { return e / V * lane_words(V) + e % V; }

// The lane's V values of a row of E, from e0 on, or `past` beyond it.  vec: whole
// 16-byte vectors (all V where those are shorter) end with the row and are
// aligned.  Otherwise long rows come in through the warp's shared memory, as a
// lane's own values are V apart from the next lane's: 600 experts 22 us without.
template <int V, typename T>
__device__ __forceinline__ void load_row(float* v, const T* row, int e0, int E, bool vec, float past,
                                         float* stage) {
  constexpr int kVec = V * static_cast<int>(sizeof(T)) >= 16 ? 16 / static_cast<int>(sizeof(T)) : V;
  const int lane = threadIdx.x & 31;
  if (kVec * sizeof(T) >= 4 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += kVec) {
      T raw[kVec];
      if (e0 + i < E) {
        if constexpr (kVec * sizeof(T) == 16)
          *reinterpret_cast<uint4*>(raw) = __ldg(reinterpret_cast<const uint4*>(row + e0 + i));
        else if constexpr (kVec * sizeof(T) == 8)
          *reinterpret_cast<uint2*>(raw) = __ldg(reinterpret_cast<const uint2*>(row + e0 + i));
        else if constexpr (kVec * sizeof(T) == 4)
          *reinterpret_cast<uint32_t*>(raw) = __ldg(reinterpret_cast<const uint32_t*>(row + e0 + i));
      }
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[i + k] = e0 + i < E ? logit_value(raw[k]) : past;
    }
  } else if constexpr (V >= 8) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 32 * i + lane;
      stage[word_of<V>(e)] = e < E ? logit_value(__ldg(row + e)) : past;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(stage + lane * lane_words(V) + i);
    __syncwarp();
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = e0 + i < E ? logit_value(__ldg(row + e0 + i)) : past;
  }
}
template <int V, typename T>
bool row_vectors(const T* rows, int E) {
  constexpr int kVec = V * static_cast<int>(sizeof(T)) >= 16 ? 16 / static_cast<int>(sizeof(T)) : V;
  return E % kVec == 0 && (reinterpret_cast<uintptr_t>(rows) & (kVec * sizeof(T) - 1)) == 0;
}

// 1 / (1 + exp(-l)): each step rounded to nearest.
__device__ __forceinline__ float sigmoid(float l) { return __frcp_rn(__fadd_rn(1.f, expf(-l))); }

// Best two of a group of experts.
struct Best {
  float a, b;
  __device__ void add(float v) {
    b = fmaxf(b, fminf(a, v));
    a = fmaxf(a, v);
  }
};

// The best two over each run of `lanes` (a power of two) lanes.
__device__ __forceinline__ Best best_of(Best best, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) {
    const float oa = __shfl_xor_sync(kFull, best.a, o), ob = __shfl_xor_sync(kFull, best.b, o);
    best.b = fmaxf(fmaxf(best.b, ob), fminf(best.a, oa));
    best.a = fmaxf(best.a, oa);
  }
  return best;
}

template <typename LogitT, int V, bool kSigmoid>
__global__ void router_topk_kernel(const TopkArgs a, const bool vec, const bool vec_bias) {
  extern __shared__ __align__(16) uint32_t s_keys[];   // [warps][32 * lane_words(V)]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  const int E = a.E, e0 = lane * V;
  constexpr int W = lane_words(V);
  uint32_t* keys = s_keys + warp * 32 * W;
  const LogitT* row = static_cast<const LogitT*>(a.logits) + static_cast<int64_t>(t) * E;
  const bool biased = a.bias != nullptr;
  const bool sums = a.groups > 1 && a.top == 2;   // groups by sums of two scores

  float l[V];
  load_row<V>(l, row, e0, E, vec, -INFINITY, reinterpret_cast<float*>(keys));
#pragma unroll
  for (int j = 0; j < V; ++j) l[j] = l[j] == l[j] ? l[j] : -INFINITY;   // NaN is masked
  // softmax: the maximum, and the sum of the exponentials (1 at the maximum
  // itself, so an infinite logit takes the whole weight).  Where the largest is
  // always among the chosen and the weights are renormalised, the sum cancels.
  float m = -INFINITY, den = 1.f;
  const bool need_sum = !kSigmoid && (biased || sums || !a.renorm);
  if (!kSigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, l[j]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  }
  auto score = [&](float x) -> float {   // for softmax before the division by the sum
    if (x == -INFINITY) return 0.f;
    if (kSigmoid) return sigmoid(x);
    return x == m ? 1.f : expf(x - m);
  };
  float s[V];
  if (need_sum || biased || sums) {
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = score(l[j]);
    if (need_sum) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) sum += s[j];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      den = fmaxf(sum, 1e-30f);
    }
  }
  // key: what chooses among experts; value: what a group is scored by
  uint32_t key[V];
  float value[V];
  if (biased) {
    float b[V];
    load_row<V>(b, a.bias, e0, E, vec_bias, 0.f, reinterpret_cast<float*>(keys));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (!kSigmoid) s[j] = __fdiv_rn(s[j], den);
      const float c = l[j] == -INFINITY ? -INFINITY : __fadd_rn(s[j], b[j]);
      key[j] = choice_key(c);
      value[j] = key[j] ? c : -INFINITY;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      key[j] = choice_key(l[j]);
      value[j] = sums ? (key[j] ? s[j] : -INFINITY) : l[j];
    }
  }

  if (a.groups > 1) {
    const int size = E / a.groups;
    const int span = size / V;   // lanes of a group, if groups begin and end with lanes
    const bool aligned = span * V == size && (span & (span - 1)) == 0 && V > 0;
    uint32_t gk = 0;   // lane g's (aligned: every lane's own) group
    Best best{-INFINITY, -INFINITY};
    if (aligned) {
#pragma unroll
      for (int j = 0; j < V; ++j) best.add(value[j]);
      best = best_of(best, span);
    } else {
      float* values = reinterpret_cast<float*>(keys);
      if constexpr (V >= 8) {
#pragma unroll
        for (int j = 0; j < V; j += 4)
          *reinterpret_cast<float4*>(values + lane * W + j) =
              make_float4(value[j], value[j + 1], value[j + 2], value[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) values[e0 + j] = value[j];
      }
      __syncwarp();
      // as many lanes a group as there are (a power of two), group after group
      const int log_lanes = __clz(a.groups - 1) - 27;
      const int g = lane >> log_lanes, lanes = 1 << log_lanes;
      if (g < a.groups)
        for (int i = lane & (lanes - 1); i < size; i += lanes)
          best.add(values[word_of<V>(g * size + i)]);
      __syncwarp();   // the keys take the values' place
      best = best_of(best, lanes);
      best.a = __shfl_sync(kFull, best.a, lane << log_lanes);   // lane g's own
      best.b = __shfl_sync(kFull, best.b, lane << log_lanes);
    }
    const bool mine = aligned ? e0 < E : lane < a.groups;
    if (mine) gk = choice_key(a.top == 2 && best.b > -INFINITY ? __fadd_rn(best.a, best.b) : best.a);
    if (aligned) {
      // the lowest lane with the best key is in the lowest such group
      const int log_span = __ffs(span) - 1, own = lane >> log_span;
      bool kept = false;
      for (int i = 0; i < a.keep; ++i) {
        const uint32_t top = __reduce_max_sync(kFull, gk);
        if (top == 0u) break;
        const int g = (__ffs(__ballot_sync(kFull, gk == top)) - 1) >> log_span;
        if (own == g) {
          kept = true;
          gk = 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = kept ? key[j] : 0u;
    } else {
      uint32_t kept = 0;
      for (int i = 0; i < a.keep; ++i) {
        const uint32_t top = __reduce_max_sync(kFull, gk);
        if (top == 0u) break;
        const int g = __ffs(__ballot_sync(kFull, gk == top)) - 1;
        kept |= 1u << g;
        if (lane == g) gk = 0u;
      }
      int g = e0 / size, left = size - (e0 - g * size);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (e0 + j < E && !((kept >> g) & 1u)) key[j] = 0u;
        if (--left == 0) {
          left = size;
          ++g;
        }
      }
    }
  }

  uint32_t lm = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) lm = max(lm, key[j]);
  // the lane's keys, which V lanes read at once: no bank twice for V <= 32
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 4)
      *reinterpret_cast<uint4*>(keys + lane * W + j) = make_uint4(key[j], key[j + 1], key[j + 2], key[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) keys[e0 + j] = key[j];
  }
  __syncwarp();
  int id = -1;
  for (int k = 0; k < a.K; ++k) {
    const uint32_t top = __reduce_max_sync(kFull, lm);
    if (top == 0u) break;
    const int src = __ffs(__ballot_sync(kFull, lm == top)) - 1;
    uint32_t v = lane < V ? keys[src * W + lane] : 0u;
    const int j = __ffs(__ballot_sync(kFull, v == top)) - 1;
    if (lane == j) {
      v = 0u;
      keys[src * W + j] = 0u;
    }
    const uint32_t rest = __reduce_max_sync(kFull, v);
    if (lane == src) lm = rest;
    if (lane == k) id = src * V + j;
    __syncwarp();
  }
  float w = 0.f;
  if (id >= 0) {
    const float x = logit_value(__ldg(row + id));
    w = score(x);
    if (need_sum) w = __fdiv_rn(w, den);
  }
  if (a.renorm) {
    float tot = w;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) tot += __shfl_xor_sync(kFull, tot, o);
    w = __fdiv_rn(w, fmaxf(tot, 1e-20f));
  }
  w *= a.scale;
  if (lane < a.K) {
    const int64_t o = static_cast<int64_t>(t) * a.K + lane;
    if (a.idx64) static_cast<int64_t*>(a.idx)[o] = id;
    else static_cast<int32_t*>(a.idx)[o] = id;
    a.w[o] = w;
  }
}

template <typename LogitT, int V>
cudaError_t launch_topk_v(const TopkArgs& a, cudaStream_t s) {
  constexpr int warps = 8;   // tokens of a block: 16384 x 64 9.1 us (one token a block 11.7, 256 tokens 3.3 and 3.4)
  const int grid = (a.T + warps - 1) / warps;
  const bool vec = row_vectors<V>(static_cast<const LogitT*>(a.logits), a.E);
  const bool vec_bias = row_vectors<V>(a.bias, a.E);
  auto* kernel = a.sigmoid ? router_topk_kernel<LogitT, V, true> : router_topk_kernel<LogitT, V, false>;
  kernel<<<grid, warps * 32, warps * 32 * lane_words(V) * 4, s>>>(a, vec, vec_bias);
  return cudaGetLastError();
}

template <typename LogitT>
cudaError_t launch_topk(const TopkArgs& a, cudaStream_t s) {
  return a.E <= 32    ? launch_topk_v<LogitT, 1>(a, s)
         : a.E <= 64  ? launch_topk_v<LogitT, 2>(a, s)
         : a.E <= 128 ? launch_topk_v<LogitT, 4>(a, s)
         : a.E <= 256 ? launch_topk_v<LogitT, 8>(a, s)
         : a.E <= 512 ? launch_topk_v<LogitT, 16>(a, s)
                      : launch_topk_v<LogitT, 32>(a, s);
}

}  // namespace

cudaError_t launch_router_topk(const void* logits, int logits_bits, const float* bias, int T,
                               int E, int K, int sigmoid, int groups, int topk_groups,
                               int group_top, int renorm, float scale, void* topk_idx,
                               int idx_bits, float* topk_w, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const TopkArgs a{logits, bias, T, E, K, sigmoid, groups, topk_groups, group_top, renorm, scale,
                   topk_idx, idx_bits == 64 ? 1 : 0, topk_w};
  return logits_bits == 16 ? launch_topk<uint16_t>(a, s)
                           : launch_topk<float>(a, s);
}

}  // namespace moe
