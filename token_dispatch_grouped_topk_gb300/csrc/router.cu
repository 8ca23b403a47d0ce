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
// sums of two, K = 8; 18 MB) take 17.5 us, 1 TB/s, at 3 instructions a clock; 256
// tokens x 64 experts 3.3 us, launch latency.  The lane with the maximum walking
// its own registers instead of shared memory: 23.5 us.
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
// The lane's V logits; -inf past E and for NaN.
template <typename LogitT, int V>
__device__ __forceinline__ void load_logits(float* l, const LogitT* row, int e0, int E, bool vec) {
  constexpr int kBytes = V * static_cast<int>(sizeof(LogitT));
  LogitT raw[V];
  if (kBytes >= 4 && vec) {
    if (e0 < E) {
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
          reinterpret_cast<uint4*>(raw)[i] = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
      } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2*>(raw) = __ldg(reinterpret_cast<const uint2*>(row + e0));
      } else if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t*>(raw) = __ldg(reinterpret_cast<const uint32_t*>(row + e0));
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = e0 < E ? logit_value(raw[j]) : -INFINITY;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = e0 + j < E ? logit_value(__ldg(row + e0 + j)) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) l[j] = l[j] == l[j] ? l[j] : -INFINITY;
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

template <typename LogitT, int V, bool kSigmoid>
__global__ void router_topk_kernel(const TopkArgs a, const bool vec, const bool vec_bias) {
  extern __shared__ __align__(16) uint32_t s_keys[];   // [warps][32 * V]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  const int E = a.E, e0 = lane * V;
  uint32_t* keys = s_keys + warp * 32 * V;
  const LogitT* row = static_cast<const LogitT*>(a.logits) + static_cast<int64_t>(t) * E;
  const bool biased = a.bias != nullptr;
  const bool sums = a.groups > 1 && a.top == 2;   // groups by sums of two scores

  float l[V];
  load_logits<LogitT, V>(l, row, e0, E, vec);
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
    if (V % 4 == 0 && vec_bias) {
      if (e0 < E) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
          reinterpret_cast<float4*>(b)[j] = __ldg(reinterpret_cast<const float4*>(a.bias + e0) + j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) b[j] = e0 + j < E ? __ldg(a.bias + e0 + j) : 0.f;
    }
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
      for (int o = 1; o < span; o <<= 1) {
        const float oa = __shfl_xor_sync(kFull, best.a, o), ob = __shfl_xor_sync(kFull, best.b, o);
        best.b = fmaxf(fmaxf(best.b, ob), fminf(best.a, oa));
        best.a = fmaxf(best.a, oa);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e0 + j < E) reinterpret_cast<float*>(keys)[e0 + j] = value[j];
      __syncwarp();
      if (lane < a.groups)
        for (int i = 0; i < size; ++i) best.add(reinterpret_cast<float*>(keys)[lane * size + i]);
      __syncwarp();
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
      *reinterpret_cast<uint4*>(keys + e0 + j) = make_uint4(key[j], key[j + 1], key[j + 2], key[j + 3]);
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
    uint32_t v = lane < V ? keys[src * V + lane] : 0u;
    const int j = __ffs(__ballot_sync(kFull, v == top)) - 1;
    if (lane == j) {
      v = 0u;
      keys[src * V + j] = 0u;
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
  constexpr int kBytes = V * static_cast<int>(sizeof(LogitT));
  const bool vec = a.E % V == 0 && (reinterpret_cast<uintptr_t>(a.logits) & (std::min(kBytes, 16) - 1)) == 0;
  const bool vec_bias = V % 4 == 0 && a.E % V == 0 && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0;
  auto* kernel = a.sigmoid ? router_topk_kernel<LogitT, V, true> : router_topk_kernel<LogitT, V, false>;
  kernel<<<grid, warps * 32, warps * 32 * V * 4, s>>>(a, vec, vec_bias);
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
