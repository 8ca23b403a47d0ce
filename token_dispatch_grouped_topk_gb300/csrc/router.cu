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
// A warp takes a token: lane i holds experts [i*V, i*V + V) in registers, so
// the lowest lane with the largest value holds the lowest id.  A choice is a
// warp maximum (redux on order-preserving integer keys) and a ballot.
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
  if (!(c > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(__fadd_rn(c, 0.f));   // -0 and +0 are one value
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0u) return -INFINITY;
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <typename LogitT>
__device__ __forceinline__ float load_logit(const LogitT* p) {
  if constexpr (sizeof(LogitT) == 2) return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
  else return __ldg(p);
}

__device__ __forceinline__ float sigmoid(float l) {
  return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-l)));
}

template <typename LogitT, int V>
__global__ void router_topk_kernel(const TopkArgs a) {
  extern __shared__ float s_val[];   // straddling groups: [warps][E]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  const int E = a.E, e0 = lane * V;
  const LogitT* row = static_cast<const LogitT*>(a.logits) + static_cast<int64_t>(t) * E;

  float l[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    l[j] = -INFINITY;
    if (e0 + j < E) {
      const float v = load_logit(row + e0 + j);
      l[j] = v == v ? v : -INFINITY;
    }
  }
  // softmax: the maximum and the sum; e = 1 at the maximum itself, so an
  // infinite logit takes the whole weight
  float m = -INFINITY, den = 1.f;
  if (!a.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, l[j]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  }
  // s: the score, for softmax before the division by the sum
  float s[V];
  uint32_t key[V];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (l[j] == -INFINITY) s[j] = 0.f;
    else if (a.sigmoid) s[j] = sigmoid(l[j]);
    else s[j] = l[j] == m ? 1.f : expf(l[j] - m);
    sum += s[j];
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    den = fmaxf(sum, 1e-30f);
  }
  float gval[V];   // what groups are scored by when two entries are added
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float c = l[j];
    gval[j] = l[j] == -INFINITY ? -INFINITY : s[j];
    if (a.bias != nullptr && l[j] != -INFINITY) {
      if (!a.sigmoid) s[j] = __fdiv_rn(s[j], den);
      c = gval[j] = __fadd_rn(s[j], __ldg(a.bias + e0 + j));
    }
    key[j] = choice_key(c);
    if (key[j] == 0u) gval[j] = -INFINITY;
    if (a.top == 1) gval[j] = key_value(key[j]);
  }
  if (a.bias != nullptr) den = 1.f;

  if (a.groups > 1) {
    const int size = E / a.groups;
    float* sv = s_val + warp * E;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e0 + j < E) sv[e0 + j] = gval[j];
    __syncwarp();
    float b1 = -INFINITY, b2 = -INFINITY;
    if (lane < a.groups) {
      for (int i = 0; i < size; ++i) {
        const float v = sv[lane * size + i];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
    }
    uint32_t gk = choice_key(a.top == 2 && b2 > -INFINITY ? __fadd_rn(b1, b2) : b1);
    if (lane >= a.groups) gk = 0u;
    uint32_t kept = 0;
    for (int i = 0; i < a.keep; ++i) {
      const uint32_t best = __reduce_max_sync(kFull, gk);
      if (best == 0u) break;
      const int src = __ffs(__ballot_sync(kFull, gk == best)) - 1;
      kept |= 1u << src;
      if (lane == src) gk = 0u;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e0 + j < E && !((kept >> ((e0 + j) / size)) & 1u)) key[j] = 0u;
  }

  uint32_t lm = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) lm = max(lm, key[j]);
  int id = -1;
  float w = 0.f;
  for (int k = 0; k < a.K; ++k) {
    const uint32_t best = __reduce_max_sync(kFull, lm);
    if (best == 0u) break;
    const int src = __ffs(__ballot_sync(kFull, lm == best)) - 1;
    int jj = 0;
    float sj = 0.f;
    if (lane == src) {
      bool found = false;
      lm = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!found && key[j] == best) {
          found = true;
          jj = j;
          sj = s[j];
          key[j] = 0u;
        }
        lm = max(lm, key[j]);
      }
    }
    const int got = __shfl_sync(kFull, e0 + jj, src);
    const float gw = __shfl_sync(kFull, sj, src);
    if (lane == k) {
      id = got;
      w = gw;
    }
  }
  w = __fdiv_rn(w, den);
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
    a.w[o] = id < 0 ? 0.f : w;
  }
}

template <typename LogitT>
cudaError_t launch_topk(const TopkArgs& a, int sm_count, cudaStream_t s) {
  const int warps = a.T >= 8 * sm_count ? 8 : a.T >= 2 * sm_count ? 4 : 1;
  const int grid = (a.T + warps - 1) / warps;
  const size_t smem = a.groups > 1 ? static_cast<size_t>(warps) * a.E * sizeof(float) : 0;
  auto kernel = a.E <= 32    ? router_topk_kernel<LogitT, 1>
                : a.E <= 64  ? router_topk_kernel<LogitT, 2>
                : a.E <= 128 ? router_topk_kernel<LogitT, 4>
                : a.E <= 256 ? router_topk_kernel<LogitT, 8>
                : a.E <= 512 ? router_topk_kernel<LogitT, 16>
                             : router_topk_kernel<LogitT, 32>;
  kernel<<<grid, warps * 32, smem, s>>>(a);   // at most 8 * 1024 * 4 bytes: 32 KB
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_router_topk(const void* logits, int logits_bits, const float* bias, int T,
                               int E, int K, int sigmoid, int groups, int topk_groups,
                               int group_top, int renorm, float scale, void* topk_idx,
                               int idx_bits, float* topk_w, int sm_count, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const TopkArgs a{logits, bias, T, E, K, sigmoid, groups, topk_groups, group_top, renorm, scale,
                   topk_idx, idx_bits == 64 ? 1 : 0, topk_w};
  return logits_bits == 16 ? launch_topk<uint16_t>(a, sm_count, s)
                           : launch_topk<float>(a, sm_count, s);
}

}  // namespace moe
