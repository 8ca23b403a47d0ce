// Routed experts for a few tokens with 4-bit weights: for every route of a
// token the gated-SiLU expert ("SGLang Expert Compute Backend", §1.1) as
// matrix-vector products, then the weighted sum over the token's routes
// ("SGLang、NCCL 与 MoE EP", §1.1):
//   g = W13[e, :I] x,  u = W13[e, I:] x,  z = SiLU(g) * u,  o = W2[e] z,
//   y[t] = bf16( sum over routes of w * o ).
// A weight is (code - 8) * scale: codes of 4 bits, two a byte (even element of
// K in the low bits), one BF16 scale per row and 128 elements of K.
//
// With a few tokens an active expert has a few rows, and the whole cost is
// reading its weights once; the products must only keep up with that stream.
// A warp takes 16 weight rows against 8 token columns with mma.sync m16n8k16
// (BF16 products, fp32 sums): the codes come straight from memory into the
// registers of the A operand, where a tensor-core tile fed from shared memory
// (tcgen05) would need the 128-row operand of dequantised weights written to
// and read from shared memory first, at four times the codes' bytes, for
// columns that are mostly empty.  A dot product may take K in any order, so
// each lane reads 16 consecutive bytes (32 codes) of its row and the token
// operand is permuted to match:
//   lane = 4 * r + q holds rows r and r + 8, codes [32q, 32q + 32) of a
//   128-group; word i of the four words gives the K pairs (8i + j, 8i + j + 4),
//   j = 0..3: nibbles j and j + 4 of one word are the halves of one register
//   after a shift and a mask.
// code - 8 is exact in BF16, so a group's sum is exact up to fp32 rounding and
// the scale multiplies it once per group, in fp32.
//
// Two launches: gate/up with the activation (z of every route, BF16, to the
// workspace), then down with the sum over routes.  z is rounded to BF16 to be
// the tensor core's operand, as the expert's input is.  Each block finds the
// active experts and their routes by itself from topk_idx.
#include "common.cuh"
#include "kernels.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = kW4Warps * 32;
constexpr int kCols = 8;     // token columns of one pass
constexpr int kRows = 16;    // weight rows of one warp tile
constexpr int kMaxRoutes = kW4MaxTokens * 32;

// The active experts in ascending order and their routes in ascending route id.
struct W4Plan {
  int off[1024 + 1];           // first route of each expert
  int pos[1024 + 1];           // scratch: counts, then next free place
  int act[1024 + 1];           // active experts (first: their prefix)
  uint16_t list[1024];         // the active experts' ids
  uint16_t route[kMaxRoutes];  // routes by expert
  int bad;
};

template <typename IdT>
__device__ void w4_plan(W4Plan* p, const IdT* __restrict__ topk_idx, int n, int E) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) p->pos[e] = 0;
  if (threadIdx.x == 0) p->bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int64_t id = static_cast<int64_t>(topk_idx[i]);
    if (id >= 0 && id < E) atomicAdd(&p->pos[id], 1);
    else if (id != -1) p->bad = 1;
  }
  __syncthreads();
  expert_prefix(p->pos, E, kMaxRoutes, 1, 1, p->off, nullptr);
  expert_prefix(p->pos, E, kMaxRoutes, kMaxRoutes, 1, p->act, nullptr);
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    if (p->off[e + 1] > p->off[e]) p->list[p->act[e]] = static_cast<uint16_t>(e);
    p->pos[e] = p->off[e];
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      int e = -1;
      if (i < n) {
        const int64_t id = static_cast<int64_t>(topk_idx[i]);
        if (id >= 0 && id < E) e = static_cast<int>(id);
      }
      const unsigned peers = __match_any_sync(0xffffffffu, e);
      if (e >= 0) p->route[p->pos[e] + __popc(peers & ((1u << lane) - 1u))] = static_cast<uint16_t>(i);
      __syncwarp();
      if (e >= 0 && lane == __ffs(peers) - 1) p->pos[e] += __popc(peers);
      __syncwarp();
    }
  }
  __syncthreads();
}

// Codes j and j + 4 of a word as the BF16 pair (code - 8): 0x4300 | code is
// the BF16 number 128 + code.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int j) {
  const uint32_t v = ((word >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ void mma_16x8x16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One row pair's codes and scales of one 128-group.
struct W4Group {
  uint4 lo, hi;
  uint16_t slo, shi;
};
__device__ __forceinline__ void w4_load(W4Group* w, const uint8_t* codes, const uint16_t* scales,
                                        int64_t row, int K, int g, int q) {
  const uint8_t* p = codes + row * (K / 2) + g * 64 + q * 16;
  w->lo = ld_stream(reinterpret_cast<const uint4*>(p));
  w->hi = ld_stream(reinterpret_cast<const uint4*>(p + 8 * static_cast<int64_t>(K / 2)));
  const uint16_t* s = scales + row * (K / kGroup) + g;
  w->slo = __ldg(s);
  w->shi = __ldg(s + 8 * (K / kGroup));
}

// The token operand of one 128-group: the lane's 32 elements of column r.
__device__ __forceinline__ void load_column(uint4* v, const uint16_t* row, int g, int q) {
  const uint4* p = reinterpret_cast<const uint4*>(row + g * kGroup + q * 32);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = row != nullptr ? p[i] : make_uint4(0, 0, 0, 0);
}

// acc += scale * (codes - 8) . column over one 128-group.
__device__ __forceinline__ void w4_dot(float* acc, const W4Group& w, const uint4* col) {
  float c[4] = {0.f, 0.f, 0.f, 0.f};
  const uint32_t lo[4] = {w.lo.x, w.lo.y, w.lo.z, w.lo.w};
  const uint32_t hi[4] = {w.hi.x, w.hi.y, w.hi.z, w.hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // elements (j, j + 4) of the column's eight
    const uint32_t b0 = __byte_perm(col[i].x, col[i].z, 0x5410);
    const uint32_t b1 = __byte_perm(col[i].x, col[i].z, 0x7632);
    const uint32_t b2 = __byte_perm(col[i].y, col[i].w, 0x5410);
    const uint32_t b3 = __byte_perm(col[i].y, col[i].w, 0x7632);
    mma_16x8x16(c, w4_pair(lo[i], 0), w4_pair(hi[i], 0), w4_pair(lo[i], 1), w4_pair(hi[i], 1), b0, b1);
    mma_16x8x16(c, w4_pair(lo[i], 2), w4_pair(hi[i], 2), w4_pair(lo[i], 3), w4_pair(hi[i], 3), b2, b3);
  }
  const float slo = __uint_as_float(static_cast<uint32_t>(w.slo) << 16);
  const float shi = __uint_as_float(static_cast<uint32_t>(w.shi) << 16);
  acc[0] = fmaf(slo, c[0], acc[0]);
  acc[1] = fmaf(slo, c[1], acc[1]);
  acc[2] = fmaf(shi, c[2], acc[2]);
  acc[3] = fmaf(shi, c[3], acc[3]);
}

struct W4Args {
  const uint16_t* x;    // BF16 [T, H]
  const void* topk_idx;
  const float* topk_w;  // [T, K]
  const uint8_t* w13;   // [E, 2I, H / 2]
  const uint16_t* s13;  // BF16 [E, 2I, H / 128]
  const uint8_t* w2;    // [E, H, I / 2]
  const uint16_t* s2;   // BF16 [E, H, I / 128]
  uint16_t* z;          // BF16 [T * K, I], by route
  uint16_t* y;          // BF16 [T, H]
  int32_t* dev_status;
  int T, H, I, K, E;
};

// Gate/up: an item is 16 gate rows and the same 16 up rows of one active
// expert; the block's warps split H.
template <typename IdT>
__global__ void __launch_bounds__(kW4Threads, 2) w4_gateup_kernel(const W4Args a) {
  __shared__ W4Plan plan;
  __shared__ float s_red[kW4Warps][2][kRows][kCols];
  w4_plan(&plan, static_cast<const IdT*>(a.topk_idx), a.T * a.K, a.E);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.dev_status[0] = plan.bad ? kDevBadExpertId : 0;
    a.dev_status[1] = 0;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, q = lane & 3;
  const int tiles = a.I / kRows;
  const int total = plan.act[a.E] * tiles;
  const int G = a.H / kGroup;
  const int g0 = G * warp / kW4Warps, g1 = G * (warp + 1) / kW4Warps;
  for (int it = blockIdx.x; it < total; it += gridDim.x) {
    const int e = plan.list[it / tiles], i0 = (it % tiles) * kRows;
    const int n = plan.off[e + 1] - plan.off[e];
    const uint16_t* routes = plan.route + plan.off[e];
    const int64_t row_g = static_cast<int64_t>(e) * 2 * a.I + i0 + r, row_u = row_g + a.I;
    for (int c0 = 0; c0 < n; c0 += kCols) {
      const uint16_t* xr =
          c0 + r < n ? a.x + static_cast<int64_t>(routes[c0 + r] / a.K) * a.H : nullptr;
      float ag[4] = {0.f, 0.f, 0.f, 0.f}, au[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
      for (int g = g0; g < g1; ++g) {
        W4Group wg, wu;
        uint4 col[4];
        w4_load(&wg, a.w13, a.s13, row_g, a.H, g, q);
        w4_load(&wu, a.w13, a.s13, row_u, a.H, g, q);
        load_column(col, xr, g, q);
        w4_dot(ag, wg, col);
        w4_dot(au, wu, col);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int rr = r + (j >> 1) * 8, cc = 2 * q + (j & 1);
        s_red[warp][0][rr][cc] = ag[j];
        s_red[warp][1][rr][cc] = au[j];
      }
      __syncthreads();
      if (threadIdx.x < kRows * kCols) {
        const int rr = threadIdx.x % kRows, cc = threadIdx.x / kRows;
        if (c0 + cc < n) {
          float gate = 0.f, up = 0.f;
#pragma unroll
          for (int w = 0; w < kW4Warps; ++w) {
            gate += s_red[w][0][rr][cc];
            up += s_red[w][1][rr][cc];
          }
          const float z = gate / (1.f + expf(-gate)) * up;
          a.z[static_cast<int64_t>(routes[c0 + cc]) * a.I + i0 + rr] =
              __bfloat16_as_ushort(__float2bfloat16_rn(z));
        }
      }
      __syncthreads();
    }
  }
}

// Down: an item is 16 rows of H for every active expert; the block's warps
// split the (expert, 128-group) units evenly and keep a sum per token.  The
// order of the sums is fixed by the routes alone.
template <typename IdT>
__global__ void __launch_bounds__(kW4Threads, 2) w4_down_kernel(const W4Args a) {
  __shared__ W4Plan plan;
  extern __shared__ float s_y[];   // [kW4Warps][T][kRows]
  w4_plan(&plan, static_cast<const IdT*>(a.topk_idx), a.T * a.K, a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, q = lane & 3;
  const int G = a.I / kGroup;
  const int units = plan.act[a.E] * G;   // at most 1024 * 128
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * warp / kW4Warps);
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (warp + 1) / kW4Warps);
  const int per = a.T * kRows;
  float* mine = s_y + warp * per;
  for (int it = blockIdx.x; it < a.H / kRows; it += gridDim.x) {
    const int h0 = it * kRows;
    for (int i = lane; i < per; i += 32) mine[i] = 0.f;
    __syncwarp();
    for (int u = u0; u < u1;) {
      const int e = plan.list[u / G];
      const int ga = u % G, gb = min(G, ga + (u1 - u));
      const int n = plan.off[e + 1] - plan.off[e];
      const uint16_t* routes = plan.route + plan.off[e];
      const int64_t row = static_cast<int64_t>(e) * a.H + h0 + r;
      for (int c0 = 0; c0 < n; c0 += kCols) {
        const uint16_t* zr =
            c0 + r < n ? a.z + static_cast<int64_t>(routes[c0 + r]) * a.I : nullptr;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int g = ga; g < gb; ++g) {
          W4Group w;
          uint4 col[4];
          w4_load(&w, a.w2, a.s2, row, a.I, g, q);
          load_column(col, zr, g, q);
          w4_dot(acc, w, col);
        }
        // column after column: a token may route to one expert twice
        for (int cc = 0; cc < min(kCols, n - c0); ++cc) {
          if (q == cc >> 1) {
            const int route = routes[c0 + cc];
            const float wt = a.topk_w[route];
            float* yt = mine + route / a.K * kRows;
            yt[r] = fmaf(wt, acc[cc & 1], yt[r]);
            yt[r + 8] = fmaf(wt, acc[2 + (cc & 1)], yt[r + 8]);
          }
          __syncwarp();
        }
      }
      u += gb - ga;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < per; i += kW4Threads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kW4Warps; ++w) v += s_y[w * per + i];
      a.y[static_cast<int64_t>(i / kRows) * a.H + h0 + i % kRows] =
          __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    __syncthreads();
  }
}

template <typename IdT>
cudaError_t launch_w4(const W4Args& a, int sm_count, cudaStream_t s) {
  const int gu = std::min(std::min(a.E, a.T * a.K) * (a.I / kRows), 2 * sm_count);
  w4_gateup_kernel<IdT><<<gu, kW4Threads, 0, s>>>(a);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const size_t smem = static_cast<size_t>(kW4Warps) * a.T * kRows * sizeof(float);
  err = cudaFuncSetAttribute(w4_down_kernel<IdT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kW4Warps * kW4MaxTokens * kRows * static_cast<int>(sizeof(float)));
  if (err != cudaSuccess) return err;
  w4_down_kernel<IdT><<<std::min(a.H / kRows, 2 * sm_count), kW4Threads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_experts_w4(const void* x, const void* topk_idx, int idx_bits,
                              const float* topk_w, int T, int H, int I, int K, int E,
                              const uint8_t* w13, const void* w13_scale, const uint8_t* w2,
                              const void* w2_scale, void* z, void* y, int32_t* dev_status,
                              int sm_count, cudaStream_t s) {
  if (T == 0) return cudaMemsetAsync(dev_status, 0, 2 * sizeof(int32_t), s);
  const W4Args a{static_cast<const uint16_t*>(x), topk_idx, topk_w, w13,
                 static_cast<const uint16_t*>(w13_scale), w2,
                 static_cast<const uint16_t*>(w2_scale), static_cast<uint16_t*>(z),
                 static_cast<uint16_t*>(y), dev_status, T, H, I, K, E};
  return idx_bits == 32 ? launch_w4<int32_t>(a, sm_count, s) : launch_w4<int64_t>(a, sm_count, s);
}

}  // namespace moe
