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
//
// Products.  A code c under a mask is already an operand: the FP16 number with
// the bits c is the subnormal c * 2^-24, and with the bits c << 4 it is c *
// 2^-20.  So a word's eight codes become four operand registers by one shift
// and four masks, with no arithmetic on them; the elements that meet the second
// kind carry a factor 2^-4.  The token operand is x * 2^k in FP16 with a power
// of two per token that takes its largest element to [2^14, 2^15): exact for
// BF16 down to 2^-27 of the largest.  Products are summed in fp32; the codes'
// offset takes 8 times the sum of the token's group off, which is kept beside
// the row.  The scale multiplies a group's result once, in fp32.
//
// A warp takes 16 weight rows (of gate and up each) against 8 token columns
// with mma.sync m16n8k16: the codes go from shared memory straight into the
// registers of the A operand, where a tensor-core tile fed from shared memory
// (tcgen05) would need the widened weights written to and read from shared
// memory once more, for columns that are mostly empty.  (The same with e4m3
// operands, whose low codes are linear too, takes fewer masks, but the
// 8-bit mma.sync is widened in software here: 2.5 times the instructions.)
// A dot product may take K in any order, so each lane reads 16 consecutive
// bytes (32 codes) of its row and the token operand is stored in the matching
// order: lane 4 * r + q holds codes [32q, 32q + 32) of a 128-group; word i of
// its four words gives the pairs (8i + j, 8i + j + 4), j = 0..3.
//
// Every warp streams its own weights: TMA boxes of 16 rows x 128 bytes (two
// groups) into a ring of its own, a few boxes ahead and over the ends of its
// items, so memory never waits for a reduction; a tile's scales, which are
// contiguous, come as one copy with the tile's first box.  The rings have one
// user and need no second barrier per slot.
//
// Four launches, each started while the one before still runs (programmatic
// dependent launch): the plan (active experts and their routes) and x as
// operand rows; gate/up with the activation; z as operand rows, once each
// route's largest z is known (z keeps eleven significant bits, where a BF16
// operand would keep eight); down with the sum over routes, whose first weights
// are on their way before z is.
#include "common.cuh"
#include "kernels.h"
#include "tensormap.h"

#include <cuda_fp16.h>

#include <algorithm>

namespace moe {
namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = kW4Warps * 32;
constexpr int kCols = 8;          // token columns of one pass
constexpr int kRows = 16;         // weight rows of one tile
constexpr int kBoxBytes = kRows * 128;  // two 128-groups of a tile's codes
constexpr int kMaxRoutes = kW4MaxTokens * 32;
constexpr int kMaxPasses = 1024 + kMaxRoutes / kCols;
constexpr int kMaxTiles = 16384 / kRows;
constexpr int kGuDepth = 2;       // ring slots per warp: a gate and an up box each
constexpr int kDnDepth = 4;       // one box each

// Passes in ascending expert, up to eight routes of one active expert each;
// routes in ascending route id.  A token's second route to one expert is
// dropped and its weight added to the first's, so the routes of a pass have
// different tokens.
struct W4Plan {
  int passes, routes;
  uint32_t pass[kMaxPasses];     // expert | routes << 10 | place of the first << 14
  uint16_t route[kMaxRoutes];
  float weight[kMaxRoutes];      // of route[i]
};
struct Pass {
  int e, n, off;
};
__device__ __forceinline__ uint32_t pack_pass(int e, int n, int off) {
  return static_cast<uint32_t>(e) | (static_cast<uint32_t>(n) << 10) | (static_cast<uint32_t>(off) << 14);
}
__device__ __forceinline__ Pass unpack_pass(uint32_t p) {
  return Pass{static_cast<int>(p & 1023u), static_cast<int>((p >> 10) & 15u),
              static_cast<int>(p >> 14)};
}

struct W4Args {
  const uint16_t* x;    // BF16 [T, H]
  const void* topk_idx;
  const float* topk_w;  // [T, K]
  const uint16_t* s13;  // BF16 [E, 2I, H / 128]
  const uint16_t* s2;   // BF16 [E, H, I / 128]
  uint16_t* y;          // BF16 [T, H]
  int32_t* dev_status;
  W4Plan* plan;
  uint8_t* xs;          // [T][2H] x as operand rows, see store_operand
  float* xscale;        // [T] 2^-k
  float* xsum;          // [T][H / 128] 8 * 2^-24 times the groups' sums of x * 2^k
  float* z;             // [T * K, I] by route
  uint32_t* zmax;       // [T * K] bits of the route's largest |z|
  uint8_t* zs;          // [T * K][2I] z as operand rows
  float* zscale;        // [T * K]
  float* zsum;          // [T * K][I / 128]
  int* done;            // [H / 16] blocks done with a tile of rows that several share
  float* part;          // [2 * blocks][T][16] their sums
  int T, H, I, K, E;
  int max_passes;       // bound of the plan's passes
};

__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The power of two that takes a row's largest magnitude (its bits) to
// [2^14, 2^15), and its inverse (a sum of products goes back by 2^24 and then
// by that).  Rows of zeros and non-finite rows keep k = 0.
__device__ __forceinline__ float operand_scale(uint32_t max_bits, float* back) {
  const int e = static_cast<int>(max_bits >> 23) - 127;   // subnormal rows: -127
  const int k = max_bits == 0 || max_bits >= 0x7f800000u ? 0 : min(14 - e, 120);
  *back = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}
// Eight elements [8i, 8i + 8) of a row, times `mult`, as the operand pairs
// (j, j + 4), the odd j times 2^-4: 16 bytes, in the row's order.  Half a warp
// stores a group together, which sums[i / 16] is of.
__device__ __forceinline__ void store_operand(uint8_t* row, float* sums, int i, const float* v,
                                              float mult) {
  float sum = 0.f;
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float u = v[j + 4 * h];
      // an infinity or NaN makes the token's sums NaN
      s[h] = fabsf(u) < INFINITY ? u * mult : __uint_as_float(0x7fffffffu);
    }
    const __half2 p = __floats2half2_rn(j & 1 ? s[0] * 0.0625f : s[0], j & 1 ? s[1] * 0.0625f : s[1]);
    const float2 f = __half22float2(p);
    sum += (f.x + f.y) * (j & 1 ? 16.f : 1.f);
    out[j] = *reinterpret_cast<const uint32_t*>(&p);
  }
  *reinterpret_cast<uint4*>(row + i * 16) = make_uint4(out[0], out[1], out[2], out[3]);
  const unsigned half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(half, sum, o);
  if (i % 16 == 0) sums[i / 16] = sum * 0x1p-21f;   // 8 * 2^-24
}

// ------------------------------------------------------------------ prepare
template <typename IdT>
__device__ void make_plan(const W4Args& a) {
  __shared__ int pos[1024 + 1];    // counts, then next free place
  __shared__ int off[1024 + 1];    // first route of each expert
  __shared__ int first[1024 + 1];  // first pass of each expert
  __shared__ int16_t ids[kMaxRoutes];
  __shared__ int s_bad;
  const IdT* topk_idx = static_cast<const IdT*>(a.topk_idx);
  const int n = a.T * a.K, E = a.E;
  for (int e = threadIdx.x; e < E; e += blockDim.x) pos[e] = 0;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int64_t id = static_cast<int64_t>(topk_idx[i]);
    const bool in = id >= 0 && id < E;
    ids[i] = in ? static_cast<int16_t>(id) : int16_t{-1};
    if (!in && id != -1) s_bad = 1;
  }
  __syncthreads();
  // a route's expert, or -1 for none and for a repeat
  auto kept = [&](int i) -> int {
    const int e = ids[i];
    for (int j = i - i % a.K; j < i; ++j)
      if (ids[j] == e) return -1;
    return e;
  };
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = kept(i);
    if (e >= 0) atomicAdd(&pos[e], 1);
  }
  __syncthreads();
  expert_prefix(pos, E, kMaxRoutes, 1, 1, off, nullptr);
  expert_prefix(pos, E, kMaxRoutes, kCols, 1, first, nullptr);
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    for (int p = first[e]; p < first[e + 1]; ++p) {
      const int o = off[e] + (p - first[e]) * kCols;
      a.plan->pass[p] = pack_pass(e, min(kCols, off[e + 1] - o), o);
    }
    pos[e] = off[e];
  }
  if (threadIdx.x == 0) {
    a.plan->passes = first[E];
    a.plan->routes = off[E];
    a.dev_status[0] = s_bad ? kDevBadExpertId : 0;
    a.dev_status[1] = 0;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int e = i < n ? kept(i) : -1;
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const int at = pos[e] + __popc(peers & ((1u << lane) - 1u));
      a.plan->route[at] = static_cast<uint16_t>(i);
      float w = a.topk_w[i];
      const int k1 = i - i % a.K + a.K;
      for (int j = i + 1; j < k1; ++j)
        if (ids[j] == e) w += a.topk_w[j];
      a.plan->weight[at] = w;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) pos[e] += __popc(peers);
    __syncwarp();
  }
}

// Block 0 plans; block 1 + t makes token t's operand row.  The counters of the later
// launches start at zero here.
template <typename IdT>
__global__ void __launch_bounds__(kW4Threads) w4_prepare_kernel(const W4Args a) {
  grid_launch_dependents();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.H / kRows; i += kW4Threads) a.done[i] = 0;
    for (int i = threadIdx.x; i < a.T * a.K; i += kW4Threads) a.zmax[i] = 0;
    make_plan<IdT>(a);
    return;
  }
  __shared__ uint32_t s_max[kW4Warps];
  const int t = blockIdx.x - 1, lane = threadIdx.x & 31;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t) * a.H);
  const int nvec = a.H / 8;
  uint32_t m = 0;
  for (int i = threadIdx.x; i < nvec; i += kW4Threads) {
    float v[8];
    bf16x8_to_f32(x[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, s_max[lane % kW4Warps]);
  float back;
  const float mult = operand_scale(m, &back);
  if (threadIdx.x == 0) a.xscale[t] = back;
  for (int i = threadIdx.x; i < nvec; i += kW4Threads) {
    float v[8];
    bf16x8_to_f32(x[i], v);
    store_operand(a.xs + static_cast<int64_t>(t) * 2 * a.H, a.xsum + t * (a.H / kGroup), i, v, mult);
  }
}

// A block per kept route.
__global__ void __launch_bounds__(128) w4_operand_z_kernel(const W4Args a) {
  grid_launch_dependents();
  grid_dependency_wait();
  if (static_cast<int>(blockIdx.x) >= a.plan->routes) return;
  const int route = a.plan->route[blockIdx.x];
  float back;
  const float mult = operand_scale(a.zmax[route], &back);
  if (threadIdx.x == 0) a.zscale[route] = back;
  const float4* z = reinterpret_cast<const float4*>(a.z + static_cast<int64_t>(route) * a.I);
  for (int i = threadIdx.x; i < a.I / 8; i += blockDim.x) {
    const float4 lo = z[2 * i], hi = z[2 * i + 1];
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    store_operand(a.zs + static_cast<int64_t>(route) * 2 * a.I, a.zsum + route * (a.I / kGroup), i, v,
                mult);
  }
}

// ----------------------------------------------------------------- products
// The lane's 64 bytes of a 128-group of its column: the pairs of words 0..3.
__device__ __forceinline__ void load_column(uint4* v, const uint8_t* row, int g, int q) {
  const uint4* p = reinterpret_cast<const uint4*>(row + g * 256 + q * 64);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = p[i];
}

__device__ __forceinline__ void mma_16x8x16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc += scale * 2^-24 * (codes - 8) . column over one 128-group; `p` is the
// lane's first row's 16 bytes in the box, sa and sb the scales of its two
// rows, s0 and s1 the sums that the offset takes off its two columns.
__device__ __forceinline__ void w4_dot(float* acc, const uint8_t* p, uint32_t sa, uint32_t sb,
                                       const uint4* col, float s0, float s1) {
  const uint4 wa = *reinterpret_cast<const uint4*>(p);
  const uint4 wb = *reinterpret_cast<const uint4*>(p + 8 * 128);
  const uint32_t ra[4] = {wa.x, wa.y, wa.z, wa.w};
  const uint32_t rb[4] = {wb.x, wb.y, wb.z, wb.w};
  float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr uint32_t even = 0x000F000Fu, odd = 0x00F000F0u;
    mma_16x8x16(c, ra[i] & even, rb[i] & even, ra[i] & odd, rb[i] & odd, col[i].x, col[i].y);
    const uint32_t ha = ra[i] >> 8, hb = rb[i] >> 8;
    mma_16x8x16(c, ha & even, hb & even, ha & odd, hb & odd, col[i].z, col[i].w);
  }
  const float fa = __uint_as_float(sa), fb = __uint_as_float(sb);
  acc[0] = fmaf(fa, c[0] - s0, acc[0]);
  acc[1] = fmaf(fa, c[1] - s1, acc[1]);
  acc[2] = fmaf(fb, c[2] - s0, acc[2]);
  acc[3] = fmaf(fb, c[3] - s1, acc[3]);
}

// The tile row of lane group r (and, plus 8, of its second row).  In TMA's
// 128-byte swizzle the 16-byte chunk c of row m lies at c ^ (m & 7); the rows
// that share a quarter of a 512-byte access differ in bit 2, so their chunks
// lie in different halves of the 128 bytes.
__device__ __forceinline__ int tile_row(int r) { return (r >> 1) | ((r & 1) << 2); }

// The scales of groups g and g + 1 (if there is one) of one row, the first in
// the low half.
__device__ __forceinline__ uint32_t load_scales(const uint16_t* row, int g, int G) {
  if ((G & 1) == 0) return *reinterpret_cast<const uint32_t*>(row + g);
  uint32_t v = row[g];
  if (g + 1 < G) v |= static_cast<uint32_t>(row[g + 1]) << 16;
  return v;
}
__device__ __forceinline__ uint32_t scale_lo(uint32_t s) { return s << 16; }
__device__ __forceinline__ uint32_t scale_hi(uint32_t s) { return s & 0xFFFF0000u; }

// Untiled copy of `bytes` (a multiple of 16, as both addresses are) into
// shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  const uint32_t a = smem_u32(p);
  return p + (((a + 1023u) & ~1023u) - a);
}

// Gate/up: an item is 16 gate rows and the same 16 up rows of one pass.  A
// team of warps takes an item: one warp where there are items enough to fill
// the GPU, else up to eight that take the item's boxes in turn.
__global__ void __launch_bounds__(kW4Threads, 2)
    w4_gateup_kernel(const __grid_constant__ CUtensorMap map, const W4Args a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ float s_red[kW4Warps][2][4][32];
  __shared__ uint64_t s_full[kW4Warps][kGuDepth], s_scale[kW4Warps][2];
  __shared__ int s_abort;
  uint8_t* ring0 = align1024(smem_raw);
  const int G = a.H / kGroup, ns = (G + 1) / 2;
  const int scale_bytes = kRows * G * 2;   // of a tile
  uint8_t* scales0 = ring0 + kW4Warps * kGuDepth * 2 * kBoxBytes;
  uint32_t* passes = reinterpret_cast<uint32_t*>(scales0 + kW4Warps * 4 * scale_bytes);
  uint16_t* routes = reinterpret_cast<uint16_t*>(passes + a.max_passes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, q = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < kGuDepth; ++i) mbar_init(&s_full[warp][i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s_scale[warp][i], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    s_abort = 0;
    tma_prefetch_desc(&map);
  }
  grid_dependency_wait();
  // only now: the launch after next reads the plan without waiting for this one
  grid_launch_dependents();
  const int np = a.plan->passes, nr = a.plan->routes;
  for (int i = threadIdx.x; i < np; i += kW4Threads) passes[i] = a.plan->pass[i];
  for (int i = threadIdx.x; i < nr; i += kW4Threads) routes[i] = a.plan->route[i];
  __syncthreads();
  const int tiles = a.I / kRows;
  const int total = np * tiles;   // at most 1280 passes x 1024 tiles
  int team = 1;
  while (team < kW4Warps && total * team * 2 <= static_cast<int>(gridDim.x) * kW4Warps) team *= 2;
  const int rank = warp & (team - 1);
  const int it0 = blockIdx.x + gridDim.x * (warp / team);
  const int it_step = gridDim.x * (kW4Warps / team);
  uint8_t* ring = ring0 + warp * kGuDepth * 2 * kBoxBytes;
  uint8_t* scales = scales0 + warp * 4 * scale_bytes;
  volatile int* abort_flag = &s_abort;

  // The warp's next box to fetch: box ps of item pit, its pj-th, whose scales
  // go to buffer pj % 2; it is at most one item ahead of the item in use, uj.
  int pit = rank < ns ? it0 : total, ps = rank, pj = 0, uj = 0, prow = 0;
  int issued = 0, used = 0;
  bool entered = false;
  auto fetch = [&]() {
    while (issued - used < kGuDepth && pit < total && pj <= uj + 1) {
      if (!entered) {
        prow = unpack_pass(passes[pit / tiles]).e * 2 * a.I + pit % tiles * kRows;
        if (lane == 0) {
          uint8_t* dst = scales + (pj & 1) * 2 * scale_bytes;
          const uint16_t* src = a.s13 + static_cast<int64_t>(prow) * G;
          mbar_arrive_expect_tx(&s_scale[warp][pj & 1], 2 * scale_bytes);
          bulk_load(dst, src, scale_bytes, &s_scale[warp][pj & 1]);
          bulk_load(dst + scale_bytes, src + static_cast<int64_t>(a.I) * G, scale_bytes,
                    &s_scale[warp][pj & 1]);
        }
        entered = true;
      }
      if (lane == 0) {
        const int slot = issued % kGuDepth;
        uint8_t* dst = ring + slot * 2 * kBoxBytes;
        mbar_arrive_expect_tx(&s_full[warp][slot], 2 * kBoxBytes);
        tma_load_2d(dst, &map, &s_full[warp][slot], ps * 128, prow);
        tma_load_2d(dst + kBoxBytes, &map, &s_full[warp][slot], ps * 128, prow + a.I);
      }
      ++issued;
      ps += team;
      if (ps >= ns) {
        ps = rank;
        pit += it_step;
        ++pj;
        entered = false;
      }
    }
  };
  fetch();

  // the lane's first row in a box, for the even and the odd group
  const int row = tile_row(r);
  const int off0 = row * 128 + ((q ^ (row & 7)) << 4), off1 = off0 ^ 64;
  int landed = 0, slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int it = it0; it < total; it += it_step) {
    const Pass pass = unpack_pass(passes[it / tiles]);
    const int i0 = it % tiles * kRows;
    const uint8_t* xr =
        r < pass.n ? a.xs + static_cast<int64_t>(routes[pass.off + r] / a.K) * 2 * a.H : nullptr;
    const float* sum0 = a.xsum + routes[pass.off + min(2 * q, pass.n - 1)] / a.K * G;
    const float* sum1 = a.xsum + routes[pass.off + min(2 * q + 1, pass.n - 1)] / a.K * G;
    float ag[4] = {0.f, 0.f, 0.f, 0.f}, au[4] = {0.f, 0.f, 0.f, 0.f};
    // columns of the even and the odd groups, each loaded while the other's
    // products run; zeros where the pass has no such column
    uint4 even[4], odd[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) even[i] = odd[i] = make_uint4(0, 0, 0, 0);
    if (xr != nullptr && rank < ns) load_column(even, xr, 2 * rank, q);
    const uint16_t* sc = reinterpret_cast<const uint16_t*>(scales + (uj & 1) * 2 * scale_bytes) + row * G;
    if (rank < ns && ok &&
        !__all_sync(0xffffffffu, mbar_wait(&s_scale[warp][uj & 1], (uj >> 1) & 1, abort_flag))) {
      ok = false;
      landed = used;
      *abort_flag = 1;
    }
    for (int s = rank; s < ns; s += team) {
      const bool two = 2 * s + 1 < G;
      if (xr != nullptr && two) load_column(odd, xr, 2 * s + 1, q);
      const uint32_t sg0 = load_scales(sc, 2 * s, G), sg1 = load_scales(sc + 8 * G, 2 * s, G);
      const uint32_t su0 = load_scales(sc + kRows * G, 2 * s, G);
      const uint32_t su1 = load_scales(sc + (kRows + 8) * G, 2 * s, G);
      if (ok && !__all_sync(0xffffffffu, mbar_wait(&s_full[warp][slot], phase, abort_flag))) {
        ok = false;
        landed = used;
        *abort_flag = 1;
      }
      const uint8_t* box = ring + slot * 2 * kBoxBytes;
      if (ok) {
        const float s0 = sum0[2 * s], s1 = sum1[2 * s];
        w4_dot(ag, box + off0, scale_lo(sg0), scale_lo(sg1), even, s0, s1);
        w4_dot(au, box + kBoxBytes + off0, scale_lo(su0), scale_lo(su1), even, s0, s1);
      }
      if (xr != nullptr && s + team < ns) load_column(even, xr, 2 * (s + team), q);
      if (ok && two) {
        const float s0 = sum0[2 * s + 1], s1 = sum1[2 * s + 1];
        w4_dot(ag, box + off1, scale_hi(sg0), scale_hi(sg1), odd, s0, s1);
        w4_dot(au, box + kBoxBytes + off1, scale_hi(su0), scale_hi(su1), odd, s0, s1);
      }
      ++used;
      if (++slot == kGuDepth) {
        slot = 0;
        phase ^= 1;
      }
      __syncwarp();   // every lane has read the slot
      if (ok) fetch();
    }
    ++uj;
    if (ok) fetch();   // the next item's scales may have waited for this one's
    if (team > 1) {   // the parts of the team's warps, in their order
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s_red[warp][0][j][lane] = ag[j];
        s_red[warp][1][j][lane] = au[j];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / team), "r"(32 * team) : "memory");
      if (rank == 0) {
        for (int w = 1; w < team; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ag[j] += s_red[warp + w][0][j][lane];
            au[j] += s_red[warp + w][1][j][lane];
          }
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / team), "r"(32 * team) : "memory");
    }
    if (rank == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int cc = 2 * q + j;
        uint32_t m = 0;
        int route = 0;
        if (cc < pass.n) {
          route = routes[pass.off + cc];
          const float back = a.xscale[route / a.K];
          float* z = a.z + static_cast<int64_t>(route) * a.I + i0 + row;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float gate = ag[2 * h + j] * 0x1p24f * back;
            const float up_v = au[2 * h + j] * 0x1p24f * back;
            const float v = gate / (1.f + expf(-gate)) * up_v;
            z[8 * h] = v;
            m = max(m, __float_as_uint(v) & 0x7fffffffu);
          }
        }
        // over the eight lanes of the column
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (r == 0 && cc < pass.n) atomicMax(a.zmax + route, m);
      }
    }
  }
  if (!ok) {
    // no copy may land after the block has ended
    for (; landed < issued; ++landed) {
      int none = 0;
      mbar_wait(&s_full[warp][landed % kGuDepth], (landed / kGuDepth) & 1, &none);
    }
    for (int j = uj; j <= pj && j <= uj + 1; ++j) {
      int none = 0;
      if (j < pj || entered) mbar_wait(&s_scale[warp][j & 1], (j >> 1) & 1, &none);
    }
    if (lane == 0) atomicOr(a.dev_status, kDevTimeout);
  }
}

// Down: 16 rows of H for every pass make a tile; the (tile, pass, box) units
// in that order are cut into equal runs, one per block, so every SM reads the
// same number of bytes whatever H and the routes are.  Inside a block the
// warps take equal runs of a tile's units and keep a sum per token.  A tile
// that one block has whole is written by it; of a tile that several blocks
// share each leaves its sums in the workspace, and the last to finish adds
// them in block order.  The order of the sums is fixed by the routes alone.
__global__ void __launch_bounds__(kW4Threads, 2)
    w4_down_kernel(const __grid_constant__ CUtensorMap map, const W4Args a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kW4Warps][kDnDepth], s_scale[kW4Warps][2];
  __shared__ int s_abort, s_last;
  uint8_t* ring0 = align1024(smem_raw);
  float* s_y = reinterpret_cast<float*>(ring0 + kW4Warps * kDnDepth * kBoxBytes);  // [warps][T][kRows]
  const int per = a.T * kRows;
  const int G = a.I / kGroup, ns = (G + 1) / 2;
  const int scale_bytes = kRows * G * 2;   // of a tile
  uint8_t* scales0 = reinterpret_cast<uint8_t*>(s_y + kW4Warps * per);
  uint32_t* passes = reinterpret_cast<uint32_t*>(scales0 + kW4Warps * 2 * scale_bytes);
  float* weights = reinterpret_cast<float*>(passes + a.max_passes);
  uint16_t* routes = reinterpret_cast<uint16_t*>(weights + a.T * a.K);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, q = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < kDnDepth; ++i) mbar_init(&s_full[warp][i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s_scale[warp][i], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    s_abort = 0;
    tma_prefetch_desc(&map);
  }
  // the plan was complete before the launch of the gate/up blocks went on, so
  // it is read (through L2) and the first weights are fetched before the wait
  const int np = __ldcg(&a.plan->passes), nr = __ldcg(&a.plan->routes);
  for (int i = threadIdx.x; i < np; i += kW4Threads) passes[i] = __ldcg(&a.plan->pass[i]);
  for (int i = threadIdx.x; i < nr; i += kW4Threads) {
    routes[i] = __ldcg(&a.plan->route[i]);
    weights[i] = __ldcg(&a.plan->weight[i]);
  }
  __syncthreads();
  const int tiles = a.H / kRows;
  const int units = np * ns;      // of a tile: at most 1280 x 64
  const int64_t all = static_cast<int64_t>(tiles) * units;
  const int nb = gridDim.x;
  auto start_of = [&](int b) { return all * b / nb; };
  const int64_t f0 = start_of(blockIdx.x), f1 = start_of(blockIdx.x + 1);
  const int t0 = units ? static_cast<int>(f0 / units) : 0;
  const int t1 = units && f1 > f0 ? static_cast<int>((f1 - 1) / units) + 1 : t0;   // tiles [t0, t1)
  // this block's units of tile t, and this warp's of those
  auto block_lo = [&](int t) { return static_cast<int>(max(f0 - static_cast<int64_t>(t) * units, int64_t{0})); };
  auto block_hi = [&](int t) {
    return static_cast<int>(min(f1 - static_cast<int64_t>(t) * units, static_cast<int64_t>(units)));
  };
  auto warp_at = [&](int t, int w) {
    const int lo = block_lo(t);
    return lo + (block_hi(t) - lo) * w / kW4Warps;
  };
  uint8_t* ring = ring0 + warp * kDnDepth * kBoxBytes;
  uint8_t* scales = scales0 + warp * 2 * scale_bytes;
  float* mine = s_y + warp * per;
  volatile int* abort_flag = &s_abort;

  // The warp's next box to fetch: unit pu of tile pt, where the warp's run ends
  // at pend.  Runs of one pass in one tile share their scales: the pj-th run's
  // are in buffer pj % 2, at most one run ahead of the run in use, uj.
  int pt = t0, pu = 0, pend = 0, pj = 0, uj = 0;
  int issued = 0, used = 0, prow = 0, prun = 0;   // prun: where the run ends
  bool entered = false;
  auto settle = [&]() {
    while (pt < t1 && pu >= pend) {
      ++pt;
      if (pt < t1) {
        pu = warp_at(pt, warp);
        pend = warp_at(pt, warp + 1);
      }
    }
  };
  auto fetch = [&]() {
    while (issued - used < kDnDepth && pt < t1 && pj <= uj + 1) {
      if (!entered) {
        const int p = pu / ns;
        prow = unpack_pass(passes[p]).e * a.H + pt * kRows;
        prun = min(pend, (p + 1) * ns);
        if (lane == 0) {
          mbar_arrive_expect_tx(&s_scale[warp][pj & 1], scale_bytes);
          bulk_load(scales + (pj & 1) * scale_bytes, a.s2 + static_cast<int64_t>(prow) * G,
                    scale_bytes, &s_scale[warp][pj & 1]);
        }
        entered = true;
      }
      if (lane == 0) {
        const int slot = issued % kDnDepth;
        mbar_arrive_expect_tx(&s_full[warp][slot], kBoxBytes);
        tma_load_2d(ring + slot * kBoxBytes, &map, &s_full[warp][slot], pu % ns * 128, prow);
      }
      ++issued;
      if (++pu == prun) {
        ++pj;
        entered = false;
        settle();
      }
    }
  };
  if (pt < t1) {
    pu = warp_at(pt, warp);
    pend = warp_at(pt, warp + 1);
    settle();
  }
  fetch();
  grid_dependency_wait();   // z
  if (units == 0) {   // no routes
    for (int t = blockIdx.x; t < tiles; t += nb)
      for (int i = threadIdx.x; i < per; i += kW4Threads)
        a.y[static_cast<int64_t>(i / kRows) * a.H + t * kRows + i % kRows] = 0;
    return;
  }

  const int row = tile_row(r);
  const int off0 = row * 128 + ((q ^ (row & 7)) << 4), off1 = off0 ^ 64;
  int landed = 0, slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int t = t0; t < t1; ++t) {
    for (int i = lane; i < per; i += 32) mine[i] = 0.f;
    __syncwarp();
    const int u1 = warp_at(t, warp + 1);
    for (int u = warp_at(t, warp); u < u1;) {
      const int p = u / ns;
      const Pass pass = unpack_pass(passes[p]);
      const int s1 = min(u1 - p * ns, ns);
      const uint8_t* zr =
          r < pass.n ? a.zs + static_cast<int64_t>(routes[pass.off + r]) * 2 * a.I : nullptr;
      const float* sum0 = a.zsum + routes[pass.off + min(2 * q, pass.n - 1)] * G;
      const float* sum1 = a.zsum + routes[pass.off + min(2 * q + 1, pass.n - 1)] * G;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      uint4 even[4], odd[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) even[i] = odd[i] = make_uint4(0, 0, 0, 0);
      int s = u - p * ns;
      u = p * ns + s1;
      if (zr != nullptr) load_column(even, zr, 2 * s, q);
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(scales + (uj & 1) * scale_bytes) + row * G;
      if (ok && !__all_sync(0xffffffffu, mbar_wait(&s_scale[warp][uj & 1], (uj >> 1) & 1, abort_flag))) {
        ok = false;
        landed = used;
        *abort_flag = 1;
      }
      for (; s < s1; ++s) {
        const bool two = 2 * s + 1 < G;
        if (zr != nullptr && two) load_column(odd, zr, 2 * s + 1, q);
        const uint32_t sa = load_scales(sc, 2 * s, G), sb = load_scales(sc + 8 * G, 2 * s, G);
        if (ok && !__all_sync(0xffffffffu, mbar_wait(&s_full[warp][slot], phase, abort_flag))) {
          ok = false;
          landed = used;
          *abort_flag = 1;
        }
        const uint8_t* box = ring + slot * kBoxBytes;
        if (ok) {
            const float s0 = sum0[2 * s], s1 = sum1[2 * s];
          w4_dot(acc, box + off0, scale_lo(sa), scale_lo(sb), even, s0, s1);
        }
        if (zr != nullptr && s + 1 < s1) load_column(even, zr, 2 * s + 2, q);
        if (ok && two) {
            const float s0 = sum0[2 * s + 1], s1 = sum1[2 * s + 1];
          w4_dot(acc, box + off1, scale_hi(sa), scale_hi(sb), odd, s0, s1);
        }
        ++used;
        if (++slot == kDnDepth) {
          slot = 0;
          phase ^= 1;
        }
        __syncwarp();   // every lane has read the slot
        if (ok) fetch();
      }
      ++uj;
      if (ok) fetch();
      // the routes of a pass have different tokens: no two lanes share a sum
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int cc = 2 * q + j;
        if (cc < pass.n) {
          const int route = routes[pass.off + cc];
          const float wt = weights[pass.off + cc] * a.zscale[route];
          float* yt = mine + route / a.K * kRows + row;
          yt[0] = fmaf(wt, acc[j] * 0x1p24f, yt[0]);
          yt[8] = fmaf(wt, acc[2 + j] * 0x1p24f, yt[8]);
        }
      }
      __syncwarp();
    }
    __syncthreads();
    const bool whole = block_lo(t) == 0 && block_hi(t) == units;
    float* part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (t > t0 ? 1 : 0)) * per;
    for (int i = threadIdx.x; i < per; i += kW4Threads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kW4Warps; ++w) v += s_y[w * per + i];
      if (whole)
        a.y[static_cast<int64_t>(i / kRows) * a.H + t * kRows + i % kRows] =
            __bfloat16_as_ushort(__float2bfloat16_rn(v));
      else
        part[i] = v;
    }
    if (!whole) {
      // blocks b0 .. b1 share the tile
      const int64_t lo = static_cast<int64_t>(t) * units, hi = lo + units;
      int b0 = static_cast<int>(lo * nb / all), b1 = static_cast<int>((hi - 1) * nb / all);
      while (start_of(b0 + 1) <= lo) ++b0;
      while (start_of(b1 + 1) <= hi - 1) ++b1;
      int sharing = 0;
      for (int b = b0; b <= b1; ++b) sharing += start_of(b + 1) > start_of(b);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) s_last = atomicAdd(a.done + t, 1) == sharing - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int i = threadIdx.x; i < per; i += kW4Threads) {
          float v = 0.f;
          for (int b = b0; b <= b1; ++b) {
            const int64_t f = start_of(b);
            if (start_of(b + 1) == f) continue;
            v += __ldcg(a.part + (static_cast<int64_t>(b) * 2 + (f / units < t ? 1 : 0)) * per + i);
          }
          a.y[static_cast<int64_t>(i / kRows) * a.H + t * kRows + i % kRows] =
              __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
      }
    }
    __syncthreads();
  }
  if (!ok) {
    for (; landed < issued; ++landed) {
      int none = 0;
      mbar_wait(&s_full[warp][landed % kDnDepth], (landed / kDnDepth) & 1, &none);
    }
    for (int j = uj; j <= pj && j <= uj + 1; ++j) {
      int none = 0;
      if (j < pj || entered) mbar_wait(&s_scale[warp][j & 1], (j >> 1) & 1, &none);
    }
    if (lane == 0) atomicOr(a.dev_status, kDevTimeout);
  }
}

// Offsets of the workspace's parts.
struct W4Workspace {
  size_t plan, xs, xscale, xsum, z, zmax, zs, zscale, zsum, done, part, total;
};
W4Workspace w4_workspace(int T, int K, int H, int I) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  const size_t n = static_cast<size_t>(T) * K;
  W4Workspace w{};
  w.plan = take(sizeof(W4Plan));
  w.xs = take(static_cast<size_t>(T) * 2 * H);
  w.xscale = take(static_cast<size_t>(T) * 4);
  w.xsum = take(static_cast<size_t>(T) * (H / kGroup) * 4);
  w.z = take(n * I * 4);
  w.zmax = take(n * 4);
  w.zs = take(n * 2 * I);
  w.zscale = take(n * 4);
  w.zsum = take(n * (I / kGroup) * 4);
  w.done = take(kMaxTiles * 4);
  w.part = take(static_cast<size_t>(kW4MaxBlocks) * 2 * T * kRows * 4);
  w.total = off;
  return w;
}

// A launch that may start while the one before in the stream still runs.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int threads, size_t smem,
                             cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

size_t experts_w4_workspace(int T, int K, int H, int I) { return w4_workspace(T, K, H, I).total; }

cudaError_t launch_experts_w4(const void* x, const void* topk_idx, int idx_bits,
                              const float* topk_w, int T, int H, int I, int K, int E,
                              const uint8_t* w13, const void* w13_scale, const uint8_t* w2,
                              const void* w2_scale, void* workspace, void* y,
                              int32_t* dev_status, int sm_count, cudaStream_t s) {
  if (T == 0) return cudaMemsetAsync(dev_status, 0, 2 * sizeof(int32_t), s);
  const int n = T * K;
  const W4Workspace w = w4_workspace(T, K, H, I);
  auto* ws = static_cast<uint8_t*>(workspace);
  W4Args a{};
  a.x = static_cast<const uint16_t*>(x);
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.s13 = static_cast<const uint16_t*>(w13_scale);
  a.s2 = static_cast<const uint16_t*>(w2_scale);
  a.y = static_cast<uint16_t*>(y);
  a.dev_status = dev_status;
  a.plan = reinterpret_cast<W4Plan*>(ws + w.plan);
  a.xs = ws + w.xs;
  a.xscale = reinterpret_cast<float*>(ws + w.xscale);
  a.xsum = reinterpret_cast<float*>(ws + w.xsum);
  a.z = reinterpret_cast<float*>(ws + w.z);
  a.zmax = reinterpret_cast<uint32_t*>(ws + w.zmax);
  a.zs = ws + w.zs;
  a.zscale = reinterpret_cast<float*>(ws + w.zscale);
  a.zsum = reinterpret_cast<float*>(ws + w.zsum);
  a.done = reinterpret_cast<int*>(ws + w.done);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.T = T;
  a.H = H;
  a.I = I;
  a.K = K;
  a.E = E;
  a.max_passes = std::min(E, n) + n / kCols;

  CUtensorMap m13, m2;
  cudaError_t err = make_map_rows128(&m13, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w13, H / 2,
                                     static_cast<uint64_t>(E) * 2 * I, kRows);
  if (err == cudaSuccess)
    err = make_map_rows128(&m2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w2, I / 2,
                           static_cast<uint64_t>(E) * H, kRows);
  const int gu_smem = 1024 + kW4Warps * (kGuDepth * 2 * kBoxBytes + 4 * kRows * (H / kGroup) * 2) +
                      4 * a.max_passes + 2 * n;
  const int dn_smem = 1024 + kW4Warps * (kDnDepth * kBoxBytes + T * kRows * 4 +
                                         2 * kRows * (I / kGroup) * 2) +
                      4 * a.max_passes + 6 * n;
  constexpr int kMaxSmem = 218 * 1024;
  static_assert(1024 + kW4Warps * (kGuDepth * 2 * kBoxBytes + 4 * kRows * 128 * 2) + 4 * kMaxPasses +
                            2 * kMaxRoutes <= kMaxSmem &&
                    1024 + kW4Warps * (kDnDepth * kBoxBytes + kW4MaxTokens * kRows * 4 +
                                       2 * kRows * 128 * 2) + 4 * kMaxPasses + 6 * kMaxRoutes <=
                        kMaxSmem,
                "shared memory of the largest call");
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(w4_gateup_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(w4_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (err != cudaSuccess) return err;
  if (idx_bits == 32) w4_prepare_kernel<int32_t><<<1 + T, kW4Threads, 0, s>>>(a);
  else w4_prepare_kernel<int64_t><<<1 + T, kW4Threads, 0, s>>>(a);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  const int blocks = std::min(kW4MaxBlocks, 2 * sm_count);
  err = launch_dependent(w4_gateup_kernel, std::min(a.max_passes * (I / kRows), blocks), kW4Threads,
                         gu_smem, s, m13, a);
  if (err == cudaSuccess) err = launch_dependent(w4_operand_z_kernel, n, 128, 0, s, a);
  if (err == cudaSuccess) err = launch_dependent(w4_down_kernel, blocks, kW4Threads, dn_smem, s, m2, a);
  return err;
}

}  // namespace moe
