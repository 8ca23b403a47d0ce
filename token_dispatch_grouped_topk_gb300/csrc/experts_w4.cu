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
// Streaming.  A block's unit is 128 weight rows (of gate and up each) x two
// groups: a producer thread brings the codes with TMA (128-byte swizzled
// boxes) and the operand rows of the pass's tokens with bulk copies through a
// ring of stages; each of eight warps takes 16 of the rows.  The launch's units
// in order (tile by tile) are cut into equal runs, one per block, so every SM
// reads the same number of bytes whatever the sizes and the routes are.  A
// tile that one block has whole is finished by it; of a tile that several
// blocks share each warp leaves its sums in the workspace, and the last to
// finish adds them in block order.  The order of every sum is fixed by the
// routes alone.
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

constexpr int kW4Warps = 8;       // that compute; one more brings the data
constexpr int kW4Threads = (kW4Warps + 1) * 32;
constexpr int kPrepThreads = 256;
constexpr int kCols = 8;          // token columns of one pass
constexpr int kRows = 16;         // weight rows of one warp
constexpr int kTileRows = kW4Warps * kRows;
constexpr int kBoxBytes = kTileRows * 128;  // two 128-groups of a tile's codes
constexpr int kOpBytes = 288;     // operand record of a group: 256 bytes, its sum, padding
constexpr int kColBytes = 2 * kOpBytes;     // one column of a unit (64 mod 128: no bank conflicts)
constexpr int kMaxStages = 5;
constexpr int kMaxRoutes = kW4MaxTokens * 32;
constexpr int kMaxPasses = 1024 + kMaxRoutes / kCols;

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
  uint8_t* xs;          // [T] operand rows of x, see store_operand
  float* xscale;        // [T] 2^-k
  float* z;             // [T * K, I] by route
  uint32_t* zmax;       // [T * K] bits of the route's largest |z|
  uint8_t* zs;          // [T * K] operand rows of z
  float* zscale;        // [T * K]
  int* done;            // [2][blocks][warps]: warps done with the tile that several blocks
                        // share and the block begins, of gate/up and of down
  float* part;          // their sums: [2 * blocks][warps][256 or T * 16]
  int T, H, I, K, E;
  int max_passes;       // bound of the plan's passes
  int stages;
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
// Bytes of an operand row: an even number of group records, so a unit's two
// are always there.
__host__ __device__ __forceinline__ int operand_row_bytes(int n) {
  return (n / kGroup + 1) / 2 * kColBytes;
}
// Eight elements [8i, 8i + 8) of a row, times `mult`, as the operand pairs
// (j, j + 4), the odd j times 2^-4.  A group's record: word by word, the 16
// bytes of the four lanes q; then 8 * 2^-24 times the group's sum.  Half a warp
// stores a group together.
__device__ __forceinline__ void store_operand(uint8_t* row, int i, const float* v, float mult) {
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
  uint8_t* rec = row + (i / 16) * kOpBytes;
  const int q = i % 16 / 4, w = i % 4;
  *reinterpret_cast<uint4*>(rec + w * 64 + q * 16) = make_uint4(out[0], out[1], out[2], out[3]);
  const unsigned half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(half, sum, o);
  if (i % 16 == 0) *reinterpret_cast<float*>(rec + 256) = sum * 0x1p-21f;
}
// The record past an odd number of groups: zeros.
__device__ __forceinline__ void store_operand_end(uint8_t* row, int n) {
  const int G = n / kGroup;
  if ((G & 1) && threadIdx.x < kOpBytes / 16)
    *reinterpret_cast<uint4*>(row + G * kOpBytes + threadIdx.x * 16) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ prepare
template <typename IdT>
__device__ void make_plan(const W4Args& a) {
  __shared__ int pos[1024 + 1];    // counts, then next free place
  __shared__ int off[1024 + 1];    // first route of each expert
  __shared__ int first[1024 + 1];  // first pass of each expert
  __shared__ int16_t ids[kMaxRoutes], kept[kMaxRoutes];
  __shared__ float weight[kMaxRoutes];
  __shared__ int s_bad;
  const IdT* topk_idx = static_cast<const IdT*>(a.topk_idx);
  const int n = a.T * a.K, E = a.E;
  for (int e = threadIdx.x; e < E; e += blockDim.x) pos[e] = 0;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int64_t id = static_cast<int64_t>(topk_idx[i]);
    weight[i] = a.topk_w[i];
    const bool in = id >= 0 && id < E;
    ids[i] = in ? static_cast<int16_t>(id) : int16_t{-1};
    if (!in && id != -1) s_bad = 1;
  }
  __syncthreads();
  // a route's expert, or -1 for none and for a repeat
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int e = ids[i];
    const int k0 = i - i % a.K;
    for (int j = k0; j < i; ++j)
      if (ids[j] == e) e = -1;
    kept[i] = static_cast<int16_t>(e);
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
    const int e = i < n ? kept[i] : -1;
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const int at = pos[e] + __popc(peers & ((1u << lane) - 1u));
      float w = weight[i];
      const int k1 = i - i % a.K + a.K;
      for (int j = i + 1; j < k1; ++j)
        if (ids[j] == e) w += weight[j];
      a.plan->route[at] = static_cast<uint16_t>(i);
      a.plan->weight[at] = w;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) pos[e] += __popc(peers);
    __syncwarp();
  }
}

// Block 0 plans; block 1 + t makes token t's operand row.  The counters of the
// later launches start at zero here.
template <typename IdT>
__global__ void __launch_bounds__(kPrepThreads) w4_prepare_kernel(const W4Args a) {
  grid_launch_dependents();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < 2 * kW4MaxBlocks * kW4Warps; i += kPrepThreads) a.done[i] = 0;
    for (int i = threadIdx.x; i < a.T * a.K; i += kPrepThreads) a.zmax[i] = 0;
    make_plan<IdT>(a);
    return;
  }
  __shared__ uint32_t s_max[kPrepThreads / 32];
  const int t = blockIdx.x - 1, lane = threadIdx.x & 31;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t) * a.H);
  const int nvec = a.H / 8;
  uint32_t m = 0;
  for (int i = threadIdx.x; i < nvec; i += kPrepThreads) {
    float v[8];
    bf16x8_to_f32(x[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, s_max[lane % (kPrepThreads / 32)]);
  float back;
  const float mult = operand_scale(m, &back);
  if (threadIdx.x == 0) a.xscale[t] = back;
  uint8_t* row = a.xs + static_cast<int64_t>(t) * operand_row_bytes(a.H);
  for (int i = threadIdx.x; i < nvec; i += kPrepThreads) {
    float v[8];
    bf16x8_to_f32(x[i], v);
    store_operand(row, i, v, mult);
  }
  store_operand_end(row, a.H);
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
  uint8_t* row = a.zs + static_cast<int64_t>(route) * operand_row_bytes(a.I);
  for (int i = threadIdx.x; i < a.I / 8; i += blockDim.x) {
    const float4 lo = z[2 * i], hi = z[2 * i + 1];
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    store_operand(row, i, v, mult);
  }
  store_operand_end(row, a.I);
}

// ----------------------------------------------------------------- products
// The lane's 64 bytes of a group record: the pairs of words 0..3.
__device__ __forceinline__ void load_column(uint4* v, const uint8_t* rec, int q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(rec + i * 64 + q * 16);
}

__device__ __forceinline__ void mma_16x8x16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
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

// The scales of groups g and g + 1 of one row, the first in the low half; zero
// for a group that is not there.
__device__ __forceinline__ uint32_t load_scales(const uint16_t* row, int g, int G) {
  if ((G & 1) == 0) return __ldg(reinterpret_cast<const uint32_t*>(row + g));
  uint32_t v = __ldg(row + g);
  if (g + 1 < G) v |= static_cast<uint32_t>(__ldg(row + g + 1)) << 16;
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

// The gate/up launch (a tile: 128 gate rows and the same up rows of one pass)
// and the down launch (a tile: 128 rows of H, for every pass).
template <bool kDown>
__global__ void __launch_bounds__(kW4Threads, 2)
    w4_stream_kernel(const __grid_constant__ CUtensorMap map, const W4Args a) {
  constexpr int kBoxes = kDown ? 1 : 2;
  constexpr int kABytes = kBoxes * kBoxBytes;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages];
  __shared__ int s_abort;
  uint8_t* ring = align1024(smem_raw);                     // [stages][kABytes]
  uint8_t* cols = ring + a.stages * kABytes;               // [stages][kCols][kColBytes]
  float* s_y = reinterpret_cast<float*>(cols + a.stages * kCols * kColBytes);  // down: [warps][T][kRows]
  const int per = kDown ? a.T * kRows : 0;
  uint32_t* passes = reinterpret_cast<uint32_t*>(s_y + kW4Warps * per);
  float* weights = reinterpret_cast<float*>(passes + a.max_passes);            // down
  uint16_t* routes = reinterpret_cast<uint16_t*>(weights + (kDown ? a.T * a.K : 0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kW4Warps);
    }
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map);
  }
  if constexpr (!kDown) {
    grid_dependency_wait();
    // only now: the launch after next reads the plan without waiting for this one
    grid_launch_dependents();
  }
  // The plan.  In the down launch it is read through L2 before the wait: it was
  // complete before the gate/up blocks let the launches after them start.
  const int np = __ldcg(&a.plan->passes), nr = __ldcg(&a.plan->routes);
  for (int i = threadIdx.x; i < np; i += kW4Threads) passes[i] = __ldcg(&a.plan->pass[i]);
  for (int i = threadIdx.x; i < nr; i += kW4Threads) {
    routes[i] = __ldcg(&a.plan->route[i]);
    if (kDown) weights[i] = __ldcg(&a.plan->weight[i]);
  }
  __syncthreads();

  const int G = (kDown ? a.I : a.H) / kGroup, ns = (G + 1) / 2;
  const int row_tiles = (kDown ? a.H : a.I) / kTileRows;
  const int tiles = kDown ? row_tiles : np * row_tiles;
  const int units = kDown ? np * ns : ns;     // of a tile
  const int64_t all = static_cast<int64_t>(tiles) * units;
  // as many blocks as there are units at most, so no run is empty
  const int nb = static_cast<int>(min(static_cast<int64_t>(gridDim.x), all));
  auto start_of = [&](int b) { return all * b / nb; };
  const bool idle = static_cast<int>(blockIdx.x) >= nb;
  const int64_t f0 = idle ? 0 : start_of(blockIdx.x), f1 = idle ? 0 : start_of(blockIdx.x + 1);
  const int t0 = f1 > f0 ? static_cast<int>(f0 / units) : 0;
  const int t1 = f1 > f0 ? static_cast<int>((f1 - 1) / units) + 1 : 0;   // tiles [t0, t1)
  // this block's units of tile t
  auto lo_of = [&](int t) { return static_cast<int>(max(f0 - static_cast<int64_t>(t) * units, int64_t{0})); };
  auto hi_of = [&](int t) {
    return static_cast<int>(min(f1 - static_cast<int64_t>(t) * units, static_cast<int64_t>(units)));
  };
  volatile int* abort_flag = &s_abort;

  if (warp == kW4Warps) {
    // ------------------------------------------------------------- producer
    // lane 0 fetches the codes, lane c the operand row of column c
    const uint8_t* ops = kDown ? a.zs : a.xs;
    const int64_t op_row = operand_row_bytes(kDown ? a.I : a.H);
    auto columns = [&](const Pass& pass, int s, int sl) {
      if (lane < pass.n) {
        const int route = routes[pass.off + lane];
        bulk_load(cols + (sl * kCols + lane) * kColBytes,
                  ops + (kDown ? route : route / a.K) * op_row + s * kColBytes, kColBytes, &s_full[sl]);
      }
    };
    // down: z, and the columns of the stages whose codes were fetched without it
    int issued = 0;
    auto late_columns = [&]() {
      grid_dependency_wait();
      int n = 0;
      for (int t = t0; t < t1 && n < issued; ++t)
        for (int u = lo_of(t); u < hi_of(t) && n < issued; ++u, ++n)
          columns(unpack_pass(passes[u / ns]), u % ns, n);
    };
    int slot = 0;
    uint32_t phase = 1;
    bool ok = true, waited = !kDown;
    for (int t = t0; t < t1 && ok; ++t) {
      const int hi = hi_of(t);
      for (int u = lo_of(t); u < hi; ++u) {
        const int p = kDown ? u / ns : t / row_tiles;
        const int s = kDown ? u - p * ns : u;
        const Pass pass = unpack_pass(passes[p]);
        if (!waited && issued == a.stages) {   // the ring is full of codes
          late_columns();
          waited = true;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&s_empty[slot], phase, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* dst = ring + slot * kABytes;
          mbar_arrive_expect_tx(&s_full[slot], kABytes + pass.n * kColBytes);
          if (kDown) {
            tma_load_2d(dst, &map, &s_full[slot], s * 128, pass.e * a.H + t * kTileRows);
          } else {
            const int row = pass.e * 2 * a.I + t % row_tiles * kTileRows;
            tma_load_2d(dst, &map, &s_full[slot], s * 128, row);
            tma_load_2d(dst + kBoxBytes, &map, &s_full[slot], s * 128, row + a.I);
          }
        }
        __syncwarp();
        if (waited) columns(pass, s, slot);
        ++issued;
        if (++slot == a.stages) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    if (!waited) late_columns();   // no more units than stages
    if (!ok) {
      // no copy may land after the block has ended
      *abort_flag = 1;
      for (int i = 0; i < min(issued, a.stages); ++i) {
        const int n = issued - 1 - i;
        int none = 0;
        mbar_wait(&s_full[n % a.stages], (n / a.stages) & 1, &none);
      }
    }
    return;
  }

  // ------------------------------------------------------------------ products
  const int r = lane >> 2, q = lane & 3;
  const int row = tile_row(r);
  // the lane's first row in a box, for the first and the second group
  const int off0 = (warp * kRows + row) * 128 + ((q ^ (row & 7)) << 4), off1 = off0 ^ 64;
  const uint16_t* scales = kDown ? a.s2 : a.s13;
  const int64_t up = kDown ? 0 : static_cast<int64_t>(a.I) * G;
  float* mine = s_y + warp * per;
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  if (kDown) {
    grid_dependency_wait();   // zscale, and y's readers before this call
    if (np == 0) {            // no routes
      for (int t = blockIdx.x; t < tiles; t += gridDim.x)
        for (int i = threadIdx.x; i < a.T * kTileRows; i += kW4Warps * 32)
          a.y[static_cast<int64_t>(i / kTileRows) * a.H + t * kTileRows + i % kTileRows] = 0;
    }
  }
  for (int t = t0; t < t1 && ok; ++t) {
    const int lo = lo_of(t), hi = hi_of(t);
    if (kDown) {
      for (int i = lane; i < per; i += 32) mine[i] = 0.f;
      __syncwarp();
    }
    float acc[kBoxes][4];
    Pass pass{};
    for (int u = lo; u < hi && ok;) {
      const int p = kDown ? u / ns : t / row_tiles;
      const int first_s = kDown ? u - p * ns : u;
      const int last_s = kDown ? min(hi - p * ns, ns) : hi;
      u += last_s - first_s;
      pass = unpack_pass(passes[p]);
      const uint16_t* sp =
          scales + static_cast<int64_t>((kDown ? pass.e * a.H + t * kTileRows
                                               : pass.e * 2 * a.I + t % row_tiles * kTileRows) +
                                        warp * kRows + row) * G;
      uint32_t next[2 * kBoxes];
      auto scales_of = [&](int s) {
#pragma unroll
        for (int b = 0; b < kBoxes; ++b) {
          next[2 * b] = load_scales(sp + b * up, 2 * s, G);
          next[2 * b + 1] = load_scales(sp + b * up + 8 * G, 2 * s, G);
        }
      };
      scales_of(first_s);
#pragma unroll
      for (int b = 0; b < kBoxes; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[b][j] = 0.f;
      for (int s = first_s; s < last_s; ++s) {
        uint32_t sc[2 * kBoxes];
#pragma unroll
        for (int j = 0; j < 2 * kBoxes; ++j) sc[j] = next[j];
        if (s + 1 < last_s) scales_of(s + 1);   // a unit ahead of their use
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[slot], phase, abort_flag))) {
          ok = false;
          break;
        }
        const uint8_t* box = ring + slot * kABytes;
        const uint8_t* col = cols + slot * kCols * kColBytes;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint4 v[4];
          load_column(v, col + r * kColBytes + g * kOpBytes, q);
          const float* sums = reinterpret_cast<const float*>(col + 2 * q * kColBytes + g * kOpBytes + 256);
          const float s0 = sums[0], s1 = sums[kColBytes / 4];
#pragma unroll
          for (int b = 0; b < kBoxes; ++b)
            w4_dot(acc[b], box + b * kBoxBytes + (g ? off1 : off0),
                   g ? scale_hi(sc[2 * b]) : scale_lo(sc[2 * b]),
                   g ? scale_hi(sc[2 * b + 1]) : scale_lo(sc[2 * b + 1]), v, s0, s1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[slot]);
        if (++slot == a.stages) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (kDown) {
        // the routes of a pass have different tokens: no two lanes share a sum
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int cc = 2 * q + j;
          if (cc < pass.n) {
            const int route = routes[pass.off + cc];
            const float wt = weights[pass.off + cc] * a.zscale[route];
            float* yt = mine + route / a.K * kRows + row;
            yt[0] = fmaf(wt, acc[0][j] * 0x1p24f, yt[0]);
            yt[8] = fmaf(wt, acc[0][2 + j] * 0x1p24f, yt[8]);
          }
        }
        __syncwarp();
      }
    }
    if (!ok) break;

    // A shared tile: leave the sums, and go on only as the last of its blocks.
    const bool whole = lo == 0 && hi == units;
    int b0 = 0, b1 = 0;
    if (!whole) {
      const int count = kDown ? per : 256;
      const int64_t first = static_cast<int64_t>(t) * units, last = first + units - 1;
      b0 = static_cast<int>(first * nb / all);
      b1 = static_cast<int>(last * nb / all);
      int64_t begin = start_of(b0);
      for (int64_t n; (n = start_of(b0 + 1)) <= first; ++b0) begin = n;
      while (start_of(b1 + 1) <= last) ++b1;
      const int sharing = b1 - b0 + 1;
      // a block's first tile is its slot 0; only b0 can have begun before this one
      const int b0_slot = begin < first ? 1 : 0;
      auto part_of = [&](int b) {
        return a.part + ((static_cast<int64_t>(b) * 2 + (b == b0 ? b0_slot : 0)) * kW4Warps + warp) * count;
      };
      float* part = part_of(blockIdx.x);
      if (kDown) {
        for (int i = lane; i < per; i += 32) part[i] = mine[i];
      } else {
#pragma unroll
        for (int b = 0; b < kBoxes; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[(b * 4 + j) * 32 + lane] = acc[b][j];
      }
      __threadfence();
      __syncwarp();
      int before = 0;
      if (lane == 0)
        before = atomicAdd(a.done + ((kDown ? kW4MaxBlocks : 0) + b0) * kW4Warps + warp, 1);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before != sharing - 1) continue;
      __threadfence();
      if (kDown) {
        for (int i = lane; i < per; i += 32) mine[i] = 0.f;
      } else {
#pragma unroll
        for (int b = 0; b < kBoxes; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[b][j] = 0.f;
      }
      for (int b = b0; b <= b1; ++b) {
        const float* from = part_of(b);
        if (kDown) {
          for (int i = lane; i < per; i += 32) mine[i] += __ldcg(from + i);
        } else {
#pragma unroll
          for (int x = 0; x < kBoxes; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[x][j] += __ldcg(from + (x * 4 + j) * 32 + lane);
        }
      }
      __syncwarp();
    }

    if constexpr (kDown) {
      for (int i = lane; i < per; i += 32)
        a.y[static_cast<int64_t>(i / kRows) * a.H + t * kTileRows + warp * kRows + i % kRows] =
            __bfloat16_as_ushort(__float2bfloat16_rn(mine[i]));
      __syncwarp();
    } else {
      const int i0 = t % row_tiles * kTileRows + warp * kRows + row;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int cc = 2 * q + j;
        uint32_t m = 0;
        int route = 0;
        if (cc < pass.n) {
          route = routes[pass.off + cc];
          const float back = a.xscale[route / a.K];
          float* z = a.z + static_cast<int64_t>(route) * a.I + i0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float gate = acc[0][2 * h + j] * 0x1p24f * back;
            const float upv = acc[kBoxes - 1][2 * h + j] * 0x1p24f * back;
            const float v = gate / (1.f + expf(-gate)) * upv;
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
    *abort_flag = 1;
    if (lane == 0) atomicOr(a.dev_status, kDevTimeout);
  }
}

// Offsets of the workspace's parts.
struct W4Workspace {
  size_t plan, xs, xscale, z, zmax, zs, zscale, done, part, total;
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
  w.xs = take(static_cast<size_t>(T) * operand_row_bytes(H));
  w.xscale = take(static_cast<size_t>(T) * 4);
  w.z = take(n * I * 4);
  w.zmax = take(n * 4);
  w.zs = take(n * operand_row_bytes(I));
  w.zscale = take(n * 4);
  w.done = take(2 * kW4MaxBlocks * kW4Warps * 4);
  w.part = take(static_cast<size_t>(kW4MaxBlocks) * 2 * kW4Warps * std::max(256, T * kRows) * 4);
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
  a.z = reinterpret_cast<float*>(ws + w.z);
  a.zmax = reinterpret_cast<uint32_t*>(ws + w.zmax);
  a.zs = ws + w.zs;
  a.zscale = reinterpret_cast<float*>(ws + w.zscale);
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
                                     static_cast<uint64_t>(E) * 2 * I, kTileRows);
  if (err == cudaSuccess)
    err = make_map_rows128(&m2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w2, I / 2,
                           static_cast<uint64_t>(E) * H, kTileRows);
  // Two blocks per SM: as many stages as half an SM's shared memory (less what
  // the system takes) holds, three at least.
  constexpr int kHalf = 113 * 1024 - 256;
  constexpr int kMaxSmem = 200 * 1024;
  constexpr int kStage = kCols * kColBytes;
  auto smem_of = [&](bool down, int stages) {
    return 1024 + stages * ((down ? 1 : 2) * kBoxBytes + kStage) + 4 * a.max_passes + 2 * n +
           (down ? kW4Warps * T * kRows * 4 + 4 * n : 0);
  };
  auto stages_of = [&](bool down) {
    int s = kMaxStages;
    while (s > 3 && smem_of(down, s) > kHalf) --s;
    return s;
  };
  static_assert(1024 + 3 * (2 * kBoxBytes + kStage) + 4 * kMaxPasses + 2 * kMaxRoutes <= kMaxSmem &&
                    1024 + 3 * (kBoxBytes + kStage) + kW4Warps * kW4MaxTokens * kRows * 4 +
                            4 * kMaxPasses + 6 * kMaxRoutes <= kMaxSmem,
                "shared memory of the largest call");
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(w4_stream_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(w4_stream_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (err != cudaSuccess) return err;
  if (idx_bits == 32) w4_prepare_kernel<int32_t><<<1 + T, kPrepThreads, 0, s>>>(a);
  else w4_prepare_kernel<int64_t><<<1 + T, kPrepThreads, 0, s>>>(a);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  const int blocks = std::min(kW4MaxBlocks, 2 * sm_count);
  a.stages = stages_of(false);
  err = launch_dependent(w4_stream_kernel<false>, blocks, kW4Threads, smem_of(false, a.stages), s, m13, a);
  if (err == cudaSuccess) err = launch_dependent(w4_operand_z_kernel, n, 128, 0, s, a);
  a.stages = stages_of(true);
  if (err == cudaSuccess)
    err = launch_dependent(w4_stream_kernel<true>, blocks, kW4Threads, smem_of(true, a.stages), s, m2, a);
  return err;
}

}  // namespace moe
