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
// kind carry a factor 2^-4.  The token operand is v * 2^k in FP16 with a power
// of two per token and 128-group that takes the group's largest element to
// [2^14, 2^15): exact for BF16 x down to 2^-27 of the largest, and eleven
// significant bits for z, where a BF16 operand would keep eight.  Products are
// summed in fp32; the codes' offset takes 8 times the sum of the token's group
// off, which is kept beside the operands with 2^-k.  The scale multiplies a
// group's result once, in fp32.
//
// A warp takes 32 weight rows against 8 token columns with mma.sync m16n8k16:
// the codes go from shared memory straight into the registers of the A
// operand, where a tensor-core tile fed from shared memory (tcgen05) would
// need the widened weights written to and read from shared memory once more,
// for columns that are mostly empty.  (The same with e4m3 operands, whose low
// codes are linear too, takes fewer masks, but the 8-bit mma.sync is widened in
// software here: 2.5 times the instructions.)  A dot product may take K in any
// order, so each lane reads 16 consecutive bytes (32 codes) of its row and the
// token operand is stored in the matching order: lane 4 * r + q holds codes
// [32q, 32q + 32) of a 128-group; word i of its four words gives the pairs
// (8i + j, 8i + j + 4), j = 0..3.
//
// Streaming.  One launch runs both products.  A unit is 256 weight rows x two
// groups of one pass (up to eight tokens of one expert): 128 gate rows and the
// same 128 up rows, then 256 rows of H.  A producer warp brings the codes with
// TMA (128-byte swizzled boxes) and the tokens' operands with bulk copies
// through a ring of stages; each of eight warps takes 2 x 16 of the rows.  The
// units of each product in order (tile by tile) are cut into equal runs, about
// one per block, so every SM reads the same number of bytes whatever the sizes
// and the routes are.  (Runs cut two or three times finer, to even out the blocks,
// were slower: 146 us to 149 and 153 with 48 tokens; so was handing the last
// quarter out in shorter runs.)  The sums of a tile are left in the workspace; of
// a tile that several runs share the last to finish adds them in run order, so
// the order of every sum is fixed by the routes alone.  A warp of its own does
// that, as a join and what follows it take about 5 us in which the ring would
// stand full (8 tokens, 64 experts of 4096 x 1536: 90 -> 85 us); where the other
// warps have nothing to do, at a run's last tile, they take a column each.  A
// finished gate/up tile is one 128-group of z, stored as operands of the down
// product; a down
// unit's codes are fetched whether or not z is there, and its operands once
// every gate/up tile of its pass has been counted.  Runs are handed out by a
// ticket, gate/up before down, to the blocks that are running, so a block
// waits only for runs that running blocks hold, which never wait themselves.
//
// A small launch before it writes x as operands, one after it adds the
// routes' rows, both overlapped (programmatic dependent launch).
//
// Measured: 48 tokens on 64 experts of 4096 x 1536 (623 MB) take 142 us, 4.4
// TB/s; one token on eight experts of 7168 x 2048 (182 MB) 54 us, 3.4 TB/s; the
// smallest calls 14 us.  About 25 us of each large call are latency: the plan and
// the first codes 6 to 9, each product's last joins 5, two launches 5.  The
// stream between them runs at 5.8 TB/s; a ninth token on an expert is a second
// pass over its codes (8 of the 48-token call's 72 passes), as one pass of
// sixteen columns needs the registers or a second read of shared memory: 190 us.
// Bringing the down product's codes into L2 while z is awaited takes bandwidth
// from the gate/up runs still under way: 148 us and more.
#include "common.cuh"
#include "kernels.h"
#include "tensormap.h"

#include <cuda_fp16.h>

#include <algorithm>

namespace moe {
namespace {

constexpr int kW4Warps = 8;       // that compute; one more brings the data, one finishes tiles
constexpr int kW4Threads = (kW4Warps + 2) * 32;
constexpr int kPrepThreads = 256;
constexpr int kCols = 8;          // token columns of one pass
constexpr int kRows = 16;         // weight rows of one warp in a box
constexpr int kBoxRows = kW4Warps * kRows;
constexpr int kBoxBytes = kBoxRows * 128;   // two 128-groups of a box's codes
constexpr int kOpBytes = 288;     // operand record of a group: 256 bytes, its tail, padding
constexpr int kColBytes = 2 * kOpBytes;     // one column of a unit (64 mod 128: no bank conflicts)
constexpr int kStageBytes = 2 * kBoxBytes + kCols * kColBytes;
constexpr int kStages = 3;        // three or two: the same within 1 % (146 and 145 us with 48 tokens)
// A run's units at least.  One token, one expert of 7168 x 2048: 24 us; with four
// 28, with eight 32; with one the joins cost more (two experts 34 us for 31).
constexpr int kRunUnits = 2;
constexpr int kMaxRoutes = kW4MaxTokens * 32;
constexpr int kMaxPasses = 1024 + kMaxRoutes / kCols;
// Columns from which on the warps share the finish of a run's last tile, and of
// both tiles of a run that is no longer than one: 48 tokens on 64 experts 146 us
// (154 with the finisher alone), 17 tokens on eight of 2560 x 896 38 (43 with only the
// last shared); one token, one column, 53.4 (54.5 shared).
constexpr int kShareColumns = 3;
constexpr int kTileRows = 2 * kBoxRows;
constexpr int kTileSums = kCols * kTileRows;   // a tile's sums, by column

// A pass: up to eight routes of one active expert.
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

struct W4Counters {
  int ticket;
  int tile[2][kW4MaxBlocks];   // runs done with the tile that several share and the run begins
  int pass[kMaxPasses];        // columns of gate/up tiles finished
};

struct W4Args {
  const uint16_t* x;    // BF16 [T, H]
  const void* topk_idx;
  const float* topk_w;  // [T, K]
  const uint16_t* s13;  // BF16 [E, 2I, H / 128]
  const uint16_t* s2;   // BF16 [E, H, I / 128]
  uint16_t* y;          // BF16 [T, H]
  int32_t* dev_status;
  uint8_t* xs;          // [T] operand rows of x
  uint8_t* zs;          // [T * K] operand rows of z, by route
  float* o;             // [T * K, H] by route
  W4Counters* count;
  float* part;          // [2][blocks][2] sums of shared tiles by run, then
                        // [blocks][2] of whole tiles, kTileSums each
  int T, H, I, K, E;
  int max_passes;       // bound of the plan's passes
};

__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Generic-proxy writes of z and async-proxy reads of it are ordered on both
// sides with a proxy fence.
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// ----------------------------------------------------------------- operands
// The power of two that takes the largest magnitude (its bits) of a group to
// [2^14, 2^15), and its inverse (a sum of products goes back by 2^24 and then
// by that).  Zeros and non-finite groups keep k = 0.
__device__ __forceinline__ float operand_scale(uint32_t max_bits, float* back) {
  const int e = static_cast<int>(max_bits >> 23) - 127;   // subnormal: -127
  const int k = max_bits == 0 || max_bits >= 0x7f800000u ? 0 : min(14 - e, 120);
  *back = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}
// An element as operand: an infinity or NaN makes the token's sums NaN.
__device__ __forceinline__ float operand_value(float v, float mult) {
  return fabsf(v) < INFINITY ? v * mult : __uint_as_float(0x7fffffffu);
}
// Bytes of an operand row: an even number of group records, so a unit's two
// are always there.
__host__ __device__ __forceinline__ int operand_row_bytes(int n) {
  return (n / kGroup + 1) / 2 * kColBytes;
}
// A group's record: word by word, the 16 bytes of the four lanes q, which are
// the pairs (j, j + 4) of eight elements, the odd j times 2^-4; then the tail.
__device__ __forceinline__ int record_word(int i) {   // of elements [8i, 8i + 8), i < 16
  return (i & 3) * 64 + (i >> 2) * 16;
}
struct RecordTail {
  float sum;    // 8 * 2^-24 times the sum of the group's v * 2^k
  float back;   // 2^-k
};

// Block t writes token t's operand row, half a warp a group.  Block 0 starts
// the counters at zero and checks the ids.
template <typename IdT>
__global__ void __launch_bounds__(kPrepThreads) w4_prepare_kernel(const W4Args a) {
  grid_launch_dependents();
  const int t = blockIdx.x;
  if (t == 0) {
    int* counters = reinterpret_cast<int*>(a.count);
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(W4Counters) / 4); i += kPrepThreads)
      counters[i] = 0;
    int bad = 0;
    for (int i = threadIdx.x; i < a.T * a.K; i += kPrepThreads) {
      const int64_t id = static_cast<int64_t>(static_cast<const IdT*>(a.topk_idx)[i]);
      bad |= id < -1 || id >= a.E;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      a.dev_status[0] = bad ? kDevBadExpertId : 0;
      a.dev_status[1] = 0;
    }
  }
  const uint4* x = reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t) * a.H);
  uint8_t* row = a.xs + static_cast<int64_t>(t) * operand_row_bytes(a.H);
  for (int i = threadIdx.x; i < a.H / 8; i += kPrepThreads) {
    float v[8];
    bf16x8_to_f32(x[i], v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    const unsigned half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(half, m, o));
    RecordTail tail;
    const float mult = operand_scale(m, &tail.back);
    float sum = 0.f;
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = j & 1 ? 0.0625f : 1.f;
      const __half2 p = __floats2half2_rn(operand_value(v[j], mult) * f, operand_value(v[j + 4], mult) * f);
      const float2 back = __half22float2(p);
      sum += (back.x + back.y) * (j & 1 ? 16.f : 1.f);
      out[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(half, sum, o);
    uint8_t* rec = row + (i >> 4) * kOpBytes;
    *reinterpret_cast<uint4*>(rec + record_word(i & 15)) = make_uint4(out[0], out[1], out[2], out[3]);
    tail.sum = sum * 0x1p-21f;
    if ((i & 15) == 0) *reinterpret_cast<RecordTail*>(rec + 256) = tail;
  }
  // the record past an odd number of groups: zeros
  const int G = a.H / kGroup;
  if ((G & 1) && threadIdx.x < kOpBytes / 16)
    *reinterpret_cast<uint4*>(row + G * kOpBytes + threadIdx.x * 16) = make_uint4(0, 0, 0, 0);
}

// --------------------------------------------------------------------- plan
// The passes in ascending expert and their routes in ascending route id.  A
// token's second route to one expert is left out (its first stands for both),
// so an expert's routes are a set of tokens, and a route's place among them the
// number of lower ones.  `scratch` holds kPlanScratch bytes and T * K shorts
// and is free again afterwards.  Returns the number of passes.  Every thread
// of the block calls it.
constexpr int kPlanScratch = 1024 * 8 + 1024 * 4 + 8 * 4;
template <typename IdT>
__device__ int w4_plan(const W4Args& a, uint32_t* passes, uint16_t* routes, uint8_t* scratch) {
  const IdT* topk_idx = static_cast<const IdT*>(a.topk_idx);
  const int n = a.T * a.K, E = a.E, tid = threadIdx.x, lane = tid & 31;
  uint64_t* tokens = reinterpret_cast<uint64_t*>(scratch);   // [1024] an expert's tokens
  int* first = reinterpret_cast<int*>(tokens + 1024);        // [1024] its first route's place
  int* warp_sum = first + 1024;                              // [8]
  int16_t* ids = reinterpret_cast<int16_t*>(warp_sum + 8);   // [n]
  for (int e = tid; e < 1024; e += blockDim.x) tokens[e] = 0;
  for (int i = tid; i < n; i += blockDim.x) {
    const int64_t id = static_cast<int64_t>(topk_idx[i]);
    ids[i] = id >= 0 && id < E ? static_cast<int16_t>(id) : int16_t{-1};
  }
  __syncthreads();
  auto kept = [&](int i, int t) {
    int e = ids[i];
    for (int j = t * a.K; j < i; ++j)
      if (ids[j] == e) e = -1;
    return e;
  };
  for (int i = tid; i < n; i += blockDim.x) {
    const int t = i / a.K, e = ids[i];
    if (e >= 0) atomicOr(reinterpret_cast<uint32_t*>(tokens + e) + (t >> 5), 1u << (t & 31));
  }
  __syncthreads();
  // prefixes of the routes (low half) and the passes (high half): thread i has
  // experts [4i, 4i + 4)
  int c[4], sum = 0, incl = 0;
  if (tid < 256) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = __popcll(tokens[4 * tid + j]);
      sum += c[j] + ((c[j] + kCols - 1) / kCols << 16);
    }
    incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sum[tid >> 5] = incl;
  }
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) total += warp_sum[w];
  if (tid < 256) {
    int at = incl - sum;
    for (int w = 0; w < tid >> 5; ++w) at += warp_sum[w];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int np = (c[j] + kCols - 1) / kCols, off = at & 0xffff;
      for (int p = 0; p < np; ++p)
        passes[(at >> 16) + p] = pack_pass(4 * tid + j, min(kCols, c[j] - p * kCols), off + p * kCols);
      first[4 * tid + j] = off;
      at += c[j] + (np << 16);
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) {
    const int t = i / a.K, e = kept(i, t);
    if (e >= 0) routes[first[e] + __popcll(tokens[e] & ((1ull << t) - 1))] = static_cast<uint16_t>(i);
  }
  // the scratch becomes a ring that TMA writes
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  return total >> 16;
}

// ----------------------------------------------------------------- products
// The lane's 64 bytes of a group record: the pairs of words 0..3.
__device__ __forceinline__ void load_column(uint4* v, const uint8_t* rec, int q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(rec + i * 64 + q * 16);
}

__device__ __forceinline__ void mma_16x8x16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc += 2^-24 * scale * (codes - 8) . column over one 128-group; `p` is the
// lane's first row's 16 bytes in the box, sa and sb the scales of its two
// rows, t0 and t1 the record tails of its two columns.
__device__ __forceinline__ void w4_dot(float* acc, const uint8_t* p, uint32_t sa, uint32_t sb,
                                       const uint4* col, const RecordTail& t0, const RecordTail& t1) {
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
  acc[0] = fmaf(fa * t0.back, c[0] - t0.sum, acc[0]);
  acc[1] = fmaf(fa * t1.back, c[1] - t1.sum, acc[1]);
  acc[2] = fmaf(fb * t0.back, c[2] - t0.sum, acc[2]);
  acc[3] = fmaf(fb * t1.back, c[3] - t1.sum, acc[3]);
}

// The box row of lane group r (and, plus 8, of its second row).  In TMA's
// 128-byte swizzle the 16-byte chunk c of row m lies at c ^ (m & 7); the rows
// that share a quarter of a 512-byte access differ in bit 2, so their chunks
// lie in different halves of the 128 bytes.
__device__ __forceinline__ int box_row(int r) { return (r >> 1) | ((r & 1) << 2); }

// The scales of groups g and g + 1 of one row, the first in the low half; zero
// for a group that is not there.
__device__ __forceinline__ uint32_t load_scales(const uint16_t* row, int g, int G) {
  if ((G & 1) == 0) return __ldg(reinterpret_cast<const uint32_t*>(row + g));
  uint32_t v = __ldg(row + g);
  if (g + 1 < G) v |= static_cast<uint32_t>(__ldg(row + g + 1)) << 16;
  return v;
}

// Untiled copy of `bytes` (a multiple of 16, as both addresses are) into
// shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Brings `bytes` (a multiple of 16, as the address is) into L2.
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// One product's tiles and runs.  A tile: a pass's 128-row (gate/up) or
// 256-row (down) block of weight rows; its units are pairs of groups.
struct Product {
  int G, units;        // groups of K, units of a tile
  int row_tiles, nb;   // tiles of a pass, runs
  int64_t all;         // units in all
  // The first unit of run b, and the run of unit u: in 32 bits wherever the
  // products fit, as 64-bit divisions take about a microsecond of every join.
  __device__ int64_t start(int b) const {
    if (all < (1 << 22)) return static_cast<uint32_t>(all) * static_cast<uint32_t>(b) / static_cast<uint32_t>(nb);
    return all * b / nb;
  }
  __device__ int run_of(int64_t u) const {
    int b = all < (1 << 22) ? static_cast<uint32_t>(u) * static_cast<uint32_t>(nb) / static_cast<uint32_t>(all)
                            : static_cast<int>(u * nb / all);
    return start(b + 1) <= u ? b + 1 : b;
  }
};
__device__ __forceinline__ Product product_of(const W4Args& a, bool down, int np) {
  Product p;
  p.G = (down ? a.I : a.H) / kGroup;
  p.units = (p.G + 1) / 2;
  p.row_tiles = down ? (a.H + 2 * kBoxRows - 1) / (2 * kBoxRows) : a.I / kBoxRows;
  p.all = static_cast<int64_t>(np) * p.row_tiles * p.units;
  p.nb = static_cast<int>(min(static_cast<int64_t>(kW4MaxBlocks), (p.all + kRunUnits - 1) / kRunUnits));
  return p;
}

// A place in a run: unit s of tile t of pass p, with `left` units to go.
struct Walk {
  int s, t, p, tile, left;
  // On from the tile's unit `end`, which the tile or the run ends at.
  __device__ void next_tile(const Product& pr, int end) {
    left -= end - s;
    s = 0;
    ++tile;
    if (++t == pr.row_tiles) {
      t = 0;
      ++p;
    }
  }
};
__device__ __forceinline__ Walk walk_of(const Product& pr, int b) {
  const int64_t f0 = pr.start(b);
  Walk w;
  w.left = static_cast<int>(pr.start(b + 1) - f0);
  w.tile = static_cast<uint32_t>(f0) / static_cast<uint32_t>(pr.units);
  w.s = static_cast<int>(f0 - static_cast<int64_t>(w.tile) * pr.units);
  w.t = w.tile % pr.row_tiles;
  w.p = w.tile / pr.row_tiles;
  return w;
}

// Where a tile's sums are: `count` runs' in order from `first` (in units of two
// slots), the first run's in slot `slot`, the others' in slot 0.
struct Sums {
  int first, count, slot;
};

// Finishes columns [c0, c0 + C) of a tile with one warp, lane i rows 4i..4i+3
// of both boxes: adds the runs' sums in order and writes the down product's
// rows, or z of the tile's 128-group as an operand record.
template <int C>
__device__ __forceinline__ void w4_finish(const W4Args& a, const Sums& from, bool down, const Walk& at,
                                          int row_tiles, const Pass& pass, const uint16_t* routes, int c0,
                                          int lane) {
  float v[C][8];
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] = 0.f;
  for (int b = 0; b < from.count; b += 4) {
    float4 in[4][C][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at_slot = (from.first + b + k) * 2 + (b + k == 0 ? from.slot : 0);
      const float4* p = reinterpret_cast<const float4*>(a.part + static_cast<int64_t>(at_slot) * kTileSums +
                                                        c0 * kTileRows) + lane;
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          in[k][j][h] = b + k < from.count && c0 + j < pass.n
                            ? __ldcg(p + j * (kTileRows / 4) + h * (kBoxRows / 4))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v[j][4 * h] += in[k][j][h].x;
          v[j][4 * h + 1] += in[k][j][h].y;
          v[j][4 * h + 2] += in[k][j][h].z;
          v[j][4 * h + 3] += in[k][j][h].w;
        }
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    if (c0 + j >= pass.n) break;
    const int64_t route = routes[pass.off + c0 + j];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] *= 0x1p24f;
    if (down) {
      float* o = a.o + route * a.H + at.t * kTileRows + 4 * lane;
      *reinterpret_cast<float4*>(o) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
      if (at.t * kTileRows + kBoxRows < a.H)
        *reinterpret_cast<float4*>(o + kBoxRows) = make_float4(v[j][4], v[j][5], v[j][6], v[j][7]);
      continue;
    }
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float gate = v[j][k];
      v[j][k] = gate / (1.f + expf(-gate)) * v[j][4 + k];
      m = max(m, __float_as_uint(v[j][k]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    RecordTail tail;
    const float mult = operand_scale(m, &tail.back);
    float sum = 0.f;
    uint32_t words[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const __half2 h = __floats2half2_rn(operand_value(v[j][2 * k], mult),
                                          operand_value(v[j][2 * k + 1], mult) * 0.0625f);
      const float2 back = __half22float2(h);
      sum += back.x + back.y * 16.f;
      words[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    // an even lane's elements and the next lane's are the record's pairs
    const uint32_t next0 = __shfl_xor_sync(0xffffffffu, words[0], 1);
    const uint32_t next1 = __shfl_xor_sync(0xffffffffu, words[1], 1);
    uint8_t* rec = a.zs + route * operand_row_bytes(a.I) + at.t * kOpBytes;
    if ((lane & 1) == 0)
      *reinterpret_cast<uint4*>(rec + record_word(lane >> 1)) =
          make_uint4(__byte_perm(words[0], next0, 0x5410), __byte_perm(words[0], next0, 0x7632),
                     __byte_perm(words[1], next1, 0x5410), __byte_perm(words[1], next1, 0x7632));
    tail.sum = sum * 0x1p-21f;
    if (lane == 0) *reinterpret_cast<RecordTail*>(rec + 256) = tail;
    // the record past an odd number of groups: zeros
    if ((row_tiles & 1) && at.t == row_tiles - 1 && lane < kOpBytes / 16)
      *reinterpret_cast<uint4*>(rec + kOpBytes + lane * 16) = make_uint4(0, 0, 0, 0);
  }
}

// Counts columns of z that the warp has written.
__device__ __forceinline__ void w4_count(int* pass_count, int columns, int lane) {
  fence_proxy_async();
  __syncwarp();
  if (lane == 0)
    asm volatile("fence.acq_rel.gpu;\n\tred.release.gpu.global.add.s32 [%0], %1;" ::"l"(pass_count), "r"(columns)
                 : "memory");
}

// ------------------------------------------------------------------- stream
struct W4Maps {
  CUtensorMap w13, w2;
};

template <typename IdT>
__global__ void __launch_bounds__(kW4Threads, 2)
    w4_stream_kernel(const __grid_constant__ W4Maps maps, const W4Args a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kStages], s_empty[kStages], s_run_full[2], s_run_empty[2];
  __shared__ uint64_t s_sums[2], s_free[2];   // a tile's sums are there, are done with
  __shared__ uint64_t s_last;                 // the sums of a run's last tile: s_from
  __shared__ Sums s_from;
  __shared__ int s_run[2], s_abort;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);   // [kStages][2 boxes]
  uint8_t* cols = ring + kStages * 2 * kBoxBytes;                // [kStages][kCols][kColBytes]
  uint32_t* passes = reinterpret_cast<uint32_t*>(cols + kStages * kCols * kColBytes);
  uint16_t* routes = reinterpret_cast<uint16_t*>(passes + a.max_passes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kW4Warps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_run_full[i], 1);
      mbar_init(&s_run_empty[i], kW4Warps + 1);
      mbar_init(&s_sums[i], kW4Warps);
      mbar_init(&s_free[i], kW4Warps);
    }
    mbar_init(&s_last, 1);
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.w13);
    tma_prefetch_desc(&maps.w2);
  }
  const int np = w4_plan<IdT>(a, passes, routes, ring);
  const Product prod[2] = {product_of(a, false, np), product_of(a, true, np)};
  const int runs = prod[0].nb + prod[1].nb;
  volatile int* abort_flag = &s_abort;
  grid_dependency_wait();   // x's operands, the counters, and the readers of old outputs
  if (warp == kW4Warps) {
    // ------------------------------------------------------------- producer
    // What this warp does between a free stage and the copies into it is on the
    // stream's critical path: coordinates and addresses are worked out per tile.
    // Lane 0 fetches the codes and lane c column c of the operands.  Lanes 0
    // and 1 also bring the two boxes' scales of a tile, which are contiguous,
    // into L2 a tile ahead: the warps read them row by row, 32 bytes at a time,
    // which behind the queue of codes takes longer than a unit's products.
    int slot = 0, issued = 0;
    uint32_t phase = 1;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      int run = 0;
      if (lane == 0) run = atomicAdd(&a.count->ticket, 1);
      run = __shfl_sync(0xffffffffu, run, 0);
      if (!__all_sync(0xffffffffu, mbar_wait(&s_run_empty[i & 1], ((i >> 1) & 1) ^ 1, abort_flag))) {
        ok = false;
        break;
      }
      if (lane == 0) {
        s_run[i & 1] = run;
        mbar_arrive(&s_run_full[i & 1]);
      }
      if (run >= runs) break;
      const bool down = run >= prod[0].nb;
      const Product pr = down ? prod[1] : prod[0];
      const CUtensorMap* map = down ? &maps.w2 : &maps.w13;
      const uint8_t* ops = down ? a.zs : a.xs;
      const int64_t op_row = operand_row_bytes(down ? a.I : a.H);
      auto prefetch_scales = [&](const Walk& v) {
        const int e = unpack_pass(passes[v.p]).e;
        const int in = down ? v.t * 2 * kBoxRows + lane * kBoxRows : v.t * kBoxRows;   // of the rows
        if (lane >= 2 || (down && in >= a.H)) return;
        const int64_t row = down ? static_cast<int64_t>(e) * a.H + in : static_cast<int64_t>(2 * e + lane) * a.I + in;
        bulk_prefetch((down ? a.s2 : a.s13) + row * pr.G, kBoxRows * pr.G * 2);
      };
      Walk w = walk_of(pr, down ? run - prod[0].nb : run);
      prefetch_scales(w);
      int have = -1;   // the pass whose z is known to be there
      while (w.left > 0 && ok) {
        const Pass pass = unpack_pass(passes[w.p]);
        const bool both = !down || w.t * 2 * kBoxRows + kBoxRows < a.H;
        const uint32_t bytes = (both ? 2 : 1) * kBoxBytes + pass.n * kColBytes;
        const int row = down ? pass.e * a.H + w.t * 2 * kBoxRows : pass.e * 2 * a.I + w.t * kBoxRows;
        const int row2 = row + (down ? kBoxRows : a.I);
        const int end = min(w.s + w.left, pr.units);
        const uint8_t* src = nullptr;
        if (lane < pass.n) {
          const int route = routes[pass.off + lane];
          src = ops + (down ? route : route / a.K) * op_row + w.s * kColBytes;
        }
        Walk after = w;
        after.next_tile(pr, end);
        if (after.left > 0) prefetch_scales(after);
        // z may not be there yet, and codes need not wait for it: as many units
        // as there are stages go out without their operands first
        const bool wait_z = down && w.p != have;
        int behind = 0;
        for (int s = w.s; s < end; ++s, ++issued) {
          if (!__all_sync(0xffffffffu, mbar_wait(&s_empty[slot], phase, abort_flag))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            uint8_t* dst = ring + slot * 2 * kBoxBytes;
            mbar_arrive_expect_tx(&s_full[slot], bytes);
            tma_load_2d(dst, map, &s_full[slot], s * 128, row);
            if (both) tma_load_2d(dst + kBoxBytes, map, &s_full[slot], s * 128, row2);
          }
          __syncwarp();   // the expected bytes stand before an operand's can land
          if (wait_z && w.p != have) {
            ++behind;
            if (behind == kStages || s + 1 == end) {
              if (!__all_sync(0xffffffffu, wait_count(&a.count->pass[w.p], prod[0].row_tiles * pass.n, abort_flag))) {
                ok = false;
                ++issued;
                break;
              }
              fence_proxy_async();
              have = w.p;
              for (int k = 0, at = slot + 1 - behind + (slot + 1 < behind ? kStages : 0); k < behind; ++k) {
                if (src != nullptr) {
                  bulk_load(cols + (at * kCols + lane) * kColBytes, src, kColBytes, &s_full[at]);
                  src += kColBytes;
                }
                if (++at == kStages) at = 0;
              }
            }
          } else if (src != nullptr) {
            bulk_load(cols + (slot * kCols + lane) * kColBytes, src, kColBytes, &s_full[slot]);
            src += kColBytes;
          }
          if (++slot == kStages) {
            slot = 0;
            phase ^= 1;
          }
        }
        w = after;
      }
    }
    if (!ok) {
      // no copy may land after the block has ended
      *abort_flag = 1;
      for (int i = 0; i < min(issued, kStages); ++i) {
        const int n = issued - 1 - i;
        int none = 0;
        mbar_wait(&s_full[n % kStages], (n / kStages) & 1, &none);
      }
      if (lane == 0) atomicOr(a.dev_status, kDevTimeout);
    }
    return;
  }

  // Where a tile's sums go: a shared tile's to its run (its first tile is slot
  // 0, its last slot 1), a whole tile's to the block.
  auto sums_of = [&](bool shared, bool down, int b, int slot) {
    const int at = shared ? (down ? kW4MaxBlocks : 0) + b : 2 * kW4MaxBlocks + static_cast<int>(blockIdx.x);
    return a.part + static_cast<int64_t>(at * 2 + slot) * kTileSums;
  };
  // A wait that ran out ends the block: the flag ends every other wait in it.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag))) return true;
    *abort_flag = 1;
    if (lane == 0) atomicOr(a.dev_status, kDevTimeout);
    return false;
  };
  if (warp == kW4Warps + 1) {
    // -------------------------------------------------------------- finisher
    // Takes the tiles' sums off the warps that compute, which go on with the
    // next tile: a join's fence and counter, the other runs' sums and z's
    // records take microseconds, in which the ring would stand full.
    for (int i = 0, tiles = 0;; ++i) {
      if (!wait(&s_run_full[i & 1], (i >> 1) & 1)) return;
      const int run = s_run[i & 1];
      __threadfence_block();   // as for a stage below
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_run_empty[i & 1]);
      if (run >= runs) return;
      const bool down = run >= prod[0].nb;
      const Product pr = down ? prod[1] : prod[0];
      const int b = down ? run - prod[0].nb : run;
      Walk w = walk_of(pr, b);
      const bool is_short = w.left <= pr.units;
      for (; w.left > 0; ++tiles) {
        const Walk at = w;
        const int end = min(w.s + w.left, pr.units);
        w.next_tile(pr, end);
        if (down && at.s == 0 && end == pr.units) {   // its rows are stored as they are
          --tiles;
          continue;
        }
        if (!wait(&s_sums[tiles & 1], (tiles >> 1) & 1)) return;
        Sums from{2 * kW4MaxBlocks + static_cast<int>(blockIdx.x), 1, tiles & 1};
        if (at.s != 0 || end != pr.units) {
          // go on only as the last of the tile's runs
          const int64_t first = static_cast<int64_t>(at.tile) * pr.units, last = first + pr.units - 1;
          const int b0 = pr.run_of(first), b1 = pr.run_of(last);
          int before = 0;
          if (lane == 0) {
            __threadfence();   // over the block's sums, which the barrier ordered before
            before = atomicAdd(&a.count->tile[down][b0], 1);
          }
          before = __shfl_sync(0xffffffffu, before, 0);
          // of the runs only b0 can have begun before the tile
          from = Sums{(down ? kW4MaxBlocks : 0) + b0, before == b1 - b0 ? b1 - b0 + 1 : 0,
                      pr.start(b0) < first ? 1 : 0};
          __threadfence();
        }
        const Pass pass = unpack_pass(passes[at.p]);
        if ((w.left == 0 || is_short) && pass.n >= kShareColumns) {
          // the other warps have nothing else to do, or little
          if (lane == 0) {
            s_from = from;
            mbar_arrive(&s_last);
          }
          continue;
        }
        if (from.count != 0) {
          for (int c0 = 0; c0 < pass.n; c0 += 2)
            w4_finish<2>(a, from, down, at, pr.row_tiles, pass, routes, c0, lane);
          if (!down) w4_count(&a.count->pass[at.p], pass.n, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_n(&s_free[tiles & 1], kW4Warps);
      }
    }
  }

  // ------------------------------------------------------------------ products
  const int r = lane >> 2, q = lane & 3;
  const int row = box_row(r);
  // the lane's first row in a box, for the first and the second group
  const int off0 = (warp * kRows + row) * 128 + ((q ^ (row & 7)) << 4), off1 = off0 ^ 64;
  int slot = 0;
  uint32_t phase = 0, last_phase = 0;
  for (int i = 0, tiles = 0;; ++i) {
    if (!wait(&s_run_full[i & 1], (i >> 1) & 1)) return;
    const int run = s_run[i & 1];
    __threadfence_block();   // as for a stage below
    __syncwarp();
    if (lane == 0) mbar_arrive(&s_run_empty[i & 1]);
    if (run >= runs) return;
    const bool down = run >= prod[0].nb;
    const Product pr = down ? prod[1] : prod[0];
    const int b = down ? run - prod[0].nb : run;
    const uint16_t* scales = down ? a.s2 : a.s13;
    const int64_t second = static_cast<int64_t>(down ? kBoxRows : a.I) * pr.G;   // the second box's rows
    // The scales of a unit are loaded one unit ahead of their use.
    uint32_t next[4];
    auto scales_of = [&](const Walk& v, int s) {
      const int e = unpack_pass(passes[v.p]).e;
      const int first = down ? e * a.H + v.t * kTileRows : e * 2 * a.I + v.t * kBoxRows;
      const uint16_t* sp = scales + static_cast<int64_t>(first + warp * kRows + row) * pr.G;
      const bool two = !down || v.t * kTileRows + kBoxRows < a.H;
      next[0] = load_scales(sp, 2 * s, pr.G);
      next[1] = load_scales(sp + 8 * pr.G, 2 * s, pr.G);
      next[2] = two ? load_scales(sp + second, 2 * s, pr.G) : 0u;
      next[3] = two ? load_scales(sp + second + 8 * pr.G, 2 * s, pr.G) : 0u;
    };
    Walk w = walk_of(pr, b);
    const bool is_short = w.left <= pr.units;
    scales_of(w, w.s);
    for (bool begun = true; w.left > 0; begun = false, ++tiles) {
      const Walk at = w;
      const int end = min(w.s + w.left, pr.units);
      w.next_tile(pr, end);
      float acc[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[k][j] = 0.f;
      for (int u = at.s; u < end; ++u) {
        uint32_t sc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = next[j];
        if (u + 1 < end) scales_of(at, u + 1);
        else if (w.left > 0) scales_of(w, 0);
        if (!wait(&s_full[slot], phase)) return;
        const uint8_t* box = ring + slot * 2 * kBoxBytes;
        const uint8_t* col = cols + slot * kCols * kColBytes;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint4 v[4];
          load_column(v, col + r * kColBytes + g * kOpBytes, q);
          const uint8_t* tails = col + 2 * q * kColBytes + g * kOpBytes + 256;
          const RecordTail tail0 = *reinterpret_cast<const RecordTail*>(tails);
          const RecordTail tail1 = *reinterpret_cast<const RecordTail*>(tails + kColBytes);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            w4_dot(acc[k], box + k * kBoxBytes + (g ? off1 : off0),
                   g ? sc[2 * k] & 0xFFFF0000u : sc[2 * k] << 16,
                   g ? sc[2 * k + 1] & 0xFFFF0000u : sc[2 * k + 1] << 16, v, tail0, tail1);
        }
        // Every lane's reads are over before lane 0 gives the stage back: without
        // the fence some were seen to come after the copy that the arrival let in.
        __threadfence_block();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[slot]);
        if (++slot == kStages) {
          slot = 0;
          phase ^= 1;
        }
      }
      // the sums of rows (row, row + 8) of both boxes and columns (2q, 2q + 1)
      const Pass pass = unpack_pass(passes[at.p]);
      if (down && at.s == 0 && end == pr.units) {
        // a whole tile of the last product needs no finish: 37 tokens on 13 experts of
        // 896 x 256, one unit a tile, 20 us (23 through the finisher)
        const bool both = at.t * kTileRows + kBoxRows < a.H;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (2 * q + j >= pass.n) continue;
          float* o = a.o + static_cast<int64_t>(routes[pass.off + 2 * q + j]) * a.H + at.t * kTileRows +
                     warp * kRows + row;
          o[0] = acc[0][j] * 0x1p24f;
          o[8] = acc[0][2 + j] * 0x1p24f;
          if (both) {
            o[kBoxRows] = acc[1][j] * 0x1p24f;
            o[kBoxRows + 8] = acc[1][2 + j] * 0x1p24f;
          }
        }
        --tiles;
        continue;
      }
      if (!wait(&s_free[tiles & 1], ((tiles >> 1) & 1) ^ 1)) return;
      const int n = pass.n;
      const bool shared = at.s != 0 || end != pr.units;
      float* out = sums_of(shared, down, b, shared ? !begun : tiles & 1) + 2 * q * kTileRows + warp * kRows + row;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (2 * q + j >= n) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) out[j * kTileRows + k * kBoxRows + 8 * h] = acc[k][2 * h + j];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_sums[tiles & 1]);
      if ((w.left == 0 || is_short) && n >= kShareColumns) {
        // a column a warp
        if (!wait(&s_last, last_phase)) return;
        last_phase ^= 1;
        const Sums from = s_from;
        if (from.count != 0 && warp < n) {
          __threadfence();
          w4_finish<1>(a, from, down, at, pr.row_tiles, pass, routes, warp, lane);
          if (!down) w4_count(&a.count->pass[at.p], 1, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[tiles & 1]);
      }
    }
  }
}

// ------------------------------------------------------------------ combine
// y[t] = bf16(sum over k ascending of w * o), a repeated expert by its first
// route; four elements of H per thread.
template <typename IdT>
__global__ void __launch_bounds__(256) w4_combine_kernel(const W4Args a) {
  __shared__ int s_row[32];
  __shared__ float s_w[32];
  const int t = blockIdx.y, K = a.K;
  if (static_cast<int>(threadIdx.x) < K) {
    const IdT* ids = static_cast<const IdT*>(a.topk_idx) + static_cast<int64_t>(t) * K;
    const int64_t id = static_cast<int64_t>(ids[threadIdx.x]);
    int k = -1;
    if (id >= 0 && id < a.E)
      for (k = 0; static_cast<int64_t>(ids[k]) != id;) ++k;
    s_row[threadIdx.x] = k < 0 ? -1 : t * K + k;
    s_w[threadIdx.x] = a.topk_w[static_cast<int64_t>(t) * K + threadIdx.x];
  }
  __syncthreads();
  grid_dependency_wait();
  const int h = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (h >= a.H) return;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < K; ++k) {
    if (s_row[k] < 0) continue;
    const float4 o = __ldcg(reinterpret_cast<const float4*>(a.o + static_cast<int64_t>(s_row[k]) * a.H + h));
    y.x = fmaf(s_w[k], o.x, y.x);
    y.y = fmaf(s_w[k], o.y, y.y);
    y.z = fmaf(s_w[k], o.z, y.z);
    y.w = fmaf(s_w[k], o.w, y.w);
  }
  *reinterpret_cast<uint2*>(a.y + static_cast<int64_t>(t) * a.H + h) =
      make_uint2(pack_bf16x2_rn(y.x, y.y), pack_bf16x2_rn(y.z, y.w));
}

// Offsets of the workspace's parts.
struct W4Workspace {
  size_t xs, zs, o, count, part, total;
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
  w.xs = take(static_cast<size_t>(T) * operand_row_bytes(H));
  w.zs = take(n * operand_row_bytes(I));
  w.o = take(n * H * 4);
  w.count = take(sizeof(W4Counters));
  w.part = take(static_cast<size_t>(kW4MaxBlocks) * 6 * kTileSums * 4);
  w.total = off;
  return w;
}

// A launch that may start while the one before in the stream still runs.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                             cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
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

template <typename IdT>
cudaError_t launch_w4(const W4Args& a, const W4Maps& maps, int sm_count, cudaStream_t s) {
  const int smem = 1024 + kStages * kStageBytes + 4 * a.max_passes + 2 * a.T * a.K;
  constexpr int kMaxSmem = 1024 + kStages * kStageBytes + 4 * kMaxPasses + 2 * kMaxRoutes;
  static_assert(kPlanScratch + 2 * kMaxRoutes <= kStages * kStageBytes && kMaxSmem <= 200 * 1024,
                "the plan's scratch fits the ring, the ring the SM");
  cudaError_t err = cudaFuncSetAttribute(w4_stream_kernel<IdT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (err != cudaSuccess) return err;
  w4_prepare_kernel<IdT><<<a.T, kPrepThreads, 0, s>>>(a);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  err = launch_dependent(w4_stream_kernel<IdT>, dim3(std::min(kW4MaxBlocks, 2 * sm_count)), kW4Threads,
                         smem, s, maps, a);
  if (err != cudaSuccess) return err;
  return launch_dependent(w4_combine_kernel<IdT>, dim3((a.H + 1023) / 1024, a.T), 256, 0, s, a);
}

}  // namespace

size_t experts_w4_workspace(int T, int K, int H, int I) { return w4_workspace(T, K, H, I).total; }

cudaError_t launch_experts_w4(const void* x, const void* topk_idx, int idx_bits,
                              const float* topk_w, int T, int H, int I, int K, int E,
                              const uint8_t* w13, const void* w13_scale, const uint8_t* w2,
                              const void* w2_scale, void* workspace, void* y,
                              int32_t* dev_status, int sm_count, cudaStream_t s) {
  if (T == 0) return cudaMemsetAsync(dev_status, 0, 2 * sizeof(int32_t), s);
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
  a.xs = ws + w.xs;
  a.zs = ws + w.zs;
  a.o = reinterpret_cast<float*>(ws + w.o);
  a.count = reinterpret_cast<W4Counters*>(ws + w.count);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.T = T;
  a.H = H;
  a.I = I;
  a.K = K;
  a.E = E;
  a.max_passes = std::min(E, T * K) + T * K / kCols;
  W4Maps maps;
  cudaError_t err = make_map_rows128(&maps.w13, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w13, H / 2,
                                     static_cast<uint64_t>(E) * 2 * I, kBoxRows);
  if (err == cudaSuccess)
    err = make_map_rows128(&maps.w2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w2, I / 2,
                           static_cast<uint64_t>(E) * H, kBoxRows);
  if (err != cudaSuccess) return err;
  return idx_bits == 32 ? launch_w4<int32_t>(a, maps, sm_count, s)
                        : launch_w4<int64_t>(a, maps, sm_count, s);
}

}  // namespace moe
