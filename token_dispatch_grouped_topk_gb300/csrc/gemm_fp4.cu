// Grouped products in microscaled 4-bit floating point on tcgen05: ragged rows
// per expert, block scales applied by the tensor cores.
//
//   P[m, n] = ga * gw[e] * sum_k (sa[m, k/B] a[m, k]) * (sw[n, k/B] w[e, n, k])
// with e2m1 codes a, w, the block scales of the format (fp4.cuh) and the fp32
// scales over the tensors:
//   down     out = bf16(P), any contraction K and output width N.  The rows are
//     BF16 between this product and the combine, as on the FP8 path: out is the
//     caller's buffer, and fp32 rows would double what both move of it (the
//     combine is bound by that).  It is a rounding of at most 2^-8 more than y's
//     own: 2.3e-3 instead of 1.7e-3 of a layer's outputs against 64 bits;
//   gate/up  Z = SiLU(G) * U with G and U the products with the first and the
//            last I rows of W13, fp32, requantised to 4 bits per block
//            ("SGLang Expert Compute Backend", §1.1 and §3.6, on other codes).
// Each expert's valid rows are tiled on their own (§2.4); only tiles that hold
// valid rows are scheduled, and only valid rows are stored.  A launch computes
// one product or, for few tiles, both ("XTuner Domino EP", HyperParallel-MoE
// section: a task starts when the tiles it needs are done).
//
// Design (one CTA per SM, persistent):
//  - tiles of 128 rows x 256 columns (gate/up: 128 gate and 128 up rows of W13),
//    one fp32 accumulator of 256 TMEM columns, N slices of one 128-row block
//    adjacent in the walk;
//  - warp 0 finds the tiles, passes them to the other warps through a ring and
//    streams their codes with TMA: stages of K = 256, 128 bytes a row, the
//    128-byte swizzle; kStages of them in a ring;
//  - warps 2-7 lay the scales of a stage out in shared memory as tcgen05.cp
//    wants them.  Scales are stored [row, K / B] like the codes, 16 (8) bytes a
//    stage and row, while the MMA takes for every 64 of K one 32-bit word a row,
//    the words of rows r, r + 32, r + 64, r + 96 side by side: a lane loads the
//    scales of those four rows, transposes 4 x 4 words in registers and stores
//    16 bytes per 64 of K.  So scales need no layout of their own: neither the
//    weights' (kept as they come) nor the activations', whose rows are ragged;
//  - warp 1 issues, per stage, the copies of the scales to TMEM and four MMAs
//    (M = 128, N = 256, K = 64).  Copies and MMAs of one thread run in order, so
//    one set of scale columns is enough.  Both issuing warps run converged up to
//    elect_one: behind a lane test each of the 16 instructions of a stage took 50
//    to 70 clocks, against 128 of an MMA (16384 tokens, 256 experts of 7168 x
//    2048: gate/up 2083 -> 1633 us with this alone);
//  - warps 8-15 take the accumulator to registers (64 gate and 64 up columns, or
//    128 columns of a row each), hand it back at once, and finish the tile while
//    the next one's products run.  A Z block lies in one thread, so its scale
//    needs no exchange.
//  - a launch of both lists all gate/up tiles, then all down tiles, and takes them
//    in that order by a ticket.  Each epilogue warp counts its part of a block's Z
//    (release); the producer passes a down tile on once its block's count is full
//    (acquire).
//
// What bounds it.  Many rows: what an SM can take in, 64 bytes a clock: 48 KB of
// codes and 6 KB of scales a stage are 850 clocks, the four MMAs 512 and the
// twelve copies about 120.  Counted on 16 full experts of 768 rows, gate/up takes
// in 55 bytes a clock over the whole launch (tensor pipe 51 %); down 42 (39 %),
// whose tiles are eight stages long, so that draining the accumulator and storing
// 64 KB of BF16 a tile weigh as well.  16384 tokens (above, 122380 rows kept):
// gate/up 1511 us, 4.8 PFLOP/s, down 968 us, 3.7; without the scale loads 8 to 15 %
// less, without code loads 1210 and 720.  Few rows: weights, 256 tokens to 64
// experts of 4096 x 1536 (both products) 112 us, 6.2 TB/s of DRAM.  One token, 8
// experts of 7168 x 2048: 46 us for 29 of weights; the rest is two products' first
// loads and last tiles.
// Every wait is bounded; on expiry the kernel raises MOE_DEV_TIMEOUT in the
// status word, drains its own copies and MMAs, frees TMEM and returns.
#include <algorithm>

#include "fp4.cuh"
#include "kernels.h"
#include "tensormap.h"

namespace moe {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 256;
constexpr int kBK = 256;         // elements of a stage: 128 bytes of codes a row
constexpr int kRowBytes = kBK / 2;
constexpr int kStages = 3;
constexpr int kScaleWarp0 = 2;   // two each for the rows' scales and both halves of the columns'
constexpr int kScaleWarps = 6;
constexpr int kEpiWarp0 = 8;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
// Register split: launched at 128 a thread; the two warpgroups that feed the
// tensor cores keep 96, the two epilogue warpgroups take 160.
constexpr int kLaunchRegs = 128;
constexpr int kCtrlRegs = 96;
constexpr int kEpiRegs = 160;
static_assert(2 * kCtrlRegs + 2 * kEpiRegs == 4 * kLaunchRegs, "register split must fit the launch");
// BF16 rows are staged per epilogue warp: 32 rows x 64 bytes, padded to 80.
constexpr int kStageRowBytes = 80;
constexpr int kStageWarpBytes = 32 * kStageRowBytes;
constexpr int kMaxExperts = 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfaCol = 256, kSfbCol = 272;   // scale columns behind the accumulator

// What a launch computes: the gate/up product, the down product (any product),
// or both, each down tile starting once its block's gate/up tiles are done.
constexpr int kGateUp = 0;
constexpr int kDown = 1;
constexpr int kBoth = 2;
// The producer finds each tile and passes it to the other warps through a ring of
// this many slots.
constexpr int kTileSlots = 8;

struct Product {
  const uint8_t* as;   // [rows, K / B] scales of the rows
  const uint8_t* ws;   // [E, weight rows, K / B] scales of the weights
  const float* ag;     // [1] scale over the rows, or null
  const float* wg;     // [E] scale over an expert's weights, or null
  int K, N;            // N: output features (gate/up: I)
  int nt;              // N slices per 128-row block
};

struct Fp4Args {
  const int32_t* counts;
  Product g[2];         // [0] gate/up, [1] down
  const float* zg;      // gate/up: [1] scale over Z, or null
  uint8_t* zq;          // gate/up: [rows, I / 2]
  uint8_t* zs;          // gate/up: [rows, I / B]
  __nv_bfloat16* out;   // down: [rows, N]
  int* sched;           // both: [0] tile ticket, [1 + b] epilogue warps done with block b
  int E, R;
  int packed;
  int early;            // the next launch of the chain may start beside this one
  long long rows;       // buffer rows
  int32_t* dev_status;
};

struct Fp4Maps {
  CUtensorMap a[2][3];   // rows: boxes of 128, 64 and 32
  CUtensorMap b[2];
};

struct Tile {
  int gu;   // a gate/up tile
  int blk, e, n_blk, rows, cols, base;
  int nkb;  // stages; 0: no tile, the list has ended
};

struct alignas(16) Control {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t tfull;
  uint64_t tempty;
  uint64_t drain;
  uint64_t tile_full[kTileSlots];
  uint64_t tile_empty[kTileSlots];
  uint32_t tmem_base;
  int abort;
  Tile tiles[kTileSlots];
  int part[3][kThreads / 32];
  int light[kMaxExperts + 1];   // prefix of the experts with one row block
  int heavy[kMaxExperts + 1];   // prefix of the row blocks of those with more
  int cnt[kMaxExperts + 1];   // prefix of the clamped counts
};

template <int kFmt>
struct Layout {
  static constexpr int kScales = kBK / kFp4Block<kFmt>;   // scale bytes of a row and stage
  static constexpr int kAtoms = kScales / 4;              // 512-byte copies per 128 rows
  static constexpr int kABytes = kBM * kRowBytes;
  static constexpr int kBBytes = kBN * kRowBytes;
  static constexpr int kSaBytes = kAtoms * 512;
  static constexpr int kSbBytes = 2 * kAtoms * 512;
  static constexpr int kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes +
                                  sizeof(Control) + kEpiWarps * kStageWarpBytes;
  static_assert(kStageBytes % 1024 == 0 && kSmem <= 232448, "shared memory of a block");
};

__device__ __forceinline__ int row_blocks(const Control* ctl, const Fp4Args& a) {
  return ctl->light[a.E] + ctl->heavy[a.E];
}

// Tile t: the N slices of one 128-row block adjacent; a launch of both lists all
// gate/up tiles before all down tiles.
// Experts of one block bring their weights from DRAM, those of more mostly reuse
// them in L2: each on its own is bound by DRAM or by the SMs' intake.  So the two
// kinds are mixed evenly over the list, each in expert order (4096 tokens to 128
// skewed experts of 4096 x 1536, gate/up 243 -> 210 us, down 155 -> 128 us).
template <int kMode>
__device__ __forceinline__ Tile decode_tile(const Control* ctl, const Fp4Args& a, int t) {
  Tile r;
  const unsigned n_light = ctl->light[a.E], blocks = row_blocks(ctl, a);
  const int gu_tiles = kMode == kBoth ? static_cast<int>(blocks) * a.g[0].nt : 0;
  r.gu = kMode == kGateUp || (kMode == kBoth && t < gu_tiles);
  const Product& g = a.g[r.gu ? 0 : 1];
  const int local = r.gu ? t : t - gu_tiles;
  r.blk = local / g.nt;
  r.n_blk = local - r.blk * g.nt;
  // light ones before this block, in 32 bits (more than 2^21 blocks go unmixed)
  const unsigned p = r.blk;
  unsigned lights = min(p, n_light);
  bool is_light = p < n_light;
  if (n_light > 0 && n_light < blocks && blocks <= (1u << 21)) {
    lights = p * n_light / blocks;
    is_light = p * n_light - lights * blocks + n_light >= blocks;   // the next block has one more
  }
  int m_blk = 0;
  if (is_light) {
    r.e = find_expert(ctl->light, a.E, lights);
  } else {
    r.e = find_expert(ctl->heavy, a.E, p - lights);
    m_blk = p - lights - ctl->heavy[r.e];
  }
  const int m0 = m_blk * kBM;
  const int count = ctl->cnt[r.e + 1] - ctl->cnt[r.e];
  r.base = (a.packed ? ctl->cnt[r.e] : r.e * a.R) + m0;
  // packed rows past the buffer, which only wrong counts claim, are no rows
  r.rows = min(min(kBM, count - m0), static_cast<int>(max(0LL, min(static_cast<long long>(kBM), a.rows - r.base))));
  r.cols = r.gu ? kBN : min(kBN, g.N - r.n_blk * kBN);   // 128 in the last slice of an odd N / 128
  r.nkb = (g.K + kBK - 1) / kBK;
  return r;
}

// First weight row of column half h of a tile.
__device__ __forceinline__ int weight_row(const Fp4Args& a, const Tile& t, int h) {
  return t.gu ? (2 * t.e + h) * a.g[0].N + t.n_blk * 128 : t.e * a.g[1].N + t.n_blk * kBN + h * 128;
}

// A warp's tile number `it` from the ring; false if the wait ran out.
__device__ __forceinline__ bool claim_tile(Control* ctl, int it, int lane, Tile* tl) {
  const int slot = it % kTileSlots;
  if (!warp_wait(&ctl->tile_full[slot], (it / kTileSlots) & 1, &ctl->abort)) return false;
  *tl = ctl->tiles[slot];
  __syncwarp();
  if (lane == 0) mbar_arrive(&ctl->tile_empty[slot]);
  return true;
}

// Z is written by ordinary stores and read by TMA, in a launch of both by
// another block: a proxy fence on either side.
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ void red_add_release_gpu(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  int dummy = 0;
  mbar_wait(bar, parity, &dummy);
}

// The prefixes over the experts of the clamped counts, of the experts with one
// 128-row block and of the others' blocks; every thread of the block calls it.
// The counts may be the launch before's, still written while this one starts:
// they are read through L2, after the wait, by all threads at once (one round
// trip); a thread adds up two experts, a warp 64.
__device__ __forceinline__ void tile_prefixes(const Fp4Args& a, Control* ctl) {
  static_assert(2 * kThreads >= kMaxExperts, "two experts a thread");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = 2 * threadIdx.x;
  // of the first expert, of both, and with the threads before
  int one[3], own[3], sum[3];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int c = e + x < a.E ? max(0, min(__ldcg(a.counts + e + x), a.R)) : 0;
    const int nb = (c + kBM - 1) / kBM;
    const int v[3] = {nb == 1 ? 1 : 0, nb > 1 ? nb : 0, c};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (x == 0) one[i] = own[i] = v[i];
      else own[i] += v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) sum[i] = own[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int u = __shfl_up_sync(0xffffffffu, sum[i], o);
      if (lane >= o) sum[i] += u;
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < 3; ++i) ctl->part[i][warp] = sum[i];
  }
  __syncthreads();
  int* const to[3] = {ctl->light, ctl->heavy, ctl->cnt};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int before = sum[i] - own[i];
    for (int w = 0; w < min(warp, (a.E + 63) / 64); ++w) before += ctl->part[i][w];
    if (e <= a.E) to[i][e] = before;
    if (e + 1 <= a.E) to[i][e + 1] = before + one[i];
    if (e + 2 == a.E) to[i][e + 2] = before + own[i];
  }
  __syncthreads();
}

// kWords 32-bit words of a row's scales (one stage's) in the widest loads that
// the row pitch aligns; past the end of the row zeros.  Through L2: the rows'
// scales are the launch before's.
template <int kWords>
__device__ __forceinline__ void load_scales(const uint8_t* row, int off, int pitch, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < kWords; ++j) w[j] = 0;
  if (kWords == 4 && (pitch & 15) == 0) {
    if (off < pitch) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(row + off));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  } else if ((pitch & 7) == 0) {
#pragma unroll
    for (int j = 0; j < kWords; j += 2)
      if (off + 4 * j < pitch) {
        const uint2 v = __ldcg(reinterpret_cast<const uint2*>(row + off + 4 * j));
        w[j] = v.x, w[j + 1] = v.y;
      }
  } else {
#pragma unroll
    for (int j = 0; j < kWords; ++j)
      if (off + 4 * j < pitch) w[j] = __ldcg(reinterpret_cast<const uint32_t*>(row + off + 4 * j));
  }
}

// One of the warps that lay scales out: block sw (0: the tile's rows, 1 and 2:
// the halves of its columns), every other pair of stages of each tile, counted
// on over the tiles.  Lanes 2i and 2i + 1 take the first and the second stage of
// rows i, 16 + i, ..., 112 + i (for NVFP4 a load asks for whole sectors), so a
// stage's words of four rows 32 apart are one lane's.
// Pairs, not more: a parity tells a slot's current use only from the one before,
// and of the stages between a warp's own, which the other warp waits for, there
// may be kStages - 1.
template <int kFmt>
__device__ __forceinline__ bool lay_out_scales(const Fp4Args& args, Control* ctl, uint8_t* smem,
                                               int sw, int par, int lane) {
  using L = Layout<kFmt>;
  static_assert(kStages >= 3, "a pair of stages may lie between a warp's own");
  const int i = lane >> 1, h = lane & 1;
  int pairs = 0, stages = 0;   // of the tiles before
  for (int it = 0;; ++it) {
    Tile tl;
    if (!claim_tile(ctl, it, lane, &tl)) return false;
    if (tl.nkb == 0) return true;
    const Product& g = args.g[tl.gu ? 0 : 1];
    const int pitch = g.K / kFp4Block<kFmt>;
    // rows past the tile's (and columns past N) repeat one: their products are
    // not stored
    const int last = sw == 0 ? max(tl.rows - 1, 0) : (sw == 2 && tl.cols < kBN ? 0 : 127);
    const long long first = sw == 0 ? min(static_cast<long long>(tl.base), args.rows - 1)
                                    : weight_row(args, tl, last ? sw - 1 : 0);
    const uint8_t* base = (sw == 0 ? g.as : g.ws) + first * pitch;
    const int nch = (tl.nkb + 1) / 2;
    for (int ch = (par ^ pairs) & 1; ch < nch; ch += 2) {
      uint32_t w[8][L::kAtoms];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        load_scales<L::kAtoms>(base + min(16 * r + i, last) * pitch, (2 * ch + h) * L::kScales, pitch, w[r]);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int kb = 2 * ch + p;
        if (kb >= tl.nkb) break;
        const int n = stages + kb, stage = n % kStages;
        if (!warp_wait(&ctl->empty[stage], ((n / kStages) & 1) ^ 1, &ctl->abort)) return false;
        if (h == p) {
          // atom j of the rows at 512 j; of column half x at 1024 j + 512 x
          uint8_t* dst = smem + stage * L::kStageBytes + L::kABytes + L::kBBytes +
                         (sw == 0 ? 0 : L::kSaBytes + 512 * (sw - 1)) + 16 * i;
          const int step = sw == 0 ? 512 : 1024;
#pragma unroll
          for (int j = 0; j < L::kAtoms; ++j) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
              *reinterpret_cast<uint4*>(dst + j * step + 256 * r) =
                  make_uint4(w[r][j], w[r + 2][j], w[r + 4][j], w[r + 6][j]);
          }
          fence_proxy_async_shared();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->full[stage]);
      }
    }
    pairs += nch;
    stages += tl.nkb;
  }
}

template <int kFmt, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_fp4_kernel(const __grid_constant__ Fp4Maps maps, const Fp4Args args) {
  using L = Layout<kFmt>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  Control* ctl = reinterpret_cast<Control*>(smem + kStages * L::kStageBytes);
  uint8_t* out_stage = smem + kStages * L::kStageBytes + sizeof(Control);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Not from a capped grid: the next launch's blocks would sit down on the SMs
  // that it leaves to other streams, and hold them until this one ends.
  if (args.early) pdl_start();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ctl->full[i], 1 + kScaleWarps / 2);   // a stage's scales: one of each two
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->tfull, 1);
    mbar_init(&ctl->tempty, kEpiWarps);
    mbar_init(&ctl->drain, 1);
    for (int i = 0; i < kTileSlots; ++i) {
      mbar_init(&ctl->tile_full[i], 1);
      mbar_init(&ctl->tile_empty[i], 1 + kScaleWarps + kEpiWarps);
    }
    ctl->abort = 0;
    fence_barrier_init();
  }
  // the maps that every launch has: the smallest boxes of rows, the weights
  if (warp == 0 && lane < 4 && (kMode == kBoth || (lane >> 1) == kMode))
    tma_prefetch_desc(lane & 1 ? &maps.b[lane >> 1] : &maps.a[lane >> 1][2]);
  if (warp == 2) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  pdl_wait();
  tile_prefixes(args, ctl);   // its barrier also publishes the mbarriers and the TMEM address
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int total = row_blocks(ctl, args) * ((kMode == kDown ? 0 : args.g[0].nt) +
                                              (kMode == kGateUp ? 0 : args.g[1].nt));
  volatile int* abort_flag = &ctl->abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    warpgroup_reg_dealloc<kCtrlRegs>();
    int issued = 0;
    bool ok = true;
    // Finds tile `it` and passes it on; false if a wait ran out.
    auto pass_on = [&](int it, Tile* tl) {
      const int slot = it % kTileSlots;
      if (!warp_wait(&ctl->tile_empty[slot], ((it / kTileSlots) & 1) ^ 1, abort_flag)) return false;
      int t = blockIdx.x + it * gridDim.x;
      if (kMode == kBoth) {
        // Tiles are taken in list order by whichever blocks run, so the gate/up
        // tiles that a down tile waits for are held by running blocks, which
        // wait on nothing before them.
        if (lane == 0) t = atomicAdd(args.sched, 1);
        t = __shfl_sync(0xffffffffu, t, 0);
      }
      *tl = Tile{};
      if (t < total) *tl = decode_tile<kMode>(ctl, args, t);
      // A down tile is passed on once its block's Z is written: who takes it from
      // the ring is then behind Z's stores.
      if (kMode == kBoth && t < total && !tl->gu) {
        if (!__all_sync(0xffffffffu, wait_count(args.sched + 1 + tl->blk, kEpiWarps * args.g[0].nt, abort_flag)))
          return false;
        fence_proxy_async_global();
        __syncwarp();
      }
      if (lane == 0) {
        ctl->tiles[slot] = *tl;
        mbar_arrive(&ctl->tile_full[slot]);
      }
      return true;
    };
    // Tiles of a fixed order are passed on one ahead, so that the scale warps need
    // not wait for a tile's last loads to begin the next; a ticket is taken when
    // its tile is due.
    Tile nx{};
    if (kMode != kBoth) ok = pass_on(0, &nx);
    for (int it = 0; ok; ++it) {
      Tile tl = nx;
      if (kMode == kBoth) ok = pass_on(it, &tl);
      if (!ok || tl.nkb == 0) break;
      const int g = tl.gu ? 0 : 1;
      const int b0 = weight_row(args, tl, 0), b1 = weight_row(args, tl, 1);
      // only the valid rows are fetched (32, 64 or 128): the rest of the A
      // tile keeps stale bytes, which reach only rows that are never stored
      const int a_box = tl.rows <= 32 ? 32 : (tl.rows <= 64 ? 64 : kBM);
      const CUtensorMap* ma = &maps.a[g][a_box == kBM ? 0 : (a_box == 64 ? 1 : 2)];
      const CUtensorMap* mb = &maps.b[g];
      const uint32_t bytes = (a_box + tl.cols) * kRowBytes;
      for (int kb = 0; kb < tl.nkb; ++kb) {
        const int stage = issued % kStages;
        if (!warp_wait(&ctl->empty[stage], ((issued / kStages) & 1) ^ 1, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + stage * L::kStageBytes;
        uint8_t* sb = sa + L::kABytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(&ctl->full[stage], bytes);
          tma_load_2d(sa, ma, &ctl->full[stage], kb * kRowBytes, tl.base);
          tma_load_2d(sb, mb, &ctl->full[stage], kb * kRowBytes, b0);
          if (tl.cols == kBN)
            tma_load_2d(sb + 128 * kRowBytes, mb, &ctl->full[stage], kb * kRowBytes, b1);
        }
        __syncwarp();
        ++issued;
        if (kMode != kBoth && kb == 0 && !pass_on(it + 1, &nx)) {
          ok = false;
          break;
        }
      }
    }
    if (!ok) *abort_flag = 1;
    // No copy may land after the block exits.  full also takes the scale
    // warps' arrivals, which an abort leaves out, so this wait is bounded too
    // and then the copies have had the whole wait limit to land.
    for (int i = 0; i < min(issued, kStages); ++i) {
      const int n = issued - 1 - i;
      drain_wait(&ctl->full[n % kStages], (n / kStages) & 1);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    warpgroup_reg_dealloc<kCtrlRegs>();
    const uint32_t acc = __shfl_sync(0xffffffffu, tmem, 0);   // uniform
    int consumed = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      Tile tl;
      ok = claim_tile(ctl, it, lane, &tl);
      if (!ok || tl.nkb == 0) break;
      const bool half_end = args.g[tl.gu ? 0 : 1].K % kBK != 0;   // the last stage holds 128 elements
      if (!warp_wait(&ctl->tempty, (it & 1) ^ 1, abort_flag)) {
        ok = false;
        break;
      }
      for (int kb = 0; kb < tl.nkb; ++kb) {
        const int stage = consumed % kStages;
        if (!warp_wait(&ctl->full[stage], (consumed / kStages) & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem) + stage * L::kStageBytes;
        const uint32_t sfa = sa + L::kABytes + L::kBBytes, sfb = sfa + L::kSaBytes;
        const uint64_t adesc = smem_desc_kmajor_sw128(sa);
        const uint64_t bdesc = smem_desc_kmajor_sw128(sa + L::kABytes);
        const int steps = half_end && kb == tl.nkb - 1 ? 2 : 4;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {   // 64 elements = 32 bytes = 2 descriptor units
            if (k >= steps) break;
            const int atom = k * L::kAtoms / 4, id = kFmt == kMxfp4 ? 2 * (k & 1) : 0;
            if (k * L::kAtoms % 4 == 0) {
              tmem_copy_scales(acc + kSfaCol + 4 * atom, smem_desc_scales(sfa + 512 * atom));
              tmem_copy_scales(acc + kSfbCol + 8 * atom, smem_desc_scales(sfb + 1024 * atom));
              tmem_copy_scales(acc + kSfbCol + 8 * atom + 4, smem_desc_scales(sfb + 1024 * atom + 512));
            }
            const uint32_t idesc = tl.cols == kBN ? idesc_fp4<kFmt>(kBM, kBN, id)
                                                  : idesc_fp4<kFmt>(kBM, 128, id);
            mma_fp4<kFmt>(acc, adesc + 2 * k, bdesc + 2 * k, idesc, acc + kSfaCol + 4 * atom,
                          acc + kSfbCol + 8 * atom, (kb | k) > 0 ? 1u : 0u);
          }
          mma_commit(&ctl->empty[stage]);
          if (kb == tl.nkb - 1) mma_commit(&ctl->tfull);
        }
        __syncwarp();
        ++consumed;
      }
    }
    if (!ok) *abort_flag = 1;
    if (consumed > 0) {
      if (elect_one()) mma_commit(&ctl->drain);
      __syncwarp();
      drain_wait(&ctl->drain, 0);
    }
  } else if (warp < kEpiWarp0) {
    // -------------------------------------------------------------- scales
    warpgroup_reg_dealloc<kCtrlRegs>();
    const int sw = warp - kScaleWarp0;
    if (!lay_out_scales<kFmt>(args, ctl, smem, sw % 3, sw / 3, lane) && lane == 0)
      *abort_flag = 1;
  } else {
    // ------------------------------------------------------------ epilogue
    warpgroup_reg_alloc<kEpiRegs>();
    const int ew = warp - kEpiWarp0;
    const int lq = warp & 3;    // TMEM lane quarter of this warp
    const int ch = ew >> 2;     // half of the tile's columns
    const int row = lq * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lq * 32) << 16);
    const float zg = kMode != kDown && args.zg ? __ldcg(args.zg) : 1.f;
    const float six_zg = __fmul_rn(6.f, zg);
    bool ok = true;
    for (int it = 0;; ++it) {
      Tile tl;
      ok = claim_tile(ctl, it, lane, &tl);
      if (!ok || tl.nkb == 0) break;
      const Product& g = args.g[tl.gu ? 0 : 1];
      const float alpha = (g.ag ? __ldcg(g.ag) : 1.f) * (g.wg ? __ldcg(g.wg + tl.e) : 1.f);
      // gate/up: gate columns 64 ch.. and up columns 128 + 64 ch..; down: 128 ch..
      const uint32_t col0 = tl.gu ? 64 * ch : 128 * ch;
      const uint32_t col1 = tl.gu ? 128 + 64 * ch : 128 * ch + 64;
      if (!warp_wait(&ctl->tfull, it & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t p0[64], p1[64];
      tmem_load64_sync(t_lane + col0, p0);
      tmem_load64_sync(t_lane + col1, p1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->tempty);
      const long long grow = static_cast<long long>(tl.base) + row;
      const bool valid = row < tl.rows;
      if (kMode == kGateUp || (kMode == kBoth && tl.gu)) {
        // SiLU with the fast exponential and division: their few ulp are far
        // below a 4-bit step
        float z[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          const float g = __uint_as_float(p0[i]) * alpha, u = __uint_as_float(p1[i]) * alpha;
          z[i] = __fdividef(g, 1.0f + __expf(-g)) * u;
        }
        constexpr int kB = kFp4Block<kFmt>;
        uint32_t codes[8], scales = 0;
#pragma unroll
        for (int b = 0; b < 64 / kB; ++b) {
          uint32_t amax = 0;
#pragma unroll
          for (int i = 0; i < kB; ++i) amax = max(amax, abs_bits(z[b * kB + i]));
          float mult;
          scales |= static_cast<uint32_t>(fp4_block_scale<kFmt>(amax, zg, six_zg, &mult)) << (8 * b);
#pragma unroll
          for (int i = 0; i < kB / 8; ++i)
            codes[b * (kB / 8) + i] = fp4_pack8(z + b * kB + 8 * i, mult);
        }
        if (valid) {
          uint4* q = reinterpret_cast<uint4*>(args.zq + grow * (g.N / 2) + tl.n_blk * 64 + ch * 32);
          q[0] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
          q[1] = make_uint4(codes[4], codes[5], codes[6], codes[7]);
          uint8_t* s = args.zs + grow * (g.N / kB) + (tl.n_blk * 128 + ch * 64) / kB;
          if constexpr (kFmt == kNvfp4) *reinterpret_cast<uint32_t*>(s) = scales;
          else *reinterpret_cast<uint16_t*>(s) = static_cast<uint16_t>(scales);
        }
        if (kMode == kBoth) {   // this warp's part of the block's Z, to the down tiles
          fence_proxy_async_global();
          __threadfence();
          __syncwarp();
          if (lane == 0) red_add_release_gpu(args.sched + 1 + tl.blk, 1);
        }
      } else if (kMode != kGateUp) {
        // BF16 rows through the warp's stage: each round the lanes leave 32
        // columns of their rows, then the warp writes 8 rows x 64 bytes per store
        const unsigned vmask = __ballot_sync(0xffffffffu, valid);
        if (128 * ch < tl.cols) {
          uint8_t* stage = out_stage + ew * kStageWarpBytes;
          uint4* srow = reinterpret_cast<uint4*>(stage + lane * kStageRowBytes);
          const int c = lane & 3;
          __nv_bfloat16* gbase = args.out + (static_cast<long long>(tl.base) + lq * 32 + (lane >> 2)) * g.N +
                                 tl.n_blk * kBN + ch * 128 + 8 * c;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t o[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int p = 32 * r + 8 * j + 2 * i;
                const float lo = __uint_as_float(p < 64 ? p0[p & 63] : p1[p & 63]) * alpha;
                const float hi = __uint_as_float(p < 64 ? p0[(p & 63) + 1] : p1[(p & 63) + 1]) * alpha;
                o[i] = pack_bf16x2_rn(lo, hi);
              }
              srow[j] = make_uint4(o[0], o[1], o[2], o[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if ((vmask >> (8 * i + (lane >> 2))) & 1u) {
                const uint4 v = *reinterpret_cast<const uint4*>(
                    stage + (8 * i + (lane >> 2)) * kStageRowBytes + 16 * c);
                *reinterpret_cast<uint4*>(gbase + static_cast<long long>(8 * i) * g.N + 32 * r) = v;
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (!ok) *abort_flag = 1;
  }

  // --------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && ctl->abort) atomicOr(args.dev_status, kDevTimeout);
}

cudaError_t make_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  return make_map_rows128(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, cols, rows, box_rows);
}

// The most 128-row blocks that a launch can have.
long long max_blocks(int E, RowLayout rl) {
  const long long padded = static_cast<long long>(E) * ((rl.R + kBM - 1) / kBM);
  return rl.packed ? std::min<long long>(padded, rl.rows / kBM + std::min<long long>(E, rl.rows)) : padded;
}

// The most 128-row blocks that a layer of so many routes can have, whatever room
// its buffers hold.
long long layer_blocks(int E, RowLayout rl, int64_t routes) {
  return std::min<long long>(max_blocks(E, rl), routes / kBM + std::min<int64_t>(E, routes));
}

// R: no tile has more rows than that, so the larger boxes may go unused.
cudaError_t product_maps(Fp4Maps* m, int g, const uint8_t* a, uint64_t rows, int R, const uint8_t* w,
                         uint64_t w_rows, int K) {
  cudaError_t err = make_map(&m->a[g][2], a, K / 2, rows, 32);
  if (err == cudaSuccess && R > 32) err = make_map(&m->a[g][1], a, K / 2, rows, 64);
  if (err == cudaSuccess && R > 64) err = make_map(&m->a[g][0], a, K / 2, rows, kBM);
  if (err == cudaSuccess) err = make_map(&m->b[g], w, K / 2, w_rows, 128);
  return err;
}

template <int kFmt, int kMode>
cudaError_t launch_impl(const Fp4Maps& maps, const Fp4Args& args, long long max_tiles, int sm_count,
                        cudaStream_t s) {
  using L = Layout<kFmt>;
  if (args.E > kMaxExperts) return cudaErrorInvalidValue;
  auto* kernel = grouped_fp4_kernel<kFmt, kMode>;
  // The register split assumes exactly kLaunchRegs a thread; with any other
  // count the epilogue's increase could wait forever, so refuse to launch.
  static const int compiled_regs = [] {
    cudaFuncAttributes attr{};
    return cudaFuncGetAttributes(&attr, grouped_fp4_kernel<kFmt, kMode>) == cudaSuccess ? attr.numRegs : -1;
  }();
  if (compiled_regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const int grid = static_cast<int>(std::min<long long>(max_tiles, sm_count));
  if (grid <= 0) return cudaSuccess;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(L::kSmem));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, args);
}

template <int kMode>
cudaError_t launch_format(int format, const Fp4Maps& maps, const Fp4Args& args, long long max_tiles,
                          int sm_count, cudaStream_t s) {
  return format == kNvfp4 ? launch_impl<kNvfp4, kMode>(maps, args, max_tiles, sm_count, s)
                          : launch_impl<kMxfp4, kMode>(maps, args, max_tiles, sm_count, s);
}

Fp4Args common_args(const int32_t* counts, int E, RowLayout rl, int32_t* dev_status, bool capped) {
  Fp4Args a{};
  a.counts = counts;
  a.E = E;
  a.R = rl.R;
  a.packed = rl.packed;
  a.early = !capped;
  a.rows = rl.rows;
  a.dev_status = dev_status;
  return a;
}

}  // namespace

cudaError_t launch_gemm_gateup_fp4(const uint8_t* xq, const uint8_t* xs, const float* xg,
                                   const int32_t* counts, int E, RowLayout rl, int H, int I,
                                   const uint8_t* w13, const uint8_t* s13, const float* g13,
                                   const float* zg, int format, uint8_t* zq, uint8_t* zs,
                                   int32_t* dev_status, int sm_count, bool capped, cudaStream_t s) {
  Fp4Maps maps{};
  cudaError_t err = product_maps(&maps, 0, xq, rl.rows, rl.R, w13, static_cast<uint64_t>(E) * 2 * I, H);
  if (err != cudaSuccess) return err;
  Fp4Args a = common_args(counts, E, rl, dev_status, capped);
  a.g[0] = Product{xs, s13, xg, g13, H, I, I / 128};
  a.zg = zg;
  a.zq = zq;
  a.zs = zs;
  return launch_format<kGateUp>(format, maps, a, max_blocks(E, rl) * a.g[0].nt, sm_count, s);
}

cudaError_t launch_grouped_gemm_fp4(const uint8_t* aq, const uint8_t* as, const float* ag,
                                    const int32_t* counts, int E, RowLayout rl, int K, int N,
                                    const uint8_t* w, const uint8_t* ws, const float* wg, int format,
                                    void* out, int32_t* dev_status, int sm_count, bool capped, cudaStream_t s) {
  Fp4Maps maps{};
  cudaError_t err = product_maps(&maps, 1, aq, rl.rows, rl.R, w, static_cast<uint64_t>(E) * N, K);
  if (err != cudaSuccess) return err;
  Fp4Args a = common_args(counts, E, rl, dev_status, capped);
  a.g[1] = Product{as, ws, ag, wg, K, N, (N + kBN - 1) / kBN};
  a.out = static_cast<__nv_bfloat16*>(out);
  return launch_format<kDown>(format, maps, a, max_blocks(E, rl) * a.g[1].nt, sm_count, s);
}

size_t gemm_fp4_sync_ints(int E, RowLayout rl, int64_t routes) {
  return 1 + static_cast<size_t>(layer_blocks(E, rl, routes));
}

bool gemm_fp4_prefer_one_launch(int E, RowLayout rl, int I, int64_t routes, int sm_count) {
  // Whole layers from call to call, one launch / two (us), by the most waves of
  // gate/up tiles: one token of 256 experts of 7168 x 2048 58 / 62 (0.8 waves),
  // 16000 of 16 of 2048 x 512 103 / 108 (3.7), 256 of 64 of 4096 x 1536 130 / 142
  // (6.3), 768 160 / 165 (8.8), 1024 178 / 172 (10.1), 2048 274 / 250 (15.2), 4096
  // skewed ones of 128 543 / 474 (30), 1000 of 1024 of 1024 x 1024 349 / 275 (56).
  // The one launch fills the last gate/up wave with down tiles and starts once, but
  // every tile costs a ticket and Z a flush.  Between 10 and 14 waves, where few of
  // many experts have rows, it can still be ahead: 16 tokens of 256 experts 337 / 347.
  return layer_blocks(E, rl, routes) * (I / 128) <= 10LL * sm_count;
}

cudaError_t launch_gemm_both_fp4(const uint8_t* xq, const uint8_t* xs, const float* xg,
                                 const int32_t* counts, int E, RowLayout rl, int H, int I,
                                 const uint8_t* w13, const uint8_t* s13, const float* g13,
                                 const uint8_t* w2, const uint8_t* s2, const float* g2,
                                 const float* zg, int format, uint8_t* zq, uint8_t* zs, void* out,
                                 int* sync, int32_t* dev_status, int sm_count, bool capped, cudaStream_t s) {
  Fp4Maps maps{};
  cudaError_t err = product_maps(&maps, 0, xq, rl.rows, rl.R, w13, static_cast<uint64_t>(E) * 2 * I, H);
  if (err == cudaSuccess)
    err = product_maps(&maps, 1, zq, rl.rows, rl.R, w2, static_cast<uint64_t>(E) * H, I);
  if (err != cudaSuccess) return err;
  Fp4Args a = common_args(counts, E, rl, dev_status, capped);
  a.g[0] = Product{xs, s13, xg, g13, H, I, I / 128};
  a.g[1] = Product{zs, s2, zg, g2, I, H, (H + kBN - 1) / kBN};
  a.zg = zg;
  a.zq = zq;
  a.zs = zs;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.sched = sync;
  return launch_format<kBoth>(format, maps, a, max_blocks(E, rl) * (a.g[0].nt + a.g[1].nt), sm_count, s);
}

}  // namespace moe
