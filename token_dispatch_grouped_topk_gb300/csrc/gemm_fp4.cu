// Grouped products in microscaled 4-bit floating point on tcgen05: ragged rows
// per expert, block scales applied by the tensor cores.
//
//   P[m, n] = ga * gw[e] * sum_k (sa[m, k/B] a[m, k]) * (sw[n, k/B] w[e, n, k])
// with e2m1 codes a, w, the block scales of the format (fp4.cuh) and the fp32
// scales over the tensors.  Two launches use it:
//   down     out = bf16(P), any contraction K and output width N;
//   gate/up  Z = SiLU(G) * U with G and U the products with the first and the
//            last I rows of W13, fp32, requantised to 4 bits per block
//            ("SGLang Expert Compute Backend", §1.1 and §3.6, on other codes).
// Each expert's valid rows are tiled on their own (§2.4); only tiles that hold
// valid rows are scheduled, and only valid rows are stored.
//
// Design (one CTA per SM, persistent):
//  - tiles of 128 rows x 256 columns (gate/up: 128 gate and 128 up rows of W13),
//    one fp32 accumulator of 256 TMEM columns, N slices of one 128-row block
//    adjacent in the walk;
//  - warp 0 streams codes with TMA: stages of K = 256, 128 bytes a row, the
//    128-byte swizzle; kStages of them in a ring;
//  - warps 4-6 lay the scales of a stage out in shared memory as tcgen05.cp
//    wants them.  Scales are stored [row, K / B] like the codes, 16 (8) bytes a
//    stage and row, while the MMA takes for every 64 of K one 32-bit word a row,
//    the words of rows r, r + 32, r + 64, r + 96 side by side: a lane loads the
//    scales of those four rows, transposes 4 x 4 words in registers and stores
//    16 bytes per 64 of K.  So scales need no layout of their own: neither the
//    weights' (kept as they come) nor the activations', whose rows are ragged;
//  - warp 1 issues, per stage, the copies of the scales to TMEM and four MMAs
//    (M = 128, N = 256, K = 64).  Copies and MMAs of one thread run in order, so
//    one set of scale columns is enough;
//  - warps 8-15 take the accumulator to registers (64 gate and 64 up columns, or
//    128 columns of a row each), hand it back at once, and finish the tile while
//    the next one's products run.  A Z block lies in one thread, so its scale
//    needs no exchange.
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
constexpr int kScaleWarp0 = 4;   // warp 4: the rows' scales, 5 and 6: the weights'
constexpr int kScaleWarps = 3;
constexpr int kEpiWarp0 = 8;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
// Register split: launched at 128 a thread; the producer's and the MMA's
// warpgroup keeps 56, the scales' 72, the two epilogue warpgroups take 192.
constexpr int kLaunchRegs = 128;
constexpr int kCtrlRegs = 56;
constexpr int kScaleRegs = 72;
constexpr int kEpiRegs = 192;
static_assert(kCtrlRegs + kScaleRegs + 2 * kEpiRegs == 4 * kLaunchRegs, "register split must fit the launch");
// BF16 rows are staged per epilogue warp: 32 rows x 64 bytes, padded to 80.
constexpr int kStageRowBytes = 80;
constexpr int kStageWarpBytes = 32 * kStageRowBytes;
constexpr int kMaxExperts = 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfaCol = 256, kSfbCol = 272;   // scale columns behind the accumulator

struct Fp4Args {
  const int32_t* counts;
  const uint8_t* as;    // [rows, K / B] scales of the rows
  const uint8_t* ws;    // [E, weight rows, K / B] scales of the weights
  const float* ag;      // [1] scale over the rows, or null
  const float* wg;      // [E] scale over an expert's weights, or null
  const float* zg;      // gate/up: [1] scale over Z, or null
  uint8_t* zq;          // gate/up: [rows, N / 2]
  uint8_t* zs;          // gate/up: [rows, N / B]
  __nv_bfloat16* out;   // down: [rows, N]
  int E, R, K, N;       // N: output features (gate/up: I)
  int nt;               // N slices per 128-row block
  int packed;
  long long rows;       // buffer rows
  int32_t* dev_status;
};

struct Fp4Maps {
  CUtensorMap a[3];   // rows: boxes of 128, 64 and 32
  CUtensorMap b;
};

struct alignas(16) Control {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t tfull;
  uint64_t tempty;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int blk_start[kMaxExperts + 1];
  int cnt[kMaxExperts + 1];   // padded: clamped counts; packed: their prefix
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

struct Tile {
  int e, m_blk, n_blk, rows, cols, base;
};

template <bool kGateUp>
__device__ __forceinline__ Tile decode_tile(const Control* ctl, const Fp4Args& a, int t) {
  Tile r;
  const int blk = t / a.nt;
  r.n_blk = t - blk * a.nt;
  r.e = find_expert(ctl->blk_start, a.E, blk);
  r.m_blk = blk - ctl->blk_start[r.e];
  const int count = a.packed ? ctl->cnt[r.e + 1] - ctl->cnt[r.e] : ctl->cnt[r.e];
  r.base = (a.packed ? ctl->cnt[r.e] : r.e * a.R) + r.m_blk * kBM;
  r.rows = min(kBM, count - r.m_blk * kBM);
  r.cols = kGateUp ? kBN : min(kBN, a.N - r.n_blk * kBN);   // 128 in the last slice of an odd N / 128
  return r;
}

// First weight row of column half h of a tile.
template <bool kGateUp>
__device__ __forceinline__ long long weight_row(const Fp4Args& a, const Tile& t, int h) {
  if (kGateUp) return static_cast<long long>(t.e) * 2 * a.N + static_cast<long long>(h) * a.N + t.n_blk * 128;
  return static_cast<long long>(t.e) * a.N + t.n_blk * kBN + h * 128;
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  int dummy = 0;
  mbar_wait(bar, parity, &dummy);
}

// First 128-row block of each expert, and its clamped count (padded) or first
// row (packed), by warp 0; every thread of the block calls it.  The counts may
// be the launch before's, still written while this one starts: they are read
// through L2, after the wait.
__device__ __forceinline__ void tile_prefixes(const Fp4Args& a, Control* ctl) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int blocks = 0, rows = 0;
    if (lane == 0) ctl->blk_start[0] = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < a.E ? max(0, min(__ldcg(a.counts + e), a.R)) : 0;
      int nb = (c + kBM - 1) / kBM, nr = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, nb, o), v = __shfl_up_sync(0xffffffffu, nr, o);
        if (lane >= o) nb += u, nr += v;
      }
      if (e < a.E) {
        ctl->blk_start[e + 1] = blocks + nb;
        if (a.packed) ctl->cnt[e + 1] = rows + nr;
        else ctl->cnt[e] = c;
      }
      blocks += __shfl_sync(0xffffffffu, nb, 31);
      rows += __shfl_sync(0xffffffffu, nr, 31);
    }
    if (a.packed && lane == 0) ctl->cnt[0] = 0;
  }
  __syncthreads();
}

// The kScales bytes of one row and stage as 32-bit words, in the widest loads
// that the row pitch aligns; past the end of the row (the last stage of an odd
// K / 128) zeros.  Through L2: the rows' scales are the launch before's.
template <int kScales>
__device__ __forceinline__ void load_scales(const uint8_t* row, int off, int pitch, uint32_t* w) {
  if constexpr (kScales == 16) {
    if ((pitch & 15) == 0) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(row + off));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(row + off));
      const uint2 u = off + 8 < pitch ? __ldcg(reinterpret_cast<const uint2*>(row + off + 8))
                                      : make_uint2(0, 0);
      w[0] = v.x, w[1] = v.y, w[2] = u.x, w[3] = u.y;
    }
  } else {
    if ((pitch & 7) == 0) {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(row + off));
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = __ldcg(reinterpret_cast<const uint32_t*>(row + off));
      w[1] = off + 4 < pitch ? __ldcg(reinterpret_cast<const uint32_t*>(row + off + 4)) : 0u;
    }
  }
}

template <int kFmt, bool kGateUp>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_fp4_kernel(const __grid_constant__ Fp4Maps maps, const Fp4Args args) {
  using L = Layout<kFmt>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  Control* ctl = reinterpret_cast<Control*>(smem + kStages * L::kStageBytes);
  uint8_t* out_stage = smem + kStages * L::kStageBytes + sizeof(Control);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_start();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ctl->full[i], 1 + kScaleWarps);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->tfull, 1);
    mbar_init(&ctl->tempty, kEpiWarps);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane < 4) tma_prefetch_desc(lane < 3 ? &maps.a[lane] : &maps.b);
  if (warp == 2) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  pdl_wait();
  tile_prefixes(args, ctl);   // its barrier also publishes the mbarriers and the TMEM address
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int total = ctl->blk_start[args.E] * args.nt;
  const int tiles = total > static_cast<int>(blockIdx.x)
                        ? (total - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  const int nkb = (args.K + kBK - 1) / kBK;
  const bool half_end = args.K % kBK != 0;   // the last stage holds 128 elements
  volatile int* abort_flag = &ctl->abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    warpgroup_reg_dealloc<kCtrlRegs>();
    if (lane == 0) {
      int issued = 0;
      bool ok = true;
      for (int it = 0; it < tiles && ok; ++it) {
        const Tile tl = decode_tile<kGateUp>(ctl, args, blockIdx.x + it * gridDim.x);
        const int b0 = static_cast<int>(weight_row<kGateUp>(args, tl, 0));
        const int b1 = static_cast<int>(weight_row<kGateUp>(args, tl, 1));
        // only the valid rows are fetched (32, 64 or 128): the rest of the A
        // tile keeps stale bytes, which reach only rows that are never stored
        const int a_box = tl.rows <= 32 ? 32 : (tl.rows <= 64 ? 64 : kBM);
        const CUtensorMap* ma = &maps.a[a_box == kBM ? 0 : (a_box == 64 ? 1 : 2)];
        const uint32_t bytes = (a_box + tl.cols) * kRowBytes;
        for (int kb = 0; kb < nkb; ++kb) {
          const int stage = issued % kStages;
          if (!mbar_wait(&ctl->empty[stage], ((issued / kStages) & 1) ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * L::kStageBytes;
          uint8_t* sb = sa + L::kABytes;
          mbar_arrive_expect_tx(&ctl->full[stage], bytes);
          tma_load_2d(sa, ma, &ctl->full[stage], kb * kRowBytes, tl.base);
          tma_load_2d(sb, &maps.b, &ctl->full[stage], kb * kRowBytes, b0);
          if (tl.cols == kBN)
            tma_load_2d(sb + 128 * kRowBytes, &maps.b, &ctl->full[stage], kb * kRowBytes, b1);
          ++issued;
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
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    warpgroup_reg_dealloc<kCtrlRegs>();
    if (lane == 0) {
      int consumed = 0;
      bool ok = true;
      for (int it = 0; it < tiles && ok; ++it) {
        const int n_blk = (blockIdx.x + it * gridDim.x) % args.nt;
        const int cols = kGateUp ? kBN : min(kBN, args.N - n_blk * kBN);
        if (!mbar_wait(&ctl->tempty, (it & 1) ^ 1, abort_flag)) {
          ok = false;
          break;
        }
        for (int kb = 0; kb < nkb; ++kb) {
          const int stage = consumed % kStages;
          if (!mbar_wait(&ctl->full[stage], (consumed / kStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * L::kStageBytes);
          const uint32_t sfa = sa + L::kABytes + L::kBBytes, sfb = sfa + L::kSaBytes;
          const uint64_t adesc = smem_desc_kmajor_sw128(sa);
          const uint64_t bdesc = smem_desc_kmajor_sw128(sa + L::kABytes);
#pragma unroll
          for (int j = 0; j < L::kAtoms; ++j) {
            tmem_copy_scales(tmem + kSfaCol + 4 * j, smem_desc_scales(sfa + 512 * j));
            tmem_copy_scales(tmem + kSfbCol + 8 * j, smem_desc_scales(sfb + 1024 * j));
            tmem_copy_scales(tmem + kSfbCol + 8 * j + 4, smem_desc_scales(sfb + 1024 * j + 512));
          }
          const int steps = half_end && kb == nkb - 1 ? 2 : 4;
#pragma unroll
          for (int k = 0; k < 4; ++k) {   // 64 elements = 32 bytes = 2 descriptor units
            if (k >= steps) break;
            const int atom = k * L::kAtoms / 4, id = kFmt == kMxfp4 ? 2 * (k & 1) : 0;
            const uint32_t idesc = cols == kBN ? idesc_fp4<kFmt>(kBM, kBN, id)
                                               : idesc_fp4<kFmt>(kBM, 128, id);
            mma_fp4<kFmt>(tmem, adesc + 2 * k, bdesc + 2 * k, idesc, tmem + kSfaCol + 4 * atom,
                          tmem + kSfbCol + 8 * atom, (kb | k) > 0 ? 1u : 0u);
          }
          mma_commit(&ctl->empty[stage]);
          ++consumed;
        }
        if (ok) mma_commit(&ctl->tfull);
      }
      if (!ok) *abort_flag = 1;
      if (consumed > 0) {
        mma_commit(&ctl->drain);
        drain_wait(&ctl->drain, 0);
      }
    }
  } else if (warp < kScaleWarp0) {
    warpgroup_reg_dealloc<kCtrlRegs>();   // warp 2 owns TMEM, warp 3 is spare
  } else if (warp < kEpiWarp0) {
    // -------------------------------------------------------------- scales
    warpgroup_reg_dealloc<kScaleRegs>();
    const int sw = warp - kScaleWarp0;   // 0: the rows, 1 and 2: halves of the columns
    if (sw < kScaleWarps) {
      constexpr int kWords = L::kAtoms;          // 32-bit words of a row and stage
      constexpr int kAhead = 2;                  // stages whose loads are in flight
      const int pitch = args.K / kFp4Block<kFmt>;
      const int n_total = tiles * nkb;
      const uint8_t* row[4];
      uint32_t w[kAhead][4][kWords];
      int l_it = 0, l_kb = 0;                    // next stage to load
      auto load = [&](uint32_t (*v)[kWords]) {
        if (l_it >= tiles) return;
        if (l_kb == 0) {
          const Tile tl = decode_tile<kGateUp>(ctl, args, blockIdx.x + l_it * gridDim.x);
          // rows past the tile's (and its columns past N) repeat its last one:
          // their products are not stored
          const int n = sw == 0 ? tl.rows : (sw == 2 && tl.cols < kBN ? 0 : 128);
          const long long first = sw == 0 ? tl.base : weight_row<kGateUp>(args, tl, n ? sw - 1 : 0);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            row[q] = (sw == 0 ? args.as : args.ws) +
                     (first + min(lane + 32 * q, max(n, 1) - 1)) * pitch;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) load_scales<L::kScales>(row[q], l_kb * L::kScales, pitch, v[q]);
        if (++l_kb == nkb) l_kb = 0, ++l_it;
      };
#pragma unroll
      for (int d = 0; d < kAhead; ++d) load(w[d]);
      bool ok = true;
      for (int n0 = 0; n0 < n_total && ok; n0 += kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const int n = n0 + d;
          if (n >= n_total || !ok) break;
          const int stage = n % kStages;
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&ctl->empty[stage], ((n / kStages) & 1) ^ 1, abort_flag));
          if (!ok) break;
          // atom j of the rows at 512 j; of column half h at 1024 j + 512 h
          uint8_t* dst = smem + stage * L::kStageBytes + L::kABytes + L::kBBytes +
                         (sw == 0 ? 0 : L::kSaBytes + 512 * (sw - 1)) + 16 * lane;
          const int step = sw == 0 ? 512 : 1024;
#pragma unroll
          for (int j = 0; j < kWords; ++j)
            *reinterpret_cast<uint4*>(dst + j * step) =
                make_uint4(w[d][0][j], w[d][1][j], w[d][2][j], w[d][3][j]);
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->full[stage]);
          load(w[d]);
        }
      }
      if (!ok && lane == 0) *abort_flag = 1;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    warpgroup_reg_alloc<kEpiRegs>();
    const int ew = warp - kEpiWarp0;
    const int lq = warp & 3;    // TMEM lane quarter of this warp
    const int ch = ew >> 2;     // half of the tile's columns
    const int row = lq * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lq * 32) << 16);
    // gate/up: gate columns 64 ch.. and up columns 128 + 64 ch..; down: 128 ch..
    const uint32_t col0 = kGateUp ? 64 * ch : 128 * ch;
    const uint32_t col1 = kGateUp ? 128 + 64 * ch : 128 * ch + 64;
    const float ag = args.ag ? __ldcg(args.ag) : 1.f;
    const float zg = kGateUp && args.zg ? __ldcg(args.zg) : 1.f;
    const float six_zg = __fmul_rn(6.f, zg);
    bool ok = true;
    for (int it = 0; it < tiles; ++it) {
      const Tile tl = decode_tile<kGateUp>(ctl, args, blockIdx.x + it * gridDim.x);
      const float alpha = args.wg ? ag * __ldg(args.wg + tl.e) : ag;
      if (!mbar_wait(&ctl->tfull, it & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      __syncwarp();
      uint32_t p0[64], p1[64];
      tmem_load64_sync(t_lane + col0, p0);
      tmem_load64_sync(t_lane + col1, p1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->tempty);
      const long long grow = static_cast<long long>(tl.base) + row;
      const bool valid = row < tl.rows && grow < args.rows;
      if constexpr (kGateUp) {
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
          uint4* q = reinterpret_cast<uint4*>(args.zq + grow * (args.N / 2) + tl.n_blk * 64 + ch * 32);
          q[0] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
          q[1] = make_uint4(codes[4], codes[5], codes[6], codes[7]);
          uint8_t* s = args.zs + grow * (args.N / kB) + (tl.n_blk * 128 + ch * 64) / kB;
          if constexpr (kFmt == kNvfp4) *reinterpret_cast<uint32_t*>(s) = scales;
          else *reinterpret_cast<uint16_t*>(s) = static_cast<uint16_t>(scales);
        }
      } else {
        // BF16 rows through the warp's stage: each round the lanes leave 32
        // columns of their rows, then the warp writes 8 rows x 64 bytes per store
        const unsigned vmask = __ballot_sync(0xffffffffu, valid);
        if (128 * ch < tl.cols) {
          uint8_t* stage = out_stage + ew * kStageWarpBytes;
          uint4* srow = reinterpret_cast<uint4*>(stage + lane * kStageRowBytes);
          const int c = lane & 3;
          __nv_bfloat16* gbase = args.out + (static_cast<long long>(tl.base) + lq * 32 + (lane >> 2)) * args.N +
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
                *reinterpret_cast<uint4*>(gbase + static_cast<long long>(8 * i) * args.N + 32 * r) = v;
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

template <int kFmt, bool kGateUp>
cudaError_t launch_impl(const uint8_t* a, const uint8_t* w, const Fp4Args& args, int sm_count,
                        cudaStream_t s) {
  using L = Layout<kFmt>;
  if (args.E > kMaxExperts) return cudaErrorInvalidValue;
  auto* kernel = grouped_fp4_kernel<kFmt, kGateUp>;
  // The register split assumes exactly kLaunchRegs a thread; with any other
  // count the epilogue's increase could wait forever, so refuse to launch.
  static const int compiled_regs = [] {
    cudaFuncAttributes attr{};
    return cudaFuncGetAttributes(&attr, grouped_fp4_kernel<kFmt, kGateUp>) == cudaSuccess ? attr.numRegs : -1;
  }();
  if (compiled_regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const long long padded = static_cast<long long>(args.E) * ((args.R + kBM - 1) / kBM);
  const long long blocks =
      args.packed ? std::min<long long>(padded, (args.rows + kBM - 1) / kBM + args.E) : padded;
  const int grid = static_cast<int>(std::min<long long>(blocks * args.nt, sm_count));
  if (grid <= 0) return cudaSuccess;
  Fp4Maps maps{};
  const uint64_t rows = static_cast<uint64_t>(args.rows), row_bytes = args.K / 2;
  cudaError_t err = make_map(&maps.a[0], a, row_bytes, rows, 128);
  if (err == cudaSuccess) err = make_map(&maps.a[1], a, row_bytes, rows, 64);
  if (err == cudaSuccess) err = make_map(&maps.a[2], a, row_bytes, rows, 32);
  if (err == cudaSuccess)
    err = make_map(&maps.b, w, row_bytes, static_cast<uint64_t>(args.E) * args.N * (kGateUp ? 2 : 1), 128);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
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

Fp4Args common_args(const uint8_t* as, const float* ag, const int32_t* counts, int E, RowLayout rl,
                    int K, int N, const uint8_t* ws, const float* wg, int32_t* dev_status) {
  Fp4Args a{};
  a.counts = counts;
  a.as = as;
  a.ag = ag;
  a.ws = ws;
  a.wg = wg;
  a.E = E;
  a.R = rl.R;
  a.K = K;
  a.N = N;
  a.packed = rl.packed;
  a.rows = rl.rows;
  a.dev_status = dev_status;
  return a;
}

}  // namespace

cudaError_t launch_gemm_gateup_fp4(const uint8_t* xq, const uint8_t* xs, const float* xg,
                                   const int32_t* counts, int E, RowLayout rl, int H, int I,
                                   const uint8_t* w13, const uint8_t* s13, const float* g13,
                                   const float* zg, int format, uint8_t* zq, uint8_t* zs,
                                   int32_t* dev_status, int sm_count, cudaStream_t s) {
  Fp4Args a = common_args(xs, xg, counts, E, rl, H, I, s13, g13, dev_status);
  a.zg = zg;
  a.zq = zq;
  a.zs = zs;
  a.nt = I / 128;
  return format == kNvfp4 ? launch_impl<kNvfp4, true>(xq, w13, a, sm_count, s)
                          : launch_impl<kMxfp4, true>(xq, w13, a, sm_count, s);
}

cudaError_t launch_grouped_gemm_fp4(const uint8_t* aq, const uint8_t* as, const float* ag,
                                    const int32_t* counts, int E, RowLayout rl, int K, int N,
                                    const uint8_t* w, const uint8_t* ws, const float* wg, int format,
                                    void* out, int32_t* dev_status, int sm_count, cudaStream_t s) {
  Fp4Args a = common_args(as, ag, counts, E, rl, K, N, ws, wg, dev_status);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.nt = (N + kBN - 1) / kBN;
  return format == kNvfp4 ? launch_impl<kNvfp4, false>(aq, w, a, sm_count, s)
                          : launch_impl<kMxfp4, false>(aq, w, a, sm_count, s);
}

}  // namespace moe
