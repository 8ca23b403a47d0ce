// The router's projection: logits[t, e] = sum_h x[t, h] * w[e, h], BF16 rows
// and weights, products and sums in fp32 on the tensor cores, fp32 logits (a
// logit rounded to BF16 would tie experts that the choice has to tell apart).
//
// A CTA computes one tile of 128 tokens x BN experts:
//  - one thread streams x and w with TMA (64 elements = one 128-byte swizzle
//    row per K block) through a ring of stages, one thread issues
//    tcgen05.mma kind::f16 into TMEM;
//  - the tensor core truncates its fp32 sums, an error that grows with the
//    number of steps (8e-6 relative over H = 7168 in one accumulator), so every
//    512 elements of H go to the other of two accumulators while eight warps
//    add the finished one to fp32 registers: 5e-7;
//  - rows past T and experts past E are TMA's zero fill; they cost no traffic
//    and are never stored.
// With few tokens one tile per SM is far from filling the GPU, so H is split
// over the CTAs of a cluster (up to 8) and the partial tiles are summed through
// distributed shared memory, each CTA summing its share of the rows in rank
// order: one launch, no workspace, the same bits on every run.
// With many tokens two CTAs compute a 256-token tile together (cta_group::2):
// each holds its own 128 rows of x and half of w, so a step of 64 brings 32 KB
// into an SM instead of 48.  An SM takes in about 64 bytes a clock and the
// products of a step last 540 clocks, so 48 KB bound the kernel (the same with w
// multicast to both CTAs, which spares L2 but not the SM's intake: 67 us).
// Measured: 16384 tokens x 256 experts of 7168 (255 MB, 60 GFLOP) take 51 us, 5 TB/s
// and 1.18 PFLOP/s (one CTA a tile: 54): about 40 us of HBM, the products' 32 behind
// it; the first loads and the epilogue of a CTA's one tile are not hidden, and 24
// of 152 SMs have none.  256 tokens x 64 experts of 4096 take 7.6 us, one token 6.7:
// launch, first load and the sum over the cluster.
// Every wait is bounded.  One that runs out makes the whole tile NaN, which the
// choice of experts masks, and raises MOE_DEV_TIMEOUT where a status is given.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tensormap.h"

namespace moe {
namespace {

constexpr int kBM = 128;
constexpr int kBK = 64;             // BF16 elements of one 128-byte swizzle row
constexpr int kABytes = kBM * 128;
constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kLogitThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr int kRingBytes = 200 * 1024;
constexpr int kPromote = 8;   // K blocks summed in TMEM before they join the registers

struct LogitArgs {
  float* out;
  int32_t* dev_status;
  int T, H, E;
  int bn, nt;      // experts per tile (a multiple of 16), tiles along E
  int stages;
  int split;       // parts of H, one per CTA of a cluster
  int acc_cols;    // TMEM columns of one accumulator
  int vec;         // 16-byte stores are possible
};

struct LogitControl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t saddr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(saddr), "r"(rank)
      : "memory");
  return v;
}
// This CTA's shared address `saddr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_cluster(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// The cta_group::2 forms of the pair: a load counted on the leader's barrier,
// TMEM columns of both CTAs, products of both, arrivals on both.
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* map, uint32_t leader_bar,
                                                 int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(smem_dst)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::
          "r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// kPair: clusters of two CTAs that compute 256 tokens together, rank 0 issuing
// the products (and split = 1); else clusters of `split` parts of H of one tile.
template <bool kPair>
__global__ void __launch_bounds__(kLogitThreads, 1)
    router_logits_kernel(const __grid_constant__ CUtensorMap map_x,
                         const __grid_constant__ CUtensorMap map_w, const LogitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ LogitControl ctl;
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w_rows = kPair ? a.bn / 2 : a.bn;   // rows of w that this CTA holds
  const int stage_bytes = kABytes + w_rows * 128;
  const int group = kPair ? 2 : a.split;
  const int rank = blockIdx.x % group;
  const int tile = blockIdx.x / group;
  const int m0 = (kPair ? tile / a.nt * 2 + rank : tile / a.nt) * kBM, n0 = tile % a.nt * a.bn;
  const int nkb = a.H / kBK;
  const int kb0 = kPair ? 0 : static_cast<int>(static_cast<int64_t>(nkb) * rank / a.split);
  const int kb1 = kPair ? nkb : static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / a.split);
  const int n_kb = kb1 - kb0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.tfull[i], 1);
      mbar_init(&ctl.tempty[i], (kPair ? 2 : 1) * kEpiWarps);
    }
    mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  if (warp == 2) {
    if (kPair) {
      tmem_alloc_pair(&ctl.tmem_base, 2 * a.acc_cols);
    } else {
      tmem_alloc(&ctl.tmem_base, 2 * a.acc_cols);
      tmem_relinquish();
    }
    tc_fence_before();
  }
  __syncwarp();
  if (kPair) cluster_sync();   // the other CTA copies into this one and signals its barriers
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;

  // accumulators of one epilogue thread: its row's columns [c0, c0 + 16 * n16)
  float acc[8][16];
  const int half16 = (a.bn / 16 + 1) / 2;
  const int ch = (warp - kEpiWarp0) >> 2;                      // half of the columns
  const int c0 = ch ? half16 * 16 : 0;
  const int n16 = ch ? a.bn / 16 - half16 : half16;
  const int lq = warp & 3;                                     // TMEM lane quarter

  // One thread's walk round the ring, without divisions: they would be a third
  // of its time per stage.
  struct Slot {
    int i;
    uint32_t phase;
    __device__ void next(int n) {
      if (++i == n) {
        i = 0;
        phase ^= 1;
      }
    }
  };
  if (warp == 0) {
    if (lane == 0) {
      Slot st{0, 1};
      const uint32_t leader = kPair ? map_cluster(smem_u32(&ctl.full[0]), 0) : 0u;
      const int wy = n0 + (kPair ? rank * w_rows : 0);
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++issued, st.next(a.stages)) {
        if (!mbar_wait(&ctl.empty[st.i], st.phase, abort_flag)) {
          *abort_flag = 1;
          break;
        }
        uint8_t* sa = smem + st.i * stage_bytes;
        if (kPair) {
          // both CTAs' copies count on the leader's barrier
          if (rank == 0) mbar_arrive_expect_tx(&ctl.full[st.i], 2 * stage_bytes);
          const uint32_t bar = leader + st.i * 8;
          tma_load_2d_pair(sa, &map_x, bar, kb * kBK, m0);
          tma_load_2d_pair(sa + kABytes, &map_w, bar, kb * kBK, wy);
        } else {
          mbar_arrive_expect_tx(&ctl.full[st.i], stage_bytes);
          tma_load_2d(sa, &map_x, &ctl.full[st.i], kb * kBK, m0);
          tma_load_2d(sa + kABytes, &map_w, &ctl.full[st.i], kb * kBK, wy);
        }
      }
      // the ring is reused below and the block may exit: no copy in flight (of a
      // pair: none that the products, which free the stages, have not read)
      for (int i = 0; i < min(issued, a.stages); ++i) {
        const int n = issued - 1 - i;
        int none = 0;
        uint64_t* bar = kPair ? &ctl.empty[n % a.stages] : &ctl.full[n % a.stages];
        if (!mbar_wait(bar, (n / a.stages) & 1, &none)) *abort_flag = 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && (!kPair || rank == 0)) {
      const uint32_t idesc = idesc_bf16_f32(kPair ? 2 * kBM : kBM, a.bn);
      auto commit = [](uint64_t* bar) {
        if (kPair) mma_commit_pair(bar);
        else mma_commit(bar);
      };
      const uint64_t ad0 = smem_desc_kmajor_sw128(smem_u32(smem));
      const uint64_t bd0 = smem_desc_kmajor_sw128(smem_u32(smem) + kABytes);
      Slot st{0, 0}, tb{0, 1};   // ring stage, accumulator
      for (int i = 0; i < n_kb; ++i, st.next(a.stages)) {
        const bool first = i % kPromote == 0, last = i % kPromote == kPromote - 1 || i + 1 == n_kb;
        if ((first && !mbar_wait(&ctl.tempty[tb.i], tb.phase, abort_flag)) ||
            !mbar_wait(&ctl.full[st.i], st.phase, abort_flag)) {
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint64_t step = static_cast<uint64_t>(st.i * stage_bytes) >> 4;   // of the descriptors' address
        const uint32_t d = tmem + tb.i * a.acc_cols;
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) {   // 16 BF16 = 32 bytes = 2 descriptor units
          const uint32_t more = !first || k > 0 ? 1u : 0u;
          if (kPair) mma_bf16_pair(d, ad0 + step + 2 * k, bd0 + step + 2 * k, idesc, more);
          else mma_bf16(d, ad0 + step + 2 * k, bd0 + step + 2 * k, idesc, more);
        }
        commit(&ctl.empty[st.i]);
        if (last) {
          commit(&ctl.tfull[tb.i]);
          tb.next(2);
        }
      }
      commit(&ctl.drain);
      int none = 0;
      if (!mbar_wait(&ctl.drain, 0, &none)) *abort_flag = 1;
    }
  } else if (warp >= kEpiWarp0) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[c][j] = 0.f;
    const int chunks = (n_kb + kPromote - 1) / kPromote;
    bool ok = true;
    for (int i = 0; i < chunks && ok; ++i) {
      const int buf = i & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.tfull[buf], (i >> 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + buf * a.acc_cols + c0 + (static_cast<uint32_t>(lq * 32) << 16);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c < n16) {   // the same for the warp
          uint32_t r[16];
          tmem_load16_sync(base + c * 16, r);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c][j] += __uint_as_float(r[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair) mbar_arrive_cluster(map_cluster(smem_u32(&ctl.tempty[buf]), 0));
        else mbar_arrive(&ctl.tempty[buf]);
      }
    }
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  __syncthreads();
  const bool ok = ctl.abort == 0;
  if (warp == 2) {
    tc_fence_after();
    if (kPair) tmem_dealloc_pair(tmem, 2 * a.acc_cols);
    else tmem_dealloc(tmem, 2 * a.acc_cols);
  }

  // The tile (or its part) to shared memory: thread = row and half the columns,
  // rows padded by 16 bytes so that eight rows' 16-byte stores hit all banks.
  float* part = reinterpret_cast<float*>(smem);
  const int pitch = a.bn + 4;
  if (warp >= kEpiWarp0) {
    float4* dst = reinterpret_cast<float4*>(part + (lq * 32 + lane) * pitch + c0);
    const float nan = __uint_as_float(0x7fffffffu);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < n16) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          dst[c * 4 + j] = ok ? make_float4(acc[c][4 * j], acc[c][4 * j + 1], acc[c][4 * j + 2], acc[c][4 * j + 3])
                              : make_float4(nan, nan, nan, nan);
      }
  }
  __syncwarp();
  const bool summed = !kPair && a.split > 1;
  if (summed) cluster_sync();
  else __syncthreads();

  // This CTA's share of the rows, summed over the parts of H in rank order.
  const int rows = summed ? kBM / a.split : kBM, r0 = summed ? rank * rows : 0;
  const int nv = a.bn / 4;
  const uint32_t part_addr = smem_u32(part);
  for (int i = threadIdx.x; i < rows * nv; i += kLogitThreads) {
    const int r = r0 + i / nv, c = (i % nv) * 4;
    const int t = m0 + r, e = n0 + c;
    if (t >= a.T || e >= a.E) continue;
    const int off = r * pitch + c;
    float4 v;
    if (summed) {
      float4 u[kMaxCluster];   // all in flight before the first sum
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p)
        if (p < a.split) u[p] = ld_cluster(part_addr + off * 4, p);
      v = u[0];
#pragma unroll
      for (int p = 1; p < kMaxCluster; ++p)
        if (p < a.split) {
          v.x += u[p].x; v.y += u[p].y; v.z += u[p].z; v.w += u[p].w;
        }
    } else {
      v = *reinterpret_cast<const float4*>(part + off);
    }
    float* o = a.out + static_cast<int64_t>(t) * a.E + e;
    if (a.vec) {
      *reinterpret_cast<float4*>(o) = v;
    } else {
      o[0] = v.x;
      if (e + 1 < a.E) o[1] = v.y;
      if (e + 2 < a.E) o[2] = v.z;
      if (e + 3 < a.E) o[3] = v.w;
    }
  }
  __syncwarp();
  // the others may still read this part, or signal this CTA's barriers
  if (kPair || summed) cluster_sync();
  if (threadIdx.x == 0 && !ok && a.dev_status != nullptr) atomicOr(a.dev_status, kDevTimeout);
}

template <bool kPair>
cudaError_t launch_logits(const CUtensorMap& mx, const CUtensorMap& mw, const LogitArgs& a,
                          unsigned grid, unsigned cluster, cudaStream_t s) {
  cudaError_t err = cudaFuncSetAttribute(router_logits_kernel<kPair>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kRingBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kLogitThreads);
  // the ring, which also takes the finished tile
  cfg.dynamicSmemBytes = 1024 + std::max(a.stages * (kABytes + (kPair ? a.bn / 2 : a.bn) * 128), kBM * (a.bn + 4) * 4);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {cluster, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, router_logits_kernel<kPair>, mx, mw, a);
}

}  // namespace

cudaError_t launch_router_logits(const void* x, const void* w, int T, int H, int E, float* logits,
                                 int32_t* dev_status, int sm_count, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const int64_t mt = (static_cast<int64_t>(T) + kBM - 1) / kBM;
  const int nkb = H / kBK;
  LogitArgs a{};
  a.out = logits;
  a.dev_status = dev_status;
  a.T = T;
  a.H = H;
  a.E = E;
  a.nt = (E + 255) / 256;
  a.split = 1;
  // H is split while the CTAs fit at once; of 152 SMs 15 clusters of eight do, 36 of
  // four.  (1024, 64 experts, 4096): 8.5 us in 8 clusters of eight, 14.6 in 16;
  // without a split 25; one token 6.7 and 22 us.
  auto fit = [&](int cluster) { return sm_count - (cluster == 8 ? 32 : cluster == 4 ? 8 : 0); };
  while (a.split < kMaxCluster && mt * a.nt * a.split * 2 <= fit(a.split * 2) && nkb >= 4 * a.split)
    a.split *= 2;
  while (mt * a.nt * a.split * 2 <= fit(a.split) && (E + a.nt - 1) / a.nt > 32) a.nt *= 2;
  a.bn = ((E + a.nt - 1) / a.nt + 15) / 16 * 16;
  a.nt = (E + a.bn - 1) / a.bn;
  const bool pair = a.split == 1 && mt > 1;
  if (pair) {   // products of a pair: experts in steps of 32
    a.bn = (a.bn + 31) / 32 * 32;
    a.nt = (E + a.bn - 1) / a.bn;
  }
  a.acc_cols = 32;
  while (a.acc_cols < a.bn) a.acc_cols *= 2;
  a.stages = std::min(kMaxStages, kRingBytes / (kABytes + (pair ? a.bn / 2 : a.bn) * 128));
  a.vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0;
  CUtensorMap mx, mw;
  cudaError_t err = make_map_rows128(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, H, T, kBM);
  if (err == cudaSuccess)
    err = make_map_rows128(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, w, H, E, pair ? a.bn / 2 : a.bn);
  if (err != cudaSuccess) return err;
  if (pair) return launch_logits<true>(mx, mw, a, static_cast<unsigned>((mt + 1) / 2 * 2 * a.nt), 2, s);
  return launch_logits<false>(mx, mw, a, static_cast<unsigned>(mt * a.nt * a.split), a.split, s);
}

}  // namespace moe
