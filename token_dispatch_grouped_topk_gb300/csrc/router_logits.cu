// The router's projection: logits[t, e] = sum_h x[t, h] * w[e, h], BF16 rows
// and weights, products and sums in fp32 on the tensor cores, fp32 logits (a
// logit rounded to BF16 would tie experts that the choice has to tell apart).
//
// A CTA computes one tile of 128 tokens x BN experts over a part of H:
//  - one thread streams x and w with TMA (64 elements = one 128-byte swizzle
//    row per K block) through a ring of stages, one thread issues
//    tcgen05.mma kind::f16 into a BN-column TMEM accumulator;
//  - rows past T and experts past E are TMA's zero fill; they cost no traffic
//    and are never stored;
//  - with few tokens one tile per SM is far from filling the GPU, so H is split
//    over the CTAs of a cluster (up to 8) and the partial tiles are summed
//    through distributed shared memory, each CTA summing its share of the rows
//    in rank order: one launch, no workspace, the same bits on every run.
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
constexpr int kLogitThreads = 128;
constexpr int kRingBytes = 200 * 1024;

struct LogitArgs {
  float* out;
  int32_t* dev_status;
  int T, H, E;
  int bn, nt;      // experts per tile (a multiple of 16), tiles along E
  int stages;
  int split;       // cluster size: parts of H
  int tmem_cols;
  int vec;         // 16-byte stores are possible
};

struct LogitControl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::
                   : "memory");
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

__global__ void __launch_bounds__(kLogitThreads, 1)
    router_logits_kernel(const __grid_constant__ CUtensorMap map_x,
                         const __grid_constant__ CUtensorMap map_w, const LogitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ LogitControl ctl;
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = kABytes + a.bn * 128;
  const int rank = blockIdx.x % a.split;
  const int tile = blockIdx.x / a.split;
  const int m0 = tile / a.nt * kBM, n0 = tile % a.nt * a.bn;
  const int nkb = a.H / kBK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / a.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / a.split);

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.done, 1);
    ctl.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  if (warp == 2) {
    tmem_alloc(&ctl.tmem_base, a.tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int st = issued % a.stages;
        if (!mbar_wait(&ctl.empty[st], ((issued / a.stages) & 1) ^ 1, abort_flag)) {
          *abort_flag = 1;
          break;
        }
        uint8_t* sa = smem + st * stage_bytes;
        mbar_arrive_expect_tx(&ctl.full[st], stage_bytes);
        tma_load_2d(sa, &map_x, &ctl.full[st], kb * kBK, m0);
        tma_load_2d(sa + kABytes, &map_w, &ctl.full[st], kb * kBK, n0);
        ++issued;
      }
      // the ring is reused below and the block may exit: no copy in flight
      for (int i = 0; i < min(issued, a.stages); ++i) {
        const int n = issued - 1 - i;
        int none = 0;
        if (!mbar_wait(&ctl.full[n % a.stages], (n / a.stages) & 1, &none)) *abort_flag = 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kBM, a.bn);
      for (int i = 0; i < kb1 - kb0; ++i) {
        const int st = i % a.stages;
        if (!mbar_wait(&ctl.full[st], (i / a.stages) & 1, abort_flag)) {
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + st * stage_bytes);
        const uint64_t ad = smem_desc_kmajor_sw128(sa);
        const uint64_t bd = smem_desc_kmajor_sw128(sa + kABytes);
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)   // 16 BF16 = 32 bytes = 2 descriptor units
          mma_bf16(tmem, ad + 2 * k, bd + 2 * k, idesc, (i > 0 || k > 0) ? 1u : 0u);
        mma_commit(&ctl.empty[st]);
      }
      // completes when every MMA issued above has
      mma_commit(&ctl.done);
      int none = 0;
      if (!mbar_wait(&ctl.done, 0, &none)) *abort_flag = 1;
    }
  }
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  const bool ok = ctl.abort == 0;

  // The tile (or its part) from TMEM to shared memory: thread = row, rows
  // padded by 16 bytes so that eight rows' 16-byte stores hit all banks.
  float* part = reinterpret_cast<float*>(smem);
  const int pitch = a.bn + 4;
  {
    const int row = warp * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float4* dst = reinterpret_cast<float4*>(part + row * pitch);
    for (int c = 0; c < a.bn; c += 16) {
      uint32_t r[16];
      if (ok) {
        tmem_load16_sync(t_lane + c, r);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = 0x7fffffffu;   // NaN
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        dst[c / 4 + j] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                     __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
    }
  }
  tc_fence_before();
  if (a.split > 1) cluster_sync();
  else __syncthreads();
  __syncwarp();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, a.tmem_cols);
  }

  // This CTA's share of the rows, summed over the parts of H in rank order.
  const int rows = kBM / a.split, r0 = rank * rows;
  const int nv = a.bn / 4;
  const uint32_t part_addr = smem_u32(part);
  for (int i = threadIdx.x; i < rows * nv; i += kLogitThreads) {
    const int r = r0 + i / nv, c = (i % nv) * 4;
    const int t = m0 + r, e = n0 + c;
    if (t >= a.T || e >= a.E) continue;
    const int off = r * pitch + c;
    float4 v;
    if (a.split > 1) {
      v = ld_cluster(part_addr + off * 4, 0);
      for (int p = 1; p < a.split; ++p) {
        const float4 u = ld_cluster(part_addr + off * 4, p);
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
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
  if (a.split > 1) cluster_sync();   // the others may still read this part
  if (threadIdx.x == 0 && !ok && a.dev_status != nullptr) atomicOr(a.dev_status, kDevTimeout);
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
  while (a.split < kMaxCluster && mt * a.nt * a.split * 2 <= sm_count && nkb >= 4 * a.split)
    a.split *= 2;
  while (mt * a.nt * a.split * 2 <= sm_count && (E + a.nt - 1) / a.nt > 32) a.nt *= 2;
  a.bn = ((E + a.nt - 1) / a.nt + 15) / 16 * 16;
  a.nt = (E + a.bn - 1) / a.bn;
  a.tmem_cols = 32;
  while (a.tmem_cols < a.bn) a.tmem_cols *= 2;
  const int stage_bytes = kABytes + a.bn * 128;
  a.stages = std::min(kMaxStages, kRingBytes / stage_bytes);
  a.vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0;
  CUtensorMap mx, mw;
  cudaError_t err = make_map_rows128(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, H, T, kBM);
  if (err == cudaSuccess)
    err = make_map_rows128(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, w, H, E, a.bn);
  if (err != cudaSuccess) return err;
  const int smem = 1024 + a.stages * stage_bytes;
  err = cudaFuncSetAttribute(router_logits_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             1024 + kRingBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(mt * a.nt * a.split));
  cfg.blockDim = dim3(kLogitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(a.split), 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, router_logits_kernel, mx, mw, a);
}

}  // namespace moe
