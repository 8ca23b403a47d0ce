// Residual addition and root-mean-square norm of token rows, the step before
// the router and the experts, with the normed row as BF16, as e4m3 codes and
// fp32 scales, or both:
//   r = x + residual                         (fp32; stored back in residual's type)
//   n = r * rsqrt(mean(r^2) + eps) * weight  (fp32)
//   y = bf16(n);  per 128: a = max(max|n|, 1e-4), yq = e4m3(n * (448 / a)), ys = a / 448
// The 8-bit row follows the quantisation rule of quant.cu and is taken from n
// itself, not from the rounded y: one rounding each.  The sum of squares, the
// norm and the scales are held in fp32.
//
// One pass: a row stays in its threads' registers between the sum of squares
// and the outputs, so every input is read once and every output written once.
// Rows up to 256 elements take a warp each (no block barrier); longer rows
// take a block, with as many threads as give each one vector of eight elements
// up to 8192 elements and two beyond: more loads in flight per thread leave
// fewer rows on an SM and were slower from one row to 16384.  A half-warp holds
// whole 128-element groups (16 lanes x 8 elements), so a group's maximum is a
// 4-step shuffle.
//
// Bound by HBM with many rows: 16384 rows of 7168 with a BF16 residual and both
// outputs, 1.06 GB, take 176 us, 6.0 TB/s.  With few rows by latency: 2 to 4 us
// (one row of 7168: 2.6).
#include "common.cuh"
#include "kernels.h"

#include <algorithm>

namespace moe {
namespace {

// Elements of a row that one warp takes.  Against a block per row: 65536 rows of
// 128 take 15 us for 35, of 256 24 for 36; of 512, the other way, 46 for 49 us.
constexpr int kWarpRowMax = 256;
constexpr int kRowWarps = 8;       // rows (= warps) per block of the warp form

struct NormArgs {
  const uint4* x;        // BF16 [T, H]
  const void* residual;  // BF16 or fp32 [T, H]; may be residual_out itself
  void* residual_out;    // null: the sum is not kept
  const void* weight;    // BF16 or fp32 [H]
  uint4* y;              // BF16 [T, H] or null
  uint2* yq;             // e4m3 [T, H] or null
  float* ys;             // fp32 [T, H / 128] or null
  int T, H;
  int weight_fp32;
  float eps;
};

// residual and residual_out may be one buffer, so these are ordinary (not
// read-only-path) accesses.
template <int kResidual>
__device__ __forceinline__ void add_residual(const NormArgs& a, int64_t v, float* f) {
  if constexpr (kResidual == 16) {
    float r[8];
    bf16x8_to_f32(static_cast<const uint4*>(a.residual)[v], r);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += r[i];
  } else if constexpr (kResidual == 32) {
    const float4* p = static_cast<const float4*>(a.residual) + 2 * v;
    const float4 lo = p[0], hi = p[1];
    f[0] += lo.x; f[1] += lo.y; f[2] += lo.z; f[3] += lo.w;
    f[4] += hi.x; f[5] += hi.y; f[6] += hi.z; f[7] += hi.w;
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* f) {
  return make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]),
                    pack_bf16x2_rn(f[4], f[5]), pack_bf16x2_rn(f[6], f[7]));
}

template <int kResidual>
__device__ __forceinline__ void store_residual(const NormArgs& a, int64_t v, const float* f) {
  if constexpr (kResidual == 16) {
    static_cast<uint4*>(a.residual_out)[v] = pack_bf16x8(f);
  } else if constexpr (kResidual == 32) {
    float4* p = static_cast<float4*>(a.residual_out) + 2 * v;
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

__device__ __forceinline__ void load_weight(const NormArgs& a, int v, float* w) {
  if (a.weight_fp32) {
    const float4* p = static_cast<const float4*>(a.weight) + 2 * v;
    const float4 lo = __ldg(p), hi = __ldg(p + 1);
    w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
    w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
  } else {
    bf16x8_to_f32(__ldg(static_cast<const uint4*>(a.weight) + v), w);
  }
}

// V vectors of 8 elements per thread; kWarp: a warp per row, else a block.
template <int kResidual, int V, bool kWarp>
__global__ void norm_kernel(const NormArgs a) {
  __shared__ float s_part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = kWarp ? blockIdx.x * kRowWarps + warp : blockIdx.x;
  if (kWarp && row >= a.T) return;
  const int tid = kWarp ? lane : threadIdx.x;
  const int nthr = kWarp ? 32 : blockDim.x;
  const int nvec = a.H / 8;
  const int64_t base = static_cast<int64_t>(row) * nvec;

  float f[V][8];
  uint4 raw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * nthr + tid;
    if (v < nvec) raw[i] = a.x[base + v];
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * nthr + tid;
    if (v >= nvec) continue;
    bf16x8_to_f32(raw[i], f[i]);
    add_residual<kResidual>(a, base + v, f[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[i][j], f[i][j], ss);
  }
  auto sum_row = [&](float v) {   // over the row, the same in every thread
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (!kWarp) {
      if (lane == 0) s_part[warp] = v;
      __syncthreads();
      v = lane < (nthr >> 5) ? s_part[lane] : 0.f;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
  };
  ss = sum_row(ss);
  float mean = ss / static_cast<float>(a.H);
  if (ss == INFINITY) {
    // The sum of up to 2^14 squares leaves the range before their mean does: once
    // more with every element times 2^-7.
    constexpr float kDown = 0x1p-7f;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i * nthr + tid >= nvec) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[i][j] * kDown, f[i][j] * kDown, ss);
    }
    if constexpr (!kWarp) __syncthreads();   // s_part has been read
    ss = sum_row(ss);
    mean = ss / static_cast<float>(a.H) * (1.f / (kDown * kDown));
  }
  const float rstd = rsqrtf(mean + a.eps);

#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * nthr + tid;
    const bool on = v < nvec;   // nvec is a multiple of 16: the same for a half-warp
    float amax = 0.f;
    if (on) {
      if (kResidual != 0 && a.residual_out != nullptr) store_residual<kResidual>(a, base + v, f[i]);
      float w[8];
      load_weight(a, v, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[i][j] = f[i][j] * rstd * w[j];
        amax = fmaxf(amax, fabsf(f[i][j]));
      }
      if (a.y != nullptr) a.y[base + v] = pack_bf16x8(f[i]);
    }
    if (a.yq != nullptr) {
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (on) {
        float mult, scale;
        fp8_group_scale(amax, &mult, &scale);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c[j] = pack_e4m3x2(__fmul_rn(f[i][2 * j], mult), __fmul_rn(f[i][2 * j + 1], mult));
        a.yq[base + v] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        if ((lane & 15) == 0) a.ys[(base + v) >> 4] = scale;
      }
    }
  }
}

template <int kResidual>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  const int nvec = a.H / 8;
  if (a.H <= kWarpRowMax) {
    const int grid = (a.T + kRowWarps - 1) / kRowWarps;
    norm_kernel<kResidual, kWarpRowMax / 256, true><<<grid, kRowWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
  }
  const int v = nvec <= 1024 ? 1 : 2;
  const int threads = ((nvec + v - 1) / v + 31) / 32 * 32;
  if (v == 1)
    norm_kernel<kResidual, 1, false><<<a.T, threads, 0, s>>>(a);
  else
    norm_kernel<kResidual, 2, false><<<a.T, threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rms_norm(const void* x, const void* residual, int residual_bits,
                                const void* weight, int weight_bits, float eps, int T, int H,
                                void* y, uint8_t* yq, float* ys, void* residual_out,
                                cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const NormArgs a{static_cast<const uint4*>(x), residual, residual_out, weight,
                   static_cast<uint4*>(y), reinterpret_cast<uint2*>(yq), ys, T, H,
                   weight_bits == 32 ? 1 : 0, eps};
  if (residual == nullptr) return launch_norm<0>(a, s);
  if (residual_bits == 16) return launch_norm<16>(a, s);
  return launch_norm<32>(a, s);
}

}  // namespace moe
