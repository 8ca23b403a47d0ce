// Rows to microscaled 4 bits and back (formats and arithmetic: fp4.cuh).
//
// Both are one pass over memory: a lane takes 16 consecutive values, one NVFP4
// block (or half an MXFP4 block, joined by one shuffle), so codes are stored as
// 8 bytes a lane, 256 a warp, and scales as one 32-bit word per four (eight)
// lanes.  The codes and scales are linear over the whole matrix (H is a
// multiple of 128), so a lane's place follows from its chunk's number alone and
// only the scale over the tensor depends on the row.  Bound by HBM: 235 M fp32
// weights to 4 bits 155 us (6.9 TB/s), back to BF16 106 us (5.7 TB/s, most of it
// writes); a few rows take the launch, 3.5 to 4.5 us.
#include <algorithm>

#include "fp4.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;   // 16-value chunks a lane has in flight

// The scale over the tensor for chunk c (per_g chunks share one; null: 1).
__device__ __forceinline__ float over_scale(const float* gscale, long long per_g, long long n_g,
                                            long long c) {
  if (gscale == nullptr) return 1.f;
  if (n_g == 1) return __ldg(gscale);
  return __ldg(gscale + (((c | per_g) >> 32) == 0
                             ? static_cast<uint32_t>(c) / static_cast<uint32_t>(per_g)
                             : c / per_g));
}

template <int kFmt, bool kF32>
__global__ void __launch_bounds__(kThreads)
    quantize_fp4_kernel(const uint4* __restrict__ x, const float* __restrict__ gscale,
                        long long per_g, long long n_g, long long chunks, uint2* __restrict__ xq,
                        uint32_t* __restrict__ xs) {
  constexpr int kVec = kF32 ? 4 : 2;   // 16-byte vectors of a chunk
  const int lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  // whole warps run on: the shuffles take every lane
  for (long long c0 = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; c0 - lane < chunks;
       c0 += step * kUnroll) {
    uint4 v[kUnroll][kVec];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long c = c0 + u * step;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        v[u][i] = c < chunks ? ld_stream(x + c * kVec + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long c = c0 + u * step;
      float f[16];
      if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[4 * i] = __uint_as_float(v[u][i].x);
          f[4 * i + 1] = __uint_as_float(v[u][i].y);
          f[4 * i + 2] = __uint_as_float(v[u][i].z);
          f[4 * i + 3] = __uint_as_float(v[u][i].w);
        }
      } else {
        bf16x8_to_f32(v[u][0], f);
        bf16x8_to_f32(v[u][1], f + 8);
      }
      const float g = c < chunks ? over_scale(gscale, per_g, n_g, c) : 1.f;
      uint32_t word;
      const uint2 codes = fp4_quantize16<kFmt>(f, g, __fmul_rn(6.f, g), lane, &word);
      if (c < chunks) {
        xq[c] = codes;
        if (kFmt == kNvfp4) {
          if ((lane & 3) == 0) xs[c >> 2] = word;
        } else {
          if ((lane & 7) == 0) xs[c >> 3] = word;
        }
      }
    }
  }
}

// A lane takes 8 values: 4 bytes of codes, its block's scale byte (shared with
// its neighbours), and 16 bytes of BF16 out, 512 consecutive ones a warp.
template <int kFmt, bool kF32>
__global__ void __launch_bounds__(kThreads)
    dequantize_fp4_kernel(const uint32_t* __restrict__ xq, const uint8_t* __restrict__ xs,
                          const float* __restrict__ gscale, long long per_g, long long n_g,
                          long long eights, uint4* __restrict__ out) {
  constexpr int kDeep = 2;   // loads a lane has in flight
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  for (long long c0 = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; c0 < eights;
       c0 += step * kDeep) {
    uint32_t q[kDeep];
    uint8_t b[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const long long c = c0 + u * step;
      if (c < eights) {
        q[u] = __ldg(xq + c);
        b[u] = __ldg(xs + c / (kFp4Block<kFmt> / 8));
      }
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const long long c = c0 + u * step;
      if (c >= eights) break;
      // 2^(b - 127) as fp32 bits (b = 0: the subnormal 2^-127; 255: NaN)
      const float s = kFmt == kNvfp4 ? e4m3_to_f32(b[u])
                                     : __uint_as_float(b[u] == 255 ? 0x7FFFFFFFu
                                                       : b[u] == 0 ? 0x00400000u
                                                                   : static_cast<uint32_t>(b[u]) << 23);
      const float g = over_scale(gscale, per_g, n_g, c >> 1);
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2(
            static_cast<__nv_fp4x2_storage_t>((q[u] >> (8 * i)) & 0xFFu), __NV_E2M1));
        // code * scale is exact (two bits times four), so one rounding by g
        const float2 p = __half22float2(h);
        f[2 * i] = p.x * s * g;
        f[2 * i + 1] = p.y * s * g;
      }
      if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          out[2 * c + i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                             __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
      } else {
        out[c] = make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]),
                                   pack_bf16x2_rn(f[4], f[5]), pack_bf16x2_rn(f[6], f[7]));
      }
    }
  }
}

// Blocks for so many threads, up to 64 an SM one after the other (235 M weights
// between two events, which add the launch: 168 and 111 us there and back, 177 and
// 128 with eight resident ones that go on).
int blocks_for(long long threads, int sm_count) {
  return static_cast<int>(std::min<long long>((threads + kThreads - 1) / kThreads, 64LL * sm_count));
}

}  // namespace

cudaError_t launch_quantize_fp4(const void* x, int x_bits, const float* gscale,
                                int64_t rows_per_gscale, int64_t rows, int H, int format,
                                uint8_t* xq, uint8_t* xs, int sm_count, cudaStream_t s) {
  const long long chunks = rows * (H / 16), per_g = rows_per_gscale * (H / 16);
  if (chunks == 0) return cudaSuccess;
  const long long n_g = (chunks + per_g - 1) / per_g;
  const int grid = blocks_for((chunks + kUnroll - 1) / kUnroll, sm_count);
  auto kernel = format == kNvfp4 ? (x_bits == 32 ? quantize_fp4_kernel<kNvfp4, true>
                                                 : quantize_fp4_kernel<kNvfp4, false>)
                                 : (x_bits == 32 ? quantize_fp4_kernel<kMxfp4, true>
                                                 : quantize_fp4_kernel<kMxfp4, false>);
  kernel<<<grid, kThreads, 0, s>>>(static_cast<const uint4*>(x), gscale, per_g, n_g, chunks,
                                   reinterpret_cast<uint2*>(xq), reinterpret_cast<uint32_t*>(xs));
  return cudaGetLastError();
}

cudaError_t launch_dequantize_fp4(const uint8_t* xq, const uint8_t* xs, const float* gscale,
                                  int64_t rows_per_gscale, int64_t rows, int H, int format,
                                  void* out, int out_bits, int sm_count, cudaStream_t s) {
  const long long chunks = rows * (H / 16), per_g = rows_per_gscale * (H / 16);
  if (chunks == 0) return cudaSuccess;
  const long long n_g = (chunks + per_g - 1) / per_g;
  const long long eights = 2 * chunks;
  const int grid = blocks_for((eights + 1) / 2, sm_count);
  auto kernel = format == kNvfp4 ? (out_bits == 32 ? dequantize_fp4_kernel<kNvfp4, true>
                                                   : dequantize_fp4_kernel<kNvfp4, false>)
                                 : (out_bits == 32 ? dequantize_fp4_kernel<kMxfp4, true>
                                                   : dequantize_fp4_kernel<kMxfp4, false>);
  kernel<<<grid, kThreads, 0, s>>>(reinterpret_cast<const uint32_t*>(xq), xs, gscale, per_g, n_g, eights,
                                   static_cast<uint4*>(out));
  return cudaGetLastError();
}

}  // namespace moe
