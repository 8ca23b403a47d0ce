// Microscaled 4-bit floating point: the number formats and the block-scaled
// tcgen05 products.
//
// A value is an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) times its
// block's scale; two codes a byte, the even element in the low four bits.
//   NVFP4: blocks of 16, the scale in e4m3, and one fp32 scale g over a tensor
//     (per expert for weights):  s = e4m3(amax / (6 g)),  q = e2m1(x / (s g)).
//   MXFP4: blocks of 32, the scale a power of two in e8m0 (2^(byte - 127)):
//     s = 2^(floor(log2 amax) - 2), the exponent of e2m1's largest binade;
//     what exceeds 6 s goes to 6 s.
// The arithmetic is fp32: 6 g, the division, s g, its reciprocal and the
// product x * (1 / (s g)) each rounded to nearest, then the code (nearest, ties
// to even, beyond 6 to 6).  The reciprocal instead of a division per element
// moves only values within 2^-23 of a midpoint.  A block whose scale rounds to
// zero has zero codes, and so has a block of zeros, whatever g is: that of a tensor
// of zeros, taken from its data, is 0.  A block with a NaN or an infinity gets the
// scale NaN (0x7F, 0xFF), which makes every product with it NaN.
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"

namespace moe {

constexpr int kNvfp4 = 0;
constexpr int kMxfp4 = 1;
template <int kFmt>
constexpr int kFp4Block = kFmt == kNvfp4 ? 16 : 32;

__device__ __forceinline__ float e4m3_to_f32(uint8_t v) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

// The scale byte of a block with largest magnitude `amax` (fp32 bits without
// the sign, so that a NaN or an infinity is the largest) and the multiplier of
// its values.
template <int kFmt>
__device__ __forceinline__ uint8_t fp4_block_scale(uint32_t amax, float g, float six_g, float* mult) {
  if constexpr (kFmt == kNvfp4) {
    if (amax == 0u || amax >= 0x7F800000u) {   // not 0 / (6 g): g may be 0
      *mult = 0.f;
      return amax == 0u ? 0 : 0x7F;
    }
    const uint8_t b = static_cast<uint8_t>(__nv_cvt_float_to_fp8(
        __fdiv_rn(__uint_as_float(amax), six_g), __NV_SATFINITE, __NV_E4M3));
    const float s = e4m3_to_f32(b);
    *mult = s > 0.f ? __frcp_rn(__fmul_rn(s, g)) : 0.f;
    return b;
  } else {
    if (amax >= 0x7F800000u) {
      *mult = 0.f;
      return 0xFF;
    }
    const int b = max(0, static_cast<int>(amax >> 23) - 2);
    *mult = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);
    return static_cast<uint8_t>(b);
  }
}

// Eight values times mult as eight codes, element 0 in the low four bits.
__device__ __forceinline__ uint32_t fp4_pack8(const float* f, float mult) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(
             make_float2(__fmul_rn(f[2 * i], mult), __fmul_rn(f[2 * i + 1], mult)), __NV_E2M1,
             cudaRoundNearest))
         << (8 * i);
  return w;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// One lane's 16 consecutive values of a row (a warp holds 512 consecutive ones)
// to 8 bytes of codes and the warp's scale bytes: *scale_word is complete in
// every fourth lane (NVFP4: the scales of 4 lanes, 64 values) or every eighth
// (MXFP4: 4 scales of 8 lanes, 128 values).  All 32 lanes call it.
template <int kFmt>
__device__ __forceinline__ uint2 fp4_quantize16(const float* f, float g, float six_g, int lane,
                                                uint32_t* scale_word) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max(amax, abs_bits(f[i]));
  if constexpr (kFmt == kMxfp4) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  float mult;
  const uint32_t b = fp4_block_scale<kFmt>(amax, g, six_g, &mult);
  constexpr int kLanes = kFp4Block<kFmt> / 16;   // lanes of a block
  uint32_t w = b << (8 * ((lane / kLanes) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, kLanes);
  w |= __shfl_xor_sync(0xffffffffu, w, 2 * kLanes);
  *scale_word = w;
  return make_uint2(fp4_pack8(f, mult), fp4_pack8(f + 8, mult));
}

// ------------------------------------------------- block-scaled tcgen05 MMA
// Instruction descriptor of kind::mxf4nvf4 with e2m1 A and B, both K-major,
// fp32 accumulator: B scale id (bits 4-5), A format (7-9) = B format (10-12) =
// 1 (E2M1), N >> 3 (17-22), scale format (23: 0 = UE4M3, 1 = UE8M0), M >> 7
// (27-28), A scale id (29-30).  The ids choose the byte of a scale's 32-bit
// column where the K = 64 of one MMA takes only part of it: MXFP4's two scales
// a row are bytes 0-1 or 2-3.
template <int kFmt>
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, int scale_id) {
  return (static_cast<uint32_t>(scale_id) << 4) | (1u << 7) | (1u << 10) |
         (static_cast<uint32_t>(N >> 3) << 17) | (kFmt == kMxfp4 ? 1u << 23 : 0u) |
         (static_cast<uint32_t>(M >> 7) << 27) | (static_cast<uint32_t>(scale_id) << 29);
}

// D[tmem] (+)= (A * sa)[smem] * (B * sb)[smem]^T over 64 elements of K, issued
// by one thread; the scales are in TMEM.
template <int kFmt>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                                        uint32_t accumulate) {
  if constexpr (kFmt == kNvfp4)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptor of 128 rows' scales as the MMA wants them in TMEM:
// 32 lanes x 16 bytes, lane r holding the 32-bit words of rows r, r + 32,
// r + 64 and r + 96; 8-lane groups 128 bytes apart (stride byte offset), no
// swizzle, descriptor version 1.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}
// Those 512 bytes to four TMEM columns of each 32-lane quarter.  Ordered before
// the MMAs that the same thread issues after it.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// One lane of a converged warp.  TMA and tcgen05 instructions take their operands
// from uniform registers; where a single lane has branched off on its own lane
// number the compiler moves every operand there one by one (50 to 70 clocks an
// instruction), where the warp runs together up to here it does not.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}
// A bounded wait of a whole warp: true in every lane, or in none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// The async proxy (TMA, tcgen05) sees this thread's shared-memory stores.
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Launch chain (programmatic dependent launch): the next kernel may start; wait
// for everything the kernels before have written.  No-ops in plain launches.
__device__ __forceinline__ void pdl_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace moe
