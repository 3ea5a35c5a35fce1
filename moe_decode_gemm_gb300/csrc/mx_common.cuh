// mx_common.cuh -- blocks of 32 numbers with a shared power of two (the OCP
// microscaling formats): scale exponents, conversions, and the tcgen05 MMA that
// takes such blocks as they are.
#pragma once

#include "tc_common.cuh"

namespace dg {

constexpr int kMxGroup = 32;       // numbers that share a scale
constexpr int kW4Tile = 128;       // weight rows of a tile, and k of a unit
constexpr int kW4Unit = kW4Tile * kW4Tile / 2;  // packed weight bytes of a unit: 128 rows x 128 k
constexpr int kW4Scales = 512;     // scale bytes of a unit: 128 rows x 4 groups

// Place of the scale byte of (row, group) in a unit's 512: what the tensor cores
// read, 32 lines of 16 bytes, line row % 32, four groups side by side.
__host__ __device__ constexpr int mx_scale_at(int row, int group) {
  return (row % 32) * 16 + (row / 32) * 4 + group;
}

// ceil(log2(a / L)) for a finite a > 0, L = (1 + FRAC / 2^23) * 2^EXP: exact, from
// the bits. Below the normal numbers it is at most the true value of the least
// normal one: callers clamp there.
template <int EXP, uint32_t FRAC>
__device__ __forceinline__ int mx_exponent(float a) {
  const uint32_t b = __float_as_uint(a);
  return (int)(b >> 23) - 127 - EXP + ((b & 0x7FFFFFu) > FRAC ? 1 : 0);
}
__device__ __forceinline__ int mx_exponent_e4m3(float a) { return mx_exponent<8, 0x600000u>(a); }  // 448
__device__ __forceinline__ int mx_exponent_e2m1(float a) { return mx_exponent<2, 0x400000u>(a); }  // 6

__device__ __forceinline__ bool not_finite(float a) {
  return (__float_as_uint(a) & 0x7F800000u) == 0x7F800000u;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2_f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// a -> low byte, b -> high byte; to the nearest e4m3, ties to even, at most 448.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(b), "f"(a));
  return y;
}

// D[tmem] (+)= (A * 2^sa)[smem] * (B * 2^sb)[smem]^T over 32 k: A 128 rows of
// e2m1 (a 16-byte line of shared memory holds 16 of them in its first 8 bytes),
// B N rows of e4m3, one scale byte per row in tensor memory. idesc_mx chooses the
// byte of the scale words.
__device__ __forceinline__ void umma_mx_elect(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b,
                                              uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "setp.ne.b32 e, %0, 0;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], %2, %3, %4, [%5], "
      "[%6], p;\n\t}" ::"r"(leader),
      "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
      : "memory");
}

// Instruction descriptor: A e2m1, B e4m3, scales that are powers of two, fp32
// sums, both operands K-major, M = 128; `group`: the byte of the scale words.
__host__ __device__ constexpr uint32_t umma_idesc_mx(int N, int group) {
  return ((uint32_t)group << 4)          // B's scale byte
         | (5u << 7)                     // A: e2m1
         | (0u << 10)                    // B: e4m3
         | ((uint32_t)(N >> 3) << 17)    // N / 8
         | (1u << 23)                    // scales: 8-bit exponents
         | ((128u >> 4) << 24)           // M / 16
         | ((uint32_t)group << 29);      // A's scale byte
}

// 512 scale bytes (32 lines of 16) from shared memory to four tensor-memory
// columns of every quarter of the lanes. MMAs issued later by the same thread
// read them.
__device__ __forceinline__ void tmem_copy_scales_elect(uint32_t leader, uint32_t taddr,
                                                       uint32_t smem_addr) {
  // no swizzle, 8 lines of 16 bytes together: 128 bytes from one such to the next
  const uint64_t d = (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 |
                     (uint64_t)1 << 46;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %0, 0;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%1], %2;\n\t}" ::"r"(leader),
      "r"(taddr), "l"(d)
      : "memory");
}

}  // namespace dg
