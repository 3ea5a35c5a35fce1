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

// Whether the phase of the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// D[tmem] (+)= (A * 2^sa)[smem] * (B * 2^sb)[smem]^T over 32 k: A 128 rows of
// e2m1 (a 16-byte line of shared memory holds 16 of them in its first 8 bytes),
// B N rows of e4m3, one scale byte per row in tensor memory. idesc_mx chooses the
// byte of the scale words.
__device__ __forceinline__ void umma_mx_elect(uint32_t leader, uint32_t d_tmem, uint32_t a_lo,
                                              uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                              uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 e, %0, 0;\n\t"
      "setp.ne.b32 p, %9, 0;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %6, [%7], "
      "[%8], p;\n\t}" ::"r"(leader),
      "r"(d_tmem), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem),
      "r"(accumulate)
      : "memory");
}

// Instruction descriptor: A e2m1, B e4m3, scales that are powers of two, fp32
// sums, both operands K-major, M = 128; `group`: the byte of the scale words
// (umma_mx_group: its bits alone).
__host__ __device__ constexpr uint32_t umma_mx_group(int group) {
  return ((uint32_t)group << 4)          // B's scale byte
         | ((uint32_t)group << 29);      // A's scale byte
}
__host__ __device__ constexpr uint32_t umma_idesc_mx(int N, int group) {
  return (5u << 7)                       // A: e2m1
         | (0u << 10)                    // B: e4m3
         | ((uint32_t)(N >> 3) << 17)    // N / 8
         | (1u << 23)                    // scales: 8-bit exponents
         | ((128u >> 4) << 24)           // M / 16
         | umma_mx_group(group);
}

// 512 scale bytes (32 lines of 16) from shared memory to four tensor-memory
// columns of every quarter of the lanes. MMAs issued later by the same thread
// read them. src: bits 0-13 hold the address / 16, the others are not used.
__device__ __forceinline__ void tmem_copy_scales_elect(uint32_t leader, uint32_t taddr, uint32_t src) {
  // no swizzle, 8 lines of 16 bytes together: 128 bytes from one such to the next
  constexpr uint32_t kHi = (128u >> 4) | 1u << 14;
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 d;\n\t"
      "setp.ne.b32 e, %0, 0;\n\t"
      "mov.b64 d, {%2, %3};\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%1], d;\n\t}" ::"r"(leader),
      "r"(taddr), "r"(src & 0x3FFFu), "r"(kHi)
      : "memory");
}

}  // namespace dg
