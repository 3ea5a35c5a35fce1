// k_norm.cu -- root-mean-square norm of the residual stream, with the residual's
// addition before it and an output in bf16 or in 8 bits with scales.
//
//   h = bf16(x + res);  y = h * rsqrt(mean(h^2) + eps) * w
//
// A row's team of threads keeps its 16-byte vectors of h packed in registers
// between the sum of squares and the output, so every value is read once; the sums
// are fp32, added up in the same order whatever the call. The team is
//   few rows    a CTA of as many threads as vectors (up to 1024): the time is latency
//   many rows   a CTA with two to four vectors a thread, several to an SM: memory
//   many short  (H <= 2048) a warp, without barriers
// The 8-bit output's groups of 32 are 4 lanes. An e4m3 has 4 significant bits, so
// an error of one fp32 step in y moves about one in a million of them to the
// other side of a rounding border, where the whole value changes by a sixteenth: for
// it the sum, the root and the product are carried in two fp32 numbers, and y is
// rounded once.
#include "launch.h"
#include "launch_util.cuh"
#include "mx_common.cuh"

namespace dg {

struct NormArgs {
  const uint16_t *x, *res, *w;   // res may be null
  uint16_t *h, *y;               // h: with res only
  uint8_t *q, *sc;               // 8-bit output
  long long ldx, ldres, ldh, ldy, ldq, ldsc;
  int H;
  float eps;
  int* status;
  int rows;
};

// The index of (row, column) in a buffer of rows ld apart, checked in DEC_DEBUG builds.
__device__ __forceinline__ long long norm_at(const NormArgs& a, long long row, long long ld, int col, int width) {
  (void)width;
  return DG_OK(a.status, row < a.rows && col >= 0 && col < width, col) ? row * ld + col : 0;
}

// A number as the sum of two fp32, the second at most half a step of the first.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add_two(Two a, float b) {  // a + b
  const float s = __fadd_rn(a.hi, b), t = __fsub_rn(s, a.hi);
  return {s, a.lo + __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two add_two(Two a, Two b) {
  Two s = add_two(a, b.hi);
  s.lo += b.lo;
  return s;
}

// 1 / sqrt(sum / n + eps): one Newton step from rsqrtf's value, whose error is taken
// exactly.
__device__ __forceinline__ Two root_two(Two sum, float n, float eps) {
  const float q = __fdiv_rn(sum.hi, n);
  const Two m = add_two(Two{q, __fdiv_rn(fmaf(-q, n, sum.hi) + sum.lo, n)}, eps);
  const float f = rsqrtf(m.hi), p = __fmul_rn(f, f), pe = fmaf(f, f, -p);
  const float e = fmaf(-m.hi, p, 1.f) - fmaf(m.hi, pe, m.lo * p);  // 1 - m f^2
  // (a mean that is not finite, or 0: f alone says what the result is)
  return {f, isfinite(e) ? 0.5f * f * e : 0.f};
}

// Two fp32 operations in one instruction.
#define DG_F32X2(name, op)                                                                      \
  __device__ __forceinline__ float2 name(float2 a, float2 b) {                                  \
    float2 y;                                                                                   \
    asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\t" op       \
        " u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"                                                \
        : "=f"(y.x), "=f"(y.y)                                                                  \
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                                              \
    return y;                                                                                   \
  }
DG_F32X2(pair_add, "add.rn.f32x2")
DG_F32X2(pair_sub, "sub.rn.f32x2")
DG_F32X2(pair_mul, "mul.rn.f32x2")
#undef DG_F32X2
template <bool RZ>
__device__ __forceinline__ float2 pair_fma(float2 a, float2 b, float2 c) {  // RZ: rounded towards 0
  float2 y;
  if constexpr (RZ)
    asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rz.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  else
    asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}

// a * f for two exact a: cut to fp32, the last bit set where something was cut off, so
// that a later rounding to fewer bits sees on which side of a border the product lies.
__device__ __forceinline__ float2 times_two(float2 a, Two f) {
  const float2 hi = make_float2(f.hi, f.hi), c = pair_mul(a, make_float2(f.lo, f.lo));
  const float2 y = pair_fma<true>(a, hi, c);
  const float2 r = pair_add(pair_fma<false>(a, hi, make_float2(-y.x, -y.y)), c);
  return make_float2(__uint_as_float(__float_as_uint(y.x) | (r.x != 0.f ? 1u : 0u)),
                     __uint_as_float(__float_as_uint(y.y) | (r.y != 0.f ? 1u : 0u)));
}

constexpr int kNormWarps = 8;   // rows of a CTA where a warp takes one

// VPT: vectors of 8 values a thread holds; MX: 8-bit output; WARP: a warp to a row.
template <int VPT, bool MX, bool WARP>
__global__ void __launch_bounds__(WARP ? kNormWarps * 32 : 1024) norm_kernel(const NormArgs a) {
  constexpr int BATCH = VPT < 4 ? VPT : 4;  // vectors loaded at once
  __shared__ float s_hi[32], s_lo[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = WARP ? lane : threadIdx.x, nt = WARP ? 32 : blockDim.x;
  const long long row = WARP ? (long long)blockIdx.x * kNormWarps + warp : blockIdx.x;
  const int nv = a.H / 8;
  griddep_launch_dependents();
  griddep_wait();
  if (WARP && row >= a.rows) return;
  uint4 h[VPT], w[VPT];
  if (VPT == 1)  // few rows: the weights' way is the same as the row's
    w[0] = t < nv ? __ldg(reinterpret_cast<const uint4*>(a.w) + t) : make_uint4(0u, 0u, 0u, 0u);
  float sum = 0.f;
  float2 sq_hi = make_float2(0.f, 0.f), sq_lo = sq_hi;  // of even and odd columns
#pragma unroll
  for (int i0 = 0; i0 < VPT; i0 += BATCH) {
    uint4 r[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int v = t + (i0 + i) * nt;
      h[i0 + i] = r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (v < nv) {
        h[i0 + i] = *reinterpret_cast<const uint4*>(a.x + norm_at(a, row, a.ldx, v * 8, a.H));
        if (a.res) r[i] = *reinterpret_cast<const uint4*>(a.res + norm_at(a, row, a.ldres, v * 8, a.H));
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int v = t + (i0 + i) * nt;
      uint32_t* hw = reinterpret_cast<uint32_t*>(&h[i0 + i]);
      const uint32_t* rw = reinterpret_cast<const uint32_t*>(&r[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (a.res) hw[j] = pack_bf16(bf16lo(hw[j]) + bf16lo(rw[j]), bf16hi(hw[j]) + bf16hi(rw[j]));
        const float2 x = make_float2(bf16lo(hw[j]), bf16hi(hw[j]));
        if (MX) {  // (the square of a bf16 is exact) what the sum's rounding takes off is kept
          const float2 q = pair_mul(x, x), s = pair_add(sq_hi, q), t = pair_sub(s, sq_hi);
          sq_lo = pair_add(sq_lo, pair_add(pair_sub(sq_hi, pair_sub(s, t)), pair_sub(q, t)));
          sq_hi = s;
        } else {
          sum = fmaf(x.x, x.x, sum);
          sum = fmaf(x.y, x.y, sum);
        }
      }
      if (a.res && v < nv)
        *reinterpret_cast<uint4*>(a.h + norm_at(a, row, a.ldh, v * 8, a.H)) = h[i0 + i];
    }
  }
  Two sum2 = {sum, 0.f};
  if (MX) sum2 = add_two(Two{sq_hi.x, sq_lo.x}, Two{sq_hi.y, sq_lo.y});
  auto reduce = [&] {
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, sum2.hi, off);
      if (MX) sum2 = add_two(sum2, Two{o, __shfl_xor_sync(0xffffffffu, sum2.lo, off)});
      else sum2.hi += o;
    }
  };
  reduce();
  if (!WARP) {
    if (lane == 0) {
      s_hi[warp] = sum2.hi;
      s_lo[warp] = sum2.lo;
    }
    __syncthreads();
    sum2.hi = lane < nt / 32 ? s_hi[lane] : 0.f;
    sum2.lo = MX && lane < nt / 32 ? s_lo[lane] : 0.f;
    reduce();
  }
  const Two f = MX ? root_two(sum2, (float)a.H, a.eps) : Two{rsqrtf(sum2.hi / (float)a.H + a.eps), 0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * nt;
    if (VPT > 1) w[i] = v < nv ? __ldg(reinterpret_cast<const uint4*>(a.w) + v) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t* hw = reinterpret_cast<const uint32_t*>(&h[i]);
    const uint32_t* ww = reinterpret_cast<const uint32_t*>(&w[i]);
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = make_float2(bf16lo(hw[j]), bf16hi(hw[j])), g = make_float2(bf16lo(ww[j]), bf16hi(ww[j]));
      if (MX) {  // (the product of two bf16 is exact)
        const float2 p = times_two(pair_mul(x, g), f);
        y[2 * j] = p.x;
        y[2 * j + 1] = p.y;
      } else {
        y[2 * j] = x.x * f.hi * g.x;
        y[2 * j + 1] = x.y * f.hi * g.y;
      }
    }
    if constexpr (MX) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      int b = 255;
      uint2 q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);  // NaN, as the scale
      if (!not_finite(__uint_as_float(m))) {
        int e = mx_exponent_e4m3(__uint_as_float(m));
        e = e < -127 ? -127 : e;
        b = e + 127;
        const float s = pow2_f(-e);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= s;
        q.x = pack_e4m3(y[0], y[1]) | pack_e4m3(y[2], y[3]) << 16;
        q.y = pack_e4m3(y[4], y[5]) | pack_e4m3(y[6], y[7]) << 16;
      }
      if (v < nv) {
        *reinterpret_cast<uint2*>(a.q + norm_at(a, row, a.ldq, v * 8, a.H)) = q;
        if (!(v & 3)) a.sc[norm_at(a, row, a.ldsc, v / 4, a.H / kMxGroup)] = (uint8_t)b;
      }
    } else if (v < nv) {
      *reinterpret_cast<uint4*>(a.y + norm_at(a, row, a.ldy, v * 8, a.H)) =
          make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                     pack_bf16(y[6], y[7]));
    }
  }
}

template <int VPT, bool WARP>
static cudaError_t run_norm(const Ctx& cx, const NormArgs& a, int threads) {
  const unsigned grid = WARP ? (unsigned)((a.rows + kNormWarps - 1) / kNormWarps) : (unsigned)a.rows;
  return a.q ? launch_k(norm_kernel<VPT, true, WARP>, dim3(grid), dim3(threads), 0, cx.stream, cx.pdl, a)
             : launch_k(norm_kernel<VPT, false, WARP>, dim3(grid), dim3(threads), 0, cx.stream, cx.pdl, a);
}

cudaError_t launch_norm(const Ctx& cx, const NormCall& c) {
  const NormArgs a = {static_cast<const uint16_t*>(c.x), static_cast<const uint16_t*>(c.res),
                      static_cast<const uint16_t*>(c.w), static_cast<uint16_t*>(c.h),
                      static_cast<uint16_t*>(c.y), static_cast<uint8_t*>(c.q), static_cast<uint8_t*>(c.sc),
                      c.ldx, c.ldres, c.ldh, c.ldy, c.ldq, c.ldsc, c.H, c.eps, cx.status, c.rows};
  const int nv = c.H / 8;
  // As few vectors a thread as all rows' threads fit on the SMs at once with, up to four
  // (3001 rows of 2048 in 8 bits: a warp of eight vectors to each 9.9 us, two warps of
  // four 8.7); short rows by a warp each, as an SM holds no more than 32 CTAs.
  int per = 1;
  while (per < 8 && (long long)c.rows * nv > 2048LL * cx.sms * per) per *= 2;
  if (nv <= 256 && (per == 8 || (nv <= 64 && c.rows > 2 * cx.sms))) {
    const int threads = kNormWarps * 32;
    if (nv <= 32) return run_norm<1, true>(cx, a, threads);
    if (nv <= 64) return run_norm<2, true>(cx, a, threads);
    if (nv <= 128) return run_norm<4, true>(cx, a, threads);
    return run_norm<8, true>(cx, a, threads);
  }
  auto threads_of = [&](int n) { return ((nv + n - 1) / n + 31) / 32 * 32; };
  if (per == 1 && nv <= 1024) return run_norm<1, false>(cx, a, threads_of(1));
  if (per <= 2 && nv <= 2048) return run_norm<2, false>(cx, a, threads_of(2));
  if (nv <= 4096) return run_norm<4, false>(cx, a, threads_of(4));
  if (nv <= 8192) return run_norm<8, false>(cx, a, threads_of(8));
  return cudaErrorInvalidValue;
}

}  // namespace dg
