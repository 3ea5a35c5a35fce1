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
// it the sum and the root are carried in two fp32 numbers, and products near a border
// are rounded from what is exact.
//
// GB300, us (in brackets the bytes at the measured copy rate): 8000 x 7168 with
// residual 67.2 (67.7), in 8 bits 66.3 (59.5: instructions, issue slots 76 % busy); 64 x
// 7168 2.5 and 2.9 (latency); 3001 x 2048 in 8 bits 7.7 (2.8: one wave, load, sum, output
// one after another). In 8 bits with every product in two numbers 73, 3.5 and 8.9.
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
  float eps, inv;  // inv = 1 / H
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

// 1 / sqrt(sum / n + eps), inv = 1 / n: one Newton step from rsqrtf's value, whose error
// is taken exactly, as is the quotient's (n has 17 bits at most).
__device__ __forceinline__ Two root_two(Two sum, float n, float inv, float eps) {
  const float q = __fmul_rn(sum.hi, inv);
  const Two m = add_two(Two{q, (fmaf(-q, n, sum.hi) + sum.lo) * inv}, eps);
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
__device__ __forceinline__ float2 pair_fma(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
      "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}

// The largest magnitude of three, NaN if one is.
__device__ __forceinline__ float most_of(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// The products of eight pairs of bf16 with f, to fp32. (Those of the pairs are exact as
// long as fp32 holds them; norm_e4m3 sees to the others.)
__device__ __forceinline__ void times_root(const uint4& h, const uint4& w, Two f, float2 (&y)[4]) {
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = pair_mul(make_float2(bf16lo(hw[j]), bf16hi(hw[j])), make_float2(bf16lo(ww[j]), bf16hi(ww[j])));
    y[j] = pair_fma(p, make_float2(f.hi, f.hi), pair_mul(p, make_float2(f.lo, f.lo)));
  }
}

// The same product, where it is not exact to the neighbour with an odd last bit, so that
// a rounding of it to fewer bits sees on which side of a border the product lies. (A rest
// of 2^-40 is the root's own error: the product is y.) The root's power of two, f's, is
// 2^k and taken apart: it goes to the smaller of x and g where it is 1 or more, else to
// the larger, so that x g f alone says whether fp32 holds what comes before it.
__device__ __forceinline__ float to_odd(float x, float g, Two f, int k) {
  const bool swap = (fabsf(x) < fabsf(g)) == (k < 0);
  const float p = (swap ? g : x) * pow2_f(k) * (swap ? x : g);
  const float y = fmaf(p, f.hi, p * f.lo), r = fmaf(p, f.hi, -y) + p * f.lo;
  uint32_t b = __float_as_uint(y);
  if (!(b & 1) && fabsf(r) > fabsf(y) * 0x1p-40f) b += (r > 0.f) == (y > 0.f) ? 1u : ~0u;
  return __uint_as_float(b);
}
__device__ __forceinline__ void to_odd(const uint4& h, const uint4& w, Two f, float2 (&y)[4]) {
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, ww[4] = {w.x, w.y, w.z, w.w};
  const int k = min(max((int)(__float_as_uint(f.hi) >> 23) - 127, -126), 126);
  const Two g = {f.hi * pow2_f(-k), f.lo * pow2_f(-k)};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    y[j] = make_float2(to_odd(bf16lo(hw[j]), bf16lo(ww[j]), g, k), to_odd(bf16hi(hw[j]), bf16hi(ww[j]), g, k));
}

// The largest magnitude (its bits) of the 32 values that four lanes hold.
__device__ __forceinline__ uint32_t group_most(const float2 (&y)[4]) {
  const float m3 = most_of(most_of(y[0].x, y[0].y, y[1].x), y[1].y, y[2].x);
  uint32_t m = __float_as_uint(most_of(most_of(m3, y[2].y, y[3].x), y[3].y, 0.f));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

__device__ __forceinline__ int group_exponent(uint32_t most) {
  const int e = mx_exponent_e4m3(__uint_as_float(most));
  return e < -127 ? -127 : e;
}

__device__ __forceinline__ uint2 to_e4m3(const float2 (&y)[4], float s) {
  const float2 ss = make_float2(s, s);
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 u = pair_mul(y[j], ss);
    q[j] = pack_e4m3(u.x, u.y);
  }
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// Eight values of a group of 32 (four lanes) in 8 bits, and the group's scale byte.
// fp32 products are off by half a step: where 2^-22 more and 2^-22 less are the same
// e4m3, so is the product. Otherwise (one warp in 700), where the largest is just what
// a scale can hold or not finite, or where products of pairs might be below fp32's
// normal numbers (the largest y below 2^-90, of which the least e4m3 is 2^-19, or a root
// above 2^12; below that a product that fp32 takes for 0 is 0 in 8 bits too), the warp
// rounds them anew from their odd neighbours.
__device__ __forceinline__ uint2 norm_e4m3(const uint4& h, const uint4& w, Two f, int* byte) {
  float2 y[4];
  times_root(h, w, f, y);
  uint32_t m = group_most(y);
  uint2 q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);  // NaN, as the scale
  *byte = 255;
  bool near = true;
  if (!not_finite(__uint_as_float(m))) {
    const int e = group_exponent(m);
    const float s = pow2_f(-e);
    q = to_e4m3(y, s * (1.f + 0x1p-22f));
    const uint2 less = to_e4m3(y, s * (1.f - 0x1p-22f));
    *byte = e + 127;
    near = q.x != less.x || q.y != less.y || (m & 0x7FFFFFu) == 0x600000u || m - 1u < 37u << 23 || f.hi > 0x1p12f;
  }
  if (__any_sync(0xffffffffu, near)) {
    to_odd(h, w, f, y);
    m = group_most(y);
    if (!not_finite(__uint_as_float(m))) {
      const int e = group_exponent(m);
      q = to_e4m3(y, pow2_f(-e));
      *byte = e + 127;
    }
  }
  return q;
}

constexpr int kNormWarps = 8;   // rows of a CTA where a warp takes one

// VPT: vectors of 8 values a thread holds; MX: 8-bit output; WARP: a warp to a row.
// 48 registers: an SM holds 20 CTAs of 64 threads, 3001 rows of 2048 run at once (in
// 8 bits 8.0 us with 57 registers, so 7.8; 8000 x 7168 69.0 and 66.6).
template <int VPT, bool MX, bool WARP>
__global__ void __maxnreg__(WARP ? 80 : VPT > 4 ? 64 : 48) norm_kernel(const NormArgs a) {
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
  if (VPT <= 4)  // on its way with the row (8000 x 7168 in 8 bits 69.7 us, so 69.0)
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
  auto reduce = [&](int lanes) {  // of each `lanes` side by side, a power of two
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      if (off >= lanes) continue;
      const float o = __shfl_xor_sync(0xffffffffu, sum2.hi, off);
      if (MX) sum2 = add_two(sum2, Two{o, __shfl_xor_sync(0xffffffffu, sum2.lo, off)});
      else sum2.hi += o;
    }
  };
  reduce(32);
  if (!WARP) {
    if (lane == 0) {
      s_hi[warp] = sum2.hi;
      s_lo[warp] = sum2.lo;
    }
    __syncthreads();
    const int warps = nt / 32, lanes = warps > 1 ? 2 << (31 - __clz(warps - 1)) : 1, from = lane & (lanes - 1);
    sum2.hi = from < warps ? s_hi[from] : 0.f;
    sum2.lo = MX && from < warps ? s_lo[from] : 0.f;
    reduce(lanes);
  }
  const Two f = MX ? root_two(sum2, (float)a.H, a.inv, a.eps) : Two{rsqrtf(sum2.hi / (float)a.H + a.eps), 0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * nt;
    if (VPT > 4 || i > 0) w[i] = v < nv ? __ldg(reinterpret_cast<const uint4*>(a.w) + v) : make_uint4(0u, 0u, 0u, 0u);
    if constexpr (MX) {
      int b;
      const uint2 q = norm_e4m3(h[i], w[i], f, &b);
      if (v < nv) {
        *reinterpret_cast<uint2*>(a.q + norm_at(a, row, a.ldq, v * 8, a.H)) = q;
        if (!(v & 3)) a.sc[norm_at(a, row, a.ldsc, v / 4, a.H / kMxGroup)] = (uint8_t)b;
      }
    } else if (v < nv) {
      const uint32_t* hw = reinterpret_cast<const uint32_t*>(&h[i]);
      const uint32_t* ww = reinterpret_cast<const uint32_t*>(&w[i]);
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = pack_bf16(bf16lo(hw[j]) * f.hi * bf16lo(ww[j]), bf16hi(hw[j]) * f.hi * bf16hi(ww[j]));
      *reinterpret_cast<uint4*>(a.y + norm_at(a, row, a.ldy, v * 8, a.H)) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

template <int VPT, bool WARP>
static cudaError_t run_norm(const Ctx& cx, const NormArgs& a, int threads) {
  const unsigned grid = WARP ? (unsigned)((a.rows - 1) / kNormWarps + 1) : (unsigned)a.rows;
  return a.q ? launch_k(norm_kernel<VPT, true, WARP>, dim3(grid), dim3(threads), 0, cx.stream, cx.pdl, a)
             : launch_k(norm_kernel<VPT, false, WARP>, dim3(grid), dim3(threads), 0, cx.stream, cx.pdl, a);
}

cudaError_t launch_norm(const Ctx& cx, const NormCall& c) {
  const NormArgs a = {static_cast<const uint16_t*>(c.x), static_cast<const uint16_t*>(c.res),
                      static_cast<const uint16_t*>(c.w), static_cast<uint16_t*>(c.h),
                      static_cast<uint16_t*>(c.y), static_cast<uint8_t*>(c.q), static_cast<uint8_t*>(c.sc),
                      c.ldx, c.ldres, c.ldh, c.ldy, c.ldq, c.ldsc, c.H, c.eps, 1.f / (float)c.H, cx.status, c.rows};
  const int nv = c.H / 8;
  // As few vectors a thread as all rows' threads fit on the SMs at once with, up to four
  // (3001 rows of 2048 in 8 bits: a warp of eight vectors to each 8.1 us, two warps of
  // four 7.8); short rows by a warp each, as an SM holds no more than 32 CTAs.
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
