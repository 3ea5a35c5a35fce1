// k_norm.cu -- root-mean-square norm of the residual stream, with the residual's
// addition before it and an output in bf16 or in 8 bits with scales.
//
//   h = bf16(x + res);  y = h * rsqrt(mean(h^2) + eps) * w
//
// A CTA per row. A thread keeps its 16-byte vectors of h packed in registers
// between the sum of squares and the output, so every value is read once; the sum
// is fp32, added up in the same order whatever the call. Few rows: as many threads
// as vectors, up to 1024, as the time is latency. Many rows: 256 threads, several
// CTAs on an SM, bound by memory. The 8-bit output's groups of 32 are 4 lanes.
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

// VPT: vectors of 8 values a thread holds; MX: 8-bit output.
template <int VPT, bool MX>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a) {
  __shared__ float s_sum[32];
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5;
  const long long row = blockIdx.x;
  const int nv = a.H / 8;
  griddep_launch_dependents();
  uint4 w[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * nt;
    w[i] = v < nv ? __ldg(reinterpret_cast<const uint4*>(a.w) + v) : make_uint4(0u, 0u, 0u, 0u);
  }
  griddep_wait();
  uint4 h[VPT], r[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * nt;
    h[i] = r[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < nv) {
      h[i] = *reinterpret_cast<const uint4*>(a.x + norm_at(a, row, a.ldx, v * 8, a.H));
      if (a.res) r[i] = *reinterpret_cast<const uint4*>(a.res + norm_at(a, row, a.ldres, v * 8, a.H));
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * nt;
    uint32_t* hw = reinterpret_cast<uint32_t*>(&h[i]);
    const uint32_t* rw = reinterpret_cast<const uint32_t*>(&r[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (a.res) hw[j] = pack_bf16(bf16lo(hw[j]) + bf16lo(rw[j]), bf16hi(hw[j]) + bf16hi(rw[j]));
      sum = fmaf(bf16lo(hw[j]), bf16lo(hw[j]), sum);
      sum = fmaf(bf16hi(hw[j]), bf16hi(hw[j]), sum);
    }
    if (a.res && v < nv)
      *reinterpret_cast<uint4*>(a.h + norm_at(a, row, a.ldh, v * 8, a.H)) = h[i];
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = lane < nt / 32 ? s_sum[lane] : 0.f;
#pragma unroll
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const float f = rsqrtf(sum / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * nt;
    const uint32_t* hw = reinterpret_cast<const uint32_t*>(&h[i]);
    const uint32_t* ww = reinterpret_cast<const uint32_t*>(&w[i]);
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[2 * j] = bf16lo(hw[j]) * f * bf16lo(ww[j]);
      y[2 * j + 1] = bf16hi(hw[j]) * f * bf16hi(ww[j]);
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
        // 2^-e in two steps: 2^127 times 2 is past the largest fp32
        const float s1 = pow2_f(-e / 2), s2 = pow2_f(-e - -e / 2);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = y[j] * s1 * s2;
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

template <int VPT>
static cudaError_t run_norm(const Ctx& cx, const NormArgs& a, int threads) {
  return a.q ? launch_k(norm_kernel<VPT, true>, dim3((unsigned)a.rows), dim3(threads), 0, cx.stream, cx.pdl, a)
             : launch_k(norm_kernel<VPT, false>, dim3((unsigned)a.rows), dim3(threads), 0, cx.stream, cx.pdl, a);
}

cudaError_t launch_norm(const Ctx& cx, const NormCall& c) {
  const NormArgs a = {static_cast<const uint16_t*>(c.x), static_cast<const uint16_t*>(c.res),
                      static_cast<const uint16_t*>(c.w), static_cast<uint16_t*>(c.h),
                      static_cast<uint16_t*>(c.y), static_cast<uint8_t*>(c.q), static_cast<uint8_t*>(c.sc),
                      c.ldx, c.ldres, c.ldh, c.ldy, c.ldq, c.ldsc, c.H, c.eps, cx.status, c.rows};
  const int nv = c.H / 8;
  const int most = c.rows <= 2 * cx.sms ? 1024 : 256;
  int threads = nv < most ? (nv + 31) / 32 * 32 : most;
  if ((nv + threads - 1) / threads > 8) threads = 1024;
  const int per = (nv + threads - 1) / threads;
  if (per <= 1) return run_norm<1>(cx, a, threads);
  if (per <= 2) return run_norm<2>(cx, a, threads);
  if (per <= 4) return run_norm<4>(cx, a, threads);
  if (per <= 8) return run_norm<8>(cx, a, threads);
  return cudaErrorInvalidValue;
}

}  // namespace dg
