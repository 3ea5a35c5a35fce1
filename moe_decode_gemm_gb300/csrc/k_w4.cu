// k_w4.cu -- projections with 4-bit weights, and the quantisation of bf16
// weights that makes them.
//
//   y = x·Wᵀ (+ res),  W[n][k] = code[n][k] * 2^(b[n][k/32] - 127)
//
// x has 1..64 tokens, in bf16 or in e4m3 with a scale for each 32 k. A call
// cannot do without N*K/2 + N*K/32 bytes of weights, 0.266 of what bf16 weights
// take, so it is bound by memory only if nothing is done per weight: unpacking
// one with ordinary instructions costs more time than reading it from 64 tokens
// down to one. So the tensor cores take the weights as they are: tcgen05.mma of
// kind mxf8f6f4 multiplies e2m1 by e4m3 and applies both scales itself; TMA
// spreads the packed weights over shared memory lines as the MMA wants them.
//
// bf16 tokens enter as two e4m3 numbers, hi + lo, with a scale each per 32 k:
// a bf16 has 8 significant bits, an e4m3 has 4. With u = x / 2^e, e the least
// exponent that brings the group's largest to 448 or less, hi = e4m3(u) and
// lo = e4m3(16 (u - hi)): the sum is x exactly down to 2^-15 of the group's
// largest value and off by at most 2^-22 of it below. The MMA treats them as
// twice as many tokens; fp32 sums of the two halves are added at the end.
//
// A unit of work is 128 weight rows x 128 k (8 KB of weights and 512 B of scales,
// each contiguous in memory). A tile of 128 rows is shared by a cluster of S CTAs,
// each with a contiguous range of its units; their fp32 tiles are summed through
// distributed shared memory in rank order (results repeat bit by bit). Two CTAs
// fit on an SM.
//
// Warps: 0 issues the weights' copies, 1 the MMAs, 2-5 convert the tokens of a
// unit into its ring slot and then drain the accumulator.
#include "launch.h"
#include "launch_util.cuh"
#include "mx_common.cuh"

namespace dg {

constexpr int kW4Threads = 6 * 32;
constexpr int kW4Conv = 128;                        // converting (and draining) threads
constexpr int kW4Slot = kW4Tile * 128;              // a unit's weights, spread: 16 KB
constexpr int kW4Smem = 115712;                     // two CTAs per SM

// Shared memory of an instantiation: ring slots of weights, NPX token rows of 128
// bytes, and the scales of both.
template <int NPX>
struct W4Shape {
  static constexpr int kX = NPX * 128;
  static constexpr int kStage = kW4Slot + kX + 2 * kW4Scales;
  static constexpr int kStages = (kW4Smem - 1024 - 256) / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + 256;
  static constexpr int kColsUsed = NPX + 8 * kStages;   // accumulator, scales of each slot
  static constexpr int kCols = kColsUsed <= 64 ? 64 : kColsUsed <= 128 ? 128 : 256;
  static_assert(kStages >= 2 && kColsUsed <= 256, "ring depth, tensor memory of two CTAs");
  static_assert(8 * (3 * kStages + 1) + 64 <= 256, "barriers and flags");
};

struct W4Args {
  const void* x;          // bf16 [M][K], or e4m3
  const uint8_t* xs;      // scale bytes of e4m3 tokens [M][K/32]
  long long ldx, ldxs;    // elements between rows
  const uint8_t* ws;      // weight scales, 512 bytes a unit
  const uint16_t* res;    // optional [M][N] bf16
  uint16_t* y;            // [M][N] bf16
  int M, N, K, KC;        // KC: units of a tile
  int half;               // token rows of one half of B: the lo rows start there (0: e4m3 tokens)
  int np;                 // token rows in all, a multiple of 16
  int* status;
  long long timeout_ns;
};

// Eight bf16 tokens' values as e4m3 hi and lo; the four lanes of a group share
// the exponent. Returns the scale byte of hi (lo's is 4 less).
__device__ __forceinline__ int split_e4m3(const uint4& v, uint2& hi, uint2& lo) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8], a = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(w[i]);
    f[2 * i + 1] = bf16hi(w[i]);
  }
  // the largest bits: the largest magnitude, and a NaN above all others
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  a = __uint_as_float(m);
  hi = lo = make_uint2(0u, 0u);
  if (not_finite(a)) return 255;  // the scale NaN: every sum of the token becomes NaN
  int e = mx_exponent_e4m3(a);
  e = e < -123 ? -123 : e;        // lo's exponent, e - 4, is at least -127
  const float s = pow2_f(-e);
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float u0 = f[2 * i] * s, u1 = f[2 * i + 1] * s;
    h[i] = pack_e4m3(u0, u1);
    uint32_t back;  // hi as two fp16, exact
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"((uint16_t)h[i]));
    float h0, h1;
    asm("{\n\t.reg .b16 p, q;\n\tmov.b32 {p, q}, %2;\n\tcvt.f32.f16 %0, p;\n\tcvt.f32.f16 %1, q;\n\t}"
        : "=f"(h0), "=f"(h1)
        : "r"(back));
    l[i] = pack_e4m3((u0 - h0) * 16.f, (u1 - h1) * 16.f);
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
  return e + 127;
}

// VPT: vectors of 16 bytes that each converting thread takes per unit; NPX: the
// most token rows (bf16: 16 VPT, tokens 8 VPT; e4m3: 16 VPT tokens).
template <int VPT, bool MX>
__global__ void __launch_bounds__(kW4Threads, 2)
    w4_linear_kernel(const __grid_constant__ CUtensorMap wmap, const W4Args a) {
  constexpr int NPX = 16 * VPT;
  using Sh = W4Shape<NPX>;
  constexpr int STAGES = Sh::kStages;
  constexpr int DEPTH = VPT == 1 ? 4 : VPT == 2 ? 2 : 1;  // units of tokens in registers ahead
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* wfull = reinterpret_cast<uint64_t*>(smem + STAGES * Sh::kStage);  // weights there
  uint64_t* xfull = wfull + STAGES;                                          // tokens there
  uint64_t* empty = xfull + STAGES;
  uint64_t* tfull = empty + STAGES;
  volatile int* s_flags = reinterpret_cast<volatile int*>(tfull + 1);  // [0] abort
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(const_cast<int*>(s_flags) + 1);
  // slot s: [weights 16 KB][token rows][weight scales][token scales]
  auto slot_x = [&](int s) { return smem + s * Sh::kStage + kW4Slot; };
  auto slot_ws = [&](int s) { return slot_x(s) + Sh::kX; };
  auto slot_xs = [&](int s) { return slot_ws(s) + kW4Scales; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&xfull[s], kW4Conv / 32);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    s_flags[0] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_taddr, Sh::kCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 64) prefetch_tmap(&wmap);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = *s_taddr;
  griddep_launch_dependents();

  const int cs = (int)cluster_size(), cr = (int)cluster_rank();
  const int tile = (int)(blockIdx.x / cs);
  const int kc0 = (int)((long long)cr * a.KC / cs);
  const int nunits = (int)((long long)(cr + 1) * a.KC / cs) - kc0;

  if (warp == 0) {
    // ---------------------------------------------------------------- weights
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      const long long unit0 = (long long)tile * a.KC + kc0;
      int i = 0;
      for (; i < nunits; ++i) {
        const int s = i % STAGES;
        if (i >= STAGES) {
          if (!mbar_wait(&empty[s], ((i / STAGES) + 1) & 1, a.timeout_ns, a.status)) s_flags[0] = 1;
        }
        if (s_flags[0]) break;
        mbar_arrive_expect_tx(&wfull[s], kW4Unit + kW4Scales);
        tma_load_2d(smem + s * Sh::kStage, &wmap, 0, (int)((unit0 + i) * kW4Tile), &wfull[s], pol);
        bulk_copy_g2s(slot_ws(s), a.ws + (unit0 + i) * kW4Scales, kW4Scales, &wfull[s]);
      }
      // Every issued copy has landed before the shared memory is used anew.
      const int issued = i;
      for (int s = 0; s < STAGES && s < issued; ++s) {
        const int uses = (issued - s + STAGES - 1) / STAGES;
        mbar_wait(&wfull[s], (uses - 1) & 1, drain_ns(a.timeout_ns), nullptr);
      }
    }
    griddep_wait();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    griddep_wait();
    const uint32_t leader = elect_one();
    for (int i = 0; i < nunits; ++i) {
      const int s = i % STAGES;
      if (!s_flags[0]) {
        if (!mbar_wait(&wfull[s], (i / STAGES) & 1, a.timeout_ns, a.status) ||
            !mbar_wait(&xfull[s], (i / STAGES) & 1, a.timeout_ns, a.status))
          s_flags[0] = 1;
      }
      __syncwarp();
      tc_fence_after();
      if (!s_flags[0]) {
        const uint32_t wb = smem_u32(smem + s * Sh::kStage), xb = smem_u32(slot_x(s));
        const uint32_t sa = taddr + NPX + 8 * s, sb = sa + 4;
        tmem_copy_scales_elect(leader, sa, smem_u32(slot_ws(s)));
        tmem_copy_scales_elect(leader, sb, smem_u32(slot_xs(s)));
#pragma unroll
        for (int g = 0; g < 4; ++g)
          umma_mx_elect(leader, taddr, umma_desc_sw128(wb + g * 32), umma_desc_sw128(xb + g * 32),
                        umma_idesc_mx(a.np, g), sa, sb, (i == 0 && g == 0) ? 0u : 1u);
      }
      __syncwarp();
      umma_commit_elect(leader, &empty[s]);
    }
    umma_commit_elect(leader, tfull);
    mbar_wait(tfull, 0, drain_ns(a.timeout_ns), nullptr);
  } else {
    // ---------------------------------------------------------------- tokens
    griddep_wait();
    const int t = threadIdx.x - 64;
    constexpr int PER = MX ? 8 : 16;       // vectors of a token's 128 k
    constexpr int EL = MX ? 16 : 8;        // elements of a vector
    const int vec = t % PER, tok0 = t / PER;
    auto load = [&](int i, int j) -> uint4 {
      const int tok = tok0 + j * (kW4Conv / PER);
      const int k = (kc0 + i) * kW4Tile + vec * EL;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (i < nunits && tok < a.M && k < a.K) {
        const long long at = tok * a.ldx + k;
        const uint8_t* p = reinterpret_cast<const uint8_t*>(a.x) + (MX ? at : 2 * at);
        v = *reinterpret_cast<const uint4*>(p);
      }
      return v;
    };
    uint4 ahead[DEPTH][VPT];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
      for (int j = 0; j < VPT; ++j) ahead[d][j] = load(d, j);
    for (int i0 = 0; i0 < nunits; i0 += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const int i = i0 + d;
        if (i >= nunits || s_flags[0]) break;
        const int s = i % STAGES;
        if (i >= STAGES) {
          if (!mbar_wait(&empty[s], ((i / STAGES) + 1) & 1, a.timeout_ns, a.status)) s_flags[0] = 1;
        }
        __syncwarp();
        uint8_t* xt = slot_x(s);
        uint8_t* xs = slot_xs(s);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int tok = tok0 + j * (kW4Conv / PER);
          if constexpr (MX) {
            if (tok < a.np)
              *reinterpret_cast<uint4*>(xt + tok * 128 + ((vec ^ (tok & 7)) << 4)) = ahead[d][j];
            const int g = vec >> 1, k = (kc0 + i) * kW4Tile + g * kMxGroup;
            if (!(vec & 1) && tok < a.np)
              xs[mx_scale_at(tok, g)] =
                  tok < a.M && k < a.K ? a.xs[tok * a.ldxs + k / kMxGroup] : (uint8_t)127;
          } else {
            uint2 hi, lo;
            const int b = split_e4m3(ahead[d][j], hi, lo);
            if (tok < a.half) {  // rows hi, then rows lo; 128-byte swizzle
              uint8_t* p = xt + tok * 128 + (((vec >> 1) ^ (tok & 7)) << 4) + (vec & 1) * 8;
              *reinterpret_cast<uint2*>(p) = hi;
              *reinterpret_cast<uint2*>(p + a.half * 128) = lo;
              if (!(vec & 3)) {
                xs[mx_scale_at(tok, vec >> 2)] = (uint8_t)b;
                xs[mx_scale_at(a.half + tok, vec >> 2)] = (uint8_t)(b == 255 ? 255 : b - 4);
              }
            }
          }
          ahead[d][j] = load(i + DEPTH, j);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&xfull[s]);
      }
    }
    if (!s_flags[0]) {
      if (!mbar_wait(tfull, 0, a.timeout_ns, a.status)) s_flags[0] = 1;
    }
    __syncwarp();
    tc_fence_after();
  }

  // Rank q owns rows q*R4 .. of the tile: each thread gives its row's sums to the
  // owner, recv[source][token][row], which adds them up in rank order.
  const int R4 = ((kW4Tile + cs - 1) / cs + 3) / 4 * 4;
  float* recv = reinterpret_cast<float*>(smem);
  const int cols = MX ? a.np : a.half;
  __syncwarp();
  cluster_sync_all();  // every rank's ring is free
  if (warp >= 2 && !s_flags[0]) {
    const int r = (warp & 3) * 32 + lane;  // row: the warp's quarter of the lanes
    const int q = r / R4, rl = r - q * R4;
    float* dst = recv + (size_t)cr * cols * R4 + rl;
    const uint32_t row = taddr + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int c = 0; c < a.M; c += 16) {
      float v[16], w[16];
      tmem_ld16_sync(row + c, v);
      if constexpr (!MX) {
        tmem_ld16_sync(row + a.half + c, w);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += w[j];
      }
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c + j < a.M) st_dsmem_f32(dst + (c + j) * R4, (uint32_t)q, v[j]);
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync_all();
  if (warp >= 2 && !s_flags[0]) {
    const int r0 = cr * R4 < kW4Tile ? cr * R4 : kW4Tile;
    const int RR = (r0 + R4 < kW4Tile ? r0 + R4 : kW4Tile) - r0;
    for (int e = threadIdx.x - 64; e < RR * a.M; e += kW4Conv) {
      const int tok = e / RR, rl = e - tok * RR;
      float sum = 0.f;
      for (int src = 0; src < cs; ++src) sum += recv[((size_t)src * cols + tok) * R4 + rl];
      const int n = tile * kW4Tile + r0 + rl;
      if (n < a.N) {
        const long long at = (long long)tok * a.N + n;
        if (a.res) sum = bf_bits2f(*DG_AT(a.status, a.res, at, (long long)a.M * a.N)) + sum;
        *DG_AT(a.status, a.y, at, (long long)a.M * a.N) = f2bf_bits(sum);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, Sh::kCols);
  }
}

template <int VPT, bool MX>
static cudaError_t run_w4(const Ctx& cx, const W4Call& c, int split) {
  using Sh = W4Shape<16 * VPT>;
  static_assert(2 * (Sh::kSmem + 1024) <= kSmemPerSm, "two CTAs per SM");
  auto kern = w4_linear_kernel<VPT, MX>;
  static DevOnce once;
  if (cudaError_t e = setup_smem(once, kern, Sh::kSmem, true); e != cudaSuccess) return e;
  const int tiles = (c.N + kW4Tile - 1) / kW4Tile, KC = (c.K + kW4Tile - 1) / kW4Tile;
  CUtensorMap wmap;
  if (!make_tmap_w4(&wmap, c.wq, (uint64_t)tiles * KC * kW4Tile)) return cudaErrorInvalidValue;
  W4Args a = {};
  a.x = c.x;
  a.xs = static_cast<const uint8_t*>(c.xs);
  a.ldx = c.ldx;
  a.ldxs = c.ldxs;
  a.ws = static_cast<const uint8_t*>(c.ws);
  a.res = static_cast<const uint16_t*>(c.res);
  a.y = static_cast<uint16_t*>(c.y);
  a.M = c.M;
  a.N = c.N;
  a.K = c.K;
  a.KC = KC;
  a.half = MX ? 0 : (c.M + 7) / 8 * 8;
  a.np = MX ? (c.M + 15) / 16 * 16 : 2 * a.half;
  a.status = cx.status;
  a.timeout_ns = cx.timeout_ns;
  return launch_kc(kern, dim3((unsigned)(tiles * split)), dim3(kW4Threads), Sh::kSmem, cx.stream, cx.pdl,
                   split, wmap, a);
}

// CTAs that share a tile of 128 rows: as many as two per SM hold, at most 8 (the
// portable cluster size) and one per unit.
static int w4_split(int N, int K, int sms) {
  const int tiles = (N + kW4Tile - 1) / kW4Tile, KC = (K + kW4Tile - 1) / kW4Tile;
  int s = 2 * sms / tiles;
  if (s > 8) s = 8;
  if (s > KC) s = KC;
  return s < 1 ? 1 : s;
}

cudaError_t launch_w4_linear(const Ctx& cx, const W4Call& c) {
  const int s = w4_split(c.N, c.K, cx.sms);
  if (c.xs) {
    if (c.M <= 16) return run_w4<1, true>(cx, c, s);
    if (c.M <= 32) return run_w4<2, true>(cx, c, s);
    return run_w4<4, true>(cx, c, s);
  }
  if (c.M <= 8) return run_w4<1, false>(cx, c, s);
  if (c.M <= 16) return run_w4<2, false>(cx, c, s);
  if (c.M <= 32) return run_w4<4, false>(cx, c, s);
  return run_w4<8, false>(cx, c, s);
}

// ------------------------------------------------------------------ quantisation
// A CTA per unit: 16 lanes take the 128 k of a row, 8 each; the four lanes of a
// group share its largest magnitude. Reads 2 bytes a weight, writes 0.53: memory.
constexpr int kQuantThreads = 256;

__global__ void __launch_bounds__(kQuantThreads)
    w4_quant_kernel(const uint16_t* W, long long ldw, uint8_t* q, uint8_t* sc, int N, int K, int KC) {
  __shared__ __align__(16) uint8_t s_sc[kW4Scales];
  const long long unit = blockIdx.x;
  const int tile = (int)(unit / KC), kc = (int)(unit - (long long)tile * KC);
  const int vec = threadIdx.x & 15, row0 = threadIdx.x >> 4;
  constexpr int ROWS = kQuantThreads / 16, STEPS = kW4Tile / ROWS;
  const int k = kc * kW4Tile + vec * 8;
  uint4 v[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int n = tile * kW4Tile + row0 + i * ROWS;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (n < N && k < K) v[i] = __ldcs(reinterpret_cast<const uint4*>(W + (long long)n * ldw + k));
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int row = row0 + i * ROWS;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    float f[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16lo(w[j]);
      f[2 * j + 1] = bf16hi(w[j]);
      m = max(m, max(__float_as_uint(f[2 * j]) & 0x7FFFFFFFu, __float_as_uint(f[2 * j + 1]) & 0x7FFFFFFFu));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float a = __uint_as_float(m);
    uint32_t codes = 0;
    int b = 255;  // a group with a value that is not finite: the scale NaN, codes 0
    if (!not_finite(a)) {
      int e = mx_exponent_e2m1(a);
      e = e < -127 ? -127 : e;
      b = e + 127;
      // 2^-e in two steps: 2^127 times 2 is past the largest fp32
      const float s1 = pow2_f(-e / 2), s2 = pow2_f(-e - -e / 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t two;  // f[2j] -> low half, f[2j+1] -> high half of a byte
        asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
            : "=r"(two)
            : "f"(f[2 * j + 1] * s1 * s2), "f"(f[2 * j] * s1 * s2));
        codes |= two << (8 * j);
      }
    }
    *reinterpret_cast<uint32_t*>(q + unit * kW4Unit + row * 64 + vec * 4) = codes;
    if (!(vec & 3)) s_sc[mx_scale_at(row, vec >> 2)] = (uint8_t)b;
  }
  __syncthreads();
  if (threadIdx.x < kW4Scales / 16)
    reinterpret_cast<uint4*>(sc + unit * kW4Scales)[threadIdx.x] =
        reinterpret_cast<const uint4*>(s_sc)[threadIdx.x];
}

cudaError_t launch_w4_quant(const Ctx& cx, const void* W, long long ldw, void* q, void* s, int N, int K) {
  const int tiles = (N + kW4Tile - 1) / kW4Tile, KC = (K + kW4Tile - 1) / kW4Tile;
  // No early start of what follows (a projection reads weights before it waits for
  // the kernel before it): this kernel never lets its dependents launch.
  w4_quant_kernel<<<(unsigned)((long long)tiles * KC), kQuantThreads, 0, cx.stream>>>(
      static_cast<const uint16_t*>(W), ldw, static_cast<uint8_t*>(q), static_cast<uint8_t*>(s), N, K, KC);
  return cudaGetLastError();
}

}  // namespace dg
