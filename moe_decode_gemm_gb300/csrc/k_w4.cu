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
// lo = e4m3(16 (u - hi)), of which the least step is 2^-13 in u: the sum is u exactly
// from 2^-6 on, and off by at most 2^-14 below; the group's largest is above 224, so
// 2^-13.8 and 2^-21.8 of it. The MMA treats them as
// twice as many tokens; fp32 sums of the two halves are added at the end.
//
// A unit of work is 128 weight rows x 128 k (8 KB of weights and 512 B of scales,
// each contiguous in memory), a ring slot a pair of them along k. One or two tiles
// of 128 rows are shared by a cluster of S CTAs, each with a contiguous range of
// their k; the fp32 sums are exchanged through distributed shared memory and added
// in rank order (results repeat bit by bit).
//
// Warps: 0 issues the weights' copies, 1 the MMAs, the others bring a pair's tokens
// into their ring (bf16 ones converted, e4m3 ones by TMA) and then drain the
// accumulators.
//
// GB300, us on the GPU (in brackets the weights' bytes at the measured copy rate):
// 7168 x 7168 with 1 / 16 / 64 tokens 7.6 / 8.3 / 12.9 (4.0), 16384 x 7168 11.8 / 13.4 /
// 19.5 (9.2), 64 tokens in 8 bits 9.4 and 15.2. About 3.5 us are start and end (first
// copies, conversion, exchange, output); 64 bf16 tokens with one tile are bound by
// the 64 bytes a clock that an SM takes in, 34 KB of tokens for 17 KB of weights.
#include <atomic>

#include "launch.h"
#include "launch_util.cuh"
#include "mx_common.cuh"

namespace dg {

constexpr int kW4Spread = kW4Tile * 128;            // a unit's weights in shared memory: 16 KB
constexpr int kPair = 2;                            // units along k whose tokens share a ring slot
static_assert(kPair * kW4Scales <= 1024, "scales of a slot");

// Where the tokens of a call come from: bf16 rows converted by each CTA, e4m3 rows
// by TMA, or bf16 rows that a kernel before has converted into images of ring slots.
enum W4Tokens : int { W4_CONVERT = 0, W4_MX = 1, W4_READY = 2 };

// Shapes of an instantiation for up to MT tokens, RT tiles a CTA, CW warps that
// bring the tokens and drain the accumulators. One CTA to an SM.
template <int MT, int RT, int MODE, int CW>
struct W4Shape {
  static constexpr int kConv = CW * 32;
  static constexpr int kThreads = 64 + kConv;
  static constexpr int kVec = (MT + CW - 1) / CW;  // tokens of a slot a warp converts
  static constexpr int kSlots = kVec == 1 ? 2 : 1;            // and slots of its turn
  static constexpr int kRows = MODE == W4_MX ? MT : 2 * MT;   // token rows: hi, then lo
  static constexpr int kXChunk = kRows * 128;                 // token rows of 128 k
  static constexpr int kXSlot = kPair * kXChunk + 1024;       // and their scales
  static constexpr int kXS = kRows <= 16 ? 4 : RT * kRows <= 128 ? 3 : 2;  // ring slots of tokens
  // A slot of weights is a pair of units: what a slot costs the copying and the
  // multiplying warp, 430 and 250 clocks, is more than half of the copies' own time.
  static constexpr int kWSlot = kPair * kW4Spread + 1024;     // and their scales
  // The sums of the rows that a CTA owns, from every rank: RT * 128 rows and 4 to spare
  // from each, MT tokens. Up to 16 tokens they have a place of their own, and no CTA
  // waits for another's rings before it sends; beyond, they take the rings' place.
  static constexpr int kSums = (RT * kW4Tile + 32) * MT * 4;
  static constexpr bool kRecvApart = MT <= 16;
  static constexpr int kFixed = 1024 + 512 + (kRecvApart ? kSums : 0);
  static constexpr int kRoom = 231424 - kFixed;
  static constexpr int kFit = (kRoom - kXS * kXSlot) / kWSlot;
  static constexpr int kWS = kFit > 6 ? 6 : kFit;             // ring slots of weights
  static constexpr int kRings = kXS * kXSlot + kWS * kWSlot;
  static constexpr int kSmem = kFixed + kRings;
  static constexpr int kTmemUsed = RT * kRows + 4 * kPair * (kXS + kWS);
  static constexpr int kTmem = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kWS >= 2 && kTmemUsed <= 512, "ring depth, tensor memory");
  static_assert(MODE != W4_CONVERT || kSlots <= kXS, "a turn takes no slot of the ring twice");
  static_assert(kSmem <= kMaxDynSmem, "shared memory");
  static_assert(8 * (2 * kWS + 2 * kXS + 1) + 16 <= 512, "barriers and flags");
  static_assert(kRecvApart || kSums <= kRings, "the sums fit in the rings");
  static_assert(CW % 4 == 0, "every quarter of the tensor-memory lanes is drained");
};

struct W4Args {
  const void* x;          // bf16 [M][K], or images of ring slots
  const uint8_t* xs;      // scale bytes of e4m3 tokens [M][K/32]
  long long ldx, ldxs;    // elements between rows
  const uint8_t* ws;      // weight scales, 512 bytes a unit
  const uint16_t* res;    // optional [M][N] bf16
  uint16_t* y;            // [M][N] bf16
  int M, N, K, KC, tiles; // KC: units of a tile
  int groups;             // converting warps: groups that take ring slots in turn
  int xarrivals;          // arrivals that complete a slot of tokens
  int* status;
  long long timeout_ns;
};

// The bits of the largest magnitude (0x7F80 or more: not finite) of the 32 bf16 that
// four lanes hold.
__device__ __forceinline__ uint32_t group_most(const uint32_t (&w)[4]) {
  auto most = [](uint32_t p, uint32_t q) {
    const __nv_bfloat162 y = __hmax2_nan(__habs2(reinterpret_cast<__nv_bfloat162&>(p)),
                                         __habs2(reinterpret_cast<__nv_bfloat162&>(q)));
    return reinterpret_cast<const uint32_t&>(y);
  };
  uint32_t m = most(most(w[0], w[1]), most(w[2], w[3]));
  m = most(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = most(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return max(m & 0xFFFFu, m >> 16);
}

// Eight values of a bf16 token as e4m3 hi and lo; the four lanes of a group share
// the exponent. Returns the scale byte of hi (lo's is 4 less). The values go
// through fp16, which holds u to 2^-25, far below what lo does.
__device__ __forceinline__ int split_e4m3(const uint4& v, uint2& hi, uint2& lo) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint32_t m = group_most(w);
  // e + 135 = the exponent field, one more where the fraction is above 1.75 (ceil(log2(a / 448)))
  int t = (int)((m + 0x1Fu) >> 7);
  t = t < 12 ? 12 : t;            // lo's exponent, e - 4, is at least -127
  const uint32_t s1 = (uint32_t)(262 - t) << 7, s = s1 | s1 << 16;  // 2^-e
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u, f, back, r;
    uint16_t a, b;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(u) : "r"(w[i]), "r"(s));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f) : "f"(bf16hi(u)), "f"(bf16lo(u)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(f));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(a));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(f), "r"(back));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x4C004C00u));  // 16, 16
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(r));
    h[i] = a;
    l[i] = b;
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
  return m >= 0x7F80u ? 255 : t - 8;  // not finite: the scale NaN, every sum of the token becomes NaN
}

// Lane's eight values of token tok in the image of a ring slot of tokens: two
// chunks of MT rows hi and MT rows lo (128 bytes each, 128-byte swizzle), then the
// scales of both chunks.
template <int MT>
__device__ __forceinline__ void put_token(uint8_t* slot, int tok, int lane, uint2 hi, uint2 lo, int b) {
  const int chunk = lane >> 4, in = lane & 15;  // vector `in` of the chunk's 128 k
  uint8_t* p = slot + (chunk * 2 * MT + tok) * 128 + (((in >> 1) ^ (tok & 7)) << 4) + (in & 1) * 8;
  *reinterpret_cast<uint2*>(p) = hi;
  *reinterpret_cast<uint2*>(p + MT * 128) = lo;
  if (!(in & 3)) {
    uint8_t* sc = slot + kPair * 2 * MT * 128 + chunk * kW4Scales;
    sc[mx_scale_at(tok, in >> 2)] = (uint8_t)b;
    sc[mx_scale_at(MT + tok, in >> 2)] = (uint8_t)(b - 4);
  }
}

// The tokens of a call as images of ring slots, a warp for each token and 256 k.
constexpr int kReadyThreads = 256;
template <int MT>
__global__ void __launch_bounds__(kReadyThreads) w4_tokens_kernel(const uint16_t* x, long long ldx, uint8_t* out,
                                                                  int M, int K, int slots) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * (kReadyThreads / 32) + (threadIdx.x >> 5);
  const int slot = item / M, tok = item - slot * M;
  if (slot >= slots) return;
  const int k = slot * kPair * kW4Tile + lane * 8;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (k < K) v = *reinterpret_cast<const uint4*>(x + tok * ldx + k);
  uint2 hi, lo;
  const int b = split_e4m3(v, hi, lo);
  put_token<MT>(out + (long long)slot * (kPair * 2 * MT * 128 + 1024), tok, lane, hi, lo, b);
}

// A thread's next outputs: a token's four rows each, threads side by side along the
// rows that the CTA owns.
template <int THREADS>
struct W4Outputs {
  static constexpr int U = 2;  // under way at once
  int quads, items, n0;        // fours of rows of a token; of all tokens; the first row
  int e;                       // the item after these
  int tok[U], quad[U];         // tok < 0: none
  uint2 res[U];
  __device__ bool any() const { return tok[0] >= 0; }
  __device__ void find(const W4Args& a, int first) {
    e = first;
#pragma unroll
    for (int u = 0; u < U; ++u, e += THREADS) {
      tok[u] = -1;
      quad[u] = 0;
      res[u] = make_uint2(0u, 0u);
      if (e >= items) continue;
      tok[u] = e / quads;
      quad[u] = e - tok[u] * quads;
      const int n = n0 + 4 * quad[u];
      if (a.res && (a.N & 3) == 0 && n < a.N)
        res[u] = *reinterpret_cast<const uint2*>(
            DG_AT(a.status, a.res, (long long)tok[u] * a.N + n, (long long)a.M * a.N - 3));
    }
  }
};

template <int MT, int RT, int MODE, int CW>
__global__ void __launch_bounds__(W4Shape<MT, RT, MODE, CW>::kThreads, 1)
    w4_linear_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap wmap1,
                     const __grid_constant__ CUtensorMap xmap, const W4Args a) {
  using Sh = W4Shape<MT, RT, MODE, CW>;
  constexpr int WS = Sh::kWS, XS = Sh::kXS, CONV = Sh::kConv;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* xring = smem + WS * Sh::kWSlot;
  float* recv = reinterpret_cast<float*>(smem + (Sh::kRecvApart ? Sh::kRings : 0));  // [source][token][row]
  uint64_t* wfull = reinterpret_cast<uint64_t*>(smem + Sh::kSmem - 1024 - 512);
  uint64_t* wempty = wfull + WS;
  uint64_t* xfull = wempty + WS;
  uint64_t* xempty = xfull + XS;
  uint64_t* tfull = xempty + XS;
  volatile int* s_flags = reinterpret_cast<volatile int*>(tfull + 1);  // [0] abort
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(const_cast<int*>(s_flags) + 1);
  auto wslot = [&](int s) { return smem + s * Sh::kWSlot; };
  auto xslot = [&](int s) { return xring + s * Sh::kXSlot; };

  const int cs = (int)cluster_size(), cr = (int)cluster_rank();
  const int tile0 = (int)(blockIdx.x / cs) * RT;
  const int nrt = RT == 1 ? 1 : (a.tiles - tile0 < RT ? a.tiles - tile0 : RT);
  const int pairs = (a.KC + kPair - 1) / kPair;  // of units; the last may be one unit
  const int kc0 = kPair * (int)((long long)cr * pairs / cs);
  const int nk = min(kPair * (int)((long long)(cr + 1) * pairs / cs), a.KC) - kc0;
  const int nx = (nk + kPair - 1) / kPair;
  // Rank q owns rows q*R4 .. of the nrt * 128.
  const int rows = nrt * kW4Tile;
  const int R4 = ((rows + cs - 1) / cs + 3) / 4 * 4;
  const int r0 = cr * R4 < rows ? cr * R4 : rows;
  const int RR = (r0 + R4 < rows ? r0 + R4 : rows) - r0;

  W4Outputs<CONV> next;
  next.quads = RR / 4;
  next.items = next.quads * a.M;
  next.n0 = tile0 * kW4Tile + r0;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < WS; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], 1);
    }
    for (int s = 0; s < XS; ++s) {
      mbar_init(&xfull[s], a.xarrivals);
      mbar_init(&xempty[s], 1);
    }
    mbar_init(tfull, 1);
    s_flags[0] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_taddr, Sh::kTmem);
    tmem_relinquish();
  }
  if (threadIdx.x == 64) {
    prefetch_tmap(&wmap);
    prefetch_tmap(&wmap1);
    if (MODE == W4_MX) prefetch_tmap(&xmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = *s_taddr;
  griddep_launch_dependents();
  if (Sh::kRecvApart && cs > 1) cluster_arrive_all();  // this CTA can be sent to

  if (warp == 0) {
    // ---------------------------------------------------------------- weights
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      int i = 0, rt = 0, s = 0, ph = 1;
      for (int kc = 0; kc < nk; ++i) {
        // The first pass over the ring finds it empty, and the kernel before perhaps
        // running; from then on the wait is for this kernel alone.
        if (i == WS) griddep_wait();
        if (i >= WS && !mbar_wait(&wempty[s], ph, a.timeout_ns, a.status)) {
          s_flags[0] = 1;
          break;
        }
        const long long unit = (long long)(tile0 + rt) * a.KC + kc0 + kc;
        const int units = nk - kc < kPair ? nk - kc : kPair;
        mbar_arrive_expect_tx(&wfull[s], units * (kW4Unit + kW4Scales));
        // a pair of units is one box; the last of an odd number has a map of its own
        tma_load_2d(wslot(s), units == kPair ? &wmap : &wmap1, 0, (int)(unit * kW4Tile), &wfull[s], pol);
        bulk_copy_g2s(wslot(s) + kPair * kW4Spread, a.ws + unit * kW4Scales, units * kW4Scales, &wfull[s]);
        if (++rt == nrt) {
          rt = 0;
          kc += kPair;
        }
        if (++s == WS) {
          s = 0;
          ph ^= 1;
        }
      }
      // Every issued copy has landed before the shared memory is used anew.
      const int issued = i;
      for (int q = 0; q < WS && q < issued; ++q) {
        const int uses = (issued - q + WS - 1) / WS;
        mbar_wait(&wfull[q], (uses - 1) & 1, drain_ns(a.timeout_ns), nullptr);
      }
    }
    griddep_wait();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    // This warp's instructions between two units are what a unit costs at least:
    // descriptors are added up from constants, the next unit's barrier is looked at
    // before it is waited for, and no flag is read on the way.
    griddep_wait();
    const uint32_t leader = elect_one();
    const uint32_t tm = __shfl_sync(~0u, taddr, 0);
    const uint32_t sfw = tm + RT * Sh::kRows, sfx = sfw + 4 * kPair * WS;
    const uint64_t desc = umma_desc_sw128(0);
    const uint32_t d_hi = (uint32_t)(desc >> 32);
    const uint32_t wa = __shfl_sync(~0u, (uint32_t)desc + (smem_u32(smem) >> 4), 0);
    const uint32_t xa = __shfl_sync(~0u, (uint32_t)desc + (smem_u32(xring) >> 4), 0);
    const uint32_t idesc = umma_idesc_mx(Sh::kRows, 0);
    int ws = 0, wp = 0, xs = 0, xp = 0;
    // A wait that runs out ends both loops: a slot that was not read is not given back,
    // or its next copy would be issued beside the one still on its way.
    bool ok = true, ready = false;
    for (int kx = 0; kx < nx; ++kx) {
      const bool two = (kx + 1) * kPair <= nk;
      ok = mbar_wait(&xfull[xs], xp, a.timeout_ns, a.status);
      if (!ok) break;
      const uint32_t xd = xa + xs * (Sh::kXSlot >> 4), sx = sfx + 4 * kPair * xs;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < kPair; ++h)
        tmem_copy_scales_elect(leader, sx + 4 * h, xd + ((kPair * Sh::kXChunk + h * kW4Scales) >> 4));
      for (int rt = 0; rt < nrt; ++rt) {
        if (!ready) ok = mbar_wait(&wfull[ws], wp, a.timeout_ns, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t wd = wa + ws * (Sh::kWSlot >> 4), sw = sfw + 4 * kPair * ws, d = tm + rt * Sh::kRows;
#pragma unroll
        for (int h = 0; h < kPair; ++h)
          if (h == 0 || two)
            tmem_copy_scales_elect(leader, sw + 4 * h, wd + ((kPair * kW4Spread + h * kW4Scales) >> 4));
#pragma unroll
        for (int h = 0; h < kPair; ++h)
          if (h == 0 || two) {
            const uint32_t wh = wd + (h * kW4Spread >> 4), xh = xd + (h * Sh::kXChunk >> 4);
#pragma unroll
            for (int g = 0; g < 4; ++g)
              umma_mx_elect(leader, d, wh + 2 * g, d_hi, xh + 2 * g, d_hi, idesc | umma_mx_group(g), sw + 4 * h,
                            sx + 4 * h, (g > 0 || h > 0 || kx > 0) ? 1u : 0u);
          }
        uint64_t* done = &wempty[ws];
        if (++ws == WS) {
          ws = 0;
          wp ^= 1;
        }
        ready = mbar_test_wait(&wfull[ws], wp);
        umma_commit_elect(leader, done);
      }
      if (!ok) break;
      umma_commit_elect(leader, &xempty[xs]);
      if (++xs == XS) {
        xs = 0;
        xp ^= 1;
      }
    }
    if (!ok) s_flags[0] = 1;
    __syncwarp();
    umma_commit_elect(leader, tfull);
    mbar_wait(tfull, 0, drain_ns(a.timeout_ns), nullptr);
  } else {
    // ---------------------------------------------------------------- tokens
    griddep_wait();
    const int t = threadIdx.x - 64;
    int xs = 0, xp = 1;  // the first pass over the ring finds it empty
    bool ok = true;
    if constexpr (MODE != W4_CONVERT) {
      if (warp == 2) {
        // the rows (and, with them in images of ring slots, the scales)
        if (lane == 0) {
          int issued = 0;
          for (int kx = 0; kx < nx; ++kx) {
            if (!mbar_wait(&xempty[xs], xp, a.timeout_ns, a.status)) {
              ok = false;
              break;
            }
            if constexpr (MODE == W4_READY) {
              mbar_arrive_expect_tx(&xfull[xs], Sh::kXSlot);
              bulk_copy_g2s(xslot(xs),
                            reinterpret_cast<const uint8_t*>(a.x) + (long long)(kc0 / kPair + kx) * Sh::kXSlot,
                            Sh::kXSlot, &xfull[xs]);
            } else {
              mbar_arrive_expect_tx(&xfull[xs], kPair * Sh::kXChunk);
#pragma unroll
              for (int h = 0; h < kPair; ++h)  // (what lies past K reads as 0)
                tma_load_2d(xslot(xs) + h * Sh::kXChunk, &xmap, (kc0 + kx * kPair + h) * kW4Tile, 0, &xfull[xs],
                            policy_evict_last());
            }
            ++issued;
            if (++xs == XS) {
              xs = 0;
              xp ^= 1;
            }
          }
          // Every issued copy has landed before the shared memory is used anew (after a
          // give-up a barrier may lack arrivals, and the wait take its whole bound).
          for (int q = 0; q < XS && q < issued; ++q)
            mbar_wait(&xfull[q], ((issued - q + XS - 1) / XS - 1) & 1, drain_ns(a.timeout_ns), nullptr);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      } else if (MODE == W4_MX && warp < 3 + (MT + 31) / 32) {
        // the scale bytes, a word of four per token and 128 k
        constexpr int DEPTH = 4;
        const int tok = t - 32;
        const uint8_t* sp = a.xs + (tok < a.M ? tok * a.ldxs : 0) + kc0 * 4;
        const bool words = ((reinterpret_cast<uintptr_t>(a.xs) | (uintptr_t)a.ldxs) & 3) == 0;
        const int ngroups = a.K / kMxGroup - kc0 * 4;  // scale bytes from here on
        auto load = [&](int kx, int h) -> uint32_t {
          const int g0 = (kx * kPair + h) * 4;
          uint32_t v = 0x7F7F7F7Fu;
          if (tok >= a.M || kx >= nx || g0 >= ngroups) return v;
          if (words && g0 + 4 <= ngroups) return *reinterpret_cast<const uint32_t*>(sp + g0);
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (g0 + g < ngroups) v = (v & ~(0xFFu << (8 * g))) | (uint32_t)sp[g0 + g] << (8 * g);
          return v;
        };
        uint32_t ahead[DEPTH][kPair];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
          for (int h = 0; h < kPair; ++h) ahead[d][h] = load(d, h);
        for (int k0 = 0; k0 < nx && ok; k0 += DEPTH) {
#pragma unroll
          for (int d = 0; d < DEPTH; ++d) {
            const int kx = k0 + d;
            if (kx >= nx || !ok) break;
            ok = __all_sync(0xffffffffu, mbar_wait(&xempty[xs], xp, a.timeout_ns, a.status));
            if (!ok) break;
            if (tok < MT) {
#pragma unroll
              for (int h = 0; h < kPair; ++h)
                *reinterpret_cast<uint32_t*>(xslot(xs) + kPair * Sh::kXChunk + h * kW4Scales + mx_scale_at(tok, 0)) =
                    ahead[d][h];
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&xfull[xs]);
#pragma unroll
            for (int h = 0; h < kPair; ++h) ahead[d][h] = load(kx + DEPTH, h);
            if (++xs == XS) {
              xs = 0;
              xp ^= 1;
            }
          }
        }
      }
    } else {
      // A warp converts a slot's 256 k of a token at a time, a chain of some 450
      // clocks; two at once (two tokens, or with up to 8 tokens two slots) hide each
      // other's latencies. The warps of a group take the tokens in turn, and with few
      // tokens groups of warps the slots. Rows past M stay as they are: what a token's
      // row holds reaches no other token's sums.
      constexpr int VEC = Sh::kVec, SLOTS = Sh::kSlots;
      constexpr int DEPTH = 2;  // turns whose tokens are in registers ahead
      const int w = warp - 2;
      const int groups = VEC == 1 ? a.groups : 1, per = VEC == 1 ? CW / groups : CW;
      const int group = w / per, tok0 = w - group * per;
      const int kend = min(a.K, (kc0 + nk) * kW4Tile);
      const int kbase = kc0 * kW4Tile + lane * 8;
      const int step = groups * SLOTS;  // slots of a turn of all groups
      // slot i of the group's turn that begins with slot kx
      auto load = [&](int kx, int i, int j) -> uint4 {
        const int tok = tok0 + j * per, k = kbase + (kx + i * groups) * (kPair * kW4Tile);
        if (tok < a.M && k < kend)
          return *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + tok * a.ldx + k);
        return make_uint4(0u, 0u, 0u, 0u);
      };
      uint4 ahead[DEPTH][SLOTS][VEC];
#pragma unroll
      for (int d = 0; d < DEPTH; ++d)
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) ahead[d][i][j] = load(group + d * step, i, j);
      const int last = tok0 < a.M ? nx : 0;  // a warp without a token has nothing to do
      for (int k0 = group; k0 < last && ok; k0 += DEPTH * step) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          const int kx = k0 + d * step;
          if (kx >= last || !ok) break;
          uint8_t* slot[SLOTS];
          int ring[SLOTS];
#pragma unroll
          for (int i = 0; i < SLOTS; ++i) {
            const int n = kx + i * groups, q = n / XS;
            ring[i] = n - q * XS;
            slot[i] = xslot(ring[i]);
            if (n < last && ok)
              ok = __all_sync(0xffffffffu, mbar_wait(&xempty[ring[i]], (q & 1) ^ 1, a.timeout_ns, a.status));
          }
          if (!ok) break;
          uint2 hi[SLOTS][VEC], lo[SLOTS][VEC];
          int b[SLOTS][VEC];
#pragma unroll
          for (int i = 0; i < SLOTS; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) b[i][j] = split_e4m3(ahead[d][i][j], hi[i][j], lo[i][j]);
#pragma unroll
          for (int i = 0; i < SLOTS; ++i) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              const int tok = tok0 + j * per;
              if (tok < a.M && kx + i * groups < last) put_token<MT>(slot[i], tok, lane, hi[i][j], lo[i][j], b[i][j]);
              ahead[d][i][j] = load(kx + DEPTH * step, i, j);
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0 && kx + i * groups < last) mbar_arrive(&xfull[ring[i]]);
          }
        }
      }
    }
    if (!ok) s_flags[0] = 1;
    next.find(a, threadIdx.x - 64);  // the first outputs' places, and their residual, meanwhile
    if (!s_flags[0]) {
      if (!mbar_wait(tfull, 0, a.timeout_ns, a.status)) s_flags[0] = 1;
    }
    __syncwarp();
    tc_fence_after();
  }

  // Each thread's row of sums goes to the rank that owns it, which adds up what it
  // got in rank order.
  __syncwarp();
  if (cs > 1) {
    if (!Sh::kRecvApart) cluster_arrive_all();
    cluster_wait_all();  // every rank can be sent to
  }
  if (warp >= 2 && !s_flags[0]) {
    constexpr int PARTS = CW / 4;  // warps that share a quarter of the lanes
    const uint32_t lanes = taddr + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int rt = 0; rt < nrt; ++rt) {
      const int r = rt * kW4Tile + (warp & 3) * 32 + lane, q = r / R4;
      float* dst = recv + (size_t)cr * a.M * R4 + (r - q * R4);
#pragma unroll 1
      for (int c = 16 * ((warp - 2) >> 2); c < a.M; c += 16 * PARTS) {
        uint32_t v[16], w[16];
        tmem_ld16(lanes + rt * Sh::kRows + c, v);
        if constexpr (MODE != W4_MX) tmem_ld16(lanes + rt * Sh::kRows + MT + c, w);
        tmem_ld_wait();
        tmem_settle<16>(v);
        if constexpr (MODE != W4_MX) tmem_settle<16>(w);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float f = __uint_as_float(v[j]);
          if constexpr (MODE != W4_MX) f += __uint_as_float(w[j]);
          if (c + j < a.M) st_dsmem_f32(dst + (c + j) * R4, (uint32_t)q, f);
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync_all();
  if (warp >= 2 && !s_flags[0]) {
    while (next.any()) {
      W4Outputs<CONV> now = next;
      next.find(a, now.e);
      float4 sum[now.U];
#pragma unroll
      for (int u = 0; u < now.U; ++u) sum[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int src = 0; src < cs; ++src) {
        const float* p = recv + (size_t)src * a.M * R4;
#pragma unroll
        for (int u = 0; u < now.U; ++u)
          if (now.tok[u] >= 0) {
            const float4 v = *reinterpret_cast<const float4*>(p + now.tok[u] * R4 + 4 * now.quad[u]);
            sum[u].x += v.x;
            sum[u].y += v.y;
            sum[u].z += v.z;
            sum[u].w += v.w;
          }
      }
#pragma unroll
      for (int u = 0; u < now.U; ++u) {
        const int n = now.n0 + 4 * now.quad[u];
        if (now.tok[u] < 0 || n >= a.N) continue;
        const long long o = (long long)now.tok[u] * a.N + n;
        const float4 v = sum[u];
        if ((a.N & 3) == 0) {  // four outputs lie in 8 aligned bytes
          const uint2 r = now.res[u];
          *reinterpret_cast<uint2*>(DG_AT(a.status, a.y, o, (long long)a.M * a.N - 3)) =
              a.res ? make_uint2(pack_bf16(bf16lo(r.x) + v.x, bf16hi(r.x) + v.y),
                                 pack_bf16(bf16lo(r.y) + v.z, bf16hi(r.y) + v.w))
                    : make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        } else {
#pragma unroll 1
          for (int j = 0; j < 4; ++j)
            if (n + j < a.N) {
              const float f = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
              const float r = a.res ? bf_bits2f(*DG_AT(a.status, a.res, o + j, (long long)a.M * a.N)) + f : f;
              *DG_AT(a.status, a.y, o + j, (long long)a.M * a.N) = f2bf_bits(r);
            }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, Sh::kTmem);
  }
}

#ifdef DEC_DEBUG
static std::atomic<int> g_w4_stall{0};  // arrivals that slots of tokens wait for in vain
int w4_stall(int on) { return g_w4_stall.exchange(on ? 1 : 0); }
#else
int w4_stall(int) { return -1; }
#endif

// CTAs that share a set of tiles: the most, up to 8 (the portable cluster size)
// and one per pair of units, for which every cluster runs at once. (A GPU's SMs come
// in groups that a cluster cannot cross: of 152 SMs, 15 clusters of 8 CTAs hold at
// most 120, 36 of 4 144.)
template <int MT, int RT, int MODE, int CW>
static cudaError_t w4_split(int sets, int pairs, int sms, int* split) {
  using Sh = W4Shape<MT, RT, MODE, CW>;
  auto kern = w4_linear_kernel<MT, RT, MODE, CW>;
  static DevOnce once;
  if (cudaError_t e = setup_smem(once, kern, Sh::kSmem, true); e != cudaSuccess) return e;
  static std::atomic<int> most[64][9];  // by device and cluster size; 0: not asked yet
  int d = 0;
  if (cudaError_t e = cudaGetDevice(&d); e != cudaSuccess) return e;
  *split = 1;
  for (int c = pairs < 8 ? pairs : 8; c > 1; --c) {
    if ((long long)sets * c > sms) continue;
    int n = d < 64 ? most[d][c].load(std::memory_order_relaxed) : 0;
    if (!n) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(c);
      cfg.blockDim = dim3(Sh::kThreads);
      cfg.dynamicSmemBytes = Sh::kSmem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)c;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg); e != cudaSuccess) return e;
      if (d < 64) most[d][c].store(n, std::memory_order_relaxed);
    }
    if (sets <= n - (n + 15) / 16) {
      *split = c;
      return cudaSuccess;
    }
  }
  return cudaSuccess;
}

template <int MT, int RT, int MODE, int CW>
static cudaError_t run_w4(const Ctx& cx, const W4Call& c) {
  using Sh = W4Shape<MT, RT, MODE, CW>;
  auto kern = w4_linear_kernel<MT, RT, MODE, CW>;
  const int tiles = (c.N + kW4Tile - 1) / kW4Tile, KC = (c.K + kW4Tile - 1) / kW4Tile;
  const int sets = (tiles + RT - 1) / RT, pairs = (KC + kPair - 1) / kPair;
  int split = 1;
  if (cudaError_t e = w4_split<MT, RT, MODE, CW>(sets, pairs, cx.sms, &split); e != cudaSuccess) return e;
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
  a.tiles = tiles;
  a.groups = 1;
  if (MODE == W4_CONVERT) {
    // (the groups' turns together take no slot of the ring twice)
    while (2 * a.groups * Sh::kSlots <= Sh::kXS && 2 * a.groups * c.M <= CW) a.groups *= 2;
    const int per = CW / a.groups;
    a.xarrivals = per < c.M ? per : c.M;  // the warps of a group that have a token
  } else {
    a.xarrivals = MODE == W4_MX ? 1 + (MT + 31) / 32 : 1;
  }
#ifdef DEC_DEBUG
  a.xarrivals += g_w4_stall.load(std::memory_order_relaxed);
#endif
  a.status = cx.status;
  a.timeout_ns = cx.timeout_ns;
  CUtensorMap wmap, wmap1, xmap;
  if (!make_tmap_w4(&wmap, c.wq, (uint64_t)tiles * KC * kW4Tile, kPair * kW4Tile) ||
      !make_tmap_w4(&wmap1, c.wq, (uint64_t)tiles * KC * kW4Tile, kW4Tile))
    return cudaErrorInvalidValue;
  xmap = wmap;
  if (MODE == W4_MX && !make_tmap_bytes(&xmap, c.x, (uint64_t)c.M, (uint64_t)c.K, (uint64_t)c.ldx, (uint32_t)MT))
    return cudaErrorInvalidValue;
  if constexpr (MODE == W4_READY) {
    const int items = pairs * c.M, per = kReadyThreads / 32;
    if (cudaError_t e = launch_k(w4_tokens_kernel<MT>, dim3((unsigned)((items + per - 1) / per)), dim3(kReadyThreads),
                                 0, cx.stream, cx.pdl, static_cast<const uint16_t*>(c.x), c.ldx,
                                 static_cast<uint8_t*>(c.work), c.M, c.K, pairs);
        e != cudaSuccess)
      return e;
    a.x = c.work;
  }
  return launch_kc(kern, dim3((unsigned)(sets * split)), dim3(Sh::kThreads), Sh::kSmem, cx.stream, cx.pdl, split,
                   wmap, wmap1, xmap, a);
}

// bf16 tokens are converted by each CTA up to 16 (one launch, no work space); beyond,
// by a kernel before (about 2 us): in each CTA 64 tokens of 16384 x 7168 took 27 us, so
// 19.5, 32 tokens 20.3 and 16.0.
constexpr int kW4Convert = 16;

size_t w4_work_bytes(int M, int K) {
  if (M <= kW4Convert || K > kW4MaxK) return 0;
  const int mt = M <= 32 ? 32 : 64, pairs = ((K + kW4Tile - 1) / kW4Tile + kPair - 1) / kPair;
  return (size_t)pairs * (kPair * 2 * mt * 128 + 1024);
}

// Ring slots of tokens that an SM goes through, with RT tiles a CTA.
template <int MT, int RT, int MODE, int CW>
static cudaError_t w4_slots(const Ctx& cx, const W4Call& c, long long* slots) {
  const int tiles = (c.N + kW4Tile - 1) / kW4Tile, pairs = ((c.K + kW4Tile - 1) / kW4Tile + kPair - 1) / kPair;
  const int sets = (tiles + RT - 1) / RT;
  int split = 1;
  const cudaError_t e = w4_split<MT, RT, MODE, CW>(sets, pairs, cx.sms, &split);
  *slots = (long long)((pairs + split - 1) / split) * ((sets * (long long)split + cx.sms - 1) / cx.sms);
  return e;
}

// One or two tiles a CTA: two where that leaves each SM at least `least` slots fewer, or
// any where there are more tiles than SMs (20000 x 4096, 157 tiles, 1 token: 15.4 us
// of one, 32 slots, 12.2 of two, 16; 64 in 8 bits 20.9 and 16.1).
// Two tiles share a slot's tokens, with twice the sums to exchange. Converting them
// takes 700 clocks a slot, longer than a pair of units; from 33 tokens on they are
// twice a pair's bytes, more than an SM takes in. us (GPU) of one / two tiles, slots
// in brackets:
//   16 tokens  16384 x 7168 20.0 (28) / 13.6 (14), 8192 x 7168 11.7 (14) / 8.7 (7),
//              2048 x 16384 9.8 (11) / 8.7 (8), 2048 x 7168 6.15 (5) / 6.07 (4), 4096 x
//              4096 5.72 (4) / 5.73 (3), 1001 x 1992 4.10 (1) / 4.35 (1)
//    8 tokens  16384 x 7168 14.4 / 13.2, 8192 x 7168 9.3 / 8.5, 2048 x 16384 8.2 / 8.2
//   64 tokens  16384 x 7168 20.1 / 19.3, 8192 x 7168 13.0 / 13.3, 2048 x 16384 11.7 / 13.1
template <int MT, int MODE, int CW>
static cudaError_t w4_tiles(const Ctx& cx, const W4Call& c, int least) {
  long long one = 0, two = 0;
  if (cudaError_t e = w4_slots<MT, 1, MODE, CW>(cx, c, &one); e != cudaSuccess) return e;
  if (cudaError_t e = w4_slots<MT, 2, MODE, CW>(cx, c, &two); e != cudaSuccess) return e;
  if ((c.N + kW4Tile - 1) / kW4Tile > cx.sms) least = 1;
  return one - two >= least ? run_w4<MT, 2, MODE, CW>(cx, c) : run_w4<MT, 1, MODE, CW>(cx, c);
}

cudaError_t launch_w4_linear(const Ctx& cx, const W4Call& c) {
  constexpr int kNever = INT32_MAX;
  if (c.xs) {
    if (c.M <= 16) return w4_tiles<16, W4_MX, 4>(cx, c, kNever);
    if (c.M <= 32) return w4_tiles<32, W4_MX, 4>(cx, c, kNever);
    return w4_tiles<64, W4_MX, 8>(cx, c, kNever);
  }
  if (c.M <= 4) return w4_tiles<8, W4_CONVERT, 8>(cx, c, kNever);  // groups of warps hide the conversion
  if (c.M <= 8) return w4_tiles<8, W4_CONVERT, 8>(cx, c, 2);
  if (c.M <= kW4Convert) return w4_tiles<16, W4_CONVERT, 8>(cx, c, 2);
  if (c.M <= 32) return w4_tiles<32, W4_READY, 4>(cx, c, kNever);
  return w4_tiles<64, W4_READY, 8>(cx, c, 12);
}

// ------------------------------------------------------------------ quantisation
// A CTA per unit: 16 lanes take the 128 k of a row, 8 each; the four lanes of a
// group share its largest magnitude. Reads 2 bytes a weight, writes 0.53: memory.
// A thread loads its eight rows' vectors at once; registers for five CTAs an SM let
// it (16384 x 7168, 43.9 us at the copy rate: 46.4; held to six CTAs 53.1, four
// vectors at once and eight CTAs 48.8).
constexpr int kQuantThreads = 256;

__global__ void __launch_bounds__(kQuantThreads, 5)
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
    const uint32_t m = group_most(w);
    uint32_t codes = 0;
    int b = 255;  // a group with a value that is not finite: the scale NaN, codes 0
    if (m < 0x7F80u) {
      int e = mx_exponent_e2m1(__uint_as_float(m << 16));
      e = e < -127 ? -127 : e;
      b = e + 127;
      const float s = pow2_f(-e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t two;  // f[2j] -> low half, f[2j+1] -> high half of a byte
        asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
            : "=r"(two)
            : "f"(bf16hi(w[j]) * s), "f"(bf16lo(w[j]) * s));
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
  return launch_k(w4_quant_kernel, dim3((unsigned)((long long)tiles * KC)), dim3(kQuantThreads), 0, cx.stream, false,
                  static_cast<const uint16_t*>(W), ldw, static_cast<uint8_t*>(q), static_cast<uint8_t*>(s), N, K, KC);
}

}  // namespace dg
