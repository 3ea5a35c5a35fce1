// k_attn_tc.cu -- attention of chunks of new tokens over a paged cache on the
// tcgen05 tensor cores (the mathematics: see k_attn.cu).
//
// A chunk of n tokens reads each key once for up to 256 rows (token, query
// head): 4 * 256 flops a byte of cache at 128 elements a head, so that the
// tensor cores bound it, not memory. A CTA works on a pair of row tiles, A and
// B, of up to 128 rows each (TMEM lanes) and a key tile of 128 positions:
//
//   S = Q·Kᵀ      128 x 128 fp32 in TMEM; Q and K from shared memory
//   P = 2^(c S - m)   by 128 threads, a row each: no shuffles; bf16 P goes
//                 back to TMEM over S
//   O += P·V      P from TMEM, V from shared memory, fp32 O in TMEM
//
// While the tensor cores do P·V and the next Q·Kᵀ of one row tile, the threads
// of the other do its softmax. TMEM: S of A and B (128 columns each), O of A
// and B: all 512 columns at 128 elements a head.
//
// m is the running maximum, but O and the sum are only rescaled when it has
// grown by more than 2^8 since: P then stays below 2^8, which bf16 and the
// fp32 sum hold as well as 1, and rescaling (a pass over O in TMEM) is rare.
//
// Warps 0-3 and 4-7: softmax and output of A and B. Warp 8 issues the MMAs,
// warp 9 the TMA loads (page by page). Warp 10 cleans value tiles at the edge
// of what the rows see: a place that no row sees may hold anything (the unused
// end of a page), and one that only some rows see may hold a NaN or infinity
// that the others' weight 0 would turn into NaN: both become 0 in shared
// memory, and the rows that do see a non-finite value get it added at the end.
//
// Every ring has a way back: a slot is filled again when the MMAs that read it
// are done and warp 10 is past it, a segment begins when all warps have left the
// one four before, and all follow the TMA warp into it. So no role, however
// late, can take a barrier's phase for the one two before.
//
// The work is split into equal ranges of (row tile pair, key tile) units, or
// drawn pair by pair where there are many, see paged.cuh.
//
// Measured (56 query and 4 key heads of 128): a chunk of 512 tokens over 32k
// positions 291 us, 1.64 PFLOP/s or 87% of what a large matrix product reaches
// (in a graph, at the highest clock; called in a row for long, under the power
// cap, 313 to 318 us, 1.5 PFLOP/s or 80%); a key tile of a pair takes 1.4 us,
// the two halves' softmax (1.1 us each) and products (0.6 us each) in turn.
// Four ragged prompts of up to 2047 tokens 148 us,
// 1.13 PFLOP/s: pairs of 1 to 16 key tiles, each with 2.5 us for its edge, its
// output and the first scores of the next. Calls of a few pairs 15 to 18 us,
// latency: 3 us until the work is split, 2.5 until the first scores, then the
// key tiles, and 3 to 5 for joining.
#include <type_traits>

#include "launch.h"
#include "launch_util.cuh"
#include "paged.cuh"
#include "tc_common.cuh"

namespace dg {

constexpr int kTcKeys = 128;         // positions of a key tile
constexpr int kTcKeysShift = 7;
constexpr int kTcRowsA = 128;        // rows of a row tile
constexpr int kTcAttnThreads = 384;
constexpr int kTcFew = 4;             // CTAs that may share a pair which one of them joins
constexpr float kTcLazy = 8.f;       // growth of the maximum (log2) that is left in P

struct TcAttnArgs {
  PagedArgs p;
  SplitShape s;
  uint16_t* out;
  float* lse;
  long long ldo;
  int group, hq, tq;   // tq: tokens of one row tile (s.tq: of the pair)
  float c;
  float* ws;
  int* ctr;            // [grid * 32 + 1] arrivals, row tile pairs drawn; zero at rest
  int4* deep;          // [grid] pairs that many CTAs share, by their first CTA; null: none is left
  long long ws_len;
  int min_units;
  long long timeout_ns;
};

// Shared memory: Q of A and B, and a ring of pairs: slot i holds the values of
// the CTA's key tile i - 1 and the keys of its tile i, which are needed and
// given back together.
template <int D>
struct TcAttnShape {
  static constexpr int kHalf = kTcKeys * 128;            // 64 columns of a 128-row tile
  static constexpr int kTile = kTcKeys * D * 2;          // a tile of Q, K or V
  static constexpr int kSlots = 64 * 1024 / kTile;       // of 2 tiles
  static constexpr int kStage = 16 * 1024;               // output rows on their way: 2 KB a warp
  // floats of a split pair's partial: for A and B o [D / 4][row][4], m and l [row]
  static constexpr int kPart = 2 * kTcRowsA * (D + 2);
  static int smem(int batch) {
    return 1024 + 2 * kTile + kSlots * 2 * kTile + kStage + 8 * (3 * kSlots + 24) + 64 + 64 +
           SplitTables::bytes(batch) + 16;
  }
};

// The 16-position steps [k0, k1) of an edge tile that some row sees (at least
// one, so that O is written).
__device__ __forceinline__ void edge_steps(const EdgeRange& er, int key0, int& k0, int& k1) {
  k0 = er.klo > key0 ? (er.klo - key0) >> 4 : 0;
  k1 = er.khi - key0 < kTcKeys ? (er.khi - key0 + 15) >> 4 : kTcKeys / 16;
  if (k0 > kTcKeys / 16 - 1) k0 = kTcKeys / 16 - 1;
  if (k1 <= k0) k1 = k0 + 1;
}

// Puts `none` (which c makes -inf) in the columns of a row of S (128 fp32 in
// TMEM, this thread's lane) outside [l0, h0]. A pass of its own over the few tiles at the edge of what
// the rows see, in few instructions: code that runs once in a while costs its
// instruction fetches.
__device__ __forceinline__ void row_mask(uint32_t ts, int l0, int h0, uint32_t none) {
#pragma unroll 1
  for (int q = 0; q < 4; ++q, ts += 32, l0 -= 32, h0 -= 32) {
    const uint32_t above = l0 <= 0 ? ~0u : (l0 > 31 ? 0u : ~0u << l0);
    const uint32_t below = h0 < 0 ? 0u : (h0 >= 31 ? ~0u : ~(~0u << (h0 + 1)));
    const uint32_t seen = above & below;
    if (__all_sync(~0u, seen == ~0u)) continue;
    uint32_t v[32];
    tmem_ld32(ts, v);
    tmem_ld_wait();
    tmem_settle<32>(v);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(seen & (1u << e))) v[e] = none;
    tmem_st32(ts, v);
  }
  tmem_st_wait();
}

// The maximum of c s over the first 32 columns of a row of S.
__device__ __forceinline__ float row_start(uint32_t ts, float c) {
  uint32_t v[32];
  tmem_ld32(ts, v);
  tmem_ld_wait();
  tmem_settle<32>(v);
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    mx0 = max3(mx0, __uint_as_float(v[e]) * c, __uint_as_float(v[e + 1]) * c);
    mx1 = max3(mx1, __uint_as_float(v[e + 2]) * c, __uint_as_float(v[e + 3]) * c);
  }
  return fmaxf(mx0, mx1);
}

// One row of S: top = max c s, the weights 2^(c s - m) as bf16 pairs in pk, and
// their fp32 sum. The next 32 columns load while the current ones are worked
// on.
__device__ __forceinline__ void row_pass(uint32_t ts, float c, float m, uint32_t* pk, float& top,
                                         float& sum) {
  alignas(8) uint32_t s[2][32];
  float mx0 = -INFINITY, mx1 = -INFINITY;
  float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
  tmem_ld32(ts, s[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t* v = s[q & 1];
    tmem_ld_wait();
    tmem_settle<32>(v);
    if (q < 3) tmem_ld32(ts + (q + 1) * 32, s[(q + 1) & 1]);
    float2* f = reinterpret_cast<float2*>(v);
    // in the order of a pipeline four pairs deep: a pair's scaling ahead of its
    // exponentials, its sum and packing behind them
#pragma unroll
    for (int e = 0; e < 16 + 8; ++e) {
      if (e < 16) f[e] = fma2(f[e], c, -m);
      if (e >= 4 && e < 20) {
        if (e & 1) mx1 = max3(mx1, f[e - 4].x, f[e - 4].y);
        else mx0 = max3(mx0, f[e - 4].x, f[e - 4].y);
        f[e - 4].x = exp2_approx(f[e - 4].x);
        f[e - 4].y = exp2_approx(f[e - 4].y);
      }
      if (e >= 8) {
        const float2 p = f[e - 8];
        if (e & 1) acc1 = add2(acc1, p);
        else acc0 = add2(acc0, p);
        pk[q * 16 + e - 8] = pack_bf16(p.x, p.y);  // weights as bf16: see k_attn.cu
      }
    }
  }
  top = fmaxf(mx0, mx1) + m;
  sum = (acc0.x + acc0.y) + (acc1.x + acc1.y);
}

template <int D>
__global__ void __launch_bounds__(kTcAttnThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
                   const TcAttnArgs a) {
  using Sh = TcAttnShape<D>;
  constexpr int kSlots = Sh::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sq = smem;                       // Q of A and B
  uint8_t* ring = smem + 2 * Sh::kTile;     // [slot] V, K
  uint8_t* stage = ring + kSlots * 2 * Sh::kTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(stage + Sh::kStage);
  uint64_t* empty = full + kSlots;
  uint64_t* v_clean = empty + kSlots;   // [slot] edge values looked over (edge tiles only)
  uint64_t* s_full = v_clean + kSlots;  // [2] S ready, and the P·V before it done
  uint64_t* p_full = s_full + 2;        // [2] P written
  uint64_t* o_full = p_full + 2;        // [2] a segment's last P·V done
  uint64_t* q_full = o_full + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* mma_done = q_empty + 1;
  uint64_t* seg_full = mma_done + 1;    // [4] a segment begun; a drawn pair is in s_seg
  uint64_t* seg_empty = seg_full + 4;   // [4] a segment left by all warps but the TMA warp
  volatile int* s_flag = reinterpret_cast<volatile int*>(full + 3 * kSlots + 24);  // [0] abort
  volatile int* s_poison = s_flag + 4;  // [4] segment number + 1 with a non-finite edge value
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(const_cast<int*>(s_flag) + 8);
  int4* s_seg = reinterpret_cast<int4*>(const_cast<int*>(s_flag) + 16);  // [4] drawn pairs
  // (four segments' worth of both: the TMA warp begins a segment when all others
  // have left the one four before, and they follow it into it)
  const SplitTables tab(s_seg + 4, a.p.batch);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);  // the MMAs done, and warp 10 past the slot
      mbar_init(&v_clean[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(mma_done, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 10);  // warps 0-7, 8 and 10
    }
    s_flag[0] = 0;
    for (int i = 0; i < 4; ++i) s_poison[i] = 0;
    fence_mbar_init();
    prefetch_tmap(&kvmap);
    prefetch_tmap(&qmap);
  }
  if (warp == 8) {
    tmem_alloc(s_taddr, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = *s_taddr;
  griddep_launch_dependents();
  griddep_wait();
  long long W, G, u0, u1;
  split_setup<true>(a.p, a.s, tab, a.min_units, blockIdx.x, gridDim.x, W, G, u0, u1);
  SplitWalk w(a.s, tab, u0, u1);
  const bool draws = tab.head[4] != 0;

  auto edges = [&]() -> EdgeRange {
    const int qn = tab.qn[w.b], t0 = w.i * a.s.tq;
    const int nt = qn - t0 < a.s.tq ? qn - t0 : a.s.tq;
    return edge_range(a.s, w.tr, tab.kv[w.b] - qn + t0, nt);
  };
  // B has rows
  auto has_b = [&] { return tab.qn[w.b] - w.i * a.s.tq > a.tq; };
  // The same result in all lanes: false once any wait of the CTA has run out.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    bool ok = true;
    if (!mbar_try_wait(bar, parity & 1)) {
      ok = !s_flag[0] && mbar_wait(bar, parity & 1, a.timeout_ns, a.p.status);
      if (!ok) s_flag[0] = 1;
    }
    return __all_sync(~0u, ok);
  };

  int drawn = 0;  // segments so far
  // To the next segment, once the TMA warp has begun it; false if a wait has run out.
  auto next = [&]() -> bool {
    const int k = drawn++;
    if (!wait(&seg_full[k & 3], k >> 2)) return false;
    if (draws) {
      const int4 e = s_seg[k & 3];
      w.jump(e.x, e.y, e.z);
    } else if (k) {
      w.next();
    }
    return true;
  };
  // This warp is done with segment k: its entries of s_seg and s_poison are free.
  auto leave = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[k & 3]);
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int x = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = taddr + lanes + x * 128, to = taddr + lanes + 256 + x * D;
    const int t = r / a.group, g = r - t * a.group;
    uint8_t* mine = stage + warp * 2048;
    const uint32_t none = a.c < 0.f ? 0x7F800000u : 0xFF800000u;
    uint32_t sn = 0, on = 0;
    int seg = 0;
    bool ok = next();
    for (; ok && w.more(); leave(seg++), ok = ok && next()) {
      if (x == 1 && !has_b()) continue;
      const EdgeRange er = edges();
      const int qn = tab.qn[w.b];
      const int t0 = w.i * a.s.tq + x * a.tq;
      const int nt = qn - t0 < a.tq ? qn - t0 : a.tq;
      const bool live = t < nt;
      const int pos = tab.kv[w.b] - qn + t0 + t;
      const int hi = live ? pos : -1;
      const int lo = live ? first_seen(a.s.window, pos) : 0;
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < w.n; ++k) {
        const int key0 = (w.j + k) * kTcKeys;
        ok = wait(&s_full[x], sn++);
        if (!ok) break;
        tc_fence_after();
        // One pass over the row with the maximum of the tiles before: weights,
        // their sum and the row's own maximum. If that has outgrown m the pass
        // is made again with the new one: S stays in TMEM until the weights
        // replace it. A segment's first tile starts from the maximum of its
        // first 32 columns.
        if (er.in(key0, kTcKeys)) row_mask(ts, lo - key0, hi - key0, none);
        uint32_t pk[64];
        float top, sum;
        if (k == 0) m = row_start(ts, a.c);
#pragma unroll 1
        for (;;) {
          row_pass(ts, a.c, m == -INFINITY ? 0.f : m, pk, top, sum);
          // (the first positions that a row sees need no other m than 0 if that is near)
          if (m == -INFINITY && fabsf(top) <= kTcLazy) m = 0.f;
          // (rows of the tile that hold no token hold whatever was there: they have
          // no say, so that results do not depend on it)
          if (!__any_sync(~0u, live && top > m + kTcLazy)) break;
          // m was -inf before the first visible position: O and l are 0 then
          const float mn = fmaxf(m, top);
          const float f = m == -INFINITY ? 0.f : exp2_approx(m - mn);
          m = mn;
          l *= f;
          if (k == 0) continue;
#pragma unroll 1
          for (int q = 0; q < D; q += 32) {
            uint32_t o[32];
            tmem_ld32(to + q, o);
            tmem_ld_wait();
            tmem_settle<32>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(to + q, o);
          }
        }
        l += sum;
        tmem_st32(ts, pk);
        tmem_st32(ts + 32, pk + 32);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      // while the last P·V runs: where the rows go and their sums. Four lanes
      // write a row, 64 bytes of it at a time.
      const long long tok0 = paged_first(a.p, w.b) + t0;
      auto inverse = [](float sum) { return sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum); };  // NaN stays NaN
      uint16_t* dst[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = (warp & 3) * 32 + e * 8 + (lane >> 2), tt = row / a.group;
        dst[e] = tt >= nt ? nullptr
                          : a.out + (tok0 + tt) * a.ldo +
                                (long long)(w.h * a.group + row - tt * a.group) * D + (lane & 3) * 8;
      }
      auto put_lse = [&](float top, float sum) {
        if (live && a.lse)
          a.lse[(tok0 + t) * a.hq + w.h * a.group + g] =
              sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      };
      // 32 columns of this warp's rows, through shared memory so that four lanes
      // write 64 bytes of a row
      auto put_rows = [&](const uint32_t* o, int q, float scale) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t* v = o + e * 8;
          auto at = [&](int n) { return __uint_as_float(v[n]) * scale; };
          *reinterpret_cast<uint4*>(mine + lane * 64 + ((e ^ (lane >> 1)) & 3) * 16) =
              make_uint4(pack_bf16(at(0), at(1)), pack_bf16(at(2), at(3)),
                         pack_bf16(at(4), at(5)), pack_bf16(at(6), at(7)));
        }
        __syncwarp();
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = e * 8 + (lane >> 2);
          v[e] = *reinterpret_cast<const uint4*>(mine + rr * 64 + (((lane & 3) ^ (rr >> 1)) & 3) * 16);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (dst[e]) *reinterpret_cast<uint4*>(dst[e] + q) = v[e];
      };
      const float inv = inverse(l);
      if (w.whole) put_lse(m, l);
      ok = wait(&o_full[x], on++);
      if (!ok) break;
      tc_fence_after();
      if (s_poison[seg & 3] == seg + 1) {
        // rows that see a non-finite edge value get it here
#pragma unroll 1
        for (int q = 0; q < D; q += 16) {
          uint32_t o[16];
          tmem_ld16(to + q, o);
          tmem_ld_wait();
          tmem_settle<16>(o);
          if (live)
            edge_values<D>(a.p, paged_row(a.p, w.b), w.h, er, lo, hi, w.j * kTcKeys,
                           (w.j + w.n) * kTcKeys, q, [&](const uint16_t* v, int) {
#pragma unroll
                             for (int e = 0; e < 16; ++e) {
                               const float f = bf_bits2f(__ldg(v + e));
                               if (!isfinite(f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
                             }
                           });
          __syncwarp();
          tmem_st16(to + q, o);
        }
        tmem_st_wait();
      }
      if (w.whole) {
#pragma unroll 1
        for (int q = 0; q < D; q += 32) {
          uint32_t o[32];
          tmem_ld32(to + q, o);
          tmem_ld_wait();
          tmem_settle<32>(o);
          put_rows(o, q, inv);
        }
        // O is read: P of the next segment may be followed by its first P·V
        tc_fence_before();
        continue;
      }
      // The pair is shared with other CTAs: the first of them ends its range with
      // it (slot 1), the others begin with it (slot 0). This warp leaves its rows'
      // O, m and sum; the last of the CTAs' warps with these rows joins them, in
      // CTA order. Above 8 CTAs in two steps, first within groups of about the
      // square root of their number, as the join of each reads 64 KB a row tile;
      // calls of few pairs leave those that more than 4 CTAs share to a second
      // kernel that spreads them over the SMs (60 tokens over 9000 positions 39
      // -> 33 us; for calls of many pairs that kernel costs more than it saves).
      const long long cf = worker_of(w.tile_unit(), W, G);
      const int nc = (int)(worker_of(w.tile_unit() + w.tr.n - 1, W, G) - cf + 1);
      auto part_of = [&](int k) -> float* {
        return a.ws + ((cf + k) * 2 + (k == 0 ? 1 : 0)) * Sh::kPart + x * (Sh::kPart / 2);
      };
      const int self = (int)(blockIdx.x - cf);
      {
        float* part = part_of(self);
#pragma unroll 1
        for (int q = 0; q < D; q += 32) {
          uint32_t o[32];
          tmem_ld32(to + q, o);
          tmem_ld_wait();
          tmem_settle<32>(o);
          float4* col = reinterpret_cast<float4*>(
              DG_AT(a.p.status, part, q * kTcRowsA + r * 4, Sh::kPart / 2 - 28 * kTcRowsA));
#pragma unroll
          for (int e = 0; e < 8; ++e)
            __stcg(col + e * kTcRowsA,
                   make_float4(__uint_as_float(o[e * 4]), __uint_as_float(o[e * 4 + 1]),
                               __uint_as_float(o[e * 4 + 2]), __uint_as_float(o[e * 4 + 3])));
        }
        __stcg(reinterpret_cast<float2*>(part + D * kTcRowsA) + r, make_float2(m, l));
      }
      tc_fence_before();
      if (a.deep && nc > kTcFew) continue;
      // the counter of a group is its first CTA's, by slot, warp and step
      auto last_of = [&](int first, int step, int count) -> bool {
        __syncwarp();
        int old = 0;
        if (lane == 0) {
          int* ctr = a.ctr + (((cf + first) * 2 + (first == 0 ? 1 : 0)) * 8 + warp) * 2 + step;
          old = atomic_add_acq_rel_gpu(ctr, 1);
          if (old == count - 1) *ctr = 0;
        }
        __syncwarp();
        return __shfl_sync(~0u, old, 0) == count - 1;
      };
      int size = nc;
      if (nc > 8)
        for (size = 3; size * size < nc;) ++size;
      const int groups = (nc + size - 1) / size;
      int first = self / size * size, stride = 1;
      int count = nc - first < size ? nc - first : size;
      bool joined = groups == 1;
#pragma unroll 1
      for (int step = 0; last_of(joined && step ? 0 : first, step, count); ++step) {
        float M = -INFINITY, L = 0.f;
        auto ml = [&](int k) {
          return __ldcg(reinterpret_cast<const float2*>(part_of(first + k * stride) + D * kTcRowsA) + r);
        };
#pragma unroll 4
        for (int k = 0; k < count; ++k) M = fmaxf(M, ml(k).x);
        // a state that has seen nothing (m = -inf) counts for nothing
        auto factor = [&](float mk) { return M == -INFINITY ? 1.f : exp2_approx(mk - M); };
#pragma unroll 4
        for (int k = 0; k < count; ++k) {
          const float2 s = ml(k);
          L += factor(s.x) * s.y;
        }
        const float inv = inverse(L);
#pragma unroll 1
        for (int q = 0; q < D; q += 32) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll 2
          for (int k = 0; k < count; ++k) {
            const float4* col =
                reinterpret_cast<const float4*>(part_of(first + k * stride) + q * kTcRowsA + r * 4);
            const float f = factor(ml(k).x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v = __ldcg(col + e * kTcRowsA);
              o[e * 4] += f * v.x;
              o[e * 4 + 1] += f * v.y;
              o[e * 4 + 2] += f * v.z;
              o[e * 4 + 3] += f * v.w;
            }
          }
          if (joined) {
            put_rows(reinterpret_cast<const uint32_t*>(o), q, inv);
          } else {
            float4* col = reinterpret_cast<float4*>(part_of(first) + q * kTcRowsA + r * 4);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              __stcg(col + e * kTcRowsA, make_float4(o[e * 4], o[e * 4 + 1], o[e * 4 + 2], o[e * 4 + 3]));
          }
        }
        if (joined) {
          put_lse(M, L);
          break;
        }
        __stcg(reinterpret_cast<float2*>(part_of(first) + D * kTcRowsA) + r, make_float2(M, L));
        // the groups' states, which the last group joins
        joined = true;
        first = 0;
        stride = size;
        count = groups;
      }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- TMA
    const uint64_t pol = policy_evict_last();
    const int rows = a.p.page < kTcKeys ? a.p.page : kTcKeys;
    const int pieces = kTcKeys / rows, page_mask = a.p.page - 1;
    const int half = lane % (D / 64), piece = (lane & 15) / (D / 64);
    const bool vlane = lane >= 16;  // lanes 0-15 load keys, 16-31 the values of the tile before
    int i = 0, seg = 0;
    int pg_prev = -1, c1_prev = 0, h_prev = 0;   // the tile before: page, place in it, head
    bool ok = true;
    // slot i: values of the tile before, keys of this one (pg < 0: none)
    auto put = [&](int pg, int c1, int h) {
      const int st = i % kSlots;
      if (i >= kSlots && !wait(&empty[st], i / kSlots + 1)) return false;
      const int vpg = __shfl_sync(~0u, pg_prev, lane & 15);
      const int my = vlane ? vpg : pg;
      const int n = __popc(__ballot_sync(~0u, my >= 0));
      if (lane == 0) mbar_arrive_expect_tx(&full[st], n * rows * 128);
      __syncwarp();
      if (my >= 0)
        tma_load_4d(ring + (st * 2 + (vlane ? 0 : 1)) * Sh::kTile + half * Sh::kHalf +
                        piece * rows * 128,
                    &kvmap, half * 64, vlane ? c1_prev : c1, vlane ? a.p.hkv + h_prev : h, my,
                    &full[st], pol);
      ++i;
      pg_prev = pg;
      c1_prev = c1;
      h_prev = h;
      return true;
    };
    // Draws the CTA's next pair for all its warps: number k of the pairs in the
    // order sequence, row tile pair (last first, as it sees most), key head; the
    // sequences whose last pair is longest first, by powers of two.
    int level = 31 - __clz((int)tab.head[5] - a.s.start), from = 0, seq = 0, base = 0, count = 0, last = 0;
    auto draw = [&] {
      const int jobs = (int)tab.head[4];
      int k = blockIdx.x;  // the first is the CTA's own
      if (drawn > 0) {
        if (lane == 0) k = gridDim.x + atomicAdd(a.ctr + 32 * gridDim.x, 1);
        k = __shfl_sync(~0u, k, 0);
        // every CTA draws until it gets none: after the last of them the counter rests
        if (lane == 0 && k == jobs + (int)gridDim.x - 1) a.ctr[32 * gridDim.x] = 0;
      }
      if (k >= jobs) {
        seq = -1;
      } else {
        while (k >= base + count) {
          base += count;
          int n = 0;
          unsigned found;
          for (;;) {
            const int b = (from & ~31) + lane;
            n = b >= from && b < a.p.batch ? (tab.qn[b] + a.s.tq - 1) / a.s.tq : 0;
            found = __ballot_sync(
                ~0u, n > 0 && 31 - __clz(tile_range(a.s, tab.qn[b], tab.kv[b], n - 1).n) == level);
            if (found || level < 0) break;
            from = (from & ~31) + 32;
            if (from >= a.p.batch) from = 0, --level;
          }
          if (level < 0) {
            seq = -1;
            break;
          }
          const int l = __ffs(found) - 1;
          seq = (from & ~31) + l;
          from = seq + 1;
          if (from >= a.p.batch) from = 0, --level;
          last = __shfl_sync(~0u, n, l) - 1;
          count = (last + 1) * a.s.hkv;
        }
      }
      const int r = k - base, up = r / a.s.hkv;
      w.jump(seq, r - up * a.s.hkv, last - up);
      if (lane == 0) s_seg[drawn & 3] = make_int4(seq, r - up * a.s.hkv, last - up, 0);
    };
    auto advance = [&] {
      if (drawn >= 4 && !wait(&seg_empty[drawn & 3], (drawn >> 2) + 1)) {
        ok = false;
        return;
      }
      if (draws) draw();
      else if (drawn) w.next();
      if (lane == 0) mbar_arrive(&seg_full[drawn & 3]);
      ++drawn;
      __syncwarp();
    };
    for (advance(); w.more() && ok; advance()) {
      const bool two = has_b();
      const int row = paged_row(a.p, w.b);
      const int32_t* trow = a.p.table + (long long)(row < 0 ? 0 : row) * a.p.table_stride;
      // this lane's piece of tile j: its entry of the page table, then its page
      // (none for a page that no row sees: a window may have left it)
      auto has = [&](int j) {
        const int pos = j * kTcKeys + piece * rows;
        return piece < pieces && pos < w.tr.khi && pos + rows > w.tr.klo;
      };
      auto entry = [&](int j) -> int {
        return has(j) ? __ldg(trow + ((j * kTcKeys + piece * rows) >> a.p.page_shift)) : -1;
      };
      auto page_of = [&](int j, int pg) -> int {
        if (!has(j)) return -1;
        // a page that does not exist reads as zeros
        if ((pg < 0 || pg >= a.p.pages) && a.p.status) atomicOr(a.p.status, kStatusBounds);
        return pg < 0 || pg >= a.p.pages ? a.p.pages : pg;
      };
      auto place = [&](int j) { return (j * kTcKeys + piece * rows) & page_mask; };
      auto load_q = [&] {
        if (lane == 0) {
          const uint32_t bytes = a.group * a.tq * 128;
          const int tok = paged_first(a.p, w.b) + w.i * a.s.tq;
          mbar_arrive_expect_tx(q_full, bytes * (D / 64) * (two ? 2 : 1));
          for (int x = 0; x < (two ? 2 : 1); ++x)
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sq + x * Sh::kTile + h * Sh::kHalf, &qmap, h * 64, w.h * a.group,
                          tok + x * a.tq, q_full, pol);
        }
        __syncwarp();
      };
      const int pg0 = entry(w.j);
      int pg_next = w.n > 1 ? entry(w.j + 1) : -1;
      // the first slot also brings the values that the segment before ends with:
      // they do not wait for that segment's last Q·Kᵀ, as its Q's place does
      if (seg == 0) load_q();
      ok = put(page_of(w.j, pg0), place(w.j), w.h);
      if (seg > 0) {
        ok = ok && wait(q_empty, seg - 1);
        if (!ok) break;
        load_q();
      }
      ++seg;
      for (int k = 1; k < w.n && ok; ++k) {
        const int pg = pg_next;
        if (k + 1 < w.n) pg_next = entry(w.j + k + 1);
        ok = put(page_of(w.j + k, pg), place(w.j + k), w.h);
      }
    }
    if (ok && i > 0) put(-1, 0, 0);
    // the copies in flight land before the CTA's shared memory is given back
    if (lane == 0) {
      if (seg > 0) mbar_wait(q_full, (seg - 1) & 1, drain_ns(a.timeout_ns), nullptr);
      for (int st = 0; st < kSlots && st < i; ++st)
        mbar_wait(&full[st], ((i - st + kSlots - 1) / kSlots - 1) & 1, drain_ns(a.timeout_ns),
                  nullptr);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA
    // One warp issues the MMAs of A and B in turn: from two warps they would
    // interleave in the tensor cores' queue, A and B would finish together and
    // the tensor cores idle while both do their softmax.
    constexpr uint32_t qk_desc = umma_idesc_bf16(128, 128);
    constexpr uint32_t pv_desc = umma_idesc_bf16(128, D) | kUmmaBMnMajor;
    // descriptors: the low word holds the address (in 16-byte units)
    const uint64_t kd = umma_desc_sw128(0), vd = umma_desc_sw128_mn(0, Sh::kHalf);
    const uint32_t k_hi = (uint32_t)(kd >> 32), v_hi = (uint32_t)(vd >> 32);
    const uint32_t leader = elect_one();
    const uint32_t tm = __shfl_sync(~0u, taddr, 0);
    const uint32_t qa = __shfl_sync(~0u, (uint32_t)kd + (smem_u32(sq) >> 4), 0);
    const uint32_t va = __shfl_sync(~0u, (uint32_t)vd + (smem_u32(ring) >> 4), 0);
    const uint32_t ka = __shfl_sync(~0u, (uint32_t)kd + (smem_u32(ring + Sh::kTile) >> 4), 0);
    auto qk = [&](auto x, int st) {
      const uint32_t k = ka + st * (2 * Sh::kTile >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * Sh::kHalf + (kk & 3) * 32) >> 4;
        umma_bf16_elect(leader, tm + x * 128, qa + x * (Sh::kTile >> 4) + off, k_hi, k + off, k_hi,
                        qk_desc, kk > 0);
      }
    };
    auto commit = [&](uint64_t* bar) { umma_commit_elect(leader, bar); };
    const std::integral_constant<int, 0> A;
    const std::integral_constant<int, 1> B;
    int i = 0, seg = 0;
    uint32_t pa = 0, pb = 0, clean = 0;  // phases: P of A and B; edge tiles of each slot
    bool ok = next() && w.more() && wait(&full[0], 0);
#pragma unroll 1
    for (; ok; leave(seg++), ok = ok && next()) {
      // the segment's first Q·Kᵀ, while the output of the one before is read
      ok = w.more() && wait(q_full, seg);
      if (!ok) break;
      tc_fence_after();
      const bool two = has_b();
      const EdgeRange er = edges();
      qk(A, i % kSlots);
      commit(&s_full[0]);
      if (two) {
        qk(B, i % kSlots);
        commit(&s_full[1]);
      }
      commit(&empty[i % kSlots]);
      if (w.n == 1) commit(q_empty);
#pragma unroll 1
      for (int k = 0; k < w.n; ++k) {
        ++i;  // the slot with this tile's values and the next tile's keys
        const int st = i % kSlots, key0 = (w.j + k) * kTcKeys;
        const bool more = k + 1 < w.n, edge = er.in(key0, kTcKeys);
        const uint32_t v = va + st * (2 * Sh::kTile >> 4), first = k == 0 ? 0u : 1u;
        auto step = [&](auto x) {
          tc_fence_after();
          const uint32_t ts = tm + x * 128, to = tm + 256 + x * D;
          if (!edge) {
#pragma unroll
            for (int kk = 0; kk < kTcKeys / 16; ++kk)
              umma_bf16_ta_elect(leader, to, ts + kk * 8, v + kk * (2048 >> 4), v_hi, pv_desc,
                                 kk > 0 ? 1u : first);
          } else {
            int k0, k1;
            edge_steps(er, key0, k0, k1);
#pragma unroll 1
            for (int kk = k0; kk < k1; ++kk)
              umma_bf16_ta_elect(leader, to, ts + kk * 8, v + kk * (2048 >> 4), v_hi, pv_desc,
                                 kk > k0 ? 1u : first);
          }
          if (more) qk(x, st);
          commit(more ? &s_full[x] : &o_full[x]);
        };
        ok = wait(&full[st], i / kSlots);
        if (edge) {
          ok = ok && wait(&v_clean[st], clean >> st);
          clean ^= 1u << st;
        }
        if (!ok || !(ok = wait(&p_full[0], pa++))) break;
        step(A);
        if (two) {
          if (!(ok = wait(&p_full[1], pb++))) break;
          step(B);
        }
        if (more) commit(&empty[st]);
        if (k + 2 == w.n) commit(q_empty);  // the segment's last Q·Kᵀ
      }
    }
    commit(mma_done);
    mbar_wait(mma_done, 0, drain_ns(a.timeout_ns), nullptr);
    __syncwarp();
  } else if (warp == 10) {
    // ---------------------------------------------------------------- edge values
    int i = 0, seg = 0;
    // the first slot's first use has no values, but its phase has to pass too:
    // fills may land out of order, and the slot's second would be taken for it
    bool ok = next() && w.more() && wait(&full[0], 0);
    if (ok && lane == 0) mbar_arrive(&empty[0]);
    for (; ok && w.more(); leave(seg++), ok = ok && next()) {
      const EdgeRange er = edges();
      for (int k = 0; k < w.n && ok; ++k) {
        ++i;
        const int key0 = (w.j + k) * kTcKeys, st = i % kSlots;
        // every tile is waited for and left, edge or not: a phase cannot be told
        // from the one two later, so the slot must not be filled again before
        ok = wait(&full[st], i / kSlots);
        if (!ok) break;
        if (!er.in(key0, kTcKeys)) {
          if (lane == 0) mbar_arrive(&empty[st]);
          continue;
        }
        uint8_t* v = ring + st * 2 * Sh::kTile;
        int k0, k1;
        edge_steps(er, key0, k0, k1);
        auto at = [&](int x) {  // 8 values: x / (D / 8) positions into the tile
          const int key = x / (D / 8), ch = x % (D / 8);
          return reinterpret_cast<uint4*>(v + (ch >> 3) * Sh::kHalf + key * 128 +
                                          (((ch & 7) ^ (key & 7)) << 4));
        };
        // positions [from, to) of the tile: 0 where no row sees them; where not
        // all do, first one look over all of them (0 * x is not 0 if x is not
        // finite)
        bool found = false;
        auto none = [&](int from, int to) {
#pragma unroll 1
          for (int x = from * (D / 8) + lane; x < to * (D / 8); x += 32) *at(x) = make_uint4(0, 0, 0, 0);
        };
        auto some = [&](int from, int to) {
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
          __nv_bfloat162 sum = zero;
#pragma unroll 4
          for (int x = from * (D / 8) + lane; x < to * (D / 8); x += 32) {
            const uint4 e = *at(x);
            const uint32_t w4[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w4[q]), zero, sum);
          }
          if (__all_sync(~0u, __low2float(sum) == 0.f && __high2float(sum) == 0.f)) return;
#pragma unroll 1
          for (int x = from * (D / 8) + lane; x < to * (D / 8); x += 32)
            found |= clean_edge_value(at(x), er, key0 + x / (D / 8));
        };
        auto within = [&](int pos) {
          const int n = pos - key0;
          return n < k0 * 16 ? k0 * 16 : (n > k1 * 16 ? k1 * 16 : n);
        };
        const int seen0 = within(er.klo), seen1 = within(er.khi);
        none(k0 * 16, seen0);
        some(seen0, within(er.all_lo < er.khi ? er.all_lo : er.khi));
        some(within(er.all_hi > er.all_lo ? er.all_hi : er.all_lo), seen1);
        none(seen1 > seen0 ? seen1 : seen0, k1 * 16);
        if (__any_sync(~0u, found) && lane == 0) s_poison[seg & 3] = seg + 1;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_clean[st]);
          mbar_arrive(&empty[st]);
        }
      }
    }
  }
  if (a.deep && threadIdx.x == 0) {
    // the pair that begins in this CTA's range and goes on past it, for the
    // second kernel: CTAs, first token, tokens, head
    SplitWalk f(a.s, tab, u0, u1);
    int4 d = make_int4(0, 0, 0, 0);
    for (; f.more(); f.next())
      if (!draws && !f.whole && f.tile_unit() >= u0) {
        const int n = (int)(worker_of(f.tile_unit() + f.tr.n - 1, W, G) - blockIdx.x + 1);
        const int t0 = f.i * a.s.tq, left = tab.qn[f.b] - t0;
        if (n > kTcFew && !s_flag[0])
          d = make_int4(n, paged_first(a.p, f.b) + t0, left < a.s.tq ? left : a.s.tq, f.h);
      }
    a.deep[blockIdx.x] = d;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(taddr, 512);
  }
}

// Joins the pairs that more than kTcFew CTAs share: block (c, y) takes 4 columns
// at a time of the pair that begins in CTA c's range, a thread for each row; the
// CTAs' parts are summed in their order.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const TcAttnArgs a) {
  using Sh = TcAttnShape<D>;
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x;
  const int4 s = __ldcg(a.deep + c);
  const int n = s.x, x = threadIdx.x >> 7, r = threadIdx.x & 127;
  const int t = r / a.group, tt = x * a.tq + t;
  if (n == 0 || t >= a.tq || tt >= s.z) return;
  auto part = [&](int k) -> const float* {
    return a.ws + ((long long)(c + k) * 2 + (k == 0 ? 1 : 0)) * Sh::kPart + x * (Sh::kPart / 2);
  };
  auto ml = [&](int k) {
    return __ldcg(reinterpret_cast<const float2*>(part(k) + D * kTcRowsA) + r);
  };
  float M = -INFINITY;
#pragma unroll 8
  for (int k = 0; k < n; ++k) M = fmaxf(M, ml(k).x);
  const long long tok = s.y + tt;
  const int head = s.w * a.group + r - t * a.group;
  for (int d = blockIdx.y * 4; d < D; d += gridDim.y * 4) {
    float v[4] = {0.f, 0.f, 0.f, 0.f}, L = 0.f;
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float2 s2 = ml(k);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(part(k) + d * kTcRowsA + r * 4));
      const float f = M == -INFINITY ? 1.f : exp2_approx(s2.x - M);
      L += f * s2.y;
      v[0] += f * o.x;
      v[1] += f * o.y;
      v[2] += f * o.z;
      v[3] += f * o.w;
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    *reinterpret_cast<uint2*>(a.out + tok * a.ldo + (long long)head * D + d) =
        make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
    if (a.lse && d == 0)
      a.lse[tok * a.hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

// ------------------------------------------------------------------ launch
template <int D>
static cudaError_t launch_tc_d(const Ctx& cx, const CUtensorMap& kv, const CUtensorMap& q,
                               const TcAttnArgs& a) {
  static DevOnce once;
  cudaError_t e = setup_smem(once, attn_tc_kernel<D>, kMaxDynSmem);
  if (e != cudaSuccess) return e;
  e = launch_k(attn_tc_kernel<D>, dim3(cx.sms), dim3(kTcAttnThreads),
               TcAttnShape<D>::smem(a.p.batch), cx.stream, cx.pdl, kv, q, a);
  if (e != cudaSuccess || !a.deep) return e;
  return launch_k(attn_join_kernel<D>, dim3(cx.sms, D / 8), dim3(256), 0, cx.stream, cx.pdl, a);
}

size_t attn_tc_ws(int dim, int sms) {
  return (size_t)sms * (2 * (2 * kTcRowsA * (size_t)(dim + 2)) * sizeof(float) + sizeof(int4));
}

cudaError_t launch_attn_tc(const Ctx& cx, const KvView& v, const AttnCall& c, float* ws, int* ctr,
                           int* kernels) {
  CUtensorMap kv, q;
  TcAttnArgs a = {};
  a.group = c.hq / v.hkv;
  a.tq = kTcRowsA / a.group;
  if (!make_tmap_kv(&kv, v, v.page < kTcKeys ? v.page : kTcKeys) ||
      !make_tmap_heads(&q, c.q, c.tokens, c.hq, v.dim, c.ldq, a.group, a.tq))
    return cudaErrorInvalidValue;
  a.p = paged_args(v, c.tokens, cx.status);
  a.s.tq = 2 * a.tq;
  a.s.bn_shift = kTcKeysShift;
  a.s.window = c.window;
  a.s.hkv = v.hkv;
  a.out = static_cast<uint16_t*>(c.out);
  a.lse = c.lse;
  a.ldo = c.ldo;
  a.hq = c.hq;
  // a scale of 0 (all weights equal): one that no score outgrows, so that masked
  // scores stay infinite
  a.c = c.scale == 0.f ? 1e-30f : c.scale * 1.4426950408889634f;
  a.ws = ws;
  a.ctr = ctr;
  a.s.start = 3;
  a.s.snap = 12;
  a.min_units = 6;
  a.timeout_ns = cx.timeout_ns;
  const long long pairs = ((long long)c.tokens / a.s.tq + v.batch) * v.hkv;
  if (pairs * 4 <= cx.sms)
    a.deep = reinterpret_cast<int4*>(ws + (size_t)cx.sms * 2 * (2 * kTcRowsA * (v.dim + 2)));
  *kernels = a.deep ? 2 : 1;
  return v.dim == 64 ? launch_tc_d<64>(cx, kv, q, a) : launch_tc_d<128>(cx, kv, q, a);
}

}  // namespace dg
