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
// The work is split into equal ranges of (row tile pair, key tile) units, see
// paged.cuh. A pair that spans several CTAs leaves its unnormalised O, m and
// sum in the workspace, and a second small kernel joins them.
#include "launch.h"
#include "launch_util.cuh"
#include "paged.cuh"
#include "tc_common.cuh"

namespace dg {

constexpr int kTcKeys = 128;         // positions of a key tile
constexpr int kTcKeysShift = 7;
constexpr int kTcRowsA = 128;        // rows of a row tile
constexpr int kTcAttnThreads = 352;
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
  int* split;          // [grid][4] the split pairs, by their first CTA
  long long ws_len;
  int min_units;
  long long timeout_ns;
};

template <int D>
struct TcAttnShape {
  static constexpr int kHalf = kTcKeys * 128;            // 64 columns of a 128-row tile
  static constexpr int kTile = kTcKeys * D * 2;          // a tile of Q, K or V
  static constexpr int kStages = 128 * 1024 / kTile;
  static constexpr int kSlot = 2 * kTcRowsA * (D + 2);   // floats of a split pair's partial
  static int smem(int batch) {
    return 1024 + 2 * kTile + kStages * kTile + 8 * (3 * kStages + 16) + 128 +
           SplitTables::bytes(batch) + 16;
  }
};

template <int D>
__global__ void __launch_bounds__(kTcAttnThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
                   const TcAttnArgs a) {
  using Sh = TcAttnShape<D>;
  constexpr int kStages = Sh::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sq = smem;                       // Q of A and B
  uint8_t* ring = smem + 2 * Sh::kTile;     // K, V, K, V, ...
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * Sh::kTile);
  uint64_t* empty = full + kStages;
  uint64_t* s_full = empty + kStages;   // [2] S ready, and everything issued before it done
  uint64_t* p_full = s_full + 2;        // [2] P written
  uint64_t* q_full = p_full + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* mma_done = q_empty + 1;
  uint64_t* v_clean = mma_done + 1;     // [kStages / 2] value stage looked over
  volatile int* s_flag = reinterpret_cast<volatile int*>(full + 3 * kStages + 16);  // [0] abort
  volatile int* s_poison = s_flag + 4;  // [4] segment number + 1 with a non-finite edge value
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(const_cast<int*>(s_flag) + 8);
  const SplitTables tab(reinterpret_cast<uint8_t*>(const_cast<int*>(s_flag)) + 128, a.p.batch);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w], 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < kStages / 2; ++i) mbar_init(&v_clean[i], 1);
    mbar_init(mma_done, 1);
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
  split_setup<kTcAttnThreads>(a.p, a.s, tab, a.min_units, W, G, u0, u1);
  SplitWalk w(a.s, tab, u0, u1);

  auto edges = [&]() -> EdgeRange {
    const int qn = tab.qn[w.b], t0 = w.i * a.s.tq;
    const int nt = qn - t0 < a.s.tq ? qn - t0 : a.s.tq;
    return edge_range(a.s, w.tr, tab.kv[w.b] - qn + t0, nt);
  };
  // B has rows
  auto has_b = [&] { return tab.qn[w.b] - w.i * a.s.tq > a.tq; };
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (s_flag[0]) return false;
    if (mbar_wait(bar, parity & 1, a.timeout_ns, a.p.status)) return true;
    s_flag[0] = 1;
    return false;
  };

  if (warp == 9) {
    // ---------------------------------------------------------------- TMA
    const uint64_t pol = policy_evict_last();
    const int rows = a.p.page < kTcKeys ? a.p.page : kTcKeys;
    const int pieces = kTcKeys / rows, page_mask = a.p.page - 1;
    const int half = lane % (D / 64), piece = lane / (D / 64);
    int it = 0, seg = 0;
    bool ok = true;
    for (; w.more() && ok; w.next(), ++seg) {
      const bool two = has_b();
      if (!__all_sync(~0u, seg == 0 || wait(q_empty, seg - 1))) break;
      if (lane == 0) {
        const uint32_t bytes = a.group * a.tq * 128;
        mbar_arrive_expect_tx(q_full, bytes * (D / 64) * (two ? 2 : 1));
        for (int x = 0; x < (two ? 2 : 1); ++x)
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sq + x * Sh::kTile + h * Sh::kHalf, &qmap, h * 64, w.h * a.group,
                        tab.q0[w.b] + w.i * a.s.tq + x * a.tq, q_full, pol);
      }
      __syncwarp();
      const int row = tab.row[w.b];
      const int32_t* trow = a.p.table + (long long)(row < 0 ? 0 : row) * a.p.table_stride;
      auto page_at = [&](int j) -> int {
        const int pos = j * kTcKeys + piece * rows;
        if (piece >= pieces || pos >= w.tr.khi) return -1;
        const int pg = __ldg(trow + (pos >> a.p.page_shift));
        // a page that does not exist reads as zeros
        if ((pg < 0 || pg >= a.p.pages) && a.p.status) atomicOr(a.p.status, kStatusBounds);
        return pg < 0 || pg >= a.p.pages ? a.p.pages : pg;
      };
      int pg_next = page_at(w.j);
      for (int k = 0; k < w.n && ok; ++k) {
        const int j = w.j + k, pg = pg_next;
        if (k + 1 < w.n) pg_next = page_at(j + 1);
        const int n = __popc(__ballot_sync(~0u, pg >= 0));
        for (int v = 0; v < 2; ++v, ++it) {
          const int st = it % kStages;
          if (it >= kStages && !wait(&empty[st], it / kStages + 1)) ok = false;
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[st], n * rows * 128);
          __syncwarp();
          if (pg >= 0)
            tma_load_4d(ring + st * Sh::kTile + half * Sh::kHalf + piece * rows * 128, &kvmap,
                        half * 64, (j * kTcKeys + piece * rows) & page_mask, v * a.p.hkv + w.h, pg,
                        &full[st], pol);
        }
      }
    }
    // the copies in flight land before the CTA's shared memory is given back
    if (lane == 0) {
      if (seg > 0) mbar_wait(q_full, (seg - 1) & 1, drain_ns(a.timeout_ns), nullptr);
      for (int st = 0; st < kStages && st < it; ++st)
        mbar_wait(&full[st], ((it - st + kStages - 1) / kStages - 1) & 1, drain_ns(a.timeout_ns),
                  nullptr);
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t qk_desc = umma_idesc_bf16(128, 128);
      constexpr uint32_t pv_desc = umma_idesc_bf16(128, D) | kUmmaBMnMajor;
      const uint32_t qa = smem_u32(sq), ra = smem_u32(ring);
      auto qk = [&](int x, uint32_t kb) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * Sh::kHalf + (kk & 3) * 32;
          umma_bf16(taddr + x * 128, umma_desc_sw128(qa + x * Sh::kTile + off),
                    umma_desc_sw128(kb + off), qk_desc, kk > 0);
        }
      };
      auto pv = [&](int x, uint32_t vb, bool first) {
#pragma unroll
        for (int kk = 0; kk < kTcKeys / 16; ++kk)
          umma_bf16_ta(taddr + 256 + x * D, taddr + x * 128 + kk * 8,
                       umma_desc_sw128_mn(vb + kk * 2048, Sh::kHalf), pv_desc, !first || kk > 0);
      };
      int it = 0, seg = 0;
      uint32_t pn[2] = {0, 0};
      bool ok = true;
      for (; w.more() && ok; w.next(), ++seg) {
        const int nx = has_b() ? 2 : 1;
        ok = wait(q_full, seg) && wait(&full[it % kStages], it / kStages);
        if (!ok) break;
        tc_fence_after();
        for (int x = 0; x < nx; ++x) {
          qk(x, ra + (it % kStages) * Sh::kTile);
          umma_commit(&s_full[x]);
        }
        umma_commit(&empty[it % kStages]);
        if (w.n == 1) umma_commit(q_empty);
        for (int k = 0; k < w.n && ok; ++k, it += 2) {
          const int vs = it + 1, ks = it + 2;  // stages of V and of the next K
          const bool more = k + 1 < w.n;
          ok = wait(&full[vs % kStages], vs / kStages);
          ok = ok && wait(&v_clean[vs % kStages / 2], vs / kStages);
          for (int x = 0; x < nx && ok; ++x) {
            ok = wait(&p_full[x], pn[x]++);
            if (!ok) break;
            tc_fence_after();
            pv(x, ra + (vs % kStages) * Sh::kTile, k == 0);
            if (more) {
              if (x == 0) {
                ok = wait(&full[ks % kStages], ks / kStages);
                if (!ok) break;
                tc_fence_after();
              }
              qk(x, ra + (ks % kStages) * Sh::kTile);
            }
            umma_commit(&s_full[x]);
          }
          umma_commit(&empty[vs % kStages]);
          if (more) umma_commit(&empty[ks % kStages]);
          if (k + 2 == w.n) umma_commit(q_empty);  // the segment's last Q·Kᵀ
        }
      }
      umma_commit(mma_done);
      mbar_wait(mma_done, 0, drain_ns(a.timeout_ns), nullptr);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---------------------------------------------------------------- edge values
    int it = 0, seg = 0;
    bool ok = true;
    for (; w.more() && ok; w.next(), ++seg) {
      const EdgeRange er = edges();
      for (int k = 0; k < w.n && ok; ++k, it += 2) {
        const int key0 = (w.j + k) * kTcKeys, vs = it + 1;
        // every tile is waited for, edge or not: a phase cannot be told from
        // the one two later
        ok = __all_sync(~0u, wait(&full[vs % kStages], vs / kStages));
        if (!ok) break;
        uint64_t* done = &v_clean[vs % kStages / 2];
        if (!er.in(key0, kTcKeys)) {
          if (lane == 0) mbar_arrive(done);
          continue;
        }
        uint8_t* v = ring + (vs % kStages) * Sh::kTile;
        bool found = false;
        auto clean = [&](int from, int to) {  // keys of the tile
          for (int x = from * (D / 8) + lane; x < to * (D / 8); x += 32) {
            const int key = x / (D / 8), ch = x % (D / 8), pos = key0 + key;
            uint4* at = reinterpret_cast<uint4*>(v + (ch >> 3) * Sh::kHalf + key * 128 +
                                                 (((ch & 7) ^ (key & 7)) << 4));
            found |= clean_edge_value(at, er, pos);
          }
        };
        const int lo_end = er.all_lo - key0 < 0 ? 0 : (er.all_lo - key0 < kTcKeys ? er.all_lo - key0 : kTcKeys);
        int hi_from = er.all_hi - key0 < 0 ? 0 : (er.all_hi - key0 < kTcKeys ? er.all_hi - key0 : kTcKeys);
        if (hi_from < lo_end) hi_from = lo_end;
        clean(0, lo_end);
        clean(hi_from, kTcKeys);
        if (__any_sync(~0u, found) && lane == 0) s_poison[seg & 3] = seg + 1;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(done);
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int x = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = taddr + lanes + x * 128, to = taddr + lanes + 256 + x * D;
    uint32_t sn = 0;
    int seg = 0;
    bool ok = true;
    for (; w.more() && ok; w.next(), ++seg) {
      if (x == 1 && !has_b()) continue;
      const EdgeRange er = edges();
      const int qn = tab.qn[w.b];
      const int t0 = w.i * a.s.tq + x * a.tq;
      const int nt = qn - t0 < a.tq ? qn - t0 : a.tq;
      const int t = r / a.group, g = r - t * a.group;
      const bool live = t < nt;
      const int pos = tab.kv[w.b] - qn + t0 + t;
      const int hi = live ? pos : -1;
      const int lo = live && a.s.window > 0 ? pos - a.s.window + 1 : 0;
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < w.n; ++k) {
        const int key0 = (w.j + k) * kTcKeys;
        ok = __all_sync(~0u, wait(&s_full[x], sn++));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, s + q * 32);
        tmem_ld_wait();
        tmem_settle<128>(s);
        if (er.in(key0, kTcKeys)) {
          const int h0 = hi - key0, l0 = lo - key0;
#pragma unroll
          for (int q = 0; q < 128; ++q)
            if (q > h0 || q < l0) s[q] = 0xFF800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int q = 0; q < 128; ++q) mx[q & 3] = fmaxf(mx[q & 3], __uint_as_float(s[q]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
        if (__any_sync(~0u, top > m + kTcLazy)) {
          // m was -inf before the first visible position: O and l are 0 then
          const float mn = fmaxf(m, top);
          const float f = m == -INFINITY ? 0.f : exp2_approx(m - mn);
          m = mn;
          l *= f;
          if (k > 0) {
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(to + q * 32, o);
              tmem_ld_wait();
              tmem_settle<32>(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(to + q * 32, o);
            }
          }
        }
        const float mb = m == -INFINITY ? 0.f : m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 128; q += 2) {
          const float p0 = exp2_approx(fmaf(__uint_as_float(s[q]), a.c, -mb));
          const float p1 = exp2_approx(fmaf(__uint_as_float(s[q + 1]), a.c, -mb));
          sum[(q >> 1) & 1] += p0;
          sum[2 + ((q >> 1) & 1)] += p1;
          // weights as bf16: see k_attn.cu
          s[q >> 1] = pack_bf16(p0, p1);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st32(ts, s);
        tmem_st32(ts + 32, s + 32);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      ok = __all_sync(~0u, wait(&s_full[x], sn++));
      if (!ok) break;
      tc_fence_after();
      // rows that see a non-finite edge value get it here
      const bool poison = s_poison[seg & 3] == seg + 1;
      const int row = tab.row[w.b];
      const long long tok = tab.q0[w.b] + t0 + t;
      const int head = w.h * a.group + g;
      const long long slot = (long long)blockIdx.x * 2 + (w.tile_unit() >= u0 ? 1 : 0);
      float* part = a.ws + slot * Sh::kSlot + x * kTcRowsA * (D + 2);
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays NaN
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(to + q * 32, o);
        tmem_ld_wait();
        tmem_settle<32>(o);
        if (poison && live && row >= 0) {
          edge_values<D>(a.p, row, w.h, er, lo, hi, w.j * kTcKeys, (w.j + w.n) * kTcKeys, q * 32,
                         [&](const uint16_t* v) {
#pragma unroll
                           for (int e = 0; e < 32; ++e) {
                             const float f = bf_bits2f(__ldg(v + e));
                             if (!isfinite(f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
                           }
                         });
        }
        if (w.whole) {
          if (live) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + tok * a.ldo + (long long)head * D + q * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t* v = o + e * 8;
              auto at = [&](int i) { return __uint_as_float(v[i]) * inv; };
              dst[e] = make_uint4(pack_bf16(at(0), at(1)), pack_bf16(at(2), at(3)),
                                  pack_bf16(at(4), at(5)), pack_bf16(at(6), at(7)));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            __stcg(DG_AT(a.p.status, part, (q * 32 + e) * kTcRowsA + r, Sh::kSlot), __uint_as_float(o[e]));
        }
      }
      if (w.whole) {
        if (live && a.lse)
          a.lse[tok * a.hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      } else {
        __stcg(part + D * kTcRowsA + r, m);
        __stcg(part + (D + 1) * kTcRowsA + r, l);
      }
      // O is read: P of the next segment may be followed by its first P·V
      tc_fence_before();
    }
  }
  // what the second kernel joins: the pair that begins in this CTA's range and
  // goes on past it
  if (threadIdx.x == 0) {
    SplitWalk f(a.s, tab, u0, u1);
    int n = 0, q0 = 0, rows = 0, h = 0;
    while (f.more()) {
      if (!f.whole && f.tile_unit() >= u0) {
        const int qn = tab.qn[f.b], t0 = f.i * a.s.tq;
        n = (int)(cta_of(f.tile_unit() + f.tr.n - 1, W, G) - blockIdx.x + 1);
        q0 = tab.q0[f.b] + t0;
        rows = (qn - t0 < a.s.tq ? qn - t0 : a.s.tq);
        h = f.h;
      }
      f.next();
    }
    int4* dst = reinterpret_cast<int4*>(a.split + blockIdx.x * 4);
    *dst = make_int4(s_flag[0] ? 0 : n, q0, rows, h);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(taddr, 512);
  }
}

// Joins the partial results of the pairs that span several CTAs: block (c, y)
// takes 4 columns at a time of the pair that begins in CTA c's range, a thread
// for each of its rows; the CTAs' parts are summed in their order.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const TcAttnArgs a) {
  using Sh = TcAttnShape<D>;
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x;
  const int4 s = __ldcg(reinterpret_cast<const int4*>(a.split + c * 4));
  const int n = s.x, x = threadIdx.x >> 7, r = threadIdx.x & 127;
  const int t = r / a.group, g = r - t * a.group, tt = x * a.tq + t;
  if (n == 0 || t >= a.tq || tt >= s.z) return;
  auto part = [&](int k) -> const float* {
    return a.ws + ((long long)(c + k) * 2 + (k == 0 ? 1 : 0)) * Sh::kSlot + x * kTcRowsA * (D + 2) + r;
  };
  float M = -INFINITY;
#pragma unroll 8
  for (int k = 0; k < n; ++k) M = fmaxf(M, __ldcg(part(k) + D * kTcRowsA));
  const long long tok = s.y + tt;
  const int head = s.w * a.group + g;
  for (int d = blockIdx.y * 4; d < D; d += gridDim.y * 4) {
    float v[4] = {0.f, 0.f, 0.f, 0.f}, L = 0.f;
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float* p = part(k);
      const float m = __ldcg(p + D * kTcRowsA), l = __ldcg(p + (D + 1) * kTcRowsA);
      const float f = M == -INFINITY ? 1.f : exp2_approx(m - M);
      L += f * l;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += f * __ldcg(p + (d + e) * kTcRowsA);
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
                               const TcAttnArgs& a, int join_y) {
  static DevOnce once;
  cudaError_t e = setup_smem(once, attn_tc_kernel<D>, kMaxDynSmem);
  if (e != cudaSuccess) return e;
  e = launch_k(attn_tc_kernel<D>, dim3(cx.sms), dim3(kTcAttnThreads), TcAttnShape<D>::smem(a.p.batch),
               cx.stream, cx.pdl, kv, q, a);
  if (e != cudaSuccess) return e;
  return launch_k(attn_join_kernel<D>, dim3(cx.sms, join_y), dim3(256), 0, cx.stream, cx.pdl, a);
}

size_t attn_tc_ws(int dim, int sms) {
  return (size_t)sms * (2 * (size_t)(2 * kTcRowsA * (dim + 2)) * sizeof(float) + 16);
}

cudaError_t launch_attn_tc(const Ctx& cx, const KvView& v, const AttnCall& c, void* ws) {
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
  a.c = c.scale * 1.4426950408889634f;
  a.split = static_cast<int*>(ws);
  a.ws = reinterpret_cast<float*>(static_cast<char*>(ws) + (size_t)cx.sms * 16);
  a.min_units = 2;
  a.timeout_ns = cx.timeout_ns;
  // few pairs, each split over many CTAs: spread each join over more blocks
  const long long pairs = ((long long)c.tokens / a.s.tq + v.batch) * v.hkv;
  const int join_y = pairs * 4 < cx.sms ? v.dim / 4 : 8;
  return v.dim == 64 ? launch_tc_d<64>(cx, kv, q, a, join_y) : launch_tc_d<128>(cx, kv, q, a, join_y);
}

}  // namespace dg
