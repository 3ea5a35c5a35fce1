// paged.cuh -- what the paged-cache kernels share: the view of a cache and a
// batch of sequences, and the split of an attention call's work over CTAs.
//
// A cache holds pages of `page` positions, [pages][2][heads][page][dim] bf16
// (keys, then values). Sequence b of a batch owns row rows[b] (or b) of the
// page table; its qn new tokens cu_q[b] .. cu_q[b+1] - 1 are the last of its
// kv_len positions. Lengths and page numbers are device data: they are clamped
// to what the caller's arrays hold, so wrong ones give wrong results and a
// status, never an access out of range.
//
// Work is counted in units: one key tile (BN positions) read for one row tile
// (tq tokens x the query heads that share a key head) of one sequence and key
// head, and `start` more at the beginning of each row tile for what it costs
// whatever its length (queries in, output out). The units of a call, in the
// order sequence, key head, row tile, key tile, are cut into equal contiguous
// ranges, one per CTA, except that a row tile of at most `snap` units is not
// cut: the cut goes to its nearer end, as joining costs more than it evens out.
// The partial softmax states of a row tile that spans several ranges are joined
// in CTA order. (The figures: one token over 8k positions 15.5 us cut without
// regard to ends, 14 with; 22 sequences of 100 to 300 positions 15 -> 10.)
#pragma once

#include "dg_common.cuh"
#include "launch.h"

namespace dg {

constexpr int kMaxBatch = 1024;   // sequences of one call

struct PagedArgs {
  const int32_t* table;
  const int32_t* rows;      // optional
  const int32_t* cu_q;
  const int32_t* kv_len;
  long long table_stride;
  int width, table_rows;    // entries of a table row, rows of the table (and of kv_len)
  const uint16_t* cache;
  long long page_stride;    // elements
  int pages, hkv, page;     // page: a power of two
  int page_shift;
  int batch, tokens;
  int* status;
};

inline PagedArgs paged_args(const KvView& v, int tokens, int* status) {
  PagedArgs p = {};
  p.table = v.table;
  p.rows = v.rows;
  p.cu_q = v.cu_q;
  p.kv_len = v.kv_len;
  p.table_stride = v.table_stride;
  p.width = v.width;
  p.table_rows = v.table_rows;
  p.cache = static_cast<const uint16_t*>(v.cache);
  p.page_stride = v.page_stride;
  p.pages = v.pages;
  p.hkv = v.hkv;
  p.page = v.page;
  while ((1 << p.page_shift) < v.page) ++p.page_shift;
  p.batch = v.batch;
  p.tokens = tokens;
  p.status = status;
  return p;
}

// Row of the table (and of kv_len) of sequence b, or -1 if there is none.
__device__ __forceinline__ int paged_row(const PagedArgs& p, int b) {
  const int r = p.rows ? __ldg(p.rows + b) : b;
  if (r >= 0 && r < p.table_rows) return r;
  if (p.status) atomicOr(p.status, kStatusBounds);
  return -1;
}

// Positions of a sequence: kv_len clamped to what its table row can hold.
__device__ __forceinline__ int paged_len(const PagedArgs& p, int row) {
  if (row < 0) return 0;
  const int n = __ldg(p.kv_len + row);
  const long long cap = (long long)p.width << p.page_shift;
  if (n >= 0 && n <= cap) return n;
  if (p.status) atomicOr(p.status, kStatusBounds);
  return n < 0 ? 0 : (int)cap;
}

// First token of sequence b, within [0, tokens].
__device__ __forceinline__ int paged_first(const PagedArgs& p, int b) {
  const int a = __ldg(p.cu_q + b);
  return a < 0 ? 0 : (a > p.tokens ? p.tokens : a);
}

// First position that a token at position pos sees. (pos may be negative, and
// window anything up to 2^31 - 1.)
__device__ __forceinline__ int first_seen(int window, int pos) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// ------------------------------------------------------------------ the split
struct SplitShape {
  int tq;        // tokens of a row tile
  int bn_shift;  // log2 of the key tile
  int window;    // 0: none
  int hkv;
  int start;     // units of a row tile before its first key tile
  int snap;      // units up to which a row tile is one CTA's
};

// Key tiles [j0, j0 + n) of row tile i of a sequence with qn new tokens and kv
// positions; n >= 1 (a tile whose rows see nothing still writes its zeros).
// klo, khi: positions that some row of the tile sees, [klo, khi).
struct TileRange {
  int j0, n, klo, khi;
};
__device__ __forceinline__ TileRange tile_range(const SplitShape& s, int qn, int kv, int i) {
  TileRange r;
  const int t0 = i * s.tq;
  const int t1 = t0 + s.tq < qn ? t0 + s.tq : qn;
  r.khi = kv - qn + t1;
  if (r.khi < 0) r.khi = 0;
  r.klo = first_seen(s.window, kv - qn + t0);
  r.j0 = r.klo >> s.bn_shift;
  r.n = ((r.khi + (1 << s.bn_shift) - 1) >> s.bn_shift) - r.j0;
  if (r.n < 1) r.n = 1;
  return r;
}

// What the rows of a row tile see of the positions.
struct EdgeRange {
  int klo, khi;          // seen by some row: [klo, khi)
  int all_lo, all_hi;    // seen by every row: [all_lo, all_hi)
  // positions [key0, key0 + n) are not all seen by every row
  __device__ bool in(int key0, int n) const { return key0 + n > all_hi || key0 < all_lo; }
};
// pos0: position of the tile's first of nt tokens
__device__ __forceinline__ EdgeRange edge_range(const SplitShape& s, const TileRange& r, int pos0,
                                                int nt) {
  return EdgeRange{r.klo, r.khi, first_seen(s.window, pos0 + nt - 1), pos0 + 1};
}

// A value of a key tile at the edge must not reach the sums of rows that do
// not see it: as 0 * NaN and 0 * inf are NaN, the kernels make 0 of what no
// row sees (the unused end of a page may hold anything), and of a non-finite
// value that only some rows see, which those rows get added at the end.
//
// Cleans 8 values of position pos in shared memory; true if one of them is
// such a non-finite value.
__device__ __forceinline__ bool clean_edge_value(uint4* at, const EdgeRange& er, int pos) {
  if (pos < er.klo || pos >= er.khi) {
    *at = make_uint4(0, 0, 0, 0);
    return false;
  }
  if (pos >= er.all_lo && pos < er.all_hi) return false;
  uint4 v = *at;
  bool any = false;
  auto finite = [&](uint32_t& e) {
    if ((e & 0x7F80u) == 0x7F80u) e &= 0xFFFF0000u, any = true;
    if ((e & 0x7F800000u) == 0x7F800000u) e &= 0xFFFFu, any = true;
  };
  finite(v.x);
  finite(v.y);
  finite(v.z);
  finite(v.w);
  if (any) *at = v;
  return any;
}

// Calls f(pointer to column d, position) for each position in [kbeg, kend) that a row
// seeing [lo, hi] sees and some other row of its tile does not.
template <int D, typename F>
__device__ __forceinline__ void edge_values(const PagedArgs& p, int row, int h, const EdgeRange& er,
                                            int lo, int hi, int kbeg, int kend, int d, const F& f) {
  if (row < 0) return;
  for (int side = 0; side < 2; ++side) {
    int from = side ? (er.all_hi > er.all_lo ? er.all_hi : er.all_lo) : er.klo;
    int to = side ? er.khi : er.all_lo;
    if (from < lo) from = lo;
    if (from < kbeg) from = kbeg;
    if (to > hi + 1) to = hi + 1;
    if (to > kend) to = kend;
    for (int key = from; key < to; ++key) {
      const int pg = __ldg(p.table + row * p.table_stride + (key >> p.page_shift));
      if (pg < 0 || pg >= p.pages) continue;
      f(p.cache + pg * p.page_stride +
        ((long long)(p.hkv + h) * p.page + (key & (p.page - 1))) * D + d, key);
    }
  }
}

// Shared-memory tables of a call's sequences (sized for the batch).
struct SplitTables {
  long long* base;   // [batch + 1] first unit of each sequence
  long long* head;   // [6] the call's units and workers, this worker's range, row tiles, the longest
  int* qn;           // [batch] new tokens
  int* kv;           // positions
  int* loc;          // [4] this worker's first sequence, head, row tile, unit in it
  static __host__ __device__ constexpr int bytes(int batch) {
    return 8 * (batch + 1) + 8 * 6 + 8 * batch + 16;
  }
  __device__ explicit SplitTables(void* smem, int batch) {
    base = reinterpret_cast<long long*>(smem);
    head = base + batch + 1;
    qn = reinterpret_cast<int*>(head + 6);
    kv = qn + batch;
    loc = kv + batch;
  }
};

// Fill the tables and find the range [u0, u1) of the W units that worker c of
// `workers` (a CTA or a cluster) has, and where it begins. Called by all
// threads of the CTA; ends with a barrier. G: workers that take part.
//
// DRAW: where there are row tiles enough and none is long, equal ranges lose
// more to their ends (a tile cut and joined, or left whole beside a range that
// is then shorter) than workers that draw whole tiles as they become free, long
// ones first (four prompts of up to 2047 tokens 168 -> 154 us, one of 2048 68 -> 59;
// modelled over 300 batches of random lengths, those that the rule takes gain 3%
// on average, the worst, of few long tiles, loses 24%). head[4] is then the number
// of row tiles of all heads (else 0), head[5] the units of the longest, and there
// is no range.
//
// One warp does it, a lane for each of 32 sequences at a time: every call waits
// for this before it can do anything else, and the other warps would add
// barriers, not speed.
template <bool DRAW>
__device__ __forceinline__ void split_setup(const PagedArgs& p, const SplitShape& s,
                                            const SplitTables& t, int min_units, long long c,
                                            long long workers, long long& W, long long& G,
                                            long long& u0, long long& u1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    constexpr int kFew = 2;  // row tiles of a sequence that one lane counts by itself
    struct Raw {
      int a, e, row, kv;
    };
    auto fetch = [&](int b) -> Raw {
      Raw r = {0, 0, 0, 0};
      if (b < p.batch) {
        r.row = p.rows ? __ldg(p.rows + b) : b;
        r.a = __ldg(p.cu_q + b);
        r.e = __ldg(p.cu_q + b + 1);
        if (r.row >= 0 && r.row < p.table_rows) r.kv = __ldg(p.kv_len + r.row);
      }
      return r;
    };
    const long long cap = (long long)p.width << p.page_shift;
    long long units = 0;
    int all_tiles = 0, longest = 0;
    Raw next = fetch(lane);
#pragma unroll 1
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const Raw r = next;
      const int b = b0 + lane;
      if (b0 + 32 < p.batch) next = fetch(b + 32);
      const int q0 = r.a < 0 ? 0 : (r.a > p.tokens ? p.tokens : r.a);
      const int q1 = r.e < q0 ? q0 : (r.e > p.tokens ? p.tokens : r.e);
      const int kv = r.kv < 0 ? 0 : (r.kv > cap ? (int)cap : r.kv), qn = q1 - q0;
      if (b < p.batch) {
        t.qn[b] = qn;
        t.kv[b] = kv;
        if (p.status && (q0 != r.a || q1 != r.e || kv != r.kv || r.row < 0 || r.row >= p.table_rows))
          atomicOr(p.status, kStatusBounds);
      }
      // (a division only where it takes one)
      int tiles = (qn > 0) + (qn > s.tq);
      if (__any_sync(~0u, qn - s.tq > s.tq)) tiles = (qn + s.tq - 1) / s.tq;
      long long u = 0;
      if (tiles <= kFew)
        for (int i = 0; i < tiles; ++i) u += tile_range(s, qn, kv, i).n + s.start;
#pragma unroll 1
      for (unsigned big = __ballot_sync(~0u, tiles > kFew); big; big &= big - 1) {
        const int l = __ffs(big) - 1, n = __shfl_sync(~0u, tiles, l);
        const int lq = __shfl_sync(~0u, qn, l), lkv = __shfl_sync(~0u, kv, l);
        long long sum = 0;
#pragma unroll 1
        for (int i = lane; i < n; i += 32) sum += tile_range(s, lq, lkv, i).n + s.start;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == l) u = sum;
      }
      u *= s.hkv;
      if (DRAW && tiles > 0) {
        const int n = tile_range(s, qn, kv, tiles - 1).n + s.start;
        if (n > longest) longest = n;
      }
      all_tiles += __reduce_add_sync(~0u, tiles);
      long long inc = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += v;
      }
      if (b < p.batch) t.base[b] = units + inc - u;
      units += __shfl_sync(~0u, inc, 31);
    }
    if (lane == 0) t.base[p.batch] = units;
    __syncwarp();
    // no more workers than give each min_units, but two for each row tile: of
    // tiles that are not cut, ranges of less than one leave no worker two
    long long g = div_small(units, min_units);
    if (g < 2LL * all_tiles * s.hkv) g = 2LL * all_tiles * s.hkv;
    if (g < 1) g = 1;
    if (g > workers) g = workers;
    if (DRAW) longest = __reduce_max_sync(~0u, longest);
    if (lane == 0) {
      t.head[0] = units;
      t.head[1] = g;
      if (DRAW) {
        const long long all = (long long)all_tiles * s.hkv;
        t.head[4] = all >= 2 * workers && all < 1 << 30 && longest * 5 * workers <= 3 * units ? all : 0;
        t.head[5] = longest;
      }
    }
  }
  __syncthreads();
  W = t.head[0];
  G = t.head[1];
  u0 = u1 = 0;
  if (DRAW && t.head[4]) return;
  // The range's two ends, a warp each: the row tile that unit u falls into, and
  // the cut moved to an end of it if it is short.
  if (warp < 2) {
    long long u = c + warp;
    u = c < G ? (u < G ? div_small(u * W, G) : W) : 0;
    if (c < G && u < W) {
      int b = -1;  // the last sequence with base <= u
#pragma unroll 1
      for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int n = __popc(
            __ballot_sync(~0u, b0 + lane < p.batch && t.base[b0 + lane < p.batch ? b0 + lane : 0] <= u));
        b += n;
        if (n < 32) break;
      }
      const long long U = div_small(t.base[b + 1] - t.base[b], s.hkv);
      const long long r = u - t.base[b];
      int h = (int)div_small(r, U);
      long long off = r - h * U;
      int i = 0, cost = 0;
      const int qn = t.qn[b], kv = t.kv[b];
#pragma unroll 1
      for (;; i += 32) {
        // past the last row tile the ranges are not used: off ends before them
        const int n = tile_range(s, qn, kv, i + lane).n + s.start;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(~0u, sum, o);
          if (lane >= o) sum += v;
        }
        const unsigned past = __ballot_sync(~0u, (long long)sum > off);
        if (past) {
          const int l = __ffs(past) - 1;
          off -= __shfl_sync(~0u, sum - n, l);
          cost = __shfl_sync(~0u, n, l);
          i += l;
          break;
        }
        off -= __shfl_sync(~0u, sum, 31);
      }
      if (off > 0 && cost <= s.snap) {
        u -= off;
        if (2 * off >= cost) {  // to the next row tile
          u += cost;
          if (++i * s.tq >= qn) {
            i = 0;
            if (++h == s.hkv) {
              h = 0;
              do ++b;
              while (b < p.batch && t.qn[b] == 0);
            }
          }
        }
        off = 0;
      }
      if (warp == 0 && lane == 0) {
        t.loc[0] = b;
        t.loc[1] = h;
        t.loc[2] = i;
        t.loc[3] = (int)off;
      }
    }
    if (lane == 0) t.head[2 + warp] = u;
  }
  __syncthreads();
  u0 = t.head[2];
  u1 = t.head[3];
}

// The worker whose equal range of the W units has unit v.
__device__ __forceinline__ long long worker_of(long long v, long long W, long long G) {
  return div_small((v + 1) * G + W - 1, W) - 1;
}

// Walks this CTA's range segment by segment: a segment is the part of one row
// tile's key tiles that the CTA has. Every warp role walks the same sequence.
struct SplitWalk {
  const SplitShape& s;
  const SplitTables& t;
  long long u, u1;
  int b, h, i, off;     // position: sequence, head, row tile, unit in it
  // the current segment
  TileRange tr;
  int step;             // units of it
  int j, n;             // key tiles [j, j + n), n >= 1
  bool whole;           // covers its row tile
  __device__ SplitWalk(const SplitShape& s_, const SplitTables& t_, long long u0, long long u1_)
      : s(s_), t(t_), u(u0), u1(u1_), b(0), h(0), i(0), off(0) {
    if (u < u1) {
      b = t.loc[0];
      h = t.loc[1];
      i = t.loc[2];
      off = t.loc[3];
      load();
    }
  }
  __device__ bool more() const { return u < u1; }
  // instead of the range: all of one row tile, or nothing (b < 0)
  __device__ void jump(int b_, int h_, int i_) {
    u = 0;
    u1 = b_ < 0 ? 0 : 1ll << 62;
    if (b_ < 0) return;
    b = b_;
    h = h_;
    i = i_;
    off = 0;
    load();
  }
  __device__ void load() {
    tr = tile_range(s, t.qn[b], t.kv[b], i);
    const long long left = u1 - u;
    step = tr.n + s.start - off;
    if (left < step) step = (int)left;
    const int first = off > s.start ? off - s.start : 0;
    j = tr.j0 + first;
    n = off + step - s.start - first;
    whole = n == tr.n;
    if (n <= 0) u = u1;  // the range ends before this row tile's first key tile
  }
  // the unit of the current row tile's first key tile
  __device__ long long tile_unit() const { return u - off + s.start; }
  __device__ void next() {
    u += step;
    if (u >= u1) return;
    // the CTA's range goes on, so the row tile has ended
    off = 0;
    if (++i * s.tq >= t.qn[b]) {
      i = 0;
      if (++h == s.hkv) {
        h = 0;
        do ++b;
        while (t.qn[b] == 0);
      }
    }
    load();
  }
};

}  // namespace dg
