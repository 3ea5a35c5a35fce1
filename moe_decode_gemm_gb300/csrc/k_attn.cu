// k_attn.cu -- attention of a batch's new tokens over a paged cache in row
// tiles of up to 32 rows (decode, a few draft tokens), on mma.sync.
//
//   s_j = scale * q·k_j,  p_j = exp(s_j - m),  o = sum_j p_j v_j / sum_j p_j,
//   lse = m + log sum_j p_j      over the positions j that a token sees:
//   j <= its own position, and within `window` of it when a window is given.
//
// The rows of a tile are (token, query head) pairs that share a key head, so
// each key and value is read from memory once per tile: with 14 query heads
// per key head one token is a tile of 14 rows. At one token per sequence a
// call reads 4*dim bytes per position and does 4*dim*14 flops on them: bound by
// memory, and the matrix instructions only have to keep up with it.
//
// One producer warp brings key tiles of 64 positions (128 of small heads; keys
// and values, 32 KB) into a ring of shared-memory stages by TMA, page by page.
// Four or eight consumer warps split the row tile (16 rows a warp) and each
// tile's positions; every one keeps the running maximum, sum and output of its
// own positions in registers, so that the main loop has no barrier between
// warps, and they are joined once at the end of a segment. Work over all
// sequences is cut into equal ranges (see paged.cuh), so that one long sequence
// is shared by all SMs; with up to 16 row tiles the ranges are clusters' of 8
// CTAs, which join their parts through distributed shared memory (one token
// over 509 positions 12 -> 7.5 us).
//
// Measured (56 query and 4 key heads of 128): 64 sequences of 2k to 32k
// positions, 1.65 GB of keys and values, 240 us = 6.9 TB/s, what a copy reaches;
// 11 sequences of 1.3k to 18k positions 28 us (27 of it their bytes). One token
// over 509 positions 7.1 us, latency: about 0.3 us until the call before is
// done, 2 for the lengths and the split, 1.5 until the queries and first keys
// are there, 1 of work, 1.5 for joining and the output. A key tile that is there
// takes a warp 0.6 to 0.7 us, one with places to mask 0.4 us more.
#include "launch.h"
#include "launch_util.cuh"
#include "paged.cuh"

namespace dg {

constexpr int attn_keys_shift(int dim) { return dim == 64 ? 7 : 6; }
constexpr int kClusterTiles = 16;   // row tiles up to which clusters are used

struct AttnArgs {
  PagedArgs p;
  SplitShape s;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  long long ldq, ldo;
  int group, hq;       // query heads per key head, query heads
  float c;             // scale * log2(e): scores in units of powers of two
  float* ws;
  int* ctr;
  long long ws_len;
  int ctr_len;
  int min_units;
  long long timeout_ns;
};

template <int D, int RT, int CL>
struct AttnShape {
  static constexpr int kKeys = 1 << attn_keys_shift(D);  // positions of a key tile: 16 KB of keys
  // warps that share a row tile's positions: 8 warps of 32 positions for two row
  // tiles of 64 columns; of 128 columns the registers allow 4 warps
  static constexpr int kKS = RT == 2 && D == 128 ? 2 : 4;
  static constexpr int kBlk = kKeys / kKS;             // positions of a warp at a time: 16 or 32
  static constexpr int kWarps = RT * kKS;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRows = 16 * RT;
  static constexpr int kHalf = kKeys * 128;        // 64 columns of a tile's keys or values
  static constexpr int kKBytes = kKeys * D * 2;
  static constexpr int kStage = 2 * kKBytes;
  static constexpr int kStages = (CL > 1 ? 96 : 128) * 1024 / kStage;
  static constexpr int kLd = D + 8;                    // floats between rows of the join scratch
  // Rows of 128 columns have their factors over the warps looked up (22 sequences
  // of 100 to 300 positions 9.8 -> 9.2 us); for those of 64, and for the parts of a
  // cluster, the barrier that takes costs more (12.7 -> 13.2, 7.2 -> 7.5).
  static constexpr bool kFactors = D == 128 && CL == 1;
  // o; m and l (or a warp's factor) of each warp's rows; of each row m, l and 1 / l
  static constexpr int kScratch =
      kWarps * 16 * kLd * 4 + kWarps * 16 * 8 + (kFactors ? kRows * 16 : 0);
  static constexpr int kItems = kRows * (D / 4);       // four columns of a row each
  static constexpr int kSlot = kItems * 6;             // floats of a partial tile: o, then m and l
  static constexpr int kMerged = CL > 1 ? kRows * (D + 2) * 4 : 0;  // a CTA's part of a cluster's tile
  static int smem(int batch) {
    return 1024 + kStages * kStage + kScratch + 2 * kMerged + (2 * kStages + 1) * 8 + 64 +
           SplitTables::bytes(batch) + 16;
  }
};

// Joins two partial softmax states (v, m, l): exact but for the rounding of the
// factors; a state that has seen nothing (m = -inf) changes nothing.
struct State {
  float4 v;
  float m, l;
  __device__ void add(float4 v2, float m2, float l2) {
    const float M = fmaxf(m, m2);
    const float f = M == -INFINITY ? 1.f : exp2_approx(m - M);
    const float g = M == -INFINITY ? 1.f : exp2_approx(m2 - M);
    v.x = v.x * f + v2.x * g;
    v.y = v.y * f + v2.y * g;
    v.z = v.z * f + v2.z * g;
    v.w = v.w * f + v2.w * g;
    l = l * f + l2 * g;
    m = M;
  }
};

// Adds the non-finite values at the edge that row r (at position pos) sees, in
// columns d .. d + 3 of this CTA's key tiles, to the part of the warp that had
// them (out of line: it hardly ever runs).
template <int D, int KEYS, int BLK, int KS>
__device__ __noinline__ void add_edge_values(const PagedArgs& p, int window, int b, int h,
                                             const EdgeRange& er, int pos, int j, int n, int rank,
                                             int step, int r, int d, float* scratch) {
  for (int k = rank; k < n; k += step)
    edge_values<D>(p, paged_row(p, b), h, er, first_seen(window, pos), pos, (j + k) * KEYS,
                   (j + k + 1) * KEYS, d, [&](const uint16_t* e, int key) {
                     const int row = ((r >> 4) * KS + key % KEYS / BLK) * 16 + (r & 15);
                     float* o = scratch + row * (D + 8) + d;
                     for (int c = 0; c < 4; ++c) {
                       const float f = bf_bits2f(__ldg(e + c));
                       if (!isfinite(f)) o[c] += f;
                     }
                   });
}

template <int D, int RT, int CL>
__global__ void __launch_bounds__(AttnShape<D, RT, CL>::kThreads, 1)
    attn_mma_kernel(const __grid_constant__ CUtensorMap kvmap, const AttnArgs a) {
  using Sh = AttnShape<D, RT, CL>;
  constexpr int kKS = Sh::kKS, kStages = Sh::kStages, kWarps = Sh::kWarps;
  constexpr int kCons = kWarps * 32;
  constexpr int kKeys = Sh::kKeys, kBlk = Sh::kBlk;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* scratch = reinterpret_cast<float*>(smem + kStages * Sh::kStage);
  float* sc_ml = scratch + kWarps * 16 * Sh::kLd;  // [warp][16][m, l]
  float4* sc_row = reinterpret_cast<float4*>(sc_ml + kWarps * 16 * 2);  // [row] m, l, 1 / l
  // [2] this CTA's part of a tile for its cluster: o [row][D], then m and l [row]
  float* merged = reinterpret_cast<float*>(smem + kStages * Sh::kStage + Sh::kScratch);
  uint64_t* full =
      reinterpret_cast<uint64_t*>(smem + kStages * Sh::kStage + Sh::kScratch + 2 * Sh::kMerged);
  uint64_t* empty = full + kStages;
  uint64_t* peers = empty + kStages;   // every CTA of the cluster has written its part
  // [0] abort [1] last [2], [3] segment number + 1 with a non-finite edge value
  volatile int* s_flag = reinterpret_cast<volatile int*>(peers + 1);
  const SplitTables tab(reinterpret_cast<uint8_t*>(peers + 1) + 64, a.p.batch);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    mbar_init(peers, CL);
    s_flag[0] = 0;
    s_flag[2] = s_flag[3] = 0;
    fence_mbar_init();
    prefetch_tmap(&kvmap);
  }
  griddep_launch_dependents();
  if (CL > 1) {  // the barriers of all its CTAs are set up
    __syncwarp();
    cluster_arrive_all();
  }
  griddep_wait();
  long long W, G, u0, u1;
  const long long worker = blockIdx.x / CL;
  const int rank = CL > 1 ? (int)cluster_rank() : 0;
  split_setup<false>(a.p, a.s, tab, a.min_units, worker, gridDim.x / CL, W, G, u0, u1);
  if (CL > 1) cluster_wait_all();
  SplitWalk w(a.s, tab, u0, u1);
  const int page_mask = a.p.page - 1;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    const uint64_t pol = policy_evict_first();
    // a tile is `pieces` boxes of `rows` positions, times keys/values, times
    // column halves: one lane each
    const int rows = a.p.page < kKeys ? a.p.page : kKeys;
    const int pieces = kKeys / rows;
    const int half = lane % (D / 64), kvsel = (lane / (D / 64)) & 1, piece = lane / (D / 64 * 2);
    int it = 0;
    bool ok = true;
    for (; w.more() && ok; w.next()) {
      const int row = paged_row(a.p, w.b);
      const int32_t* trow = a.p.table + (long long)(row < 0 ? 0 : row) * a.p.table_stride;
      auto page_at = [&](int j) -> int {
        // (pages that no row sees are not looked up: a window may have left them)
        const int pos = j * kKeys + piece * rows;
        if (piece >= pieces || pos >= w.tr.khi || pos + rows <= w.tr.klo) return -1;
        const int pg = __ldg(trow + (pos >> a.p.page_shift));
        // a page that does not exist reads as zeros
        if ((pg < 0 || pg >= a.p.pages) && a.p.status) atomicOr(a.p.status, kStatusBounds);
        return pg < 0 || pg >= a.p.pages ? a.p.pages : pg;
      };
      int pg_next = rank < w.n ? page_at(w.j + rank) : -1;
      for (int k = rank; k < w.n; k += CL, ++it) {
        const int j = w.j + k, pg = pg_next;
        if (k + CL < w.n) pg_next = page_at(j + CL);
        const int st = it % kStages;
        if (it >= kStages && !mbar_wait(&empty[st], ((it / kStages) + 1) & 1, a.timeout_ns, a.p.status))
          s_flag[0] = 1;
        __syncwarp();
        if (s_flag[0]) {
          ok = false;
          break;
        }
        const int n = __popc(__ballot_sync(~0u, pg >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], n * rows * 128);
        __syncwarp();
        if (pg >= 0)
          tma_load_4d(smem + st * Sh::kStage + kvsel * Sh::kKBytes + half * Sh::kHalf +
                          piece * rows * 128,
                      &kvmap, half * 64, (j * kKeys + piece * rows) & page_mask,
                      kvsel * a.p.hkv + w.h, pg, &full[st], pol);
      }
    }
    // the copies in flight land before the CTA's shared memory is given back
    if (lane == 0)
      for (int st = 0; st < kStages && st < it; ++st)
        mbar_wait(&full[st], ((it - st + kStages - 1) / kStages - 1) & 1, drain_ns(a.timeout_ns),
                  nullptr);
    __syncwarp();
  } else {
  // ------------------------------------------------------------------ consumers
  const int rt = warp / kKS, ks = warp % kKS;   // row tile of 16, share of the positions
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  int it = 0, seg = 0;
  for (; w.more(); w.next(), ++seg) {
    const int qn = tab.qn[w.b], kv = tab.kv[w.b];
    const int q0 = paged_first(a.p, w.b), t0 = w.i * a.s.tq;
    const int nt = qn - t0 < a.s.tq ? qn - t0 : a.s.tq;
    const int rows = nt * a.group;
    const int pos0 = kv - qn + t0;               // position of the tile's first token
    // the two rows of this thread: query fragments and the positions they see
    uint32_t qf[D / 16][4];
    int hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = rt * 16 + r0 + e * 8;
      const bool live = r < rows;
      const int t = live ? r / a.group : 0;
      const uint16_t* src = a.q + (long long)(q0 + t0 + t) * a.ldq +
                            (long long)(w.h * a.group + (live ? r - t * a.group : 0)) * D;
      hi[e] = live ? pos0 + t : -1;
      lo[e] = live ? first_seen(a.s.window, pos0 + t) : 0;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][e] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + c0)) : 0u;
        qf[kk][e + 2] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + c0)) : 0u;
      }
    }
    const EdgeRange er = edge_range(a.s, w.tr, pos0, nt);
    bool found = false;  // a non-finite value that only some rows see
    float o[D / 8][4];
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int k = rank; k < w.n; k += CL, ++it) {
      const int st = it % kStages, key0 = (w.j + k) * kKeys;
      if (!mbar_try_wait(&full[st], (it / kStages) & 1) && !s_flag[0] &&
          !mbar_wait(&full[st], (it / kStages) & 1, a.timeout_ns, a.p.status))
        s_flag[0] = 1;
      const uint32_t kb = smem_u32(smem + st * Sh::kStage), vb = kb + Sh::kKBytes;
      const bool edge = er.in(key0, kKeys);
      const int kr = ks * kBlk;  // first position of this warp in the tile
      if (key0 + kr < w.tr.khi && key0 + kr + kBlk > w.tr.klo) {
        float s[kBlk / 8][4];
#pragma unroll
        for (int t = 0; t < kBlk / 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
        {
          // matrices: positions 0-7 / 8-15 (lane bit 4), column chunks 0 / 1 (bit 3)
          const int key = kr + (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int chunk = (kk & 3) * 2 + ch;
#pragma unroll
            for (int t = 0; t < kBlk / 16; ++t) {
              uint32_t b0, b1, b2, b3;
              ldmatrix_x4(b0, b1, b2, b3, kb + (kk >> 2) * Sh::kHalf + (key + t * 16) * 128 +
                                              ((chunk ^ (key & 7)) << 4));
              mma_bf16_16816(s[2 * t], qf[kk], b0, b1);
              mma_bf16_16816(s[2 * t + 1], qf[kk], b2, b3);
            }
          }
        }
        if (edge) {
          // values that no row sees (the unused end of a page may hold
          // anything), and non-finite ones that only some rows see, become 0.
          // Warps of other row tiles may do the same to the same values.
          auto within = [&](int pos) {
            const int n = pos - key0;
            return n < kr ? kr : (n > kr + kBlk ? kr + kBlk : n);
          };
          auto at = [&](int x) {  // 8 values: x / (D / 8) positions into the tile
            const int key = x / (D / 8), ch = x % (D / 8);
            return reinterpret_cast<uint4*>(smem + st * Sh::kStage + Sh::kKBytes +
                                            (ch >> 3) * Sh::kHalf + key * 128 +
                                            (((ch & 7) ^ (key & 7)) << 4));
          };
          const int seen0 = within(er.klo), seen1 = within(er.khi);
          // before and past what is seen; then what not all rows see
#pragma unroll 1
          for (int side = 0; side < 2; ++side) {
            const int from = side ? (seen1 > seen0 ? seen1 : seen0) : kr, to = side ? kr + kBlk : seen0;
#pragma unroll 1
            for (int x = from * (D / 8) + lane; x < to * (D / 8); x += 32)
              *at(x) = make_uint4(0, 0, 0, 0);
            const int some0 =
                side ? within(er.all_hi > er.all_lo ? er.all_hi : er.all_lo) : seen0;
            const int some1 = side ? seen1 : within(er.all_lo < er.khi ? er.all_lo : er.khi);
#pragma unroll 1
            for (int x = some0 * (D / 8) + lane; x < some1 * (D / 8); x += 32)
              found |= clean_edge_value(at(x), er, key0 + x / (D / 8));
          }
          fence_async_shared();
          __syncwarp();
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < kBlk / 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] *= a.c;  // before the mask: c may be 0 or negative
        if (edge)
#pragma unroll
          for (int t = 0; t < kBlk / 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + kr + t * 8 + c0 + (e & 1);
              if (key > hi[e >> 1] || key < lo[e >> 1]) s[t][e] = -INFINITY;
            }
#pragma unroll
        for (int t = 0; t < kBlk / 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[t][e]);
        bool grew = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(~0u, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(~0u, mx[e], 2));
          grew |= mx[e] > m[e];
        }
        if (__any_sync(~0u, grew)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // a row that has seen nothing yet has o = l = 0 whatever the factor
            const float mn = fmaxf(m[e], mx[e]);
            const float f = m[e] == -INFINITY ? 0.f : exp2_approx(m[e] - mn);
            m[e] = mn;
            l[e] *= f;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              o[d][2 * e] *= f;
              o[d][2 * e + 1] *= f;
            }
          }
        }
        uint32_t pf[kBlk / 16][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mb = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
          for (int t = 0; t < kBlk / 8; ++t) {
            const float p0 = exp2_approx(s[t][2 * e] - mb);
            const float p1 = exp2_approx(s[t][2 * e + 1] - mb);
            l[e] += p0 + p1;
            // weights enter the product with the values as bf16: a relative
            // error of at most 2^-8 each, of the size of the output's own
            // rounding; the sum l takes them unrounded
            pf[t / 2][(t & 1) * 2 + e] = pack_bf16(p0, p1);
          }
        }
        {
          // matrices: positions 0-7 / 8-15 (lane bit 3), column chunks 0 / 1 (bit 4)
          const int key = kr + (lane & 15), ch = lane >> 4;
#pragma unroll
          for (int t = 0; t < kBlk / 16; ++t)
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              uint32_t b0, b1, b2, b3;
              const int chunk = (d & 3) * 2 + ch;
              ldmatrix_x4_trans(b0, b1, b2, b3, vb + (d >> 2) * Sh::kHalf + (key + t * 16) * 128 +
                                                    ((chunk ^ (key & 7)) << 4));
              mma_bf16_16816(o[2 * d], pf[t], b0, b1);
              mma_bf16_16816(o[2 * d + 1], pf[t], b2, b3);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // the warps' parts to shared memory
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(~0u, l[e], 1);
      l[e] += __shfl_xor_sync(~0u, l[e], 2);
      if ((lane & 3) == 0) {
        sc_ml[(warp * 16 + r0 + e * 8) * 2] = m[e];
        sc_ml[(warp * 16 + r0 + e * 8) * 2 + 1] = l[e];
      }
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        *reinterpret_cast<float2*>(scratch + (warp * 16 + r0 + e * 8) * Sh::kLd + d * 8 + c0) =
            make_float2(o[d][2 * e], o[d][2 * e + 1]);
    }
    if (found) s_flag[2 + (seg & 1)] = seg + 1;
    named_bar_sync(1, kCons);
    const int ct = threadIdx.x, items = rows * (D / 4);
    if (s_flag[2 + (seg & 1)] == seg + 1) {
      for (int x = ct; x < items; x += kCons)
        add_edge_values<D, kKeys, kBlk, kKS>(a.p, a.s.window, w.b, w.h, er,
                                             pos0 + x / (D / 4) / a.group, w.j, w.n, rank, CL,
                                             x / (D / 4), (x % (D / 4)) * 4, scratch);
      named_bar_sync(1, kCons);
    }
    const bool aborted = s_flag[0] != 0;
    const long long ut = w.tile_unit();
    auto inverse = [](float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); };  // NaN stays NaN
    auto store_lse = [&](int r, float m, float l) {
      const int t = r / a.group, g = r - t * a.group;
      if (a.lse)
        a.lse[(long long)(q0 + t0 + t) * a.hq + w.h * a.group + g] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    };
    auto store = [&](int r, int d, const State& s, float inv, bool lse) {
      const int t = r / a.group, g = r - t * a.group;
      *reinterpret_cast<uint2*>(a.out + (long long)(q0 + t0 + t) * a.ldo +
                                (long long)(w.h * a.group + g) * D + d) =
          make_uint2(pack_bf16(s.v.x * inv, s.v.y * inv), pack_bf16(s.v.z * inv, s.v.w * inv));
      if (lse && d == 0) store_lse(r, s.m, s.l);
    };
    // a row's part of warp k of those that share it
    auto part_at = [&](int r, int k) { return (r >> 4) * kKS * 16 + (r & 15) + k * 16; };
    // a row's maximum and sum over its warps, and the warps' factors
    auto row_state = [&](int r, float* f) -> float2 {
      float2 ml[kKS];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int k = 0; k < kKS; ++k) {
        ml[k] = *reinterpret_cast<const float2*>(sc_ml + part_at(r, k) * 2);
        M = fmaxf(M, ml[k].x);
      }
#pragma unroll
      for (int k = 0; k < kKS; ++k) {
        f[k] = M == -INFINITY ? 1.f : exp2_approx(ml[k].x - M);
        L += f[k] * ml[k].y;
      }
      return make_float2(M, L);
    };
    if (Sh::kFactors) {
      if (ct < rows) {
        float f[kKS];
        const float2 ml = row_state(ct, f);
#pragma unroll
        for (int k = 0; k < kKS; ++k) sc_ml[part_at(ct, k) * 2] = f[k];
        sc_row[ct] = make_float4(ml.x, ml.y, inverse(ml.y), 0.f);
        if (w.whole && !aborted) store_lse(ct, ml.x, ml.y);
      }
      named_bar_sync(1, kCons);
    }
    // four columns of a row over the warps that share the row tile
    auto own = [&](int r, int d) -> State {
      State s = {make_float4(0.f, 0.f, 0.f, 0.f), 0.f, 0.f};
      float f[kKS];
      if (Sh::kFactors) {
        const float4 row = sc_row[r];
        s.m = row.x, s.l = row.y;
#pragma unroll
        for (int k = 0; k < kKS; ++k) f[k] = sc_ml[part_at(r, k) * 2];
      } else {
        const float2 ml = row_state(r, f);
        s.m = ml.x, s.l = ml.y;
      }
#pragma unroll
      for (int k = 0; k < kKS; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(scratch + part_at(r, k) * Sh::kLd + d);
        s.v.x += f[k] * v.x;
        s.v.y += f[k] * v.y;
        s.v.z += f[k] * v.z;
        s.v.w += f[k] * v.w;
      }
      return s;
    };
    // A tile shared with other workers: its first one ends its range with it
    // (slot 1), the others begin with it (slot 0). The CTAs of rank r of each
    // see to the same columns, so that the last of them joins these.
    auto slot_of = [&](long long c, bool first) { return a.ws + (c * 2 + (first ? 1 : 0)) * Sh::kSlot; };
    float* mine = slot_of(worker, ut >= u0);
    auto put = [&](int x, const State& s, float inv, bool lse) {
      if (w.whole) {
        if (!aborted) store(x / (D / 4), (x % (D / 4)) * 4, s, inv, lse);
      } else {
        __stcg(reinterpret_cast<float4*>(DG_AT(a.p.status, mine, x * 4, Sh::kSlot - 3)), s.v);
        __stcg(reinterpret_cast<float2*>(mine + Sh::kItems * 4 + x * 2), make_float2(s.m, s.l));
      }
    };
    // In a cluster this CTA's part goes to shared memory first. Two buffers:
    // whoever writes one again has seen every CTA arrive for the other, after
    // reading this one.
    float* buf = merged + (seg & 1) * (Sh::kMerged / 4);
    constexpr int kBatch = 4;  // items whose loads are in flight together
#pragma unroll 1
    for (int x0 = ct; x0 < items; x0 += kBatch * kCons) {
      State s[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int x = x0 + q * kCons < items ? x0 + q * kCons : x0;
        s[q] = own(x / (D / 4), (x % (D / 4)) * 4);
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int x = x0 + q * kCons, r = x / (D / 4), d = (x % (D / 4)) * 4;
        if (x >= items) break;
        if (CL == 1) {
          put(x, s[q], Sh::kFactors ? sc_row[r].z : inverse(s[q].l), !Sh::kFactors);
        } else {
          *reinterpret_cast<float4*>(buf + r * D + d) = s[q].v;
          if (d == 0)
            *reinterpret_cast<float2*>(buf + Sh::kRows * D + r * 2) = make_float2(s[q].m, s[q].l);
        }
      }
    }
    // the items this CTA sees to: in a cluster one run of them, joined over all
    // its CTAs, two lanes to an item with half of the CTAs each
    const int per = CL > 1 ? (items + CL - 1) / CL : items;
    const int first = rank * per, last = first + per < items ? first + per : items;
    if (CL > 1) {
      named_bar_sync(1, kCons);
      if (ct < CL) mbar_arrive_remote(peers, ct);
      if (!mbar_wait_cluster(peers, seg & 1, a.timeout_ns, a.p.status)) s_flag[0] = 1;
#pragma unroll 1
      for (int x0 = first; x0 < last; x0 += kCons / 2) {
        const int x = x0 + ct / 2, xr = x < last ? x : first;
        const int r = xr / (D / 4), d = (xr % (D / 4)) * 4;
        float4 v[CL / 2 + 1];
        float2 ml[CL / 2 + 1];
#pragma unroll
        for (int k = 0; k < CL / 2; ++k) {
          const uint32_t cta = (ct & 1) * (CL / 2) + k;
          v[k] = ld_dsmem_f32x4(buf + r * D + d, cta);
          ml[k] = ld_dsmem_f32x2(buf + Sh::kRows * D + r * 2, cta);
        }
        State s = {v[0], ml[0].x, ml[0].y};
#pragma unroll
        for (int k = 1; k < CL / 2; ++k) s.add(v[k], ml[k].x, ml[k].y);
        const float4 v2 = make_float4(__shfl_xor_sync(~0u, s.v.x, 1), __shfl_xor_sync(~0u, s.v.y, 1),
                                      __shfl_xor_sync(~0u, s.v.z, 1), __shfl_xor_sync(~0u, s.v.w, 1));
        const float m2 = __shfl_xor_sync(~0u, s.m, 1), l2 = __shfl_xor_sync(~0u, s.l, 1);
        if (x >= last || (ct & 1)) continue;
        s.add(v2, m2, l2);
        put(x, s, inverse(s.l), true);
      }
    }
    if (w.whole) {
      named_bar_sync(1, kCons);
      continue;
    }
    named_bar_sync(1, kCons);
    const long long cf = worker_of(ut, W, G);
    const int nc = (int)(worker_of(ut + w.tr.n - 1, W, G) - cf + 1);
    if (ct == 0) {
      // the tile's counters are its first worker's (which is first for no other)
      int* cp = DG_AT(a.p.status, a.ctr, cf * CL + rank, a.ctr_len);
      const int old = atomic_add_acq_rel_gpu(cp, 1);
      const int last = old == nc - 1 ? 1 : 0;
      if (last) *cp = 0;
      s_flag[1] = last;
    }
    named_bar_sync(1, kCons);
    if (s_flag[1] && !aborted) {
      // parts, and items of each, whose loads are in flight together (two items
      // where the registers last: 11 sequences 31.2 -> 27.8 us)
      constexpr int kAhead = 4, kItemsAhead = kWarps > 4 ? 1 : 2;
#pragma unroll 1
      for (int x0 = first + ct; x0 < last; x0 += kItemsAhead * kCons) {
        State s[kItemsAhead];
#pragma unroll
        for (int i = 0; i < kItemsAhead; ++i) s[i] = {make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
#pragma unroll 1
        for (int k0 = 0; k0 < nc; k0 += kAhead) {
          float4 v[kItemsAhead][kAhead];
          float2 ml[kItemsAhead][kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (k0 + k < nc) {
              const float* p = slot_of(cf + k0 + k, k0 + k == 0);
#pragma unroll
              for (int i = 0; i < kItemsAhead; ++i) {
                const int x = x0 + i * kCons < last ? x0 + i * kCons : x0;
                v[i][k] = __ldcg(reinterpret_cast<const float4*>(p + x * 4));
                ml[i][k] = __ldcg(reinterpret_cast<const float2*>(p + Sh::kItems * 4 + x * 2));
              }
            }
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (k0 + k < nc)
#pragma unroll
              for (int i = 0; i < kItemsAhead; ++i) s[i].add(v[i][k], ml[i][k].x, ml[i][k].y);
        }
#pragma unroll
        for (int i = 0; i < kItemsAhead; ++i) {
          const int x = x0 + i * kCons;
          if (x < last) store(x / (D / 4), (x % (D / 4)) * 4, s[i], inverse(s[i].l), true);
        }
      }
    }
    named_bar_sync(1, kCons);
  }
  }
  if (CL > 1) cluster_sync_all();  // no CTA ends while another may read its part
}

// ------------------------------------------------------------------ launch
// Clusters of the kernel that fit on the device at once (0: none).
template <int D, int RT, int CL>
static int clusters_at_once(int smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL);
  cfg.blockDim = dim3(AttnShape<D, RT, CL>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {CL, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, attn_mma_kernel<D, RT, CL>, &cfg) == cudaSuccess ? n : 0;
}

template <int D, int RT, int CL>
static cudaError_t launch_rt(const Ctx& cx, const CUtensorMap& map, const AttnArgs& a) {
  using Sh = AttnShape<D, RT, CL>;
  static DevOnce once;
  cudaError_t e = setup_smem(once, attn_mma_kernel<D, RT, CL>, kMaxDynSmem);
  if (e != cudaSuccess) return e;
  if (CL == 1)
    return launch_k(attn_mma_kernel<D, RT, CL>, dim3(cx.sms), dim3(Sh::kThreads),
                    Sh::smem(a.p.batch), cx.stream, cx.pdl, map, a);
  static DevOnce asked;
  static int at_once[64];
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  int n = 0;
  if (dev < 64) {
    e = asked.run([&]() -> cudaError_t {
      at_once[dev] = clusters_at_once<D, RT, CL>(Sh::smem(kMaxBatch));
      return cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    n = at_once[dev];
  }
  if (n < 1) n = 1;
  if (n > cx.sms / CL) n = cx.sms / CL;
  return launch_kc(attn_mma_kernel<D, RT, CL>, dim3(n * CL), dim3(Sh::kThreads),
                   Sh::smem(a.p.batch), cx.stream, cx.pdl, CL, map, a);
}

size_t attn_mma_ws(int dim, int rt, int sms) {
  return (size_t)sms * 2 * 16 * rt * (dim / 4) * 6 * sizeof(float);
}

cudaError_t launch_attn_mma(const Ctx& cx, const KvView& v, int rt, const AttnCall& c, float* ws,
                            int* ctr) {
  CUtensorMap map;
  const int keys = 1 << attn_keys_shift(v.dim);
  if (!make_tmap_kv(&map, v, v.page < keys ? v.page : keys))
    return cudaErrorInvalidValue;
  AttnArgs a = {};
  a.p = paged_args(v, c.tokens, cx.status);
  a.group = c.hq / v.hkv;
  a.hq = c.hq;
  a.s.tq = 16 * rt / a.group;
  a.s.bn_shift = attn_keys_shift(v.dim);
  a.s.window = c.window;
  a.s.hkv = v.hkv;
  a.q = static_cast<const uint16_t*>(c.q);
  a.out = static_cast<uint16_t*>(c.out);
  a.lse = c.lse;
  a.ldq = c.ldq;
  a.ldo = c.ldo;
  a.c = c.scale * 1.4426950408889634f;
  a.ws = ws;
  a.ctr = ctr;
  a.ws_len = cx.ws_len;
  a.ctr_len = (int)cx.ctr_len;
  a.s.start = 4;
  a.s.snap = 20;
  a.min_units = 8;
  a.timeout_ns = cx.timeout_ns;
  const bool d64 = v.dim == 64;
  // Few row tiles: a cluster of 8 CTAs for each part of one, so that the parts
  // are joined through distributed shared memory and only a few partial tiles
  // go through the workspace. Its key tiles are read 8 at a time, so that what
  // a row tile costs at its start weighs 8 times as many.
  const long long tiles =
      (c.max_q > 0 && c.max_q <= a.s.tq ? v.batch : (long long)c.tokens / a.s.tq + v.batch) * v.hkv;
  if (tiles <= kClusterTiles) {
    a.s.start = 40;
    a.s.snap = 100;
    a.min_units = 96;
  }
  if (rt == 1 && tiles <= kClusterTiles)
    return d64 ? launch_rt<64, 1, 8>(cx, map, a) : launch_rt<128, 1, 8>(cx, map, a);
  if (tiles <= kClusterTiles)
    return d64 ? launch_rt<64, 2, 8>(cx, map, a) : launch_rt<128, 2, 8>(cx, map, a);
  if (rt == 1) return d64 ? launch_rt<64, 1, 1>(cx, map, a) : launch_rt<128, 1, 1>(cx, map, a);
  return d64 ? launch_rt<64, 2, 1>(cx, map, a) : launch_rt<128, 2, 1>(cx, map, a);
}

}  // namespace dg
