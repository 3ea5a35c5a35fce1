// k_attn.cu -- attention of a batch's new tokens over a paged cache for row
// tiles of up to 64 rows (decode, draft tokens, short chunks), on mma.sync.
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
// One producer warp brings key tiles of 64 positions (keys and values) into a
// ring of shared-memory stages by TMA, page by page. The 4*RT (2*RT at RT = 4)
// consumer warps split each tile's positions among them; every one keeps the
// running maximum, sum and output of its own positions in registers, so that
// the main loop has no barrier between warps, and they are joined once at the
// end of a segment. Work over all sequences is cut into equal ranges (see
// paged.cuh), so that one long sequence is shared by all SMs.
#include "launch.h"
#include "launch_util.cuh"
#include "paged.cuh"

namespace dg {

constexpr int kAttnKeys = 64;  // positions of a key tile
constexpr int kAttnKeysShift = 6;

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

template <int D, int RT>
struct AttnShape {
  static constexpr int kKS = RT == 4 ? 2 : 4;          // warps that share a row tile's positions
  static constexpr int kWarps = RT * kKS;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRows = 16 * RT;
  static constexpr int kHalf = kAttnKeys * 128;        // 64 columns of a tile's keys or values
  static constexpr int kKBytes = kAttnKeys * D * 2;
  static constexpr int kStage = 2 * kKBytes;
  static constexpr int kStages = 128 * 1024 / kStage;
  static constexpr int kLd = D + 8;                    // floats between rows of the join scratch
  static constexpr int kScratch = kWarps * 16 * kLd * 4 + kWarps * 16 * 8;
  static constexpr int kSlot = kRows * (D + 2);        // floats of a partial tile
  static int smem(int batch) {
    return 1024 + kStages * kStage + kScratch + 2 * kStages * 8 + 64 + SplitTables::bytes(batch) + 16;
  }
};

template <int D, int RT>
__global__ void __launch_bounds__(AttnShape<D, RT>::kThreads, 1)
    attn_mma_kernel(const __grid_constant__ CUtensorMap kvmap, const AttnArgs a) {
  using Sh = AttnShape<D, RT>;
  constexpr int kKS = Sh::kKS, kStages = Sh::kStages, kWarps = Sh::kWarps;
  constexpr int kCons = kWarps * 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* scratch = reinterpret_cast<float*>(smem + kStages * Sh::kStage);
  float* sc_ml = scratch + kWarps * 16 * Sh::kLd;  // [warp][16][m, l]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * Sh::kStage + Sh::kScratch);
  uint64_t* empty = full + kStages;
  // [0] abort [1] last [2], [3] segment number + 1 with a non-finite edge value
  volatile int* s_flag = reinterpret_cast<volatile int*>(empty + kStages);
  const SplitTables tab(reinterpret_cast<uint8_t*>(empty + kStages) + 64, a.p.batch);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    s_flag[0] = 0;
    s_flag[2] = s_flag[3] = 0;
    fence_mbar_init();
    prefetch_tmap(&kvmap);
  }
  griddep_launch_dependents();
  griddep_wait();
  long long W, G, u0, u1;
  split_setup<Sh::kThreads>(a.p, a.s, tab, a.min_units, W, G, u0, u1);
  SplitWalk w(a.s, tab, u0, u1);
  const int page_mask = a.p.page - 1;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    const uint64_t pol = policy_evict_first();
    // a tile is `pieces` boxes of `rows` positions, times keys/values, times
    // column halves: one lane each
    const int rows = a.p.page < kAttnKeys ? a.p.page : kAttnKeys;
    const int pieces = kAttnKeys / rows;
    const int half = lane % (D / 64), kvsel = (lane / (D / 64)) & 1, piece = lane / (D / 64 * 2);
    int it = 0;
    bool ok = true;
    for (; w.more() && ok; w.next()) {
      const int row = paged_row(a.p, w.b);
      const int32_t* trow = a.p.table + (long long)(row < 0 ? 0 : row) * a.p.table_stride;
      auto page_at = [&](int j) -> int {
        const int pos = j * kAttnKeys + piece * rows;
        if (piece >= pieces || pos >= w.tr.khi) return -1;
        const int pg = __ldg(trow + (pos >> a.p.page_shift));
        // a page that does not exist reads as zeros
        if ((pg < 0 || pg >= a.p.pages) && a.p.status) atomicOr(a.p.status, kStatusBounds);
        return pg < 0 || pg >= a.p.pages ? a.p.pages : pg;
      };
      int pg_next = page_at(w.j);
      for (int k = 0; k < w.n; ++k, ++it) {
        const int j = w.j + k, pg = pg_next;
        if (k + 1 < w.n) pg_next = page_at(j + 1);
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
                      &kvmap, half * 64, (j * kAttnKeys + piece * rows) & page_mask,
                      kvsel * a.p.hkv + w.h, pg, &full[st], pol);
      }
    }
    // the copies in flight land before the CTA's shared memory is given back
    if (lane == 0)
      for (int st = 0; st < kStages && st < it; ++st)
        mbar_wait(&full[st], ((it - st + kStages - 1) / kStages - 1) & 1, drain_ns(a.timeout_ns),
                  nullptr);
    return;
  }

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
      lo[e] = live && a.s.window > 0 ? pos0 + t - a.s.window + 1 : 0;
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

    for (int k = 0; k < w.n; ++k, ++it) {
      const int st = it % kStages, key0 = (w.j + k) * kAttnKeys;
      if (!s_flag[0] && !mbar_wait(&full[st], (it / kStages) & 1, a.timeout_ns, a.p.status))
        s_flag[0] = 1;
      const uint32_t kb = smem_u32(smem + st * Sh::kStage), vb = kb + Sh::kKBytes;
      const bool edge = er.in(key0, kAttnKeys);
#pragma unroll
      for (int blk = 0; blk < kAttnKeys / 16 / kKS; ++blk) {
        const int kr = (blk * kKS + ks) * 16;  // first position of this block in the tile
        if (key0 + kr >= w.tr.khi || key0 + kr + 16 <= w.tr.klo) continue;
        float s[2][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = 0.f;
        {
          // matrices: positions 0-7 / 8-15 (lane bit 4), column chunks 0 / 1 (bit 3)
          const int key = kr + (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b0, b1, b2, b3;
            const int chunk = (kk & 3) * 2 + ch;
            ldmatrix_x4(b0, b1, b2, b3,
                        kb + (kk >> 2) * Sh::kHalf + key * 128 + ((chunk ^ (key & 7)) << 4));
            mma_bf16_16816(s[0], qf[kk], b0, b1);
            mma_bf16_16816(s[1], qf[kk], b2, b3);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[t][e] *= a.c;  // before the mask: c may be 0 or negative
            const int key = key0 + kr + t * 8 + c0 + (e & 1);
            if (edge && (key > hi[e >> 1] || key < lo[e >> 1])) s[t][e] = -INFINITY;
          }
        float base[2];
        bool grew = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
          const float mn = fmaxf(m[e], mx);
          grew |= mn > m[e];
          base[e] = mn;
        }
        if (__any_sync(~0u, grew)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // a row that has seen nothing yet has o = l = 0 whatever the factor
            const float f = m[e] == -INFINITY ? 0.f : exp2_approx(m[e] - base[e]);
            m[e] = base[e];
            l[e] *= f;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              o[d][2 * e] *= f;
              o[d][2 * e + 1] *= f;
            }
          }
        }
        uint32_t pf[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mb = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float p0 = exp2_approx(s[t][2 * e] - mb);
            const float p1 = exp2_approx(s[t][2 * e + 1] - mb);
            l[e] += p0 + p1;
            // weights enter the product with the values as bf16: a relative
            // error of at most 2^-8 each, of the size of the output's own
            // rounding; the sum l takes them unrounded
            pf[t * 2 + e] = pack_bf16(p0, p1);
          }
        }
        if (edge) {
          // values that no row sees (the unused end of a page may hold
          // anything), and non-finite ones that only some rows see, become 0.
          // Warps of other row tiles may do the same to the same values.
          for (int x = lane; x < 16 * (D / 8); x += 32) {
            const int key = kr + x / (D / 8), ch = x % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(smem + st * Sh::kStage + Sh::kKBytes +
                                                 (ch >> 3) * Sh::kHalf + key * 128 +
                                                 (((ch & 7) ^ (key & 7)) << 4));
            found |= clean_edge_value(at, er, key0 + key);
          }
          fence_async_shared();
          __syncwarp();
        }
        {
          // matrices: positions 0-7 / 8-15 (lane bit 3), column chunks 0 / 1 (bit 4)
          const int key = kr + (lane & 15), ch = lane >> 4;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t b0, b1, b2, b3;
            const int chunk = (d & 3) * 2 + ch;
            ldmatrix_x4_trans(b0, b1, b2, b3,
                              vb + (d >> 2) * Sh::kHalf + key * 128 + ((chunk ^ (key & 7)) << 4));
            mma_bf16_16816(o[2 * d], pf, b0, b1);
            mma_bf16_16816(o[2 * d + 1], pf, b2, b3);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // join the warps that share this row tile's positions
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
    const bool aborted = s_flag[0] != 0;
    const bool poison = s_flag[2 + (seg & 1)] == seg + 1;
    const int ct = threadIdx.x;
    const long long c = blockIdx.x;
    const long long ut = w.tile_unit();
    // the tile's first CTA ends its range with it, the others begin with it
    const long long slot = c * 2 + (ut >= u0 ? 1 : 0);
    float* mine = a.ws + slot * Sh::kSlot;
    auto store = [&](int r, int d, float4 v, float mm, float ll) {
      const int t = r / a.group, g = r - t * a.group;
      const long long tok = q0 + t0 + t;
      const int head = w.h * a.group + g;
      const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);  // NaN stays NaN
      uint2 pk = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
      *reinterpret_cast<uint2*>(a.out + tok * a.ldo + (long long)head * D + d) = pk;
      if (a.lse && d == 0)
        a.lse[tok * a.hq + head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
    };
    for (int x = ct; x < rows * (D / 4); x += kCons) {
      const int r = x / (D / 4), d = (x % (D / 4)) * 4;
      const int wr = (r >> 4) * kKS, rr = r & 15;
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kKS; ++k) M = fmaxf(M, sc_ml[((wr + k) * 16 + rr) * 2]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int k = 0; k < kKS; ++k) {
        const float mk = sc_ml[((wr + k) * 16 + rr) * 2];
        const float f = M == -INFINITY ? 1.f : exp2_approx(mk - M);
        const float4 q4 =
            *reinterpret_cast<const float4*>(scratch + ((wr + k) * 16 + rr) * Sh::kLd + d);
        L += f * sc_ml[((wr + k) * 16 + rr) * 2 + 1];
        v.x += f * q4.x;
        v.y += f * q4.y;
        v.z += f * q4.z;
        v.w += f * q4.w;
      }
      if (poison) {
        const int t = r / a.group, p = pos0 + t;
        edge_values<D>(a.p, paged_row(a.p, w.b), w.h, er, a.s.window > 0 ? p - a.s.window + 1 : 0, p,
                       w.j * kAttnKeys, (w.j + w.n) * kAttnKeys, d, [&](const uint16_t* e) {
                         const uint2 pk = __ldg(reinterpret_cast<const uint2*>(e));
                         const float f[4] = {bf16lo(pk.x), bf16hi(pk.x), bf16lo(pk.y), bf16hi(pk.y)};
                         if (!isfinite(f[0])) v.x += f[0];
                         if (!isfinite(f[1])) v.y += f[1];
                         if (!isfinite(f[2])) v.z += f[2];
                         if (!isfinite(f[3])) v.w += f[3];
                       });
      }
      if (w.whole) {
        if (!aborted) store(r, d, v, M, L);
      } else {
        __stcg(reinterpret_cast<float4*>(DG_AT(a.p.status, mine, r * D + d, Sh::kSlot - 3)), v);
        if (d == 0)
          __stcg(reinterpret_cast<float2*>(mine + Sh::kRows * D + r * 2), make_float2(M, L));
      }
    }
    named_bar_sync(1, kCons);
    if (!w.whole) {
      const long long cf = cta_of(ut, W, G), cl = cta_of(ut + w.tr.n - 1, W, G);
      const int nc = (int)(cl - cf + 1);
      if (ct == 0) {
        // the tile's counter is its first CTA's (which is first for no other)
        int* cp = DG_AT(a.p.status, a.ctr, cf, a.ctr_len);
        const int old = atomic_add_acq_rel_gpu(cp, 1);
        const int last = old == nc - 1 ? 1 : 0;
        if (last) *cp = 0;
        s_flag[1] = last;
      }
      named_bar_sync(1, kCons);
      if (s_flag[1] && !aborted) {
        auto slot_of = [&](int k) -> const float* {
          return a.ws + ((cf + k) * 2 + (k == 0 ? 1 : 0)) * Sh::kSlot;
        };
        for (int x = ct; x < rows * (D / 4); x += kCons) {
          const int r = x / (D / 4), d = (x % (D / 4)) * 4;
          float M = -INFINITY;
          for (int k = 0; k < nc; ++k) M = fmaxf(M, __ldcg(slot_of(k) + Sh::kRows * D + r * 2));
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          float L = 0.f;
#pragma unroll 4
          for (int k = 0; k < nc; ++k) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(slot_of(k) + Sh::kRows * D + r * 2));
            const float4 q4 = __ldcg(reinterpret_cast<const float4*>(slot_of(k) + r * D + d));
            const float f = M == -INFINITY ? 1.f : exp2_approx(ml.x - M);
            L += f * ml.y;
            v.x += f * q4.x;
            v.y += f * q4.y;
            v.z += f * q4.z;
            v.w += f * q4.w;
          }
          store(r, d, v, M, L);
        }
      }
      named_bar_sync(1, kCons);
    }
  }
}

// ------------------------------------------------------------------ launch
template <int D, int RT>
static cudaError_t launch_rt(const Ctx& cx, const CUtensorMap& map, const AttnArgs& a, int grid) {
  using Sh = AttnShape<D, RT>;
  static DevOnce once;
  cudaError_t e = setup_smem(once, attn_mma_kernel<D, RT>, kMaxDynSmem);
  if (e != cudaSuccess) return e;
  return launch_k(attn_mma_kernel<D, RT>, dim3(grid), dim3(Sh::kThreads), Sh::smem(a.p.batch),
                  cx.stream, cx.pdl, map, a);
}

size_t attn_mma_ws(int dim, int rt, int sms) {
  return (size_t)sms * 2 * 16 * rt * (dim + 2) * sizeof(float);
}

cudaError_t launch_attn_mma(const Ctx& cx, const KvView& v, int rt, const AttnCall& c, float* ws,
                            int* ctr) {
  CUtensorMap map;
  if (!make_tmap_kv(&map, v, v.page < kAttnKeys ? v.page : kAttnKeys))
    return cudaErrorInvalidValue;
  AttnArgs a = {};
  a.p = paged_args(v, c.tokens, cx.status);
  a.group = c.hq / v.hkv;
  a.hq = c.hq;
  a.s.tq = 16 * rt / a.group;
  a.s.bn_shift = kAttnKeysShift;
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
  a.s.start = 3;
  a.min_units = 7;
  a.timeout_ns = cx.timeout_ns;
  const bool d64 = v.dim == 64;
  if (rt == 1) return d64 ? launch_rt<64, 1>(cx, map, a, cx.sms) : launch_rt<128, 1>(cx, map, a, cx.sms);
  if (rt == 2) return d64 ? launch_rt<64, 2>(cx, map, a, cx.sms) : launch_rt<128, 2>(cx, map, a, cx.sms);
  return d64 ? launch_rt<64, 4>(cx, map, a, cx.sms) : launch_rt<128, 4>(cx, map, a, cx.sms);
}

}  // namespace dg
