// k_kv.cu -- what goes into a paged cache and how its pages are managed: the
// norm and rotation of a step's queries and keys with the append of its keys
// and values, and the calls that change, fork, copy and compact the pages of
// a cache of several layers.
#include "launch.h"
#include "launch_util.cuh"
#include "paged.cuh"

namespace dg {

// ------------------------------------------------------------------ append
//   y = x * rsqrt(mean(x^2) + eps) * w    per query and key head (w: wq or wk)
//   (a, c) -> (a cos - c sin, c cos + a sin)   on the head's first rot elements,
//   pairs (i, i + rot/2), or (2i, 2i + 1) interleaved
// in fp32, rounded once to bf16; values are copied. Queries go to q, keys and
// values to the places of their positions in the cache. Each head is read and
// written once: bound by memory at many tokens, by the latency of one chain of
// dependent loads (sequence, page, row of angles) at few.
//
// D/8 lanes hold a head, 8 elements each, so that the sum of squares is a few
// shuffles and a pair's other half is in this lane or one shuffle away. A CTA
// has one token's heads, or some of them: where the token goes and its angles
// are looked up once, and a lane keeps the angles and weights of its elements
// for all its heads. (Heads of any token on any lane, each with its own places
// and angles, took twice the instructions and were bound by them: 80 us for
// 7.9k tokens of 64 heads of 128.)
//
// Measured: those 7.9k tokens, half of each head rotated, 262 MB in 49 us =
// 5.3 TB/s, 79% of a copy's rate, instructions and memory about even; one token
// 2.5 us, 64 tokens 3.3 us. Four loads in flight to a lane need 64 heads of 128
// (128 of 64) to a token; with fewer a CTA's lanes are that much emptier: 24 + 16
// heads of 128, 2793 tokens, 14.9 us (8.5 at a copy's rate), 32 + 16 of 64, 7153
// tokens, 28.7 (13.0).
constexpr int kAppendThreads = 256;

struct AppendArgs {
  PagedArgs p;
  const uint16_t* qkv;
  const uint16_t* wq;
  const uint16_t* wk;
  const float* rope;
  const int32_t* positions;
  uint16_t* q;
  uint16_t* cache;
  long long ldqkv, ldq;
  int hq, rope_len, rot;
  float eps;
};

template <int D, int U, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads, U > 1 && INTERLEAVED ? 5 : 4) append_kernel(const AppendArgs a) {
  constexpr int LG = D / 8;                      // lanes of a head
  constexpr int kGroups = kAppendThreads / LG;   // heads at a time
  const int H = a.hq + 2 * a.p.hkv;
  const int tid = threadIdx.x, l = tid % LG, tok = blockIdx.x;
  const int head0 = blockIdx.y * (kGroups * U) + tid / LG;
  griddep_launch_dependents();
  griddep_wait();

  uint4 x[U];
  const uint16_t* src = a.qkv + tok * a.ldqkv + head0 * D + l * 8;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    x[k] = make_uint4(0, 0, 0, 0);
    if (head0 + k * kGroups < H) x[k] = *reinterpret_cast<const uint4*>(src + k * kGroups * D);
  }
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (a.wq) {
    wq = __ldg(reinterpret_cast<const uint4*>(a.wq) + l);
    wk = __ldg(reinterpret_cast<const uint4*>(a.wk) + l);
  }
  // the token's sequence: as many as end at or before it come first
  int b = 0;
  for (int i = 0; i < a.p.batch; i += kAppendThreads)
    b += __syncthreads_count(i + tid < a.p.batch && __ldg(a.p.cu_q + i + tid + 1) <= tok);
  if (b >= a.p.batch) return;  // past the last sequence
  const int first = __ldg(a.p.cu_q + b), end = __ldg(a.p.cu_q + b + 1);
  if (first > tok || end <= tok) {  // before the first sequence, or cu_q does not rise
    if (b > 0 && a.p.status) atomicOr(a.p.status, kStatusBounds);
    return;
  }
  const int row = paged_row(a.p, b);
  const int pos = paged_len(a.p, row) - end + tok;
  int rp = a.positions ? __ldg(a.positions + tok) : (pos < 0 ? 0 : pos);
  int page = -1;
  if (row >= 0 && pos >= 0) {
    page = __ldg(a.p.table + row * a.p.table_stride + (pos >> a.p.page_shift));
    if (page >= a.p.pages) page = -1;
  }
  if (a.p.status && (page < 0 || rp < 0 || rp >= a.rope_len)) atomicOr(a.p.status, kStatusBounds);
  rp = rp < 0 ? 0 : (rp >= a.rope_len ? a.rope_len - 1 : rp);

  // this lane's cosines and sines: of its 8 elements, or of its 4 pairs
  const int half = a.rot >> 1;
  const bool turned = l * 8 < a.rot, second = !INTERLEAVED && l * 8 >= half;
  const int other = turned ? (second ? l - half / 8 : l + half / 8) : l;
  float c[INTERLEAVED ? 4 : 8], s[INTERLEAVED ? 4 : 8];
  if (turned) {
    const float* at = a.rope + (long long)rp * a.rot + (INTERLEAVED ? l * 4 : l * 8 - (second ? half : 0));
#pragma unroll
    for (int q = 0; q < (INTERLEAVED ? 1 : 2); ++q) {
      const float4 cs = __ldg(reinterpret_cast<const float4*>(at) + q);
      const float4 sn = __ldg(reinterpret_cast<const float4*>(at + half) + q);
      const float sign = INTERLEAVED || second ? 1.f : -1.f;
      c[q * 4] = cs.x, c[q * 4 + 1] = cs.y, c[q * 4 + 2] = cs.z, c[q * 4 + 3] = cs.w;
      s[q * 4] = sign * sn.x, s[q * 4 + 1] = sign * sn.y;
      s[q * 4 + 2] = sign * sn.z, s[q * 4 + 3] = sign * sn.w;
    }
  }
  // the lanes of this head: heads of one warp may take different branches
  const unsigned gmask = ((1u << LG) - 1) << (tid & 31 & ~(LG - 1));
  uint16_t* const qdst = a.q + tok * a.ldq + l * 8;
  // key heads, then value heads, as the cache has them
  const long long step = (long long)a.p.page * D;
  uint16_t* const kdst = a.cache + (page < 0 ? 0 : page) * a.p.page_stride +
                         (long long)(pos & (a.p.page - 1)) * D + l * 8;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int head = head0 + k * kGroups;
    if (head >= H) break;
    uint4 out = x[k];
    if (head < a.hq + a.p.hkv) {
      float y[8];
      unpack8(out, y);
      if (a.wq) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
        for (int o = LG / 2; o; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o, LG);
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        float w[8];
        unpack8(head < a.hq ? wq : wk, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * r * w[e];
      }
      if (INTERLEAVED) {
        if (turned) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = y[2 * e], q = y[2 * e + 1];
            y[2 * e] = p * c[e] - q * s[e];
            y[2 * e + 1] = q * c[e] + p * s[e];
          }
        }
      } else {
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = __shfl_sync(gmask, y[e], other, LG);
        if (turned) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = y[e] * c[INTERLEAVED ? 0 : e] + z[e] * s[INTERLEAVED ? 0 : e];
        }
      }
      out = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                       pack_bf16(y[6], y[7]));
    }
    if (head < a.hq) *reinterpret_cast<uint4*>(qdst + head * D) = out;
    else if (page >= 0) *reinterpret_cast<uint4*>(kdst + (head - a.hq) * step) = out;
  }
}

template <int D, bool INTERLEAVED>
static cudaError_t launch_append_d(const Ctx& cx, const AppendArgs& a) {
  constexpr int kGroups = kAppendThreads / (D / 8);
  const int heads = a.hq + 2 * a.p.hkv;
  // few tokens: a head for each thread group, spread over the SMs; many: four,
  // whose loads are in flight together
  if ((long long)a.p.tokens * heads <= 2LL * cx.sms * kGroups)
    return launch_k(append_kernel<D, 1, INTERLEAVED>,
                    dim3((unsigned)a.p.tokens, (unsigned)((heads + kGroups - 1) / kGroups)),
                    dim3(kAppendThreads), 0, cx.stream, cx.pdl, a);
  return launch_k(append_kernel<D, 4, INTERLEAVED>,
                  dim3((unsigned)a.p.tokens, (unsigned)((heads + 4 * kGroups - 1) / (4 * kGroups))),
                  dim3(kAppendThreads), 0, cx.stream, cx.pdl, a);
}

cudaError_t launch_append(const Ctx& cx, const KvView& v, const AppendCall& c) {
  AppendArgs a = {};
  a.p = paged_args(v, c.tokens, cx.status);
  a.qkv = static_cast<const uint16_t*>(c.qkv);
  a.wq = static_cast<const uint16_t*>(c.wq);
  a.wk = static_cast<const uint16_t*>(c.wk);
  a.rope = c.rope;
  a.positions = c.positions;
  a.q = static_cast<uint16_t*>(c.q);
  a.cache = static_cast<uint16_t*>(v.cache);
  a.ldqkv = c.ldqkv;
  a.ldq = c.ldq;
  a.hq = c.hq;
  a.rope_len = c.rope_len;
  a.rot = c.rot;
  a.eps = c.eps;
  if (c.interleaved)
    return v.dim == 64 ? launch_append_d<64, true>(cx, a) : launch_append_d<128, true>(cx, a);
  return v.dim == 64 ? launch_append_d<64, false>(cx, a) : launch_append_d<128, false>(cx, a);
}

// ------------------------------------------------------------------ page copies
// Pages move in chunks of 16 KB (256 threads): a chunk of one page of one layer
// for each pass of a CTA, 64 bytes in flight per thread. Bound by memory: 701 pages
// of four layers (735 MB read and written) 120 us = 6.1 TB/s.
constexpr int kCopyThreads = 256;
constexpr int kCopyChunk = kCopyThreads * 64;

template <int NT, typename Pair>
__device__ __forceinline__ void copy_pages(const KvPool& p, int n, const Pair& pair) {
  constexpr int kChunk = NT * 64;
  const int chunks = (int)((p.page_bytes + kChunk - 1) / kChunk);
  const long long total = (long long)n * p.layers * chunks;
  for (long long x = blockIdx.x; x < total; x += gridDim.x) {
    const int i = (int)(x / ((long long)p.layers * chunks));
    const int rest = (int)(x - (long long)i * p.layers * chunks);
    const int layer = rest / chunks;
    const long long at = (long long)(rest - layer * chunks) * kChunk;
    int src, dst;
    if (!pair(i, src, dst)) continue;
    const uint8_t* s = p.data + layer * p.layer_stride + src * p.page_stride + at;
    uint8_t* d = p.data + layer * p.layer_stride + dst * p.page_stride + at;
    const long long left = p.page_bytes - at;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int o = (k * NT + threadIdx.x) * 16;
      if (o < left) v[k] = __ldcs(reinterpret_cast<const uint4*>(s + o));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int o = (k * NT + threadIdx.x) * 16;
      if (o < left) __stcs(reinterpret_cast<uint4*>(d + o), v[k]);
    }
  }
}

// ------------------------------------------------------------------ page state
// refs[page] counts the table entries that hold a page; 0 is free. A call's
// new pages are the lowest free ones, in the order of its requests: a rank
// over refs and a prefix sum over the requests. One thread-block cluster does
// the whole call: each CTA ranks a slice of refs, the slices' counts are
// exchanged through distributed shared memory, and the cluster's barriers
// separate reading refs, giving pages back and taking new ones. The state is
// a few hundred KB at most, so that a call is bound by latency, not by bytes.
// Measured: 4 to 5 us a call of 64 sequences of a pool of 4096 pages.
constexpr int kPoolCtas = 8;
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;

struct PoolArgs {
  KvPool p;
  const int32_t* seqs;  // resize: the sequences; fork: the copies (dst)
  const int32_t* src;   // fork
  const int32_t* len;   // resize: new lengths, null for 0
  int n;
  int32_t* pairs;       // [2 n] pages to copy: from (-1: none), to
  int* status;
};

// Exclusive prefix of v over the CTA's threads; total in all threads.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int w = s_warp[lane];  // kPoolWarps == 32
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(~0u, w, o);
    if (lane >= o) w += t;
  }
  total = __shfl_sync(~0u, w, 31);
  const int before = __shfl_sync(~0u, w, warp ? warp - 1 : 0);
  __syncthreads();
  return inc - v + (warp ? before : 0);
}

// This thread's run of pages [first, first + per) and, in bits, which of them
// are free (per <= 64).
struct PageRun {
  int first, count;
  unsigned long long bits;
  __device__ PageRun(const KvPool& p, uint32_t rank, bool want_free) {
    const int per = (p.pages + kPoolCtas * kPoolThreads - 1) / (kPoolCtas * kPoolThreads);
    const long long f = ((long long)rank * kPoolThreads + threadIdx.x) * per;
    first = f < p.pages ? (int)f : p.pages;
    count = p.pages - first < per ? p.pages - first : per;
    bits = 0;
    for (int k = 0; k < count; ++k)
      if ((__ldcg(p.refs + first + k) <= 0) == want_free) bits |= 1ull << k;
  }
};

template <bool FORK>
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    kv_change_kernel(const PoolArgs a) {
  __shared__ int s_start[kMaxBatch + 1];  // new pages before each request
  __shared__ int s_col[kMaxBatch];        // first table column that gets a new page
  __shared__ int s_cow[kMaxBatch];        // page to copy into it, or -1
  __shared__ int s_row[kMaxBatch];        // the sequence, or -1 (a request that is left out)
  __shared__ int s_src[FORK ? kMaxBatch : 1];
  __shared__ int s_old[kMaxBatch], s_new[kMaxBatch];  // columns held before, after
  __shared__ int s_warp[32], s_cnt[kPoolCtas], s_rel[kPoolCtas], s_mine;
  const KvPool& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int mask = (1 << p.page_shift) - 1;
  if (tid == 0) s_mine = 0;
  griddep_launch_dependents();
  __syncwarp();
  cluster_arrive_all();  // this CTA's shared memory may be written by the others
  griddep_wait();

  auto blocks = [&](int n) { return (int)(((long long)n + mask) >> p.page_shift); };
  auto bad = [&] {
    if (a.status) atomicOr(a.status, kStatusBounds);
  };
  auto length = [&](int s) -> int {  // a sequence's length, within its table row
    const int n = __ldcg(p.lens + s);
    const long long cap = (long long)p.width << p.page_shift;
    return n < 0 ? 0 : (n > cap ? (int)cap : n);
  };
  auto entry = [&](int s, int col) -> int {
    return __ldcg(p.table + (long long)s * p.table_stride + col);
  };
  auto is_page = [&](int pg) { return pg >= 0 && pg < p.pages; };

  // request tid
  int need = 0, cow = 0, newlen = 0;
  if (tid < a.n) {
    int row = __ldg(a.seqs + tid), from = -1, col = 0, nold = 0, nnew = 0;
    if (row < 0 || row >= p.seqs) row = -1;
    if (FORK) {
      const int s = __ldg(a.src + tid);
      if (s < 0 || s >= p.seqs || s == row) row = -1;
      s_src[tid] = s;
      if (row >= 0) {
        newlen = length(s);
        nold = blocks(length(row));
        col = newlen >> p.page_shift;  // full pages are shared
        nnew = blocks(newlen);
        need = nnew - col;
        if (need) from = entry(s, col);
      }
    } else {
      newlen = a.len ? __ldg(a.len + tid) : 0;
      if (newlen < 0 || newlen > ((long long)p.width << p.page_shift)) row = -1;
      if (row >= 0) {
        const int was = length(row);
        nold = blocks(was);
        nnew = blocks(newlen);
        col = nold;
        if (nnew > nold) need = nnew - nold;
        if (newlen < was && (newlen & mask)) {
          // the last page stays in part: if others hold it too, a page of its
          // own, for what will be written after its end
          const int pg = entry(row, nnew - 1);
          if (is_page(pg) && __ldcg(p.refs + pg) > 1) {
            from = pg;
            col = nnew - 1;
            need = 1;
          }
        }
      }
    }
    if (row < 0) bad();
    if (from >= 0 && !is_page(from)) {
      bad();
      from = -1;
    }
    cow = from >= 0;
    s_row[tid] = row;
    s_cow[tid] = from;
    s_col[tid] = col;
    s_old[tid] = nold;
    s_new[tid] = nnew;
  }
  const PageRun run(p, rank, true);
  int total, mine, copies;
  const int start = block_scan(need, s_warp, total);
  if (tid < a.n) s_start[tid] = start;
  block_scan(cow, s_warp, copies);
  const int before = block_scan(__popcll(run.bits), s_warp, mine);
  cluster_wait_all();  // all CTAs of the cluster have started
  if (tid < kPoolCtas) st_dsmem_s32(&s_cnt[rank], tid, mine);
  cluster_sync_all();  // every CTA has read refs, lengths and the entries above

  int offset = before, free_pages = 0;
  for (int r = 0; r < kPoolCtas; ++r) {
    if (r < (int)rank) offset += s_cnt[r];
    free_pages += s_cnt[r];
  }
  const int lacking = total > free_pages ? total - free_pages : 0;
  if (rank == 0 && tid < a.n && a.pairs && (!cow || lacking)) a.pairs[2 * tid] = -1;
  const int wid = (int)rank * kPoolWarps + warp;
  if (!lacking) {
    if (FORK) {
      for (int i = wid; i < a.n; i += kPoolCtas * kPoolWarps)
        if (s_row[i] >= 0)
          for (int c = lane; c < s_col[i]; c += 32) {
            const int pg = entry(s_src[i], c);
            if (is_page(pg)) atomicAdd(p.refs + pg, 1);
            else bad();
          }
    }
  }
  if (FORK) cluster_sync_all();  // a page is added to before it is taken from
  if (!lacking) {
    int freed = 0;
    auto release = [&](int pg) {
      if (!is_page(pg)) bad();
      else if (atomicSub(p.refs + pg, 1) == 1) ++freed;
    };
    for (int i = wid; i < a.n; i += kPoolCtas * kPoolWarps) {
      const int row = s_row[i];
      if (row < 0) continue;
      int32_t* t = p.table + (long long)row * p.table_stride;
      if (FORK) {
        const int end = s_old[i] > s_new[i] ? s_old[i] : s_new[i];
        for (int c = lane; c < end; c += 32) {
          if (c < s_old[i]) release(__ldcg(t + c));
          t[c] = c < s_col[i] ? entry(s_src[i], c) : -1;
        }
      } else {
        for (int c = s_new[i] + lane; c < s_old[i]; c += 32) {
          release(__ldcg(t + c));
          t[c] = -1;
        }
        if (lane == 0 && s_cow[i] >= 0) release(s_cow[i]);
      }
    }
    freed = __reduce_add_sync(~0u, freed);
    if (lane == 0 && freed) atomicAdd(&s_mine, freed);
  }
  __syncthreads();
  if (tid == 0) st_dsmem_s32(&s_rel[rank], 0, s_mine);
  cluster_sync_all();
  if (!lacking) {
    if (rank == 0 && tid < a.n && s_row[tid] >= 0) p.lens[s_row[tid]] = newlen;
    int r = offset;
    for (unsigned long long m = run.bits; m && r < total; m &= m - 1, ++r) {
      const int pg = run.first + __ffsll(m) - 1;
      int lo = 0, hi = a.n - 1;  // the last request that starts at or before r
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= r) lo = mid;
        else hi = mid - 1;
      }
      p.refs[pg] = 1;
      p.table[(long long)s_row[lo] * p.table_stride + s_col[lo] + (r - s_start[lo])] = pg;
      if (s_cow[lo] >= 0 && a.pairs) {
        a.pairs[2 * lo] = s_cow[lo];
        a.pairs[2 * lo + 1] = pg;
      }
    }
  }
  if (rank == 0 && tid == 0 && p.info) {
    int freed = 0;
    for (int r = 0; r < kPoolCtas; ++r) freed += s_rel[r];
    p.info[0] = lacking;
    p.info[1] = lacking ? free_pages : free_pages - total + freed;
    p.info[2] = lacking ? 0 : copies;
  }
  // A cut sequence's copies of pages that others hold are few, mostly none:
  // this cluster makes them itself, where a second kernel would cost every
  // call 2 us and its launch. A fork copies a page for most of its sequences:
  // that takes the whole device. Measured, pages of 128 KB a layer, us beyond a
  // call without copies (and what their bytes take): 1 / 8 / 64 pages of 4 layers
  // 3 / 14 / 90 (0.2 / 1.2 / 10), of 60 layers 23 / 166 / 1285 (2.3 / 18 / 148).
  if (!FORK && copies && !lacking) {
    cluster_sync_all();
    copy_pages<kPoolThreads>(p, a.n, [&](int i, int& s, int& d) {
      s = __ldcg(a.pairs + 2 * i);
      d = __ldcg(a.pairs + 2 * i + 1);
      return s >= 0;
    });
  }
}

__global__ void __launch_bounds__(kCopyThreads)
    kv_copy_kernel(const KvPool p, const int32_t* src, const int32_t* dst, int step, int n, int* status) {
  griddep_launch_dependents();
  griddep_wait();
  copy_pages<kCopyThreads>(p, n, [&](int i, int& s, int& d) {
    s = __ldcg(src + (long long)i * step);
    if (s == -1) return false;
    d = __ldcg(dst + (long long)i * step);
    if (s >= 0 && s < p.pages && d >= 0 && d < p.pages) return s != d;
    if (status) atomicOr(status, kStatusBounds);
    return false;
  });
}

// ------------------------------------------------------------------ compact
// The live pages at or past n = (number of live pages) move, in order, to the
// free pages before n. ws: [0] live pages before page n, [1] moves, then
// holes[pages], movers[pages] (indexed by the live pages before them) and
// rank[pages] (live pages before a page). Bound by memory for a large pool: 9000
// pages of four layers, half of them live in small holes, 1.14 GB in 186 us = 6.1 TB/s.
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    kv_rank_kernel(const KvPool p, int* ws) {
  __shared__ int s_warp[32], s_cnt[kPoolCtas];
  const uint32_t rank = cluster_rank();
  griddep_launch_dependents();
  cluster_arrive_all();  // this CTA's shared memory may be written by the others
  griddep_wait();
  int* holes = ws + 2;
  int* movers = holes + p.pages;
  int* ranks = movers + p.pages;
  const PageRun run(p, rank, false);
  int mine;
  int before = block_scan(__popcll(run.bits), s_warp, mine);
  cluster_wait_all();  // all CTAs of the cluster have started
  if (threadIdx.x < kPoolCtas) st_dsmem_s32(&s_cnt[rank], threadIdx.x, mine);
  cluster_sync_all();
  int n = 0;
  for (int r = 0; r < kPoolCtas; ++r) {
    if (r < (int)rank) before += s_cnt[r];
    n += s_cnt[r];
  }
  auto write_head = [&](int live_before) {
    ws[0] = live_before;
    ws[1] = n - live_before;
    if (p.info) {
      p.info[0] = 0;
      p.info[1] = p.pages - n;
      p.info[2] = n - live_before;
    }
  };
  for (int k = 0; k < run.count; ++k) {
    const int pg = run.first + k;
    const bool live = (run.bits >> k) & 1;
    if (pg == n) write_head(before);
    if (pg < n) {
      if (!live) holes[pg - before] = pg;
    } else {
      ranks[pg] = before;
      if (live) movers[before] = pg;
    }
    before += live;
  }
  if (n == p.pages && rank == 0 && threadIdx.x == 0) write_head(n);
}

__global__ void __launch_bounds__(kCopyThreads) kv_move_kernel(const KvPool p, const int* ws) {
  griddep_launch_dependents();
  griddep_wait();
  const int l0 = __ldcg(ws), moves = __ldcg(ws + 1), n = l0 + moves;
  const int* holes = ws + 2;
  const int* movers = holes + p.pages;
  const int* ranks = movers + p.pages;
  const long long tid = (long long)blockIdx.x * kCopyThreads + threadIdx.x;
  const long long threads = (long long)gridDim.x * kCopyThreads;
  for (long long i = tid; i < moves; i += threads) {
    const int from = __ldcg(movers + l0 + i), to = __ldcg(holes + i);
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
  }
  const long long entries = (long long)p.seqs * p.width;
  for (long long i = tid; i < entries; i += threads) {
    const long long s = i / p.width;
    int32_t* t = p.table + s * p.table_stride + (i - s * p.width);
    const int pg = *t;
    if (pg < n || pg >= p.pages) continue;
    // live pages at or past n only: an entry of a page that refs calls free
    // would be a mistake of the caller's; its rank is still within the lists
    const int m = __ldcg(ranks + pg) - l0;
    if (m < moves) *t = __ldcg(holes + m);
  }
  copy_pages<kCopyThreads>(p, moves, [&](int i, int& s, int& d) {
    s = __ldcg(movers + l0 + i);
    d = __ldcg(holes + i);
    return true;
  });
}

// ------------------------------------------------------------------ launches
static int copy_grid(const Ctx& cx, const KvPool& p, long long n) {
  const long long chunks = n * p.layers * ((p.page_bytes + kCopyChunk - 1) / kCopyChunk);
  const long long most = 8LL * cx.sms;
  return (int)(chunks < 1 ? 1 : (chunks < most ? chunks : most));
}

cudaError_t launch_kv_copy(const Ctx& cx, const KvPool& p, const int32_t* src, const int32_t* dst,
                           int step, int n) {
  return launch_k(kv_copy_kernel, dim3(copy_grid(cx, p, n)), dim3(kCopyThreads), 0, cx.stream, cx.pdl,
                  p, src, dst, step, n, cx.status);
}

cudaError_t launch_kv_resize(const Ctx& cx, const KvPool& p, const int32_t* seqs,
                             const int32_t* len, int n, int* pairs) {
  PoolArgs a = {p, seqs, nullptr, len, n, pairs, cx.status};
  return launch_k(kv_change_kernel<false>, dim3(kPoolCtas), dim3(kPoolThreads), 0, cx.stream, cx.pdl,
                  a);
}

cudaError_t launch_kv_fork(const Ctx& cx, const KvPool& p, const int32_t* src, const int32_t* dst,
                           int n, int* pairs) {
  PoolArgs a = {p, dst, src, nullptr, n, pairs, cx.status};
  cudaError_t e = launch_k(kv_change_kernel<true>, dim3(kPoolCtas), dim3(kPoolThreads), 0, cx.stream,
                           cx.pdl, a);
  if (e != cudaSuccess) return e;
  return launch_kv_copy(cx, p, pairs, pairs + 1, 2, n);
}

cudaError_t launch_kv_compact(const Ctx& cx, const KvPool& p, int* ws) {
  cudaError_t e = launch_k(kv_rank_kernel, dim3(kPoolCtas), dim3(kPoolThreads), 0, cx.stream, cx.pdl,
                           p, ws);
  if (e != cudaSuccess) return e;
  return launch_k(kv_move_kernel, dim3(copy_grid(cx, p, p.pages / 2 + 1)), dim3(kCopyThreads), 0,
                  cx.stream, cx.pdl, p, ws);
}

}  // namespace dg
