// api_kv.cu -- the C ABI of the paged cache: argument checks, the choice of
// the attention kernel, and the workspace that its calls share.
#include <cmath>
#include <cstdlib>
#include <cstring>

#include "../../include/decgemm.h"
#include "launch.h"

namespace dg {

// Positions of a table row: the end of a key tile past the last is still 32 bits.
constexpr int64_t kMaxPositions = INT32_MAX - 255;

static thread_local int t_last_attention = DEC_REGIME_NONE;

static bool al(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

static int result(cudaError_t e, int launches) {
  if (e != cudaSuccess) return DEC_ECUDA;
  count_launches(launches);
  return DEC_OK;
}

// The view in the library's own terms, checked.
static int view_of(const dec_kv_view* kv, KvView* v) {
  if (!kv || !kv->cache || !kv->table || !kv->cu_q || !kv->kv_len) return DEC_EINVAL;
  if (kv->pages < 1 || kv->heads < 1 || kv->page_size < 1 || kv->dim < 1 || kv->batch < 1 ||
      kv->width < 1 || kv->table_rows < 1 || kv->max_q < 0)
    return DEC_EINVAL;
  if (!kv->rows && kv->table_rows < kv->batch) return DEC_EINVAL;
  if (!al(kv->cache, 16) || !al(kv->table, 4) || !al(kv->cu_q, 4) || !al(kv->kv_len, 4) ||
      !al(kv->rows, 4))
    return DEC_EINVAL;
  const int64_t page_elems = 2LL * kv->heads * kv->page_size * kv->dim;
  if (kv->page_stride < page_elems || kv->page_stride % 8 || kv->table_stride < kv->width)
    return DEC_EINVAL;
  if (kv->page_size & (kv->page_size - 1)) return DEC_EINVAL;
  if (kv->page_size < 16 || kv->page_size > 256 || (kv->dim != 64 && kv->dim != 128) ||
      kv->batch > 1024 || (int64_t)kv->width * kv->page_size > kMaxPositions)
    return DEC_EUNSUPPORTED;
  *v = {kv->cache, kv->page_stride, kv->pages,  kv->heads,      kv->page_size, kv->dim, kv->table,
        kv->table_stride, kv->width, kv->table_rows, kv->rows, kv->cu_q, kv->kv_len, kv->batch};
  return DEC_OK;
}

static int attention(const dec_kv_view* kv, const AttnCall& c, void* stream) {
  KvView v;
  int rc = view_of(kv, &v);
  if (rc) return rc;
  if (!c.q || !c.out || c.tokens < 1 || c.hq < 1 || c.hq % v.hkv || c.window < 0) return DEC_EINVAL;
  if (!std::isfinite(c.scale)) return DEC_EINVAL;
  const int64_t qw = (int64_t)c.hq * v.dim;
  if (c.ldq < qw || c.ldq % 8 || c.ldo < qw || c.ldo % 8) return DEC_EINVAL;
  if (!al(c.q, 16) || !al(c.out, 16) || !al(c.lse, 4)) return DEC_EINVAL;
  const int group = c.hq / v.hkv;
  if (group > 64) return DEC_EUNSUPPORTED;
  const int sms = kv_sms();
  if (!sms) return DEC_ENODEV;
  Ctx cx;
  void* ws;
  int* ctr;
  // Rows (token, query head) of the longest chunk. Up to 32: mma.sync, a row tile
  // of 16 or 32. Above, mma.sync reads the keys once for every 32 rows where
  // tcgen05 reads them once, but starts and joins sooner: it stays while the
  // reading does not count. us of mma.sync / tcgen05 over 64, 512, 2048 and 8192
  // positions:
  //   28 rows, 8 sequences of 4 key heads of 128   9/13  14/18  20/28  33/39
  //   56 rows, the same                            9/13  14/18  21/28  42/39
  //   56 rows, 40 sequences                       15/13  25/23  62/48 187/120
  //   64 rows, 8 sequences of 8 key heads of 64    8/9   11/13  21/22  45/42
  //   64 rows, 40 sequences                       20/25  32/34  68/71 196/210
  //   126 rows, 1 sequence of 4 key heads of 128   9/12  14/17  20/26  30/27
  //   128 rows, 1 sequence of 8 key heads of 64    8/10  10/14  16/21  22/26
  //   128 rows, 8 sequences of them               13/9   19/13  30/22  70/42
  //   120 rows, 1 sequence of 8 key heads of 128  10/13  14/18  21/27  35/28
  // From 65 rows on that is up to about 20 row tiles of 128 columns, or 40 of 64,
  // a little more than the clusters take. (The last line has 32 and goes to
  // tcgen05: slower below some 4096 positions, faster above.)
  const int64_t longest = kv->max_q > 0 ? kv->max_q : c.tokens, rows = longest * group;
  bool tc = rows > 32;
  if (tc && group <= 32 && rows <= 128) {
    const int tq = 32 / group;
    const int64_t tiles = (longest + tq - 1) / tq * v.batch * v.hkv;
    if (rows <= 64) tc = v.dim == 128 && tiles * 2 > sms;
    else tc = tiles * v.dim > 17 * sms;
  }
  const char* force = std::getenv("DEC_FORCE");
  if (force && !std::strcmp(force, "mma") && group <= 32) tc = false;
  if (force && !std::strcmp(force, "tc")) tc = true;
  if (tc) {
    if ((rc = kv_context(stream, attn_tc_ws(v.dim, sms), attn_tc_ctrs(sms), &cx, &ws, &ctr))) return rc;
    t_last_attention = DEC_REGIME_TC;
    int kernels = 0;
    const cudaError_t e = launch_attn_tc(cx, v, c, static_cast<float*>(ws), ctr, &kernels);
    return result(e, kernels);
  }
  const int rt = rows <= 16 && group <= 16 ? 1 : 2;
  if ((rc = kv_context(stream, attn_mma_ws(v.dim, rt, sms), sms, &cx, &ws, &ctr))) return rc;
  t_last_attention = DEC_REGIME_MMA;
  return result(launch_attn_mma(cx, v, rt, c, static_cast<float*>(ws), ctr), 1);
}

static int pool_of(const dec_kv_pool* pool, KvPool* p) {
  if (!pool || !pool->data || !pool->refs || !pool->table || !pool->lens) return DEC_EINVAL;
  if (pool->layers < 1 || pool->pages < 1 || pool->page_size < 1 || pool->seqs < 1 ||
      pool->width < 1 || pool->page_bytes < 16 || pool->page_bytes % 16)
    return DEC_EINVAL;
  if (pool->page_size & (pool->page_size - 1)) return DEC_EINVAL;
  if (pool->page_stride < pool->page_bytes || pool->page_stride % 16 || pool->layer_stride % 16 ||
      (pool->layers > 1 && pool->layer_stride < pool->page_bytes) || pool->table_stride < pool->width)
    return DEC_EINVAL;
  if (!al(pool->data, 16) || !al(pool->refs, 4) || !al(pool->table, 4) || !al(pool->lens, 4) ||
      !al(pool->info, 4))
    return DEC_EINVAL;
  if (pool->pages > kMaxPages || (int64_t)pool->width * pool->page_size > INT32_MAX)
    return DEC_EUNSUPPORTED;
  int shift = 0;
  while ((1 << shift) < pool->page_size) ++shift;
  *p = {static_cast<uint8_t*>(pool->data), pool->layer_stride, pool->page_stride, pool->page_bytes,
        pool->layers, pool->pages, shift, pool->refs, pool->table, pool->table_stride, pool->width,
        pool->lens, pool->seqs, pool->info};
  return DEC_OK;
}

}  // namespace dg

using namespace dg;

extern "C" {

int kv_append(const dec_kv_view* kv, const void* qkv, int64_t ldqkv, const void* wq, const void* wk,
              float eps, const float* rope, int rope_len, int rot, int interleaved,
              const int32_t* positions, void* q, int64_t ldq, int tokens, int q_heads, void* stream) {
  KvView v;
  int rc = view_of(kv, &v);
  if (rc) return rc;
  if (!qkv || !q || !rope || (!wq) != (!wk) || tokens < 1 || q_heads < 1 || rope_len < 1)
    return DEC_EINVAL;
  if (rot < 16 || rot % 16 || rot > v.dim || !std::isfinite(eps) || eps < 0.f) return DEC_EINVAL;
  if (ldqkv < (int64_t)(q_heads + 2 * v.hkv) * v.dim || ldqkv % 8 || ldq < (int64_t)q_heads * v.dim ||
      ldq % 8)
    return DEC_EINVAL;
  if (!al(qkv, 16) || !al(q, 16) || !al(rope, 16) || !al(wq, 16) || !al(wk, 16) || !al(positions, 4))
    return DEC_EINVAL;
  if ((int64_t)q_heads + 2 * v.hkv > 32768) return DEC_EUNSUPPORTED;
  Ctx cx;
  if ((rc = kv_context(stream, 0, 0, &cx, nullptr, nullptr))) return rc;
  const AppendCall c = {qkv, wq, wk, rope, positions, q, ldqkv, ldq, tokens, q_heads, rope_len, rot,
                        interleaved != 0, eps};
  return result(launch_append(cx, v, c), 1);
}

int kv_attention(const dec_kv_view* kv, const void* q, int64_t ldq, void* out, int64_t ldo, float* lse,
                 int tokens, int q_heads, float scale, int window, void* stream) {
  const AttnCall c = {q, out, lse, ldq, ldo, tokens, q_heads, window, kv ? kv->max_q : 0, scale};
  return attention(kv, c, stream);
}

int kv_last_attention(void) { return t_last_attention; }

int kv_resize(const dec_kv_pool* pool, const int32_t* seqs, const int32_t* lens, int n, void* stream) {
  KvPool p;
  int rc = pool_of(pool, &p);
  if (rc) return rc;
  if (!seqs || !lens || n < 1 || !al(seqs, 4) || !al(lens, 4)) return DEC_EINVAL;
  if (n > 1024) return DEC_EUNSUPPORTED;
  Ctx cx;
  void* ws;
  if ((rc = kv_context(stream, (size_t)2 * n * sizeof(int), 0, &cx, &ws, nullptr))) return rc;
  return result(launch_kv_resize(cx, p, seqs, lens, n, static_cast<int*>(ws)), 1);
}

int kv_free(const dec_kv_pool* pool, const int32_t* seqs, int n, void* stream) {
  KvPool p;
  int rc = pool_of(pool, &p);
  if (rc) return rc;
  if (!seqs || n < 1 || !al(seqs, 4)) return DEC_EINVAL;
  if (n > 1024) return DEC_EUNSUPPORTED;
  Ctx cx;
  if ((rc = kv_context(stream, 0, 0, &cx, nullptr, nullptr))) return rc;
  return result(launch_kv_resize(cx, p, seqs, nullptr, n, nullptr), 1);
}

int kv_fork(const dec_kv_pool* pool, const int32_t* src, const int32_t* dst, int n, void* stream) {
  KvPool p;
  int rc = pool_of(pool, &p);
  if (rc) return rc;
  if (!src || !dst || n < 1 || !al(src, 4) || !al(dst, 4)) return DEC_EINVAL;
  if (n > 1024) return DEC_EUNSUPPORTED;
  Ctx cx;
  void* ws;
  if ((rc = kv_context(stream, (size_t)2 * n * sizeof(int), 0, &cx, &ws, nullptr))) return rc;
  return result(launch_kv_fork(cx, p, src, dst, n, static_cast<int*>(ws)), 2);
}

int kv_copy(const dec_kv_pool* pool, const int32_t* src, const int32_t* dst, int n, void* stream) {
  KvPool p;
  int rc = pool_of(pool, &p);
  if (rc) return rc;
  if (!src || !dst || n < 1 || !al(src, 4) || !al(dst, 4)) return DEC_EINVAL;
  Ctx cx;
  if ((rc = kv_context(stream, 0, 0, &cx, nullptr, nullptr))) return rc;
  return result(launch_kv_copy(cx, p, src, dst, 1, n), 1);
}

int kv_compact(const dec_kv_pool* pool, void* stream) {
  KvPool p;
  int rc = pool_of(pool, &p);
  if (rc) return rc;
  Ctx cx;
  void* ws;
  if ((rc = kv_context(stream, ((size_t)3 * p.pages + 2) * sizeof(int), 0, &cx, &ws, nullptr)))
    return rc;
  return result(launch_kv_compact(cx, p, static_cast<int*>(ws)), 2);
}

}  // extern "C"
