// api_w4.cu -- the C ABI of the norm and of the projections with 4-bit weights:
// argument checks.
#include <cmath>

#include "../../include/decgemm.h"
#include "launch.h"

namespace dg {

static bool al(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

static int result(cudaError_t e, int launches = 1) {
  if (e != cudaSuccess) return DEC_ECUDA;
  count_launches(launches);
  return DEC_OK;
}

static int norm(NormCall c, void* stream) {
  if (!c.x || !c.w || (!c.y && !c.q) || (c.res && !c.h)) return DEC_EINVAL;
  if (c.rows < 1 || c.H < 8 || c.H % (c.q ? 32 : 8) || !std::isfinite(c.eps) || c.eps < 0.f)
    return DEC_EINVAL;
  const void* ptrs[] = {c.x, c.res, c.w, c.h, c.y, c.q};
  for (const void* p : ptrs)
    if (!al(p, 16)) return DEC_EINVAL;
  if (c.ldx < c.H || c.ldx % 8 || (c.res && (c.ldres < c.H || c.ldres % 8 || c.ldh < c.H || c.ldh % 8)))
    return DEC_EINVAL;
  if (c.y && (c.ldy < c.H || c.ldy % 8 || c.y == c.h)) return DEC_EINVAL;
  if (c.q && (!c.sc || c.ldq < c.H || c.ldq % 16 || c.ldsc < c.H / 32)) return DEC_EINVAL;
  if (c.H > kNormMaxWidth) return DEC_EUNSUPPORTED;
  // In place row by row only: other rows would be written before they are read.
  auto in_place = [&](const void* out, long long ld, const void* in, long long ldin) {
    return out && out == in && c.rows > 1 && ld != ldin;
  };
  if (in_place(c.h, c.ldh, c.x, c.ldx) || in_place(c.h, c.ldh, c.res, c.ldres) ||
      in_place(c.y, c.ldy, c.x, c.ldx) || in_place(c.y, c.ldy, c.res, c.ldres))
    return DEC_EINVAL;
  if (c.h == c.w || c.y == c.w) return DEC_EINVAL;
  for (const void* p : {c.x, c.res, c.w, static_cast<const void*>(c.h)})
    if (c.q && (c.q == p || c.sc == p || c.q == c.sc)) return DEC_EINVAL;
  Ctx cx;
  if (int rc = kv_context(stream, 0, 0, &cx, nullptr, nullptr)) return rc;
  return result(launch_norm(cx, c));
}

static int linear(const W4Call& c, void* stream) {
  if (!c.x || !c.wq || !c.ws || !c.y) return DEC_EINVAL;
  if (c.M < 1 || c.N < 1 || c.K < 8 || c.K % (c.xs ? 32 : 8)) return DEC_EINVAL;
  if (c.ldx < c.K || c.ldx % (c.xs ? 16 : 8) || (c.xs && c.ldxs < c.K / 32)) return DEC_EINVAL;
  if (!al(c.x, 16) || !al(c.wq, 128) || !al(c.ws, 16) || !al(c.res, 16) || !al(c.y, 16)) return DEC_EINVAL;
  if (c.M > 64 || !w4_fits(c.N, c.K)) return DEC_EUNSUPPORTED;
  const bool work = !c.xs && w4_work_bytes(c.M, c.K) > 0;
  if (work && (!c.work || !al(c.work, 16))) return DEC_EINVAL;
  // Outputs are written while other CTAs still read tokens, the work space before that.
  if (c.y == c.x || c.y == c.xs || (work && (c.work == c.x || c.work == c.y || c.work == c.res)))
    return DEC_EINVAL;
  Ctx cx;
  if (int rc = kv_context(stream, 0, 0, &cx, nullptr, nullptr)) return rc;
  return result(launch_w4_linear(cx, c), work ? 2 : 1);
}

}  // namespace dg

using namespace dg;

extern "C" {

int dec_rmsnorm(const void* x, int64_t ldx, const void* res, int64_t ldres, const void* w, float eps,
                void* h, int64_t ldh, void* y, int64_t ldy, int rows, int H, void* stream) {
  if (!y) return DEC_EINVAL;
  return norm({x, res, w, h, y, nullptr, nullptr, ldx, ldres, ldh, ldy, 0, 0, rows, H, eps}, stream);
}

int dec_rmsnorm_mx(const void* x, int64_t ldx, const void* res, int64_t ldres, const void* w, float eps,
                   void* h, int64_t ldh, void* q, int64_t ldq, void* scales, int64_t ldscales, int rows,
                   int H, void* stream) {
  if (!q) return DEC_EINVAL;
  return norm({x, res, w, h, nullptr, q, scales, ldx, ldres, ldh, 0, ldq, ldscales, rows, H, eps}, stream);
}

int dec_quant_w4(const void* W, int64_t ldw, void* q, void* scales, int N, int K, void* stream) {
  if (!W || !q || !scales || N < 1 || K < 8 || K % 8 || ldw < K || ldw % 8) return DEC_EINVAL;
  if (!al(W, 16) || !al(q, 128) || !al(scales, 16)) return DEC_EINVAL;
  if (!w4_fits(N, K)) return DEC_EUNSUPPORTED;
  Ctx cx;
  if (int rc = kv_context(stream, 0, 0, &cx, nullptr, nullptr)) return rc;
  return result(launch_w4_quant(cx, W, ldw, q, scales, N, K));
}

size_t dec_linear_w4_work(int M, int K) { return M < 1 || M > 64 || K < 1 ? 0 : w4_work_bytes(M, K); }

int dec_linear_w4(const void* x, int64_t ldx, const void* wq, const void* wscales, const void* res,
                  void* y, int M, int N, int K, void* work, void* stream) {
  return linear({x, nullptr, wq, wscales, res, y, ldx, 0, M, N, K, work}, stream);
}

int dec_linear_w4_mx(const void* x, int64_t ldx, const void* xscales, int64_t ldxscales, const void* wq,
                     const void* wscales, const void* res, void* y, int M, int N, int K, void* stream) {
  if (!xscales) return DEC_EINVAL;
  return linear({x, xscales, wq, wscales, res, y, ldx, ldxscales, M, N, K, nullptr}, stream);
}

int dec_debug_stall(int on) {
  const int old = w4_stall(on);
  return old < 0 ? DEC_EUNSUPPORTED : old;
}

}  // extern "C"
