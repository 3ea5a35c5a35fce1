"""Outputs over operands that other CTAs still read are refused by the C ABI of the
norm and of the 4-bit projections, before any kernel."""
import pytest

import moe_decode_gemm_gb300 as dg

A = [(i + 1) << 24 for i in range(8)]   # aligned fake pointers: never dereferenced


@pytest.fixture(scope="module")
def L():
    from moe_decode_gemm_gb300 import build
    build.build()
    return dg.lib()


def _linear(L, M=2, x=A[0], y=A[3], work=A[4], res=A[5], mx=False, xs=A[6]):
    if mx:
        return L.dec_linear_w4_mx(x, 64, xs, 2, A[1], A[2], res, y, M, 64, 64, None)
    return L.dec_linear_w4(x, 64, A[1], A[2], res, y, M, 64, 64, work, None)


@pytest.mark.parametrize("kw", [
    dict(y=A[0]), dict(y=A[0], M=40), dict(y=A[0], M=1), dict(M=40, work=A[0]), dict(M=40, work=A[3]),
    dict(M=40, work=A[5]), dict(mx=True, y=A[0]), dict(mx=True, y=A[6])])
def test_linear(L, kw):
    assert _linear(L, **kw) == dg.DEC_EINVAL


def _norm(L, mx=False, x=A[0], ldx=64, res=A[1], ldres=64, w=A[2], h=A[3], ldh=64, y=A[4], ldy=64, s=A[5]):
    if mx:
        return L.dec_rmsnorm_mx(x, ldx, res, ldres, w, 1e-6, h, ldh, y, ldy, s, 2, 2, 64, None)
    return L.dec_rmsnorm(x, ldx, res, ldres, w, 1e-6, h, ldh, y, ldy, 2, 64, None)


@pytest.mark.parametrize("kw", [
    dict(h=A[0], ldx=128), dict(h=A[1], ldh=128), dict(h=A[2]), dict(y=A[0], ldx=128), dict(y=A[1], ldres=72),
    dict(y=A[2]), dict(mx=True, y=A[0]), dict(mx=True, y=A[1]), dict(mx=True, y=A[3]), dict(mx=True, s=A[0]),
    dict(mx=True, s=A[4]), dict(mx=True, h=A[0], ldx=128)])
def test_norm(L, kw):
    assert _norm(L, **kw) == dg.DEC_EINVAL


@pytest.mark.gpu
def test_through_the_binding(L):
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    W = dg.dec_quant_w4(torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(dg.DecError):
        dg.dec_linear_w4(x, W, y=x)


@pytest.mark.parametrize("M,K", [(64, 2 ** 31 - 8), (17, 2 ** 29 + 8), (64, 2 ** 31 - 1)])
def test_no_work_space_for_what_is_refused(L, M, K):
    assert L.dec_linear_w4_work(M, K) == 0
    assert L.dec_linear_w4_work(M, 2 ** 29) > 2 * M * 2 ** 29
