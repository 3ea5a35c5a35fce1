"""Refusals of the norm and of the projections with 4-bit weights, before any
kernel: by the binding (tensors that the C ABI would misread) and by the C ABI
(codes as documented). CPU only."""
import ctypes

import pytest

import _w4 as ref
import moe_decode_gemm_gb300 as dg

torch = pytest.importorskip("torch")

BF, F8, E8, U8 = ref.BF, ref.F8, ref.E8, torch.uint8


@pytest.fixture(scope="module")
def L():
    from moe_decode_gemm_gb300 import build
    build.build()
    return dg.lib()


def _t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=torch.uint8).to(dtype)


def _w4(n=16, k=64):
    return dg.W4(torch.zeros((-(-n // 128), -(-k // 128), 128, 64), dtype=U8),
                 torch.zeros((-(-n // 128), -(-k // 128), 32, 4, 4), dtype=U8), n, k)


def _mx(t=2, h=64):
    return dg.MX8(_t(t, h, dtype=F8), _t(t, h // 32, dtype=U8))


# ------------------------------------------------------------------ the binding
@pytest.mark.parametrize("kw,exc,msg", [
    (dict(x=_t(2, 64, dtype=torch.float32)), TypeError, "x: expected torch.bfloat16"),
    (dict(x=[1.0]), TypeError, "x: expected a torch tensor"),
    (dict(x=_t(2, 32)), ValueError, "x: expected shape [any, 64]"),
    (dict(x=_t(64)), ValueError, "x: expected shape [any, 64]"),
    (dict(x=_t(64, 2).t()), ValueError, "x: needs unit column stride"),
    (dict(x=_t(2, 68)[:, :64]), ValueError, "x: needs a row stride that is a multiple of 8"),
    (dict(x=_t(1, 64).expand(2, 64)), ValueError, "x: its rows overlap"),
    (dict(x=_mx(2, 32)), ValueError, "x: expected shape [any, 64]"),
    (dict(W=_t(16, 64)), TypeError, "W: expected a W4"),
    (dict(y=_t(2, 15)), ValueError, "y: expected shape [2, 16]"),
    (dict(y=_t(2, 32)[:, :16]), ValueError, "y: must be contiguous"),
    (dict(residual=_t(3, 16)), ValueError, "residual: expected shape [2, 16]"),
    (dict(residual=_t(2, 16, dtype=torch.float16)), TypeError, "residual: expected torch.bfloat16"),
    (dict(), ValueError, "x: expected a CUDA tensor"),
    (dict(x=_mx()), ValueError, "x: expected a CUDA tensor"),
])
def test_linear_w4_rejects(kw, exc, msg):
    a = dict(x=_t(2, 64), W=_w4(), y=None, residual=None)
    a.update(kw)
    with pytest.raises(exc) as e:
        dg.dec_linear_w4(a["x"], a["W"], a["y"], residual=a["residual"])
    assert msg in str(e.value)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kw,exc,msg", [
    (dict(x=_t(2, 64, dtype=torch.float32)), TypeError, "x: expected torch.bfloat16"),
    (dict(x=_t(2, 2, 64)), ValueError, "x: expected shape [any, any]"),
    (dict(x=_t(2, 68)[:, :64]), ValueError, "x: needs a row stride that is a multiple of 8"),
    (dict(w=_t(63)), ValueError, "w: expected shape [64]"),
    (dict(w=_t(64, dtype=torch.float32)), TypeError, "w: expected torch.bfloat16"),
    (dict(w=_t(128)[::2]), ValueError, "w: needs unit column stride"),
    (dict(residual=_t(2, 32)), ValueError, "residual: expected shape [2, 64]"),
    (dict(residual=[1.0]), TypeError, "residual: expected a torch tensor"),
    (dict(x=_t(1, 64).expand(2, 64)), ValueError, "x: its rows overlap"),
    (dict(residual=_t(2, 64), h=_t(3, 64)), ValueError, "h: expected shape [2, 64]"),
    (dict(h=_t(2, 64)), ValueError, "h: given without a residual"),
    (dict(), ValueError, "x: expected a CUDA tensor"),
])
def test_norm_rejects(mx, kw, exc, msg):
    a = dict(x=_t(2, 64), w=_t(64), residual=None, h=None)
    a.update(kw)
    with pytest.raises(exc) as e:
        (dg.dec_rmsnorm_mx if mx else dg.dec_rmsnorm)(a["x"], a["w"], a["residual"], h=a["h"])
    assert msg in str(e.value)


@pytest.mark.parametrize("args,exc,msg", [
    ((_t(2, 64, dtype=U8), _t(2, 2, dtype=U8)), TypeError, "q: expected torch.float8_e4m3fn"),
    ((_t(2, 48, dtype=F8), _t(2, 1, dtype=U8)), ValueError, "multiple of 32"),
    ((_t(2, 64, dtype=F8), _t(2, 1, dtype=U8)), ValueError, "s: expected shape [2, 2]"),
    ((_t(2, 64, dtype=F8), _t(2, 2)), TypeError, "s: expected torch.float8_e8m0fnu"),
    ((_t(2, 72, dtype=F8)[:, :64], _t(2, 2, dtype=U8)), ValueError, "q: needs a row stride that is a multiple of 16"),
])
def test_mx8_rejects(args, exc, msg):
    with pytest.raises(exc) as e:
        dg.MX8(*args)
    assert msg in str(e.value)


@pytest.mark.parametrize("n,k,q,s,exc", [
    (16, 60, (1, 1, 128, 64), (1, 1, 32, 4, 4), ValueError),
    (0, 64, (1, 1, 128, 64), (1, 1, 32, 4, 4), ValueError),
    (129, 64, (1, 1, 128, 64), (1, 1, 32, 4, 4), ValueError),
    (16, 136, (1, 1, 128, 64), (1, 2, 32, 4, 4), ValueError),
    (16, 136, (1, 2, 128, 64), (1, 1, 32, 4, 4), ValueError),
])
def test_w4_rejects_shapes(n, k, q, s, exc):
    with pytest.raises(exc):
        dg.W4(torch.zeros(q, dtype=U8), torch.zeros(s, dtype=U8), n, k)


def test_w4_rejects_types_and_strides():
    with pytest.raises(TypeError):
        dg.W4(torch.zeros((1, 1, 128, 64), dtype=torch.int8), torch.zeros((1, 1, 32, 4, 4), dtype=U8), 16, 64)
    with pytest.raises(ValueError, match="contiguous"):
        dg.W4(torch.zeros((1, 1, 128, 128), dtype=U8)[..., :64], torch.zeros((1, 1, 32, 4, 4), dtype=U8), 16, 64)


@pytest.mark.parametrize("W,exc,msg", [
    (_t(16, 64, dtype=torch.float32), TypeError, "W: expected torch.bfloat16"),
    (_t(16, 60), ValueError, "multiple of 8"),
    (_t(64, 16).t(), ValueError, "W: needs unit column stride"),
    (_t(16, 64), ValueError, "W: expected a CUDA tensor"),
])
def test_quant_rejects(W, exc, msg):
    with pytest.raises(exc) as e:
        dg.dec_quant_w4(W)
    assert msg in str(e.value)


@pytest.mark.parametrize("n,k", [(1, 8), (130, 200), (300, 1000)])
def test_pack_is_the_documented_layout(n, k):
    codes, scales = ref.random_codes(1, n, k)
    w = dg.W4.pack(codes, scales)
    got = ref.unpack(w.q, w.s, n, k)
    assert torch.equal(got[0], codes) and torch.equal(got[1], scales)
    pad = torch.ones(-(-n // 128) * 128, -(-k // 128) * 128, dtype=torch.bool)
    pad[:n, :k] = False
    assert not ref.unpack(w.q, w.s, *pad.shape)[0][pad].any()


def test_pack_rejects_what_is_no_code():
    codes, scales = ref.random_codes(1, 20, 64)
    codes[3, 5] = 16
    with pytest.raises(ValueError, match="expected 0 to 15, got 16"):
        dg.W4.pack(codes, scales)


# ------------------------------------------------------------------ the C ABI
A = 1 << 20               # aligned fake pointers: never dereferenced
MIS = (1 << 20) + 8


def _norm(L, mx=False, **kw):
    a = dict(x=A, ldx=64, res=None, ldres=0, w=A, eps=1e-6, h=None, ldh=0, y=A, ldy=64, s=A, lds=2, rows=2, H=64)
    a.update(kw)
    if mx:
        return L.dec_rmsnorm_mx(a["x"], a["ldx"], a["res"], a["ldres"], a["w"], a["eps"], a["h"], a["ldh"], a["y"],
                                a["ldy"], a["s"], a["lds"], a["rows"], a["H"], None)
    return L.dec_rmsnorm(a["x"], a["ldx"], a["res"], a["ldres"], a["w"], a["eps"], a["h"], a["ldh"], a["y"],
                         a["ldy"], a["rows"], a["H"], None)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), dg.DEC_EINVAL), (dict(w=None), dg.DEC_EINVAL), (dict(y=None), dg.DEC_EINVAL),
    (dict(res=A, ldres=64), dg.DEC_EINVAL),                     # a residual needs h
    (dict(res=A, ldres=63, h=A, ldh=64), dg.DEC_EINVAL),
    (dict(res=A, ldres=64, h=A, ldh=56), dg.DEC_EINVAL),
    (dict(rows=0), dg.DEC_EINVAL), (dict(H=0), dg.DEC_EINVAL), (dict(H=60), dg.DEC_EINVAL),
    (dict(ldx=56), dg.DEC_EINVAL), (dict(ldx=68), dg.DEC_EINVAL), (dict(ldy=56), dg.DEC_EINVAL),
    (dict(eps=-1.0), dg.DEC_EINVAL), (dict(eps=float("nan")), dg.DEC_EINVAL),
    (dict(x=MIS), dg.DEC_EINVAL), (dict(w=MIS), dg.DEC_EINVAL), (dict(y=MIS), dg.DEC_EINVAL),
    (dict(H=65568, ldx=65568, ldy=65568, lds=2049), dg.DEC_EUNSUPPORTED),
])
def test_norm_codes(L, mx, kw, code):
    assert _norm(L, mx, **kw) == code


@pytest.mark.parametrize("kw", [dict(H=72, ldx=72, ldy=80, lds=3), dict(ldy=72), dict(lds=1), dict(s=None)])
def test_norm_mx_codes(L, kw):
    assert _norm(L, True, **kw) == dg.DEC_EINVAL


def test_norm_output_is_not_the_stream(L):
    assert _norm(L, res=A, ldres=64, h=2 * A, ldh=64, y=2 * A) == dg.DEC_EINVAL


def _linear(L, mx=False, **kw):
    a = dict(x=A, ldx=64, xs=A, ldxs=2, q=A, s=A, res=None, y=A, M=2, N=16, K=64, work=A)
    a.update(kw)
    if mx:
        return L.dec_linear_w4_mx(a["x"], a["ldx"], a["xs"], a["ldxs"], a["q"], a["s"], a["res"], a["y"], a["M"],
                                  a["N"], a["K"], None)
    return L.dec_linear_w4(a["x"], a["ldx"], a["q"], a["s"], a["res"], a["y"], a["M"], a["N"], a["K"], a["work"], None)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), dg.DEC_EINVAL), (dict(q=None), dg.DEC_EINVAL), (dict(s=None), dg.DEC_EINVAL),
    (dict(y=None), dg.DEC_EINVAL), (dict(M=0), dg.DEC_EINVAL), (dict(N=0), dg.DEC_EINVAL),
    (dict(K=60), dg.DEC_EINVAL), (dict(K=0), dg.DEC_EINVAL), (dict(ldx=48), dg.DEC_EINVAL),
    (dict(ldx=68), dg.DEC_EINVAL), (dict(x=MIS), dg.DEC_EINVAL), (dict(q=A + 64), dg.DEC_EINVAL),
    (dict(s=MIS), dg.DEC_EINVAL), (dict(res=MIS), dg.DEC_EINVAL), (dict(y=MIS), dg.DEC_EINVAL),
    (dict(M=65), dg.DEC_EUNSUPPORTED), (dict(N=1 << 30, K=1 << 12, ldx=1 << 12, ldxs=128), dg.DEC_EUNSUPPORTED),
])
def test_linear_codes(L, mx, kw, code):
    assert _linear(L, mx, **kw) == code


@pytest.mark.parametrize("kw", [dict(K=40), dict(ldx=72), dict(ldxs=1), dict(xs=None)])
def test_linear_mx_codes(L, kw):
    assert _linear(L, True, **kw) == dg.DEC_EINVAL


def test_linear_work(L):
    """A few tokens need no work space; more have to be given it, 16-byte aligned."""
    assert L.dec_linear_w4_work(1, 4096) == 0 and L.dec_linear_w4_work(64, 4096) > 2 * 64 * 4096
    assert L.dec_linear_w4_work(0, 4096) == 0 and L.dec_linear_w4_work(65, 4096) == 0
    for work in (None, MIS):
        assert _linear(L, M=64, work=work) == dg.DEC_EINVAL


@pytest.mark.parametrize("args,code", [
    ((None, 64, A, A, 16, 64), dg.DEC_EINVAL), ((A, 64, None, A, 16, 64), dg.DEC_EINVAL),
    ((A, 64, A, None, 16, 64), dg.DEC_EINVAL), ((A, 64, A, A, 0, 64), dg.DEC_EINVAL),
    ((A, 64, A, A, 16, 60), dg.DEC_EINVAL), ((A, 56, A, A, 16, 64), dg.DEC_EINVAL),
    ((A, 68, A, A, 16, 64), dg.DEC_EINVAL), ((MIS, 64, A, A, 16, 64), dg.DEC_EINVAL),
    ((A, 64, A + 64, A, 16, 64), dg.DEC_EINVAL), ((A, 64, A, MIS, 16, 64), dg.DEC_EINVAL),
    ((A, 1 << 12, A, A, 1 << 30, 1 << 12), dg.DEC_EUNSUPPORTED),
])
def test_quant_codes(L, args, code):
    assert L.dec_quant_w4(*args, None) == code
