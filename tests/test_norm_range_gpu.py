"""The 8-bit norm where a product of a value and its weight leaves fp32's normal
numbers and the norm itself does not: every value and scale is the
definition's."""
import pytest

import _w4 as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_decode_gemm_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


import moe_decode_gemm_gb300 as dg  # noqa: E402

BF = ref.BF


def _exact(x, w, eps, res=None):
    """Values and exponents of the definition in 64 bits; the sum of squares is one of
    fp32, and where that is infinite the root is 0."""
    h, want = ref.norm(x, w, res, eps=eps)
    want = torch.where(h.square().sum(1, keepdim=True) >= 2.0 ** 128, torch.zeros_like(want), want)
    g = want.reshape(x.shape[0], -1, 32)
    e = ref.least_exponent(g.abs().amax(2), 448.0)
    v = g / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1e-30))).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).reshape(x.shape), e


def _same(x, w, eps=1e-6, res=None):
    got = dg.dec_rmsnorm_mx(x.cuda(), w.cuda(), None if res is None else res.cuda(), eps=eps)
    got = got if res is None else got[0]
    assert dg.sync_check() == dg.DEC_OK
    q, e = _exact(x, w, eps, res)
    assert torch.equal(got.s.view(torch.uint8).cpu().double() - 127, e)
    assert torch.equal(got.q.double().cpu(), q)


# (rows, width): a warp a row, a CTA a row with one, two and four values a thread
SHAPES = [(700, 96), (3, 1024), (4, 7168), (40, 16384)]


@pytest.mark.parametrize("rows,H", SHAPES)
@pytest.mark.parametrize("px,pw,eps", [
    (60, 70, 1e-6),      # products past the largest fp32
    (50, 100, 1e-6),
    (-40, -90, 0.0),     # below the least normal one, with a large root
    (-40, -80, 0.0),
    (-20, -110, 0.0),
    (0, -118, 1e-6),     # tiny outputs
    (30, -118, 1e-6),    # a small root: products far above the outputs
])
def test_far_products(rows, H, px, pw, eps):
    x = (ref.normal(H, rows, H).double() * 2.0 ** px).to(BF)
    w = ((1 + ref.normal(2, H, std=0.3).double()) * 2.0 ** pw).to(BF)
    _same(x, w, eps)


@pytest.mark.parametrize("rows,H", SHAPES)
def test_weights_of_very_different_size(rows, H):
    """Each group of 32 has a range of its own, within one row of large values."""
    x = (ref.normal(H, rows, H).double() * 2.0 ** 40).to(BF)
    p = torch.arange(H // 32).repeat_interleave(32) * 23 % 200 - 90
    w = ((1 + ref.normal(3, H, std=0.3).double()) * torch.exp2(p.double())).to(BF)
    _same(x, w, res=(ref.normal(4, rows, H).double() * 2.0 ** 38).to(BF))


def test_equal_values_of_2_to_60():
    x = torch.full((2, 32), 2.0 ** 60).to(BF)
    w = torch.full((32,), 2.0 ** 70).to(BF)
    got = dg.dec_rmsnorm_mx(x.cuda(), w.cuda())
    assert (got.s.view(torch.uint8) == 127 + 70 - 8).all() and (got.q.float() == 256).all()
    assert (dg.dec_rmsnorm(x.cuda(), w.cuda()) == 2.0 ** 70).all()


def test_rows_whose_sum_of_squares_is_past_fp32():
    """Both forms give 0 for finite values, as the root is 0."""
    x = torch.full((2, 64), 3e38).to(BF)
    x[1, 5] = float("inf")
    w = torch.full((64,), 2.0).to(BF)
    got, plain = dg.dec_rmsnorm_mx(x.cuda(), w.cuda()), dg.dec_rmsnorm(x.cuda(), w.cuda())
    s = got.s.view(torch.uint8).cpu()
    assert (got.q[0].float() == 0).all() and (s[0] == 0).all() and (plain[0] == 0).all()
    assert s[1, 0] == 255 and s[1, 1] == 0 and got.q[1, :32].float().isnan().all()
    assert plain[1, 5].isnan() and plain[1].isnan().sum() == 1


@pytest.mark.parametrize("eps", [2.0 ** -20, 2.0 ** -30, 2.0 ** -60])
def test_products_that_fp32_takes_for_0(eps):
    """Groups whose products of value and weight are below fp32's least number, under a
    root of up to 2^30."""
    x = (ref.normal(6, 8, 256).double() * 2.0 ** -60).to(BF)
    w = ((1 + ref.normal(7, 256, std=0.3).double()) * 2.0 ** -92).to(BF)
    _same(x, w, eps)
