"""bf16 tokens as two e4m3 numbers: what the split keeps of them, restated here, and
that the projection takes them so. Weights of 1 on the diagonal give each value
back as the tensor cores saw it."""
import pytest

import _w4 as ref

torch = pytest.importorskip("torch")

BF, F8 = ref.BF, ref.F8
LARGEST = [225.0, 240.0, 256.0, 300.0, 447.0, 448.0, 450.0, 1.0]


def _split(x):
    """The sum of the two numbers of each value of bf16 x [M, K], and its 2^e."""
    v = x.double().reshape(x.shape[0], -1, 32)
    e = ref.least_exponent(v.abs().amax(2), 448.0).clamp(min=-123)[..., None]
    u = v / torch.exp2(e)
    hi = u.float().to(F8).double()
    lo = (16 * (u - hi)).float().to(F8).double()
    scale = torch.exp2(e).expand_as(u)
    return ((hi + lo / 16) * scale).reshape(x.shape), scale.reshape(x.shape)


def _tokens(power):
    """Groups of 32 with a given largest value and all sizes below it down to 2^-26 of it."""
    g = torch.Generator().manual_seed(7)
    rows = []
    for most in LARGEST:
        m = 1 + torch.randint(0, 128, (128,), generator=g) / 128.0
        p = torch.randint(-18, 8, (128,), generator=g).double()
        row = (m * torch.exp2(p)).clamp(max=most) * (1 - 2 * torch.randint(0, 2, (128,), generator=g))
        row[::32] = most
        rows.append(row)
    return (torch.stack(rows) * 2.0 ** power).to(BF)


@pytest.mark.parametrize("power", [-60, 0, 90])
def test_bounds(power):
    x = _tokens(power)
    got, scale = _split(x)
    v, err = x.double(), (got - x.double()).abs()
    most = v.abs().reshape(len(x), -1, 32).amax(2).repeat_interleave(32, 1)
    assert (err[v.abs() >= 2.0 ** -6 * scale] == 0).all()
    assert (err <= 2.0 ** -14 * scale).all() and (err > 2.0 ** -22 * most).any()
    assert (err <= 2.0 ** -14 / 224 * most).all()
    assert (err[v.abs() >= 2.0 ** -6 / 224 * most] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("copies", [1, 2, 4, 8])   # 8 to 64 tokens: each way that they are taken
@pytest.mark.parametrize("power", [-60, 0, 90])
def test_projection_takes_them_so(copies, power):
    import moe_decode_gemm_gb300 as dg
    from moe_decode_gemm_gb300 import build
    build.build()
    W = dg.W4.pack((2 * torch.eye(128)).to(torch.uint8).cuda(), torch.full((128, 4), 127, dtype=torch.uint8).cuda())
    x = _tokens(power).repeat(copies, 1)
    want, _ = _split(x)
    # the two parts are products of their own, their sum is exact in fp32, and rounded once
    assert torch.equal(dg.dec_linear_w4(x.cuda(), W).cpu(), want.float().to(BF))
    assert dg.sync_check() == dg.DEC_OK
