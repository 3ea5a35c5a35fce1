"""W4 and MX8 do not go on with memory that their tensors no longer have."""
import pytest

import _w4 as ref
import moe_decode_gemm_gb300 as dg

torch = pytest.importorskip("torch")

U8 = torch.uint8


def _w4():
    return dg.W4.pack(*ref.random_codes(1, 200, 64))


def _mx():
    return dg.MX8(torch.zeros((3, 64)).to(ref.F8), torch.zeros((3, 2), dtype=U8))


@pytest.mark.parametrize("make,names", [(_w4, "qsnk"), (_mx, ("q", "s", "shape"))])
def test_their_parts_are_not_exchanged(make, names):
    handle = make()
    for name in names:
        with pytest.raises(AttributeError):
            setattr(handle, name, getattr(handle, name))


@pytest.mark.parametrize("make", [_w4, _mx])
@pytest.mark.parametrize("part", ["q", "s"])
def test_tensors_with_other_memory(make, part):
    handle = make()
    old = handle._at()
    t = getattr(handle, part)
    t.data = t.clone()
    assert t.data_ptr() in handle._at() and handle._at() != old
    t.data = t[:1].clone()                                 # of another shape: no such handle
    with pytest.raises(ValueError, match="expected"):
        handle._at()


@pytest.mark.gpu
@pytest.mark.parametrize("mx", [False, True])
def test_calls_see_it(mx):
    N, K = 200, 256
    (c0, s0), (c1, s1) = ref.random_codes(1, N, K), ref.random_codes(2, N, K)
    a, b = dg.W4.pack(c0.cuda(), s0.cuda()), dg.W4.pack(c1.cuda(), s1.cuda())
    x = ref.normal(3, 5, K).cuda()
    if mx:
        x = dg.dec_rmsnorm_mx(x, torch.ones(K, dtype=ref.BF, device="cuda"))
    want = dg.dec_linear_w4(x, b)
    a.q.data, a.s.data = b.q.clone(), b.s.clone()
    assert torch.equal(dg.dec_linear_w4(x, a), want)
    if mx:
        other = dg.dec_rmsnorm_mx(ref.normal(4, 5, K).cuda(), torch.ones(K, dtype=ref.BF, device="cuda"))
        want = dg.dec_linear_w4(other, b)
        x.q.data, x.s.data = other.q.clone(), other.s.clone()
        assert torch.equal(dg.dec_linear_w4(x, a), want)
