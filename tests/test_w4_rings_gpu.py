"""Projections with 4-bit weights of two tiles a CTA that go round their rings
several times, alone and in clusters: the kernels of the largest matrices."""
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


@pytest.fixture(scope="module")
def matrix():
    made = {}

    def get(N, K):
        if (N, K) not in made:
            made.clear()
            codes, scales = ref.random_codes(N + K, N, K)
            made[N, K] = dg.W4.pack(codes.cuda(), scales.cuda()), ref.weights(codes, scales)
        return made[N, K]

    return get


# 16384 x 7168: 64 pairs of tiles in clusters of two, 14 ring slots a CTA; 16300: the last
# pair's second tile is cut. 20000 x 4104: 157 tiles, an odd number, no clusters, an odd
# number of units.
@pytest.mark.parametrize("N,K", [(16384, 7168), (16300, 7160), (20000, 4104)])
@pytest.mark.parametrize("M", [1, 8, 16, 20, 32, 33, 64])
def test_bf16_tokens(matrix, M, N, K):
    W, w = matrix(N, K)
    x, res = ref.activations(M, M, K), ref.normal(M + 1, M, N, std=3.0)
    xd, rd = x.cuda(), res.cuda()
    y = dg.dec_linear_w4(xd, W, residual=rd)
    for _ in range(5):
        assert torch.equal(dg.dec_linear_w4(xd, W, residual=rd), y)
    assert dg.sync_check() == dg.DEC_OK
    want, a, spread = ref.linear(x, w, res)
    # as linear_bound, with what two 8-bit numbers may lose: 2^-21.8 of the group's largest
    bound = ref.linear_bound(want, a, spread, K, True) + 2.0 ** -21.8 * spread
    assert ((y.double().cpu() - want).abs() <= bound).all()


@pytest.mark.parametrize("N,K", [(16384, 7168), (20000, 4128)])
@pytest.mark.parametrize("M", [5, 31, 64])
def test_8_bit_tokens(matrix, M, N, K):
    W, w = matrix(N, K)
    q = ref.normal(M, M, K, std=60.0).float().clamp(-448, 448).to(ref.F8)
    s = torch.randint(110, 130, (M, K // 32), generator=torch.Generator().manual_seed(M)).to(torch.uint8)
    x = dg.MX8(q.cuda(), s.cuda())
    y = dg.dec_linear_w4(x, W)
    for _ in range(5):
        assert torch.equal(dg.dec_linear_w4(x, W), y)
    assert dg.sync_check() == dg.DEC_OK
    want, a, spread = ref.linear(ref.mx8_values(q, s), w)
    assert ((y.double().cpu() - want).abs() <= ref.linear_bound(want, a, spread, K, True)).all()
