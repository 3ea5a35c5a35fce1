"""Sizes that the C ABI's 32 bits do not hold are refused by the binding of the
projections and the MoE block, not cut to them. CPU only: tensors without memory."""
import pytest

import moe_decode_gemm_gb300 as dg

torch = pytest.importorskip("torch")

FAR = (1 << 32) + 8


def _t(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="meta")


@pytest.mark.parametrize("M,N,K", [(FAR, 16, 64), (2, FAR, 64), (2, 16, FAR), (1 << 31, 16, 64)])
def test_projections(M, N, K):
    x, W, y = _t(M, K), _t(N, K), _t(M, N)
    for call in (lambda: dg.dec_linear(x, W, y), lambda: dg.dec_linear_splitk(x, W, 2, y),
                 lambda: dg.dec_linear_noalloc(x, W, y)):
        with pytest.raises(ValueError, match="%d does not fit 32 bits" % max(M, N, K)):
            call()


def test_forced_split():
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        dg.dec_linear_splitk(_t(2, 64), _t(16, 64), (1 << 32) + 2)


@pytest.mark.parametrize("M,topk", [(FAR, 2), (4, (1 << 32) + 2)])
def test_moe_block(M, topk):
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        dg.moe_decode(_t(M, 64), _t(8, 64), _t(8, 32, 64), _t(8, 64, 16), None, None, topk)
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        dg.moe_decode_latent(_t(M, 64), _t(40, 64), _t(8, 32, 32), _t(8, 32, 16), _t(64, 32), None, None, topk)
