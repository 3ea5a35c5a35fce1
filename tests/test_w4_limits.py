"""Sizes that the C ABI's 32 bits do not hold are refused by the binding of the norm
and of the 4-bit projections, not cut to them. CPU only: tensors without memory."""
import pytest

import moe_decode_gemm_gb300 as dg

torch = pytest.importorskip("torch")

BF, F8, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8
FAR = 1 << 32


def _t(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


def _w4(n=16, k=64):
    return dg.W4(_t(-(-n // 128), -(-k // 128), 128, 64, dtype=U8), _t(-(-n // 128), -(-k // 128), 32, 4, 4, dtype=U8),
                 n, k)


@pytest.mark.parametrize("call", [dg.dec_rmsnorm, dg.dec_rmsnorm_mx])
@pytest.mark.parametrize("rows,width", [(1, FAR + 32), (FAR + 3, 32), (1, 1 << 31), (1 << 31, 64)])
def test_norm(call, rows, width):
    with pytest.raises(ValueError, match="x: %d does not fit 32 bits" % max(rows, width)):
        call(_t(rows, width), _t(width))


@pytest.mark.parametrize("tokens", [FAR + 1, 1 << 31])
def test_linear(tokens):
    with pytest.raises(ValueError, match="x: %d does not fit 32 bits" % tokens):
        dg.dec_linear_w4(_t(tokens, 64), _w4())
    with pytest.raises(ValueError, match="%d does not fit 32 bits" % tokens):
        dg.dec_linear_w4(dg.MX8(_t(tokens, 64, dtype=F8), _t(tokens, 2, dtype=U8)), _w4())


@pytest.mark.parametrize("n,k", [(FAR + 16, 64), (16, FAR + 64), (1 << 31, 8)])
def test_weights(n, k):
    with pytest.raises(ValueError, match="%d does not fit 32 bits" % max(n, k)):
        dg.dec_quant_w4(_t(n, k))
    with pytest.raises(ValueError, match="%d does not fit 32 bits" % max(n, k)):
        _w4(n, k)


def test_sizes_below_are_looked_at_further():
    for rows, width in ((1, (1 << 31) - 8), ((1 << 31) - 1, 8)):
        with pytest.raises(ValueError, match="x: expected a CUDA tensor"):
            dg.dec_rmsnorm(_t(rows, width), _t(width))
