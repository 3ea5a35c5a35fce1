"""Integers past 32 bits are refused, not cut to 32 bits on their way to the C ABI."""
import pytest

import _paged as pg
import moe_decode_gemm_gb300 as dg
from moe_decode_gemm_gb300 import paged

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1, -(1 << 32) + 5])
def test_integers_past_32_bits(n):
    with pytest.raises(ValueError) as e:
        paged._int32("window", n)
    assert "window: %d does not fit 32 bits" % n in str(e.value)


@pytest.mark.parametrize("n", [0, 5, (1 << 31) - 1, -(1 << 31)])
def test_integers_of_32_bits(n):
    assert paged._int32("window", n) == n


def test_a_window_is_whole():
    with pytest.raises(TypeError):
        paged._int32("window", 2.5)


@pytest.mark.gpu
def test_calls_refuse_them():
    from moe_decode_gemm_gb300 import build
    build.build()
    bt = pg.Batch([1, 2], [30, 40], 4, 2, 64, 16, seed=120)
    kv, q = bt.device(dg), bt.q.cuda()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731

    def hint():
        kv.max_q = 1 << 32

    for call in (lambda: dg.kv_attention(q, kv, window=(1 << 32) + 5),
                 lambda: bt.device(dg, max_q=(1 << 32) + 1), hint,
                 lambda: dg.KVPool(kv.cache[None], z(bt.pages), z(2, 4), z(2),
                                   page_size=(1 << 32) + 16)):
        with pytest.raises(ValueError) as e:
            call()
        assert "does not fit 32 bits" in str(e.value)
    with pytest.raises(dg.DecError):
        dg.kv_attention(q, kv, window=-1)
    lse = torch.empty((3, 4), device="cuda")
    pg.check_attention(bt, dg.kv_attention(q, kv, window=(1 << 31) - 1, lse=lse), lse)
