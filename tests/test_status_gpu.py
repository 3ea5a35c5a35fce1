"""A wait that gave up is reported even where wrong device data was met as well,
and calls after a report of wrong data are right."""
import pytest

import _paged as pg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_decode_gemm_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


import moe_decode_gemm_gb300 as dg  # noqa: E402


def _wrong_append():
    bt = pg.Batch([2, 3], [20, 40], 4, 2, 64, 16, seed=100)
    bt.table[0, 1] = -1
    dg.kv_append(pg.normal(pg.gen(1), 5, 8 * 64).cuda(), bt.device(dg),
                 torch.zeros(64, 64, device="cuda"))


@pytest.mark.parametrize("first", ["time-out", "bounds"])
def test_time_out_is_not_hidden_by_a_bounds_report(first):
    if first == "bounds":
        _wrong_append()
    dg.selftest_timeout(2_000_000)
    if first == "time-out":
        _wrong_append()
    assert dg.sync_check() == dg.DEC_ETIMEOUT
    assert dg.sync_check() == dg.DEC_EBOUNDS
    assert dg.sync_check() == dg.DEC_OK


def test_bounds_report_alone_and_calls_after_it():
    _wrong_append()
    assert dg.sync_check() == dg.DEC_EBOUNDS
    assert dg.sync_check() == dg.DEC_OK
    bt = pg.Batch([1, 70], [3000, 200], 14, 1, 128, 64, seed=101)
    for max_q in (1, 70):
        lse = torch.empty((bt.tokens, 14), device="cuda")
        out = dg.kv_attention(bt.q.cuda(), bt.device(dg, max_q=max_q), lse=lse)
        assert dg.sync_check() == dg.DEC_OK
        pg.check_attention(bt, out, lse)
