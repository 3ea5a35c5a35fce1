"""Windows and positions near 2^31."""
import ctypes

import pytest

import _paged as pg
import moe_decode_gemm_gb300 as dg
from moe_decode_gemm_gb300 import paged

torch = pytest.importorskip("torch")

A = 1 << 20          # an aligned fake pointer: never dereferenced


@pytest.mark.parametrize("page", [16, 64, 256])
def test_rows_whose_last_key_tile_would_end_past_32_bits(page):
    from moe_decode_gemm_gb300 import build
    build.build()
    for width, ok in (((1 << 31) // page - 1, False), ((1 << 31) // page - 256 // page, True)):
        if page == 256 and not ok:
            continue   # (2^31 / 256 - 1) pages end 256 positions before 2^31
        v = paged._View(cache=A, page_stride=2 * page * 64, pages=10, heads=1, page_size=page, dim=64,
                        table=A, table_stride=width, width=width, table_rows=1, rows=None, cu_q=A,
                        kv_len=A, batch=1, max_q=1)
        # (tokens = 0: an allowed view is refused for that, before anything runs)
        rc = dg.lib().kv_attention(ctypes.byref(v), A, 64, A, 64, None, 0, 1, 0.1, 0, None)
        assert rc == (dg.DEC_EINVAL if ok else dg.DEC_EUNSUPPORTED)


@pytest.mark.gpu
@pytest.mark.parametrize("force", ["mma", "tc"])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 20, 1 << 30])
def test_largest_windows_where_some_tokens_see_nothing(monkeypatch, force, window):
    # chunks longer than their sequences: the first tokens' positions are negative
    from moe_decode_gemm_gb300 import build
    build.build()
    monkeypatch.setenv("DEC_FORCE", force)
    bt = pg.Batch([60, 3, 90, 1, 5], [20, 3, 61, 0, 100], 8, 2, 64, 16, seed=130)
    lse = torch.empty((bt.tokens, 8), device="cuda")
    out = dg.kv_attention(bt.q.cuda(), bt.device(dg, max_q=90), lse=lse, window=window)
    assert dg.sync_check() == dg.DEC_OK and dg.last_attention() == force
    pg.check_attention(bt, out, lse)
