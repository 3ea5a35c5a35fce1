"""Windows over a cache that has dropped the pages before them: their table
entries are -1 and their contents gone, which no row can tell.
"""
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


@pytest.mark.parametrize("force", ["mma", "tc"])
@pytest.mark.parametrize("dim,page", [(128, 16), (128, 32), (64, 16), (64, 64), (128, 256)])
@pytest.mark.parametrize("window", [1, 17, 50, 300])
def test_dropped_pages_are_not_looked_up(monkeypatch, force, dim, page, window):
    monkeypatch.setenv("DEC_FORCE", force)
    new = [1, 1, 3, 1, 2, 40, 1]
    total = [700, 513, 260, 128, 97, 640, 30]
    bt = pg.Batch(new, total, 14, 1, dim, page, seed=95)
    for b, (n, m) in enumerate(zip(new, total)):
        first = max(0, m - n - window + 1)       # the first position that its first token sees
        gone = first // page
        bt.cache[bt.table[b, :gone].long()] = float("nan")
        bt.table[b, :gone] = -1
    kv, q = bt.device(dg, max_q=max(new)), bt.q.cuda()
    lse = torch.empty((bt.tokens, 14), device="cuda")
    out = dg.kv_attention(q, kv, lse=lse, window=window)
    assert dg.sync_check() == dg.DEC_OK and dg.last_attention() == force
    pg.check_attention(bt, out, lse, window)
