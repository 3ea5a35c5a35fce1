"""The tcgen05 attention kernel's warps at different paces: a CTA that has a pair
of row tiles whose second one has non-finite values to add, place by place,
before many pairs that have no second row tile and are over at once. The warps
of the second row tile come last to everything that is written per segment; the
kernel has to wait for them.
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


@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8)])
@pytest.mark.parametrize("long", [0, 30000])   # pairs drawn one by one; equal ranges
def test_second_row_tile_slower_than_many_short_pairs(hq, hkv, long):
    one = 128 // (hq // hkv)                   # tokens of a row tile
    n = 300
    new = [1 + b % 7 for b in range(n)]
    total = [new[b] + b % 30 for b in range(n)]
    slow = [0, 100, 101, 200]
    for b in slow:
        new[b] = total[b] = 2 * one
    if long:
        new[150], total[150] = 3, long
    bt = pg.Batch(new, total, hq, hkv, 64, 64, seed=90)
    for b in slow:
        k, v = bt.k[b], bt.v[b]
        v[:, one // 2::7, 3] = float("inf")
        v[:, one::5, 40] = float("nan")
        bt.put(b, k, v)
    kv, q = bt.device(dg, max_q=2 * one), bt.q.cuda()
    ref, rl, ab = pg.attention(bt)
    fine = ref.isfinite()
    first = None
    for _ in range(4):
        lse = torch.empty((bt.tokens, hq), device="cuda")
        out = dg.kv_attention(q, kv, lse=lse)
        assert dg.sync_check() == dg.DEC_OK and dg.last_attention() == "tc"
        o = out.double().cpu()
        assert torch.equal(o.isnan(), ref.isnan()) and torch.equal(o.isfinite(), fine)
        err = (o - ref)[fine].abs()
        assert bool((err <= (pg.U * ref.abs() + (pg.U + 2.0 ** -12) * ab)[fine]).all())
        assert bool(((lse.double().cpu() - rl).abs() <= 2.0 ** -16 * (1 + rl.abs())).all())
        bits = out.view(torch.int16)
        assert first is None or torch.equal(bits, first)
        first = bits


@pytest.mark.parametrize("hq,hkv,dim,new,total", [
    (14, 1, 128, 300, 9000), (8, 2, 64, 200, 7000), (28, 2, 128, 40, 20000)])
def test_long_chunks_in_a_row(hq, hkv, dim, new, total):
    # each call begins while the one before still reads memory as fast as it
    # can, so that the first key tiles land in any order
    bt = pg.Batch([new], [total], hq, hkv, dim, 64, seed=91)
    kv, q = bt.device(dg, max_q=new), bt.q.cuda()
    outs = [torch.empty((new, hq * dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lse = torch.empty((new, hq), device="cuda")
    for i in range(200):
        dg.kv_attention(q, kv, out=outs[i > 0], lse=lse)
    assert dg.sync_check() == dg.DEC_OK and dg.last_attention() == "tc"
    assert torch.equal(*outs)
    pg.check_attention(bt, outs[1], lse)
