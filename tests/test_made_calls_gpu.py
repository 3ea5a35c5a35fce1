"""Projections, the MoE block and the paged cache's calls on a stream that is not the
current one: what they make themselves is not memory that the current stream
still reads."""
import pytest

import _paged as pg
import _w4 as ref
import workloads as wl

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_decode_gemm_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


import moe_decode_gemm_gb300 as dg  # noqa: E402

PAUSE = 100_000_000   # clocks: about 50 ms


def _call(name):
    x = ref.normal(1, 4, 512).cuda()
    if name in ("linear", "splitk"):
        W = ref.normal(2, 768, 512, std=0.03).cuda()
        if name == "linear":
            return lambda s: dg.dec_linear(x, W, stream=s)
        return lambda s: dg.dec_linear_splitk(x, W, 2, stream=s)
    if name == "moe":
        L = wl.LayerWeights(0, "cuda", H=512, KV=256, E=16, I=128)
        return lambda s: dg.moe_decode(x, L.Wr, L.W13, L.W2, L.Ws13, L.Ws2, 4, stream=s)
    if name == "add":
        return lambda s: dg.dec_add(x, x, stream=s)
    bt = pg.Batch([2, 3], [20, 40], 4, 2, 64, 16, seed=100)
    kv = bt.device(dg)
    if name == "append":
        rope = torch.ones(64, 64, device="cuda")
        qkv = pg.normal(pg.gen(1), 5, 8 * 64).cuda()
        return lambda s: dg.kv_append(qkv, kv, rope, stream=s)
    q = bt.q.cuda()
    return lambda s: dg.kv_attention(q, kv, stream=s)


@pytest.mark.parametrize("name", ["linear", "splitk", "moe", "add", "append", "attention"])
def test_a_freed_block_is_not_written_while_it_is_read(name):
    call = _call(name)
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.full_like(want.view(torch.int16), 77) for _ in range(4)]
    kept = [torch.empty_like(t) for t in blocks]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(PAUSE)
    for k, t in zip(kept, blocks):
        k.copy_(t)
    del blocks, t
    got = call(side)
    torch.cuda.synchronize()
    assert dg.sync_check() == dg.DEC_OK
    assert all(bool((k == 77).all()) for k in kept) and torch.equal(got, want)
