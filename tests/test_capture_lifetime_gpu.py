"""A captured graph stays valid when later calls need more of the library's
workspace: what its kernels' arguments point to is neither freed nor laid out
anew, and its arrival counters are zero at rest.

Each test captures a small call, makes larger ones, and only then replays: the
replay's bits are those of the eager call. For the paged cache it is first
checked, before anything is replayed, that the larger calls took no device
memory (their workspace has one size).
"""
import math

import pytest

import _paged as pg
import workloads as wl

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_decode_gemm_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


import moe_decode_gemm_gb300 as dg  # noqa: E402

BF = torch.bfloat16


def _capture(call):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def _replayed(g, outs, want):
    for t in outs:
        t.fill_(0)
    g.replay()
    torch.cuda.synchronize()
    assert dg.sync_check() == dg.DEC_OK
    for t, w in zip(outs, want):
        assert torch.equal(t, w)


def _attention(seed, new, total, hq, hkv, dim):
    bt = pg.Batch(new, total, hq, hkv, dim, 64, seed=seed)
    kv, q = bt.device(dg, max_q=max(new)), bt.q.cuda()
    out = torch.zeros((bt.tokens, hq * dim), dtype=BF, device="cuda")
    lse = torch.zeros((bt.tokens, hq), device="cuda")
    return (lambda: dg.kv_attention(q, kv, out=out, lse=lse)), [out, lse]


@pytest.mark.parametrize("new,total,hq,hkv,dim", [
    ([1], [3000], 8, 1, 64), ([1] * 20, [900] * 20, 14, 1, 64), ([40], [2000], 8, 2, 64)])
def test_attention_outlives_larger_paged_calls(new, total, hq, hkv, dim):
    small, outs = _attention(80, new, total, hq, hkv, dim)
    larger = [_attention(81, [100], [2500], 14, 1, 128)[0],
              _attention(82, [2] * 30, [700] * 30, 14, 2, 128)[0],
              _attention(83, [1], [9000], 28, 2, 128)[0]]
    pool = pg.random_pool(84, seqs=40, width=9, page=16, pages=9001, layers=1, fill=0.02)
    pool = dg.KVPool(*(t.cuda() for t in pool))
    larger.append(lambda: dg.kv_compact(pool))

    def grow():
        for call in larger:
            call()
        torch.cuda.synchronize()
    small()
    grow()            # every kernel's code is on the device
    dg.shutdown()     # and no workspace is
    small()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    g = _capture(small)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    grow()
    assert torch.cuda.mem_get_info()[0] > free - (1 << 20)
    _replayed(g, outs, want)
    grow()            # and the larger ones outlive the replay
    _replayed(g, outs, want)


def _block(M, H, E, I, k, key):
    n = lambda *a: wl.normal_bf16_cuda(*a)  # noqa: E731
    x, Wr = n((M, H), 1.0, *key, "x"), n((E, H), 1.0 / math.sqrt(H), *key, "Wr")
    W13, W2 = n((E, 2 * I, H), 0.02, *key, "W13"), n((E, H, I), 0.02, *key, "W2")
    S13, S2 = n((2 * I, H), 0.02, *key, "S13"), n((H, I), 0.02, *key, "S2")
    out = torch.zeros((M, H), dtype=BF, device="cuda")
    return (lambda: dg.moe_decode(x, Wr, W13, W2, S13, S2, k, out=out)), [out]


@pytest.mark.parametrize("M", [1, 6, 40])
def test_block_outlives_blocks_with_more_experts_and_tokens(M):
    dg.shutdown()
    small, outs = _block(M, 512, 16, 128, 4, ("life", M))
    small()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    g = _capture(small)
    # more tiles' counters; then a layout that the present buffer might hold
    for shape in ((64, 512, 16, 128, 4), (64, 512, 18, 128, 4), (64, 2048, 64, 256, 8)):
        big, big_outs = _block(*shape, ("life", shape))
        big()
        torch.cuda.synchronize()
        big_want = [t.clone() for t in big_outs]
        for _ in range(2):
            _replayed(g, outs, want)
        big()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(big_outs, big_want))


def test_projection_outlives_larger_ones():
    dg.shutdown()
    x, W = wl.normal_bf16_cuda((20, 1000), 1.0, "life", "x"), wl.normal_bf16_cuda((600, 1000), 0.02, "life", "W")
    y = torch.zeros((20, 600), dtype=BF, device="cuda")
    small = lambda: dg.dec_linear_splitk(x, W, 3, y=y)  # noqa: E731
    small()
    torch.cuda.synchronize()
    want = y.clone()
    g = _capture(small)
    for n in (4000, 16384):
        dg.dec_linear(wl.normal_bf16_cuda((64, 1000), 1.0, "life", n),
                      wl.normal_bf16_cuda((n, 1000), 0.02, "life", n, "W"))
        _replayed(g, [y], [want])


def test_replay_after_a_time_out_and_a_larger_block():
    dg.shutdown()
    small, outs = _block(2, 512, 16, 128, 4, ("life", "reset"))
    small()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    g = _capture(small)
    _block(64, 2048, 64, 256, 8, ("life", "reset", "big"))[0]()
    dg.selftest_timeout(2_000_000)   # 2 ms on a barrier nobody completes
    assert dg.sync_check() == dg.DEC_ETIMEOUT
    _replayed(g, outs, want)
