"""Calls on a stream that is not the current one, with the caching allocator's
freed blocks at hand: a block that the current stream still reads is not written
by the call, and an output that the current stream still reads is not written by
the next call."""
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

BF = torch.bfloat16
M, N, K = 40, 1024, 1024
PAUSE = 100_000_000   # clocks: about 50 ms


def _flat(got):
    if isinstance(got, (tuple, list)):
        return [t for g in got for t in _flat(g)]
    if isinstance(got, dg.MX8):
        return [got.q.view(torch.uint8), got.s.view(torch.uint8)]
    if isinstance(got, dg.W4):
        return [got.q, got.s]
    return [got]


@pytest.fixture(scope="module")
def calls():
    x, res, w = ref.normal(1, M, K).cuda(), ref.normal(2, M, K).cuda(), ref.normal(3, K).cuda()
    W = ref.normal(4, N, K, std=0.03).cuda()
    w4, mx = dg.dec_quant_w4(W), dg.dec_rmsnorm_mx(x, w)
    return {
        "norm": lambda s: dg.dec_rmsnorm(x, w, res, stream=s),
        "norm_mx": lambda s: dg.dec_rmsnorm_mx(x, w, res, stream=s),
        "linear": lambda s: dg.dec_linear_w4(x[:9], w4, stream=s),
        "linear with work space": lambda s: dg.dec_linear_w4(x, w4, stream=s),
        "linear_mx": lambda s: dg.dec_linear_w4(mx, w4, stream=s),
        "quant": lambda s: dg.dec_quant_w4(W, stream=s),
    }


NAMES = ["norm", "norm_mx", "linear", "linear with work space", "linear_mx", "quant"]


@pytest.mark.parametrize("name", NAMES)
def test_a_freed_block_is_not_written_while_it_is_read(calls, name):
    call = calls[name]
    want = [t.clone() for t in _flat(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' and the work space's sizes, freed while they are still to be read
    sizes = [t.numel() * t.element_size() for t in want] + [dg.lib().dec_linear_w4_work(M, K)]
    blocks = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    kept = [torch.empty_like(t) for t in blocks]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(PAUSE)
    for k, t in zip(kept, blocks):
        k.copy_(t)
    del blocks, t
    got = _flat(call(side))
    torch.cuda.synchronize()
    assert all(bool((k == 77).all()) for k in kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_an_output_is_not_written_anew_while_it_is_read(calls, name):
    call = calls[name]
    want = [t.clone() for t in _flat(call(None))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _flat(call(side))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(PAUSE)
    kept = [t.clone() for t in got]
    sizes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):   # what the stream's next calls write
        again = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(4)]
    more = _flat(call(side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
    assert all(torch.equal(a, b) for a, b in zip(more, want)) and len(again) == 4 * len(want)


@pytest.mark.parametrize("name", NAMES)
def test_captured_on_a_stream_beside_the_capturing_one(calls, name):
    """The call's tensors are of the graph's own memory, and each replay writes them."""
    call = calls[name]
    want = [t.clone() for t in _flat(call(None))]
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in _flat(got):
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_flat(got), want))
