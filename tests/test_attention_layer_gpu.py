"""The decode layer with its attention over a paged cache, step by step.

Each stage is checked on the GPU's own bf16 input to it: the attention and the
append against the 64-bit plain forms, the projections against the fp64 oracle,
the MoE block against the same block called by itself (equal bits).
"""
import pytest

import _paged as pg
import oracle
import workloads as wl
from _util import assert_within_tol, to_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_decode_gemm_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


import moe_decode_gemm_gb300 as dg  # noqa: E402
from moe_decode_gemm_gb300.stack import attention_layer  # noqa: E402

BF = torch.bfloat16
H, HQ, HKV, DIM, PAGE, E, I, K = 512, 4, 1, 128, 16, 16, 128, 4
KV = 2 * HKV * DIM


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_two_layers(graph):
    layers = [wl.LayerWeights(l, "cuda", H=H, KV=KV, E=E, I=I) for l in range(2)]
    g = pg.gen(60)
    w = [(pg.normal(g, DIM), pg.normal(g, DIM)) for _ in layers]
    wd = [(a.cuda(), b.cuda()) for a, b in w]
    ang = torch.rand(200, DIM // 2, generator=g, dtype=torch.float64) * 6.28
    rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    rd = rope.cuda()
    data = torch.full((2, 40, 2, HKV, PAGE, DIM), float("nan"), dtype=BF, device="cuda")
    pool = dg.KVPool(data, _i32([0] * 40), torch.full((3, 8), -1, dtype=torch.int32, device="cuda"),
                     _i32([0] * 3))
    past = [[[None, None] for _ in range(3)] for _ in layers]
    lens = [0, 0, 0]
    stream = torch.cuda.Stream()

    def step(new, replay):
        M = sum(new)
        for s, n in enumerate(new):
            lens[s] += n
        dg.kv_resize(pool, _i32([0, 1, 2]), _i32(lens))
        cu = _i32([0] + torch.tensor(new).cumsum(0).tolist())
        x = [pg.normal(g, M, H).cuda()] + [torch.empty(M, H, dtype=BF, device="cuda") for _ in layers]
        b = [dict(qkv=torch.empty(M, H + KV, dtype=BF, device="cuda"), o=torch.empty_like(x[0]),
                  r=torch.empty_like(x[0])) for _ in layers]
        raw = []

        def run(st):
            for l, L in enumerate(layers):
                kv = pool.layer(l, cu, max_q=max(new))
                attention_layer(L, x[l], kv, rd, b[l]["qkv"], b[l]["o"], b[l]["r"], x[l + 1], K,
                                *wd[l], stream=st)

        torch.cuda.synchronize()
        run(stream)
        stream.synchronize()
        if replay:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=stream):
                run(stream)
            want = [t.clone() for t in x[1:]]
            for t in x[1:]:
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            gr.replay()
            torch.cuda.synchronize()
            for t, u in zip(x[1:], want):
                assert torch.equal(t, u)
        assert dg.sync_check() == dg.DEC_OK
        for l, L in enumerate(layers):
            raw = dg.dec_linear(x[l], L.Wqkv)          # before the in-place norm and rotation
            ref, A = oracle.linear(wl.torch_to_bits(x[l]), wl.torch_to_bits(L.Wqkv))
            assert_within_tol(to_f64(raw), ref, A, "q|k|v")
            pos = torch.tensor([lens[s] - n + t for s, n in enumerate(new) for t in range(n)])
            y = pg.append(raw.cpu(), w[l], rope, pos, DIM, HQ, HKV, DIM, False)
            q = b[l]["qkv"][:, :H].double().cpu().view(M, HQ, DIM)
            big = y[:, :HQ].abs().amax(-1, keepdim=True)
            assert bool(((q - y[:, :HQ]).abs() <= pg.U * y[:, :HQ].abs() + 2.0 ** -18 * big).all())
            assert torch.equal(b[l]["qkv"][:, H:], raw[:, H:])
            bt = pg.Batch(new, lens, HQ, HKV, DIM, PAGE)
            cache = data[l].cpu()
            table = pool.table.cpu()
            bt.q = b[l]["qkv"][:, :H].cpu()
            for s in range(3):
                pages = table[s, :-(-lens[s] // PAGE)].long()
                rows = cache[pages].movedim(0, 2).flatten(2, 3)[:, :, :lens[s]]
                bt.k[s], bt.v[s] = rows[0], rows[1]
                old = past[l][s]
                if old[0] is not None:   # what was there stays
                    n = old[0].shape[1]
                    assert torch.equal(bt.k[s][:, :n], old[0]) and torch.equal(bt.v[s][:, :n], old[1])
                past[l][s] = [rows[0].clone(), rows[1].clone()]
            kref = y[:, HQ:HQ + HKV]
            at = 0
            for s, n in enumerate(new):
                got = bt.k[s][:, lens[s] - n:].transpose(0, 1).double()
                kb = kref[at:at + n]
                lim = pg.U * kb.abs() + 2.0 ** -18 * kb.abs().amax(-1, keepdim=True)
                assert bool(((got - kb).abs() <= lim).all())
                at += n
            ref, _, ab = pg.attention(bt)
            o = b[l]["o"].double().cpu()
            assert bool(((o - ref).abs() <= pg.U * ref.abs() + (pg.U + 2.0 ** -12) * ab).all())
            oo, oA = oracle.linear(wl.torch_to_bits(b[l]["o"]), wl.torch_to_bits(L.Wo))
            rref, rA = oracle.residual(wl.torch_to_bits(x[l]), oo, oA)
            assert_within_tol(to_f64(b[l]["r"]), rref, rA, "r")
            r = b[l]["r"]
            again = dg.moe_decode(r, L.Wr, L.W13, L.W2, L.Ws13, L.Ws2, K, residual=r)
            assert torch.equal(again, x[l + 1])

    step([20, 5, 33], False)      # prompts
    step([1, 1, 1], graph)        # one token each
    step([3, 0, 2], graph)        # a few drafts, one sequence idle
