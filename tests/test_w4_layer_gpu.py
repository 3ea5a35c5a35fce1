"""The decode layer with its norms and 4-bit projections, stage by stage: each is
checked on the GPU's own bf16 input to it, the norm and the projections against
the definitions in 64 bits, the others against the same calls by themselves."""
from types import SimpleNamespace

import pytest

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
from moe_decode_gemm_gb300.stack import w4_layer  # noqa: E402

BF = torch.bfloat16
H, HQ, HKV, DIM, PAGE, E, I, K = 512, 4, 1, 128, 16, 16, 128, 4
QKV = (HQ + 2 * HKV) * DIM


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _near(got, want, bound):
    assert ((got.double().cpu() - want).abs() <= bound).all()


@pytest.mark.parametrize("mx", [False, True])
def test_steps(mx):
    moe = wl.LayerWeights(0, "cuda", H=H, KV=2 * HKV * DIM, E=E, I=I)
    Wqkv, Wo = ref.normal(1, QKV, H, std=0.04), ref.normal(2, H, HQ * DIM, std=0.04)
    w1, w2 = ((1 + ref.normal(s, H, std=0.2).float()).to(BF) for s in (3, 4))
    L = SimpleNamespace(Wqkv=dg.dec_quant_w4(Wqkv.cuda()), Wo=dg.dec_quant_w4(Wo.cuda()), w1=w1.cuda(), w2=w2.cuda(),
                        Wr=moe.Wr, W13=moe.W13, W2=moe.W2, Ws13=moe.Ws13, Ws2=moe.Ws2)
    vqkv = ref.weights(*ref.unpack(L.Wqkv.q, L.Wqkv.s, QKV, H))
    vo = ref.weights(*ref.unpack(L.Wo.q, L.Wo.s, H, HQ * DIM))
    angle = torch.rand(100, DIM // 2, generator=torch.Generator().manual_seed(5), dtype=torch.float64) * 6.28
    rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    pool = dg.KVPool(torch.zeros((1, 20, 2, HKV, PAGE, DIM), dtype=BF, device="cuda"), _i32([0] * 20),
                     torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), _i32([0, 0]))
    lens = [0, 0]
    for turn, new in enumerate(([20, 33], [1, 1], [3, 0])):
        M = sum(new)
        lens = [a + b for a, b in zip(lens, new)]
        dg.kv_resize(pool, _i32([0, 1]), _i32(lens))
        kv = pool.layer(0, _i32([0, new[0], M]), max_q=max(new))
        x = ref.activations(10 + turn, M, H).cuda()
        qkv = torch.empty(M, QKV, dtype=BF, device="cuda")
        o, a, r, out = (torch.empty(M, H, dtype=BF, device="cuda") for _ in range(4))
        got = w4_layer(L, x, kv, rope, qkv, o, a, r, out, K, mx=mx)
        assert got is out and dg.sync_check() == dg.DEC_OK
        # on a stream of its own, its passing tensors' memory wanted at once by another
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        q2, o2, a2, r2, out2 = (torch.empty_like(t) for t in (qkv, o, a, r, out))
        for _ in range(8):
            w4_layer(L, x, kv, rope, q2, o2, a2, r2, out2, K, mx=mx, stream=side)
            torch.full((M, 4 * H), float("nan"), dtype=BF, device="cuda")
            torch.full((M, H), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out2, out) and torch.equal(a2, a) and dg.sync_check(side) == dg.DEC_OK
        # the norm and the first projection
        n = (dg.dec_rmsnorm_mx if mx else dg.dec_rmsnorm)(x, L.w1)
        values = ref.mx8_values(n.q.cpu(), n.s.cpu()) if mx else n.cpu()
        _, want = ref.norm(x.cpu(), w1)
        step = torch.exp2(n.s.view(torch.uint8).cpu().double() - 127).repeat_interleave(32, 1) if mx else 0
        _near(values, want, (ref.HALF_E4M3 if mx else ref.HALF_BF) * 1.001 * want.abs() + 2.0 ** -10 * step + 1e-30)
        raw = dg.dec_linear_w4(n, L.Wqkv)
        want, s, spread = ref.linear(values, vqkv)
        _near(raw, want, ref.linear_bound(want, s, spread, H, mx))
        assert torch.equal(raw[:, HQ * DIM:], qkv[:, HQ * DIM:])       # keys and values as projected
        assert torch.equal(dg.kv_attention(qkv[:, :HQ * DIM], kv), o)
        # the second projection, the residual and its norm
        want, s, spread = ref.linear(o.cpu(), vo)
        _near(a, want, ref.linear_bound(want, s, spread, HQ * DIM, False))
        h, want = ref.norm(a.cpu(), w2, x.cpu())
        assert torch.equal(r.double().cpu(), h)
        n2 = dg.dec_rmsnorm(r, L.w2)
        _near(n2, want, ref.HALF_BF * 1.001 * want.abs() + 1e-30)
        assert torch.equal(dg.moe_decode(n2, L.Wr, L.W13, L.W2, L.Ws13, L.Ws2, K, residual=r), out)
