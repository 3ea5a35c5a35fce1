"""A single row's stride means nothing: a step of one token may pass a row of a
tensor of any width."""
import pytest

import _paged as pg
import moe_decode_gemm_gb300 as dg
from moe_decode_gemm_gb300 import paged

torch = pytest.importorskip("torch")

BF = torch.bfloat16


class _Handle:          # a handle's device, for tensors on the CPU
    device, _index = torch.device("cpu"), -1


@pytest.mark.parametrize("wide", [64, 65, 100, 128])
def test_stride_of_one_row(wide):
    t = torch.zeros((1, wide), dtype=BF)[:, :64]
    assert paged._rows("q", _Handle, t, BF) == (1, 64, 64)
    t = torch.zeros((3, wide), dtype=BF)[:, :64]
    assert paged._rows("q", _Handle, t, BF) == (3, 64, wide)


@pytest.mark.gpu
def test_one_token_of_wider_rows():
    from moe_decode_gemm_gb300 import build
    build.build()
    bt = pg.Batch([1], [70], 4, 2, 64, 16, seed=110)
    odd = lambda n, dtype=BF: torch.zeros((1, n + 3), dtype=dtype, device="cuda")[:, :n]  # noqa: E731
    kv = bt.device(dg)
    qkv, q, out, lse = odd(8 * 64), odd(4 * 64), odd(4 * 64), odd(4, torch.float32)
    x = pg.normal(pg.gen(1), 1, 8 * 64)
    qkv.copy_(x)
    rope = torch.zeros((71, 64), device="cuda")
    rope[:, :32] = 1
    dg.kv_append(qkv, kv, rope, q=q)
    dg.kv_attention(q, kv, out=out, lse=lse)
    assert dg.sync_check() == dg.DEC_OK
    k, v = x.view(8, 1, 64)[4:6], x.view(8, 1, 64)[6:]
    bt.k[0] = torch.cat([bt.k[0][:, :69], k], 1)
    bt.v[0] = torch.cat([bt.v[0][:, :69], v], 1)
    bt.q = x[:, :4 * 64]
    assert torch.equal(q.cpu(), bt.q)
    pg.check_attention(bt, out, lse)
