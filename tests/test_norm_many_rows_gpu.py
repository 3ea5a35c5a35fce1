"""The norm of as many rows as 32 bits count."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_decode_gemm_gb300 as dg  # noqa: E402


def test_norm_of_2_to_31_rows():
    from moe_decode_gemm_gb300 import build
    build.build()
    rows, H, size = (1 << 31) - 1, 8, 2
    if torch.cuda.mem_get_info()[0] < 3 * rows * H * size:
        pytest.skip("needs 100 GB")
    x = torch.full((rows, H), 2.0, dtype=torch.bfloat16, device="cuda")
    w = torch.arange(1, H + 1, device="cuda").to(torch.bfloat16)
    x[-1] = -4.0
    y = dg.dec_rmsnorm(x, w, eps=0.0)
    assert dg.sync_check() == dg.DEC_OK
    assert torch.equal(y[-1], -w)
    for first in range(0, rows - 1, 1 << 28):
        part = y[first:min(first + (1 << 28), rows - 1)]
        assert bool((part == w).all())
    del x, y, part
    torch.cuda.empty_cache()
