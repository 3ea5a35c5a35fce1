"""Projections with 4-bit weights that stall: every CTA waits for tokens that never
come, gives up within its bound, says so and ends, and the next call is right.
Each source of the tokens, with one CTA to a tile and with clusters, and more
ring slots than the rings hold."""
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


@pytest.mark.parametrize("M,N,K,mx", [
    (1, 2048, 4096, False), (7, 20000, 5120, False), (12, 8192, 4096, False), (12, 130, 264, False),
    (40, 1024, 4096, False), (20, 20000, 2560, False), (64, 1024, 4096, True), (9, 20000, 2560, True)])
def test_stalled_call(M, N, K, mx):
    codes, scales = ref.random_codes(1, N, K)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    x = ref.activations(M, M, K).cuda()
    if mx:
        x = dg.dec_rmsnorm_mx(x, torch.ones(K, dtype=ref.BF, device="cuda"))
    first = dg.dec_linear_w4(x, W)
    assert dg.sync_check() == dg.DEC_OK
    old = dg.use_library(dg._load(dg.DEBUG_LIB_PATH))
    L = dg.lib()
    limit = dg.set_wait_timeout_ns(2_000_000)
    try:
        assert L.dec_debug_stall(1) == 0
        for _ in range(2):
            dg.dec_linear_w4(x, W)
            assert dg.sync_check() == dg.DEC_ETIMEOUT
        assert L.dec_debug_stall(0) == 1
        dg.set_wait_timeout_ns(limit)
        assert torch.equal(dg.dec_linear_w4(x, W), first)
        assert dg.sync_check() == dg.DEC_OK
    finally:
        L.dec_debug_stall(0)
        dg.set_wait_timeout_ns(limit)
        torch.cuda.synchronize()
        dg.use_library(old)
    assert torch.equal(dg.dec_linear_w4(x, W), first) and dg.sync_check() == dg.DEC_OK
