"""Projections with 4-bit weights, their quantisation, and the norm before them,
against the definitions in 64 bits."""
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

BF, F8, E8 = ref.BF, ref.F8, ref.E8


def _check(y, want, bound):
    assert dg.sync_check() == dg.DEC_OK
    y = y.double().cpu()
    bad = ~((y - want).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%d of %d outside the bound, first at %s: %r, want %r within %r"
                             % (int(bad.sum()), bad.numel(), i, y[i].item(), want[i].item(),
                                bound[i].item()))


def _strided(t, gap):
    """The same rows, further apart, NaN between them."""
    if not gap:
        return t.cuda()
    wide = torch.full((t.shape[0], t.shape[1] + gap), float("nan"), device="cuda").to(t.dtype)
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def _mx8(seed, m, k, gap=0):
    q = ref.normal(seed, m, k, std=60.0).float().clamp(-448, 448).to(F8)
    s = torch.randint(110, 130, (m, k // 32), generator=torch.Generator().manual_seed(seed)).to(torch.uint8)
    return dg.MX8(_strided(q, gap), s.cuda()), ref.mx8_values(q, s)


# ------------------------------------------------------------------ products
SHAPES = [(1, 8), (5, 40), (127, 120), (128, 128), (129, 136), (300, 1000), (1001, 1992), (520, 4104),
          (2048, 1024), (7168, 256), (40, 9000)]


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 40, 57, 64])
@pytest.mark.parametrize("N,K", SHAPES)
def test_linear(M, N, K):
    codes, scales = ref.random_codes(N + K, N, K)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    x = ref.activations(M, M, K)
    res = ref.normal(M + 1, M, N, std=3.0) if (M + N) % 2 else None
    y = dg.dec_linear_w4(_strided(x, 8 * (M % 3)), W, residual=None if res is None else res.cuda())
    want, a, spread = ref.linear(x, ref.weights(codes, scales), res)
    _check(y, want, ref.linear_bound(want, a, spread, K, False))


@pytest.mark.parametrize("M", [1, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(1, 32), (129, 160), (300, 1024), (1001, 1984), (7168, 256), (40, 9024)])
def test_linear_of_8_bit_tokens(M, N, K):
    codes, scales = ref.random_codes(N + K, N, K)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    x, values = _mx8(M, M, K, gap=16 * (M % 3))
    res = ref.normal(M + 1, M, N, std=3.0) if (M + N) % 2 else None
    y = dg.dec_linear_w4(x, W, residual=None if res is None else res.cuda())
    want, a, spread = ref.linear(values, ref.weights(codes, scales), res)
    _check(y, want, ref.linear_bound(want, a, spread, K, True))


@pytest.mark.parametrize("M", [1, 8, 16, 32, 64])
def test_linear_large(M):
    N, K = 8192 + 77, 7168
    codes, scales = ref.random_codes(9, N, K)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    x = ref.activations(M, M, K)
    y = dg.dec_linear_w4(x.cuda(), W)
    want, a, spread = ref.linear(x, ref.weights(codes, scales))
    _check(y, want, ref.linear_bound(want, a, spread, K, False))
    for _ in range(3):
        assert torch.equal(dg.dec_linear_w4(x.cuda(), W), y)  # the same bits from run to run


@pytest.mark.parametrize("M,mx", [(1, False), (6, False), (16, False), (32, False), (64, False), (11, True),
                                  (25, True), (64, True)])
def test_linear_of_more_tiles_than_sms(M, mx):
    """153 tiles of 128 outputs, an odd number, the last of 44."""
    N, K = 152 * 128 + 44, 640
    codes, scales = ref.random_codes(10, N, K)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    x = _mx8(M, M, K) if mx else (ref.activations(M, M, K),) * 2
    y = dg.dec_linear_w4(x[0] if mx else x[0].cuda(), W)
    want, a, spread = ref.linear(x[1], ref.weights(codes, scales))
    _check(y, want, ref.linear_bound(want, a, spread, K, mx))


def test_linear_of_tokens_with_a_far_larger_value():
    """Elements down to 2^-15 of the largest of their 32 are taken exactly: with
    a weight of 0 under the largest, only fp32 sums and the output round."""
    M, N, K = 3, 64, 256
    codes, scales = ref.random_codes(3, N, K)
    codes[:, ::32] = 0
    x = ref.normal(5, M, K).abs() + 1
    x[:, ::32] = 2.0 ** 14 * 1.5
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    y = dg.dec_linear_w4(x.to(BF).cuda(), W)
    want, a, _ = ref.linear(x.to(BF), ref.weights(codes, scales))
    _check(y, want, ref.linear_bound(want, a, torch.zeros_like(a), K, False))


@pytest.mark.parametrize("M", [3, 20])
def test_linear_of_the_largest_bf16(M):
    """The weights bring the products back: nothing overflows on the way."""
    N, K = 100, 256
    codes, scales = ref.random_codes(8, N, K)
    x = ref.normal(9, M, K).sign() * 3.3e38
    y = dg.dec_linear_w4(x.to(BF).cuda(), dg.W4.pack(codes.cuda(), (scales - 20).cuda()))
    want, a, spread = ref.linear(x.to(BF), ref.weights(codes, scales - 20))
    _check(y, want, ref.linear_bound(want, a, spread, K, False))


@pytest.mark.parametrize("power", [-120, -60, 60, 100])
def test_linear_of_tokens_near_the_ends_of_bf16(power):
    M, N, K = 5, 200, 512
    codes, scales = ref.random_codes(4, N, K)
    x = (ref.normal(6, M, K).double() * 2.0 ** power).to(BF)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    y = dg.dec_linear_w4(x.cuda(), W)
    want, a, spread = ref.linear(x, ref.weights(codes, scales))
    # below the normal numbers of fp32 and bf16: a step of theirs
    _check(y, want, ref.linear_bound(want, a, spread, K, False) + 2.0 ** -126)


def test_linear_of_tokens_that_are_not_finite():
    """The token's outputs are NaN, the others' are as without it."""
    M, N, K = 9, 300, 700 // 8 * 8
    codes, scales = ref.random_codes(5, N, K)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    x = ref.normal(7, M, K)
    clean = dg.dec_linear_w4(x.cuda(), W)
    x[2, 130], x[5, 0], x[8, K - 1] = float("inf"), float("nan"), float("-inf")
    y = dg.dec_linear_w4(x.cuda(), W)
    bad = torch.tensor([2, 5, 8])
    good = torch.tensor([0, 1, 3, 4, 6, 7])
    assert y[bad].isnan().all()
    assert torch.equal(y[good], clean[good])


def test_linear_of_weights_that_are_not_finite():
    N, K = 200, 256
    codes, scales = ref.random_codes(6, N, K)
    scales[17, 3] = 255
    y = dg.dec_linear_w4(ref.normal(8, 4, K).cuda(), dg.W4.pack(codes.cuda(), scales.cuda()))
    assert y[:, 17].isnan().all() and y.isnan().sum() == 4


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("N,K", [(1, 8), (3, 40), (128, 128), (130, 264), (1000, 1000), (257, 4104)])
def test_quant(N, K):
    W = ref.normal(N + K, N, K, std=0.02)
    W[0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])   # halfway, scale 1
    if K > 40:
        W[N // 2, 32:64] = 0
        W[N - 1, 0:32] *= 2.0 ** -118                                       # subnormal
        W[N - 1, 32:40] = 3e38
    w4 = dg.dec_quant_w4(_strided(W, 24))
    assert dg.sync_check() == dg.DEC_OK
    codes, scales = ref.quantise(W.double())
    got = ref.unpack(w4.q, w4.s, N, K)
    assert torch.equal(got[1], scales)
    assert torch.equal(got[0], codes)
    # what lies past N and K, through the layout's own words
    again = dg.W4.pack(codes, scales)
    assert torch.equal(w4.q.cpu(), again.q) and torch.equal(w4.s.cpu(), again.s)


def test_quant_of_weights_that_are_not_finite():
    W = ref.normal(1, 40, 128)
    W[3, 40], W[7, 100] = float("inf"), float("nan")
    w4 = dg.dec_quant_w4(W.cuda())
    codes, scales = ref.unpack(w4.q, w4.s, 40, 128)
    assert scales[3, 1] == 255 and scales[7, 3] == 255 and (scales == 255).sum() == 2
    assert (codes[3, 32:64] == 0).all() and (codes[7, 96:] == 0).all()


# ------------------------------------------------------------------ the norm
WIDTHS = [8, 32, 40, 96, 1000, 1024, 2048, 7168, 8200, 16384, 40000, 65536]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 310])
def test_norm(rows, H):
    if rows * H > 4000000:
        rows = 17
    x, w = ref.activations(H, rows, H), (1 + ref.normal(2, H, std=0.3).float()).to(BF)
    # fp32: a sum of squares with a chain of at most 64 + 10 roundings (half of
    # it in the root), rsqrtf (2 steps), three products
    rel = ref.HALF_BF + 48 * 2.0 ** -24
    h, want = ref.norm(x, w)
    _check(dg.dec_rmsnorm(_strided(x, 8), w.cuda()), want, rel * want.abs() + 1e-38)
    res = ref.normal(3, rows, H)
    h, want = ref.norm(x, w, res)
    y, hh = dg.dec_rmsnorm(x.cuda(), w.cuda(), _strided(res, 16))
    _check(y, want, rel * want.abs() + 1e-38)
    assert torch.equal(hh.double().cpu(), h)


def _check_mx(got, want):
    assert dg.sync_check() == dg.DEC_OK
    s = got.s.view(torch.uint8).cpu().double() - 127
    a = want.reshape(want.shape[0], -1, 32).abs().amax(2)
    e = ref.least_exponent(a, 448.0)
    # a group's largest value may lie so near a border that fp32 sees it beyond
    near = ((a / (448 * torch.exp2(e)) - 1).abs() < 2.0 ** -18) | ((a / (224 * torch.exp2(e)) - 1).abs() < 2.0 ** -18)
    assert ((s == e) | near).all()
    v = ref.mx8_values(got.q.cpu(), got.s.cpu())
    step = torch.exp2(s).repeat_interleave(32, 1)
    bound = torch.maximum((ref.HALF_E4M3 + 2.0 ** -18) * want.abs(), 2.0 ** -10 * step)
    assert ((v - want).abs() <= bound).all()


@pytest.mark.parametrize("H", [32, 96, 1024, 2048, 7168, 8224, 16384, 40000, 65536])
@pytest.mark.parametrize("rows", [1, 3, 310])
def test_norm_in_8_bits(rows, H):
    if rows * H > 4000000:
        rows = 17
    x, w = ref.activations(H, rows, H), (1 + ref.normal(2, H, std=0.3).float()).to(BF)
    x[0, :32] = 0
    h, want = ref.norm(x, w)
    _check_mx(dg.dec_rmsnorm_mx(_strided(x, 24), w.cuda()), want)
    res = ref.normal(3, rows, H)
    h, want = ref.norm(x, w, res)
    y, hh = dg.dec_rmsnorm_mx(x.cuda(), w.cuda(), res.cuda())
    _check_mx(y, want)
    assert torch.equal(hh.double().cpu(), h)


@pytest.mark.parametrize("rows,H", [(2, 7168), (400, 1024), (1000, 2048), (40, 16384)])
def test_norm_in_8_bits_is_rounded_once(rows, H):
    """Every value and scale is the definition's: fp32 alone puts one in a million on
    the other side of a rounding border."""
    x, w, res = ref.activations(H, rows, H), ref.normal(2, H), ref.normal(3, rows, H)
    got, _ = dg.dec_rmsnorm_mx(x.cuda(), w.cuda(), res.cuda())
    _, want = ref.norm(x, w, res)
    g = want.reshape(rows, -1, 32)
    e = ref.least_exponent(g.abs().amax(2), 448.0)
    v = g / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1e-30))).clamp(min=-6) - 3)
    assert torch.equal(got.s.view(torch.uint8).cpu().double() - 127, e)
    assert torch.equal(got.q.double().cpu(), (torch.round(v / step) * step).reshape(rows, H))


def test_norm_of_exact_products():
    """Where nothing is cut off nothing is marked as cut off: borders and scales of
    exact values (mean 1, eps 0)."""
    x = ref.normal(4, 3, 64).sign()
    w = torch.tensor([1.75, 1.0625, 1.1875, 0.4375, 0.0, 1.0, -1.0625, 0.5] * 8).to(BF)
    got = dg.dec_rmsnorm_mx(x.cuda(), w.cuda(), eps=0.0)
    v = x.float() * w.float()
    assert (got.s.view(torch.uint8) == 127 - 8).all()      # 1.75 = 448 * 2^-8
    assert torch.equal(got.q.cpu().view(torch.uint8), (v * 256).to(F8).view(torch.uint8))


def test_norm_of_rows_of_one_size():
    """Roots that are rational (rows of +-c, eps 0): products that lie on a border are
    neither rounded up nor given a larger scale."""
    c = torch.arange(1, 128, 2).to(BF)[:, None]
    x = c * ref.normal(5, 64, 96).sign()
    w = torch.tensor([1.75, 1.0625, 1.1875, 0.4375, 0.0, 1.0, -1.0625, 0.5] * 12).to(BF)
    got = dg.dec_rmsnorm_mx(x.cuda(), w.cuda(), eps=0.0)
    v = x.float().sign() * w.float()
    assert (got.s.view(torch.uint8) == 127 - 8).all()
    assert torch.equal(got.q.cpu().float(), (v * 256).to(F8).float())


def test_norm_of_the_least_products():
    """Where products are below fp32's normal numbers the 8-bit values still are the
    definition's, as near as fp32's least step."""
    x, w = ref.normal(6, 16, 256), (ref.normal(7, 256).float() * 2.0 ** -124).to(BF)
    x[8:] *= 2.0 ** -4
    _, want = ref.norm(x, w)
    got = dg.dec_rmsnorm_mx(x.cuda(), w.cuda())
    s = got.s.view(torch.uint8).cpu().double() - 127
    have = got.q.double().cpu().reshape(16, 8, 32) * torch.exp2(s)[..., None]
    want = want.reshape(16, 8, 32)
    # half a step of an e4m3 (2^-4 of the value, 2^-10 of the scale below the normal
    # ones) and a step of fp32's least numbers
    assert ((have - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * torch.exp2(s)[..., None] + 2.0 ** -148).all()


@pytest.mark.parametrize("mx", [False, True])
def test_norm_in_place(mx):
    """h over the residual or x, y over x; rows behind the last are left alone."""
    x, res, w = ref.normal(1, 6, 512).cuda(), ref.normal(2, 8, 512).cuda(), ref.normal(3, 512).cuda()
    call = dg.dec_rmsnorm_mx if mx else dg.dec_rmsnorm
    y0, h0 = call(x, w, res[:6])
    tail = res[6:].clone()
    keep = x.clone()
    if mx:
        out = dg.MX8(torch.zeros((6, 512), device="cuda").to(F8), torch.zeros((6, 16), dtype=torch.uint8, device="cuda"))
        y, h = call(x, w, res[:6], h=res[:6], out=out)
        assert y is out and torch.equal(y.q.view(torch.uint8), y0.q.view(torch.uint8))
        assert torch.equal(y.s.view(torch.uint8), y0.s.view(torch.uint8)) and torch.equal(x, keep)
    else:
        y, h = call(x, w, res[:6], h=res[:6], y=x)
        assert y is x and torch.equal(y, y0)
    assert torch.equal(h, h0) and torch.equal(res[:6], h0) and torch.equal(res[6:], tail)


def test_norm_of_rows_that_are_not_finite():
    x, w = ref.normal(1, 4, 128), torch.ones(128, dtype=BF)
    clean = dg.dec_rmsnorm_mx(x.cuda(), w.cuda())
    x[1, 40], x[2, 3] = float("nan"), float("inf")
    got = dg.dec_rmsnorm_mx(x.cuda(), w.cuda())
    s = got.s.view(torch.uint8).cpu()
    assert (s[1] == 255).all() and s[2, 0] == 255 and (s[2, 1:] == 0).all()  # inf: the others are 0
    assert got.q.cpu().float()[1].isnan().all()
    for r in (0, 3):
        assert torch.equal(got.q[r].view(torch.uint8), clean.q[r].view(torch.uint8))


def test_norm_of_zeros_and_of_a_zero_eps():
    w = torch.ones(64, dtype=BF, device="cuda")
    assert (dg.dec_rmsnorm(torch.zeros((2, 64), dtype=BF, device="cuda"), w) == 0).all()
    x = ref.normal(1, 2, 64)
    _, want = ref.norm(x, w.cpu(), eps=0.0)
    _check(dg.dec_rmsnorm(x.cuda(), w, eps=0.0), want, (ref.HALF_BF + 2.0 ** -18) * want.abs())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("M", [1, 8, 20, 64])
def test_norm_and_projections_in_a_row(M):
    """norm -> 4-bit projection -> norm in 8 bits -> 4-bit projection with the
    residual, and the same as a captured graph, replayed on other tokens."""
    H, N = 1024, 768
    w1, w2 = (ref.normal(i, H, std=0.2).float().add(1).to(BF) for i in (1, 2))
    Wa, Wb = ref.normal(3, H, H, std=0.03), ref.normal(4, H, H, std=0.03)
    qa, qb = dg.dec_quant_w4(Wa.cuda()), dg.dec_quant_w4(Wb.cuda())
    va, vb = (ref.weights(*ref.unpack(w.q, w.s, H, H)) for w in (qa, qb))
    x = torch.empty((M, H), dtype=BF, device="cuda")
    w1d, w2d = w1.cuda(), w2.cuda()

    def step():
        y = dg.dec_rmsnorm(x, w1d)
        a = dg.dec_linear_w4(y, qa)
        z, h = dg.dec_rmsnorm_mx(a, w2d, x)
        return y, a, z, h, dg.dec_linear_w4(z, qb, residual=h)

    def check(x0, got):
        y, a, z, h, out = got
        _, want = ref.norm(x0, w1)
        _check(y, want, (ref.HALF_BF + 2.0 ** -18) * want.abs())
        want, s, spread = ref.linear(y.cpu(), va)
        _check(a, want, ref.linear_bound(want, s, spread, H, False))
        hw, want = ref.norm(a.cpu(), w2, x0)
        assert torch.equal(h.double().cpu(), hw)
        _check_mx(z, want)
        want, s, spread = ref.linear(ref.mx8_values(z.q.cpu(), z.s.cpu()), vb, h.cpu())
        _check(out, want, ref.linear_bound(want, s, spread, H, True))

    x0 = ref.activations(5, M, H)
    x.copy_(x0)
    check(x0, step())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (6, 7):
        x0 = ref.activations(seed, M, H)
        x.copy_(x0)
        g.replay()
        torch.cuda.synchronize()
        check(x0, got)


def test_on_another_stream():
    """Two streams with calls of their own at once."""
    N, K = 640, 1024
    codes, scales = ref.random_codes(1, N, K)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    xs = [ref.normal(i, 20, K).cuda() for i in range(2)]
    w = torch.ones(K, dtype=BF, device="cuda")
    want = [dg.dec_linear_w4(dg.dec_rmsnorm(x, w), W) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(dg.dec_linear_w4(dg.dec_rmsnorm(xs[i], w, stream=s), W, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


# ------------------------------------------------------------------ the index-checking build
def test_index_checks():
    """Every kind of call through the build that checks its indexes."""
    dbg = dg._load(dg.DEBUG_LIB_PATH)
    old = dg.use_library(dbg)
    try:
        for M, N, K in ((1, 130, 264), (7, 2048, 1024), (16, 1001, 520), (30, 300, 1000), (64, 257, 512)):
            W = ref.normal(N, N, K, std=0.05)
            w4 = dg.dec_quant_w4(W.cuda())
            x, res = ref.activations(M, M, K), ref.normal(M + 1, M, N)
            y = dg.dec_linear_w4(x.cuda(), w4, residual=res.cuda())
            want, a, spread = ref.linear(x, ref.weights(*ref.unpack(w4.q, w4.s, N, K)), res)
            _check(y, want, ref.linear_bound(want, a, spread, K, False))
        for rows, H in ((1, 40), (5, 7168), (700, 96), (700, 2048), (330, 8200)):
            x, w, res = ref.activations(H, rows, H), ref.normal(1, H), ref.normal(2, rows, H)
            h, want = ref.norm(x, w, res)
            y, hh = dg.dec_rmsnorm(_strided(x, 8), w.cuda(), res.cuda())
            _check(y, want, (ref.HALF_BF + 48 * 2.0 ** -24) * want.abs() + 1e-38)
            if H % 32 == 0:
                _check_mx(dg.dec_rmsnorm_mx(x.cuda(), w.cuda(), res.cuda())[0], want)
        x, values = _mx8(3, 33, 1024)
        codes, scales = ref.random_codes(3, 300, 1024)
        y = dg.dec_linear_w4(x, dg.W4.pack(codes.cuda(), scales.cuda()))
        want, a, spread = ref.linear(values, ref.weights(codes, scales))
        _check(y, want, ref.linear_bound(want, a, spread, 1024, True))
    finally:
        torch.cuda.synchronize()
        dg.use_library(old)


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("M,N,K,mx", [(1, 2048, 4096, False), (12, 8192, 4096, False), (40, 1024, 4096, False),
                                      (64, 1024, 4096, True)])
def test_waits_that_run_out(M, N, K, mx):
    """With no time to wait the kernel gives up, says so and ends; the next call is right."""
    codes, scales = ref.random_codes(1, N, K)
    W = dg.W4.pack(codes.cuda(), scales.cuda())
    if mx:
        x, values = _mx8(M, M, K)
    else:
        values = ref.activations(M, M, K)
        x = values.cuda()
    first = dg.dec_linear_w4(x, W)
    assert dg.sync_check() == dg.DEC_OK
    old = dg.set_wait_timeout_ns(0)
    try:
        dg.dec_linear_w4(x, W)
        assert dg.sync_check() in (dg.DEC_OK, dg.DEC_ETIMEOUT)
    finally:
        dg.set_wait_timeout_ns(old)
    assert torch.equal(dg.dec_linear_w4(x, W), first)
    assert dg.sync_check() == dg.DEC_OK
    want, a, spread = ref.linear(values, ref.weights(codes, scales))
    _check(first, want, ref.linear_bound(want, a, spread, K, mx))
