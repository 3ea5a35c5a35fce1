"""64-bit definitions of the norm and of the projections with 4-bit weights, on
the CPU, and their inputs."""
from __future__ import annotations

import torch

BF, F8, E8 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu
HALF_BF = 2.0 ** -8     # half a bf16 step, relative to the value
HALF_E4M3 = 2.0 ** -4   # half an e4m3 step, relative to a normal value
VALUES = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                      dtype=torch.float64)


def normal(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(BF)


def activations(seed, rows, width):
    """Columns of very different size, as in a residual stream."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(0.9 * torch.randn(width, generator=g))
    return (torch.randn((rows, width), generator=g) * size).to(BF)


def random_codes(seed, n, k):
    """Every code, and scale bytes of sizes that weights have."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
    scales = torch.randint(112, 125, (n, -(-k // 32)), generator=g, dtype=torch.uint8)
    return codes, scales


def weights(codes, scales):
    """The weights' values: float64 [N, K]."""
    w = VALUES[codes.long()] * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :codes.shape[1]]
    return w


def unpack(q, s, n, k):
    """Codes [N, K] and scale bytes [N, ceil(K/32)] from the packed form, place by place."""
    q, s = q.cpu(), s.cpu()
    i, j = torch.arange(n)[:, None], torch.arange(k)[None]
    byte = q[i // 128, j // 128, i % 128, (j % 128) // 2]
    g = torch.arange(-(-k // 32))[None]
    return (torch.where(j % 2 == 1, byte >> 4, byte & 15),
            s[i // 128, g // 4, i % 32, i % 128 // 32, g % 4])


def least_exponent(a, largest):
    """The least e >= -127 with a <= largest * 2^e."""
    e = torch.full(a.shape, -127, dtype=torch.float64)
    for _ in range(300):
        more = a > largest * torch.exp2(e)
        if not more.any():
            return e
        e = e + more.double()
    raise AssertionError("not finite")


def quantise(W):
    """dec_quant_w4's definition: codes and scale bytes of float64 weights."""
    n, k = W.shape
    g = torch.nn.functional.pad(W, (0, -k % 32)).reshape(n, -1, 32)
    e = least_exponent(g.abs().amax(2), 6.0)
    v = (g / torch.exp2(e)[..., None]).reshape(n, -1)[:, :k]
    d = (v.abs()[..., None] - VALUES[:8]).abs()
    # the nearest; of two equally near the even code
    odd = torch.arange(8) % 2 * 1e-9
    code = (d + odd).argmin(-1)
    return (code + 8 * torch.signbit(v)).to(torch.uint8), (e + 127).to(torch.uint8)


def linear(x, w, res=None):
    """(y, sum of |products|, largest of each 32 k times |w|) in float64."""
    x = x.double()
    m, k = x.shape
    y = x @ w.t()
    most = torch.nn.functional.pad(x.abs(), (0, -k % 32)).reshape(m, -1, 32).amax(2)
    spread = most.repeat_interleave(32, 1)[:, :k] @ w.abs().t()
    a = x.abs() @ w.abs().t()
    if res is not None:
        y, a = y + res.double(), a + res.double().abs()
    return y, a, spread


def linear_bound(y, a, spread, k, mx):
    """Half a bf16 step of the result; fp32 sums (at most one rounding, of a whole
    step, for each MMA of 32 k, for the 32 products in it, for the ranks of a
    cluster and the halves: 2^-23 each of the sum of magnitudes); and what a
    bf16 token may lose as two e4m3 numbers: 2^-22 of its group's largest."""
    return HALF_BF * y.abs() + (k / 32 + 48) * 2.0 ** -23 * a + (0 if mx else 2.0 ** -22) * spread + 1e-37


def mx8_values(q, s):
    return q.double() * torch.exp2(s.view(torch.uint8).double() - 127).repeat_interleave(32, 1)


def norm(x, w, res=None, eps=1e-6):
    """(h, y) in float64; h is kept in bf16."""
    h = x.double()
    if res is not None:
        h = (h + res.double()).to(BF).double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * w.double()
    return h, y
