"""Cases that measure the norm of the residual stream and the projections with 4-bit weights.

Three groups of calls that a decode layer with 4-bit weights makes:

  norm    the residual's addition and the root-mean-square norm, with an output in bf16 or in
          8 bits with a scale for each 32 values
  linear  y = x W^T with 4-bit weights and a scale for each 32 of a row, 1 to 64 tokens; x in
          bf16, or in 8 bits with scales as the norm gives it
  quant   bf16 weights to 4-bit weights with scales, in the layout that `linear` reads

`run` computes them with elementary torch operations in 32 bits, or, where `own` is true, by the
framework's calls. Widths are those of the layer stack and the projection table (2048, 4096, 7168,
8192, 16384), or generic odd ones.

4-bit weights: code c has its sign in bit 3 and stands for one of 0, .5, 1, 1.5, 2, 3, 4, 6 times
2^(b - 127), b the scale byte of its 32 weights. Codes lie as [N/128, K/128, 128 rows, 64 bytes],
element 2i of a row in the low half of byte i; scale bytes as [N/128, K/128, row % 32, row / 32, 4].
What lies past N and K is zero.
"""
import math

import torch

own = False

BF, F8, E8 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's token between two projections: the smallest call, all latency
        dict(name="norm_1_row", kind="norm", rows=1, width=7168, residual=True, mx=False, gap=0),
        # a full decode batch, for projections that take 8-bit activations
        dict(name="norm_64_rows_8bit", kind="norm", rows=64, width=7168, residual=True, mx=True, gap=0),
        # the tokens of a long prompt: bandwidth
        dict(name="norm_prompt", kind="norm", rows=8000, width=7168, residual=True, mx=False, gap=0),
        # part of a wider projection's columns, no residual
        dict(name="norm_slice_8bit", kind="norm", rows=3001, width=2048, residual=False, mx=True, gap=512),
        # one user: the output projection with the residual
        dict(name="linear_1_token", kind="linear", tokens=1, n=7168, k=7168, residual=True, mx=False, gap=0),
        # a few users' long reductions, few outputs
        dict(name="linear_8_tokens", kind="linear", tokens=8, n=2048, k=16384, residual=False, mx=False, gap=0),
        # the fused q|k|v projection of a medium batch
        dict(name="linear_16_tokens", kind="linear", tokens=16, n=8192, k=7168, residual=False, mx=False, gap=0),
        # the largest projection at the largest batch
        dict(name="linear_64_tokens", kind="linear", tokens=64, n=16384, k=7168, residual=False, mx=False, gap=0),
        # the same batch after a norm with 8-bit output
        dict(name="linear_64_8bit", kind="linear", tokens=64, n=7168, k=7168, residual=True, mx=True, gap=0),
        # a small odd head, read from a slice of a wider activation
        dict(name="linear_odd", kind="linear", tokens=5, n=1001, k=1992, residual=True, mx=False, gap=1000),
        # an odd matrix of a small model
        dict(name="quant_odd", kind="quant", n=1000, k=4008),
        # the largest projection, when a model is loaded
        dict(name="quant_large", kind="quant", n=16384, k=7168),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    kind = rng.choice(["norm", "linear", "linear", "quant"])
    mx = rng.random() < 0.4
    step = 32 if mx else 8
    if kind == "norm":
        return dict(kind=kind, rows=_loguniform(rng, 1, 8000), width=step * _loguniform(rng, 2, 16384 // step),
                    residual=rng.random() < 0.7, mx=mx, gap=8 * rng.choice([0, 0, 1, 37]))
    k = step * _loguniform(rng, 2, 16384 // step)
    n = _loguniform(rng, 16, 16384)
    if kind == "quant":
        return dict(kind=kind, n=n, k=8 * _loguniform(rng, 4, 1024))
    return dict(kind=kind, tokens=_loguniform(rng, 1, 64), n=n, k=k, residual=rng.random() < 0.5, mx=mx,
                gap=32 * rng.choice([0, 0, 1, 9]))


def work(case):
    if case["kind"] == "norm":
        t = case["rows"] * case["width"]
        out = t + t // 32 if case["mx"] else 2 * t
        return {"bytes": 2 * t + (4 * t if case["residual"] else 0) + out + 2 * case["width"], "flops": 4 * t}
    nk = case["n"] * case["k"]
    w4 = nk // 2 + nk // 32
    if case["kind"] == "quant":
        return {"bytes": 2 * nk + w4, "flops": 2 * nk}
    m, n, k = case["tokens"], case["n"], case["k"]
    x = m * k + m * k // 32 if case["mx"] else 2 * m * k
    return {"bytes": w4 + x + 2 * m * n * (2 if case["residual"] else 1), "flops": 2 * m * nk}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 250)


def draw(rng):
    most = max(_cost(c) for c in listed())
    case = _draw(rng)
    while _cost(case) > most:
        case = _draw(rng)
    return case


# ------------------------------------------------------------------ inputs
def _activations(gen, rows, width, gap):
    """A residual stream: most columns near one size, a few far larger; rows gap elements further apart."""
    x = torch.empty((rows, width + gap), dtype=BF, device="cuda").normal_(0.0, 1.0, generator=gen)
    size = torch.empty(width + gap, device="cuda").normal_(0.0, 0.7, generator=gen).exp_()
    return x.mul_(size.to(BF))[:, :width]


def _weights(gen, n, k):
    """A projection's weights: rows of different size, normal within."""
    w = torch.empty((n, k), dtype=BF, device="cuda").normal_(0.0, 0.02, generator=gen)
    return w.mul_(torch.empty((n, 1), device="cuda").uniform_(0.5, 2.0, generator=gen).to(BF))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = dict(case=case)
    if case["kind"] == "norm":
        st["x"] = _activations(gen, case["rows"], case["width"], case["gap"])
        st["w"] = torch.empty(case["width"], dtype=BF, device="cuda").normal_(1.0, 0.2, generator=gen)
        if case["residual"]:
            st["res"] = _activations(gen, case["rows"], case["width"], 0)
    elif case["kind"] == "quant":
        st["W"] = _weights(gen, case["n"], case["k"])
    else:
        st["q"], st["s"] = _quantise(_weights(gen, case["n"], case["k"]))
        x = _activations(gen, case["tokens"], case["k"], case["gap"])
        if case["mx"]:
            wide = case["k"] + case["gap"]
            st["x"] = torch.empty((case["tokens"], wide), dtype=F8, device="cuda")[:, :case["k"]]
            q, st["xs"] = _to_mx8(x.float())
            st["x"].copy_(q)
        else:
            st["x"] = x
        if case["residual"]:
            st["res"] = _activations(gen, case["tokens"], case["n"], 0)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if own:
        import moe_decode_gemm_gb300 as dg
        if case["kind"] == "norm":
            call = dg.dec_rmsnorm_mx if case["mx"] else dg.dec_rmsnorm
            got = call(st["x"], st["w"], st.get("res"), eps=EPS)
            y, h = got if case["residual"] else (got, None)
            out = dict(q=y.q, scale=y.s) if case["mx"] else dict(y=y)
            return dict(out, h=h) if case["residual"] else out
        if case["kind"] == "quant":
            w = dg.dec_quant_w4(st["W"])
            return dict(q=w.q, s=w.s)
        # the handles over weights and activations, which a program makes once and keeps
        if "w4" not in st:
            st["w4"] = dg.W4(st["q"], st["s"], case["n"], case["k"])
            st["in"] = dg.MX8(st["x"], st["xs"]) if case["mx"] else st["x"]
        return dg.dec_linear_w4(st["in"], st["w4"], residual=st.get("res"))
    if case["kind"] == "norm":
        return _norm(st)
    if case["kind"] == "quant":
        q, s = _quantise(st["W"])
        return dict(q=q, s=s)
    return _linear(st)


# ------------------------------------------------------------------ plain forms
def _pow2(e):
    """2^e in fp32 for -126 <= e <= 127, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(a, largest):
    """ceil(log2(a / largest)) without rounding, at least -127; largest = 1.75 * 2^8 or 1.5 * 2^2."""
    f, p = torch.frexp(a)
    g, r = math.frexp(largest)
    e = p - r + (f > g).int()
    return torch.where(a == 0, torch.full_like(e, -127), e.clamp(min=-127))


def _to_mx8(y):
    """fp32 [T, H] as e4m3 values and a power of two for each 32."""
    v = y.view(y.shape[0], -1, 32)
    e = _exponent(v.abs().amax(-1), 448.0)
    # in two steps, as 2^-e alone may not be a normal number
    half = -e // 2
    q = v * _pow2(half)[..., None] * _pow2(-e - half)[..., None]
    return q.to(F8).view(y.shape), (e + 127).to(torch.uint8).view(E8)


def _norm(st):
    case, x = st["case"], st["x"]
    out = {}
    if case["residual"]:
        out["h"] = (x.float() + st["res"].float()).to(BF)
        x = out["h"]
    h = x.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["w"].float()
    if case["mx"]:
        out["q"], out["scale"] = _to_mx8(y)
    else:
        out["y"] = y.to(BF)
    return out


def _quantise(W):
    """bf16 [N, K] as codes and scale bytes in the layout that the projections read."""
    n, k = W.shape
    nt, kc = -(-n // 128), -(-k // 128)
    w = torch.zeros((nt * 128, kc * 128), device="cuda")
    w[:n, :k] = W
    v = w.view(nt * 128, kc * 4, 32)
    e = _exponent(v.abs().amax(-1), 6.0)
    half = -e // 2
    v = v * _pow2(half)[..., None] * _pow2(-e - half)[..., None]
    a = v.abs()
    # halfway between two values: to the one whose last bit is 0
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code = (code | (torch.signbit(v).byte() << 3)).view(nt, 128, kc, 64, 2)
    q = (code[..., 0] | (code[..., 1] << 4)).permute(0, 2, 1, 3).contiguous()
    s = (e + 127).byte().view(nt, 4, 32, kc, 4).permute(0, 3, 2, 1, 4).contiguous()
    return q, s


def _dequantise(q, s, n, k):
    nt, kc = q.shape[:2]
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    code = torch.stack([q & 15, q >> 4], -1).view(nt, kc, 128, 4, 32)
    e = s.permute(0, 1, 3, 2, 4).reshape(nt, kc, 128, 4).int() - 127
    w = value[code.int()] * _pow2(e)[..., None]
    return w.view(nt, kc, 128, 128).permute(0, 2, 1, 3).reshape(nt * 128, kc * 128)[:n, :k]


def _linear(st):
    case = st["case"]
    w = _dequantise(st["q"], st["s"], case["n"], case["k"])
    x = st["x"].float()
    if case["mx"]:
        e = st["xs"].view(torch.uint8).int() - 127
        x = (x.view(x.shape[0], -1, 32) * _pow2(e)[..., None]).view(x.shape)
    y = torch.matmul(x, w.t())
    if case["residual"]:
        y = y + st["res"].float()
    return y.to(BF)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _ceil_log2(a, largest):
    """The least e, at least -127, with a <= largest * 2^e: by trial around the logarithm."""
    e = torch.floor(torch.log2(a.clamp(min=1e-300) / largest)) - 1
    e = e + (a > largest * torch.exp2(e)).double()
    e = e + (a > largest * torch.exp2(e)).double()
    e = e + (a > largest * torch.exp2(e)).double()
    return torch.clamp(e, min=-127.0)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "norm":
        return _exact_norm(case, st)
    if case["kind"] == "quant":
        return _exact_quant(case, st)
    n, k = case["n"], case["k"]
    rows, cols = torch.arange(n, device="cuda")[:, None], torch.arange(k, device="cuda")[None]
    byte = st["q"][rows // 128, cols // 128, rows % 128, cols % 128 // 2]
    code = torch.where(cols % 2 == 1, byte >> 4, byte & 15).double()
    sign, m = torch.where(code >= 8, -1.0, 1.0), code % 8
    # 0, 1/2 in steps of 1/2 up to 2, then 3, 4, 6
    size = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    scale = st["s"][rows // 128, cols // 128, rows % 32, rows % 128 // 32, cols % 128 // 32].double()
    w = sign * size * torch.exp2(scale - 127)
    x = st["x"].double()
    if case["mx"]:
        x = x * torch.exp2(st["xs"].view(torch.uint8).double() - 127).repeat_interleave(32, 1)
    y = x @ w.T
    return y + st["res"].double() if case["residual"] else y


def _exact_norm(case, st):
    h = st["x"].double()
    out = {}
    if case["residual"]:
        h = (h + st["res"].double()).to(BF).double()  # the residual stream is kept in bf16
        out["h"] = h
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["width"] + EPS) * st["w"].double()
    if not case["mx"]:
        return dict(out, y=y)
    g = y.unflatten(1, (-1, 32))
    e = _ceil_log2(g.abs().amax(2), 448.0)
    v = g / torch.exp2(e)[..., None]
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=1e-300))), min=-6.0) - 3)
    return dict(out, q=(torch.round(v / step) * step).flatten(1), scale=torch.exp2(e))


def _exact_quant(case, st):
    n, k = case["n"], case["k"]
    nt, kc = (n + 127) // 128, (k + 127) // 128
    w = torch.nn.functional.pad(st["W"].double(), (0, kc * 128 - k, 0, nt * 128 - n))
    w = w.reshape(nt, 128, kc, 4, 32)
    e = _ceil_log2(w.abs().amax(4), 6.0)
    v = w / torch.exp2(e)[..., None]
    del w
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=1e-300))), min=0.0) - 1)
    a = (torch.round(v / step) * step).abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)) + 8 * torch.signbit(v)
    del v, step, a
    code = code.reshape(nt, 128, kc, 64, 2)
    q = code[..., 0] + 16 * code[..., 1]
    return dict(q=q.transpose(1, 2).long(), s=(e + 127).reshape(nt, 4, 32, kc, 4).permute(0, 3, 2, 1, 4).long())
