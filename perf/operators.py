"""Cases that measure the paged key/value cache's operators.

Three groups of calls that a decode step with attention makes:

  append     the heads of a fused q|k|v projection are normalised and rotated,
             and the new keys and values go to their places in a paged cache
  attention  the new tokens' queries over the cache: one token per sequence,
             a few draft tokens, a chunk over a long past, whole prompts
  pages      growing and rolling back sequences, forking, copying and
             compacting the pages of a cache of several layers

`run` computes them with elementary torch operations in 32 bits, or, where
`own` is true, by the framework's calls. Heads are those of the layer stack
(56 query heads of 128, 4 key/value heads: q 7168 wide, k|v 1024 wide) or
generic (32 and 8 heads of 64).
"""
import math
import random

import numpy as np
import torch

own = False

BF = torch.bfloat16
STACK = dict(hq=56, hkv=4, dim=128)   # q 7168 = 56 x 128, kv 1024 = 2 x 4 x 128
SMALL = dict(hq=32, hkv=8, dim=64)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user, a short past: the smallest call of a decode step, all latency
        dict(name="attn_1_token_short", kind="attention", batch=1, q=1, past_lo=508, past_hi=508,
             page=64, window=0, mix=1, **STACK),
        # a full decode batch with long pasts of very different lengths: bandwidth
        dict(name="attn_64_tokens_long", kind="attention", batch=64, q=1, past_lo=2000,
             past_hi=32000, page=64, window=0, mix=2, **STACK),
        # a few draft tokens for each sequence, small heads, a sliding window
        dict(name="attn_drafts_window", kind="attention", batch=24, q=5, past_lo=1, past_hi=9000,
             page=16, window=1024, mix=3, **SMALL),
        # one chunk of a long prompt over what is cached already
        dict(name="attn_chunk_over_32k", kind="attention", batch=1, q=512, past_lo=32300,
             past_hi=32300, page=64, window=0, mix=4, **STACK),
        # whole prompts of ragged lengths, nothing cached before them
        dict(name="attn_prompts_ragged", kind="attention", batch=4, q=2047, past_lo=0, past_hi=0,
             page=128, window=0, mix=5, **STACK),
        # the new token of one user
        dict(name="append_1_token", kind="append", batch=1, q=1, past_lo=700, past_hi=700, page=64,
             rot=128, interleaved=False, norm=True, mix=6, **STACK),
        # a full decode batch
        dict(name="append_64_tokens", kind="append", batch=64, q=1, past_lo=1, past_hi=250,
             page=16, rot=128, interleaved=False, norm=True, mix=7, **STACK),
        # the chunks of several prompts, half of each head rotated
        dict(name="append_chunks", kind="append", batch=5, q=1999, past_lo=0, past_hi=600, page=32,
             rot=64, interleaved=True, norm=True, mix=8, **STACK),
        # rejected draft tokens rolled back and room made for the next step's
        dict(name="pages_step", kind="step", layers=4, seqs=64, width=64, page=16, pool=4096,
             fill=0.6, n=64, mix=9, **STACK),
        # beams dropped and forked anew from the best ones
        dict(name="pages_fork", kind="fork", layers=4, seqs=64, width=64, page=32, pool=3000,
             fill=0.5, n=48, mix=10, **STACK),
        # pages taken to other places, as for swapping
        dict(name="pages_copy", kind="copy", layers=4, seqs=16, width=64, page=64, pool=2500,
             fill=0.5, n=701, mix=11, **STACK),
        # a pool that has run for long, half of it free in small holes
        dict(name="pages_compact", kind="compact", layers=4, seqs=96, width=128, page=32,
             pool=9000, fill=0.5, n=0, mix=12, **STACK),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    heads = rng.choice([STACK, STACK, SMALL, dict(hq=24, hkv=8, dim=128), dict(hq=8, hkv=8, dim=64)])
    kind = rng.choice(["token", "drafts", "chunk", "prompts", "append", "append", "step", "fork",
                       "copy", "compact"])
    page, mix = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 30)
    if kind in ("token", "drafts", "chunk", "prompts"):
        batch = {"token": _loguniform(rng, 1, 64), "drafts": _loguniform(rng, 1, 32),
                 "chunk": rng.randint(1, 3), "prompts": rng.randint(1, 4)}[kind]
        q = {"token": 1, "drafts": rng.randint(2, 6), "chunk": _loguniform(rng, 20, 700),
             "prompts": _loguniform(rng, 100, 2047)}[kind]
        hi = 0 if kind == "prompts" else _loguniform(rng, 100, 32000)
        lo = 0 if kind == "prompts" else max(1, hi // rng.randint(1, 16))
        return dict(kind="attention", batch=batch, q=q, past_lo=lo, past_hi=hi, page=page,
                    window=rng.choice([0, 0, 0, 300, 2000]), mix=mix, **heads)
    if kind == "append":
        batch = _loguniform(rng, 1, 64)
        return dict(kind="append", batch=batch, q=max(1, _loguniform(rng, 1, 8000) // batch),
                    past_lo=0, past_hi=rng.randint(0, 300), page=page,
                    rot=rng.choice([heads["dim"], heads["dim"] // 2]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.75, mix=mix, **heads)
    pool = _loguniform(rng, 300, 6000) * 32 // page
    seqs = rng.randint(8, min(96, pool // 6))
    width = max(2, min(128, 2 * pool // seqs))
    n = {"step": rng.randint(1, seqs), "fork": rng.randint(1, max(1, seqs // 2)),
         "copy": rng.randint(1, pool // 3), "compact": 0}[kind]
    return dict(kind=kind, layers=rng.randint(1, 4), seqs=seqs, width=width, page=page, pool=pool,
                fill=rng.uniform(0.2, 0.5), n=n, mix=mix, **heads)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 250)


def draw(rng):
    most = max(_cost(c) for c in listed())
    case = _draw(rng)
    while _cost(case) > most:
        case = _draw(rng)
    return case


def _lengths(case):
    """New tokens and total length (with them) of each sequence."""
    rng = random.Random(case["mix"])
    b, q = case["batch"], case["q"]
    lo, hi = case["past_lo"], case["past_hi"]
    past = [_loguniform(rng, lo + 1, hi + 1) - 1 for _ in range(b)]
    new = [q if q == 1 else rng.randint(max(1, q // 2), q) for _ in range(b)]
    new[0], past[0] = q, hi
    if b >= 8:
        new[b // 2] = 0            # a sequence that takes no part in this step
    return new, [p + n for p, n in zip(past, new)]


def _pool_lengths(case):
    """Length of each sequence of a pool: about `fill` of its pages in use."""
    rng = random.Random(case["mix"])
    per = case["fill"] * case["pool"] / case["seqs"]
    most = case["width"] * case["page"]
    return [max(1, min(most, int(per * case["page"] * rng.uniform(0.4, 1.6))))
            for _ in range(case["seqs"])]


def _shared(lens, s, page):
    """Full pages that sequence s has in common with the one before it: every third sequence
    begins with the same prompt."""
    return min(lens[s], lens[s - 1]) // page // 2 if s % 3 == 2 else 0


def _parts(case):
    """Sequences of a pool case: those that the call works on."""
    n, s = case["n"], case["seqs"]
    return list(range(n)), list(range(s - n, s))


# ------------------------------------------------------------------ inputs
def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(gen, *shape, std=1.0):
    return torch.empty(shape, dtype=BF, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 31))
    if case["kind"] in ("attention", "append"):
        return _prepare_batch(case, gen, rng)
    return _prepare_pool(case, gen, rng)


def _prepare_batch(case, gen, rng):
    new, total = _lengths(case)
    page, dim, hq, hkv = case["page"], case["dim"], case["hq"], case["hkv"]
    blocks = [-(-n // page) for n in total]
    pages = sum(blocks) + 3
    order = rng.permutation(pages)
    table = np.full((len(new), max(blocks) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    tokens = sum(new)
    st = dict(case=case, table=torch.from_numpy(table).cuda(),
              cu_q=_i32([0] + list(np.cumsum(new))), kv_len=_i32(total),
              cache=_normal(gen, pages, 2, hkv, page, dim))
    if case["kind"] == "attention":
        st["q"] = _normal(gen, tokens, hq * dim)
    else:
        # a projection's output: the columns of a few heads larger than the others
        st["qkv"] = _normal(gen, tokens, (hq + 2 * hkv) * dim, std=0.7)
        st["wq"] = (1.0 + 0.2 * _normal(gen, dim).float()).to(BF) if case["norm"] else None
        st["wk"] = (1.0 + 0.2 * _normal(gen, dim).float()).to(BF) if case["norm"] else None
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        angle = torch.arange(max(total) + 1, dtype=torch.float64)[:, None] * freq
        st["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    return st


def _prepare_pool(case, gen, rng):
    page, pool, width = case["page"], case["pool"], case["width"]
    lens = _pool_lengths(case)
    order = rng.permutation(pool)
    table = np.full((case["seqs"], width), -1, dtype=np.int32)
    refs = np.zeros(pool, dtype=np.int32)
    at = 0
    for s, n in enumerate(lens):
        blocks = -(-n // page)
        common = _shared(lens, s, page)
        table[s, :common] = table[s - 1, :common]
        table[s, common:blocks] = order[at:at + blocks - common]
        at += blocks - common
        np.add.at(refs, table[s, :blocks], 1)
    st = dict(case=case, table=torch.from_numpy(table).cuda(), refs=torch.from_numpy(refs).cuda(),
              lens=_i32(lens), info=torch.zeros(4, dtype=torch.int32, device="cuda"),
              data=_normal(gen, case["layers"], pool, 2, case["hkv"], page, case["dim"]))
    first, last = _parts(case)
    if case["kind"] == "step":
        # k tokens rolled back (0 to 5), then room for up to 40 more
        back = [max(0, lens[s] - int(rng.randint(0, 6))) for s in first]
        st["seqs"], st["back"] = _i32(first), _i32(back)
        st["ahead"] = _i32([min(width * page, n + 1 + int(rng.randint(0, 40))) for n in back])
    elif case["kind"] == "fork":
        left = case["seqs"] - case["n"]
        st["src"], st["dst"] = _i32(rng.randint(0, left, case["n"])), _i32(last)
    elif case["kind"] == "copy":
        pages = rng.permutation(pool)[:2 * case["n"]]
        st["src"], st["dst"] = _i32(pages[:case["n"]]), _i32(pages[case["n"]:])
    else:
        st["table0"], st["refs0"] = st["table"].clone(), st["refs"].clone()
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        import moe_decode_gemm_gb300 as dg
        # the handle over the cache, which a program makes once and keeps
        if "kv" not in st:
            st["kv"] = (dg.PagedKV(st["cache"], st["table"], st["cu_q"], st["kv_len"],
                                   max_q=case["q"])
                        if kind in ("attention", "append") else
                        dg.KVPool(st["data"], st["refs"], st["table"], st["lens"], st["info"]))
        kv = st["kv"]
    if kind == "attention":
        lse = torch.empty((st["q"].shape[0], case["hq"]), dtype=torch.float32, device="cuda")
        if own:
            return dg.kv_attention(st["q"], kv, window=case["window"], lse=lse), lse
        return _attention(st, lse)
    if kind == "append":
        if own:
            q = dg.kv_append(st["qkv"], kv, st["rope"], st["wq"], st["wk"],
                             interleaved=case["interleaved"])
            return q, st["cache"]
        return _append(st), st["cache"]
    if kind == "step":
        if own:
            dg.kv_resize(kv, st["seqs"], st["back"])
            dg.kv_resize(kv, st["seqs"], st["ahead"])
        else:
            _resize(st, st["seqs"], st["back"])
            _resize(st, st["seqs"], st["ahead"])
    elif kind == "fork":
        if own:
            dg.kv_free(kv, st["dst"])
            dg.kv_fork(kv, st["src"], st["dst"])
        else:
            _resize(st, st["dst"], torch.zeros_like(st["dst"]))
            _fork(st)
    elif kind == "copy":
        if own:
            dg.kv_copy(kv, st["src"], st["dst"])
        else:
            st["data"][:, st["dst"].long()] = st["data"][:, st["src"].long()]
    else:
        # the scattered state again, so that every pass has the same to move
        st["table"].copy_(st["table0"])
        st["refs"].copy_(st["refs0"])
        if own:
            dg.kv_compact(kv)
        else:
            _compact(st)
    out = dict(data=st["data"], table=st["table"], refs=st["refs"], lens=st["lens"])
    if kind != "copy":
        out["info"] = st["info"]
    return out


# ------------------------------------------------------------------ plain forms
def _places(st, tokens):
    """Sequence, place in its chunk and position in its cache of each new token."""
    cu = st["cu_q"].long()
    tok = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    t = tok - cu[b]
    return b, t, st["kv_len"].long()[b] - (cu[1:] - cu[:-1])[b] + t


def _attention(st, lse):
    case, q = st["case"], st["q"]
    page, dim, hq, hkv = case["page"], case["dim"], case["hq"], case["hkv"]
    tokens, batch, most = q.shape[0], case["batch"], st["table"].shape[1] * case["page"]
    b, t, pos = _places(st, tokens)
    rows = torch.zeros((batch, case["q"], hkv, hq // hkv, dim), device="cuda")
    rows[b, t] = q.float().view(tokens, hkv, hq // hkv, dim)
    at = torch.full((batch, case["q"]), -1, dtype=torch.long, device="cuda")
    at[b, t] = pos
    kv = st["cache"][st["table"].long().clamp(min=0)]                 # [B, W, 2, hkv, page, dim]
    k, v = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, batch, hkv, most, dim).float()
    key = torch.arange(most, device="cuda")
    live = key < st["kv_len"].long()[:, None]                         # [B, most]
    zero = torch.zeros((), device="cuda")
    k = torch.where(live[:, None, :, None], k, zero)
    v = torch.where(live[:, None, :, None], v, zero)
    rows = rows.permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, dim)   # rows: group, then token
    s = torch.matmul(rows * (1.0 / math.sqrt(dim)), k.transpose(2, 3))
    seen = (key <= at[:, :, None]) & live[:, None, :]                 # [B, q, most]
    if case["window"]:
        seen &= key > at[:, :, None] - case["window"]
    s = s.view(batch, hkv, hq // hkv, case["q"], most)
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), zero, m)
    s = s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(batch, hkv, -1, most), v).view(batch, hkv, hq // hkv, case["q"], dim)
    o = torch.where(l > 0, o / l, zero)
    lse.copy_((m + l.log())[..., 0].permute(0, 3, 1, 2)[b, t].reshape(tokens, hq))
    return o.permute(0, 3, 1, 2, 4)[b, t].reshape(tokens, hq * dim).to(BF), lse


def _append(st):
    case, qkv = st["case"], st["qkv"]
    page, dim, hq, hkv, rot = case["page"], case["dim"], case["hq"], case["hkv"], case["rot"]
    tokens = qkv.shape[0]
    b, _, pos = _places(st, tokens)
    x = qkv.view(tokens, hq + 2 * hkv, dim)
    y = x[:, :hq + hkv].float()
    if case["norm"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
        y = torch.cat([y[:, :hq] * st["wq"].float(), y[:, hq:] * st["wk"].float()], 1)
    cos, sin = st["rope"][pos][:, None].split(rot // 2, -1)
    r = y[..., :rot]
    if case["interleaved"]:
        a, c = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2)
    else:
        a, c = r.chunk(2, -1)
        r = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
    y = torch.cat([r, y[..., rot:]], -1).to(BF)
    where = st["table"][b, pos // page].long()
    st["cache"][where, 0, :, pos % page] = y[:, hq:]
    st["cache"][where, 1, :, pos % page] = x[:, hq + hkv:]
    return y[:, :hq].reshape(tokens, hq * dim)


def _free_first(refs):
    """Page numbers, the free ones first and ascending, and how many are free."""
    return torch.sort((refs > 0).int(), stable=True)[1], (refs == 0).sum()


def _note(st, lacking, copied):
    st["info"][0] = lacking
    st["info"][1] = (st["refs"] == 0).sum()
    st["info"][2] = copied


def _take(st, seqs, old, new, drop, alloc, source):
    """Table rows `old` of `seqs` become: -1 where `drop`, the lowest free pages in order where
    `alloc`, else `new`. Pages of `source` (or -1) are copied to where they are replaced."""
    order, free = _free_first(st["refs"])
    total = alloc.sum()
    ok = total <= free
    rank = alloc.flatten().cumsum(0).view(alloc.shape) - 1
    fresh = order[rank.clamp(0, order.numel() - 1)].int()
    rows = torch.where(alloc, fresh, torch.where(drop, torch.full_like(new, -1), new))
    rows = torch.where(ok, rows, old)
    st["refs"].index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).int().flatten())
    st["refs"].index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).int().flatten())
    copy = alloc & (source >= 0) & ok
    st["data"][:, rows[copy].long()] = st["data"][:, source[copy].long()]
    st["table"][seqs] = rows
    return ok, torch.where(ok, 0, total - free), copy.sum()


def _resize(st, seqs, length):
    seqs, page = seqs.long(), st["case"]["page"]
    was, rows = st["lens"][seqs], st["table"][seqs]
    old, new = -(-was // page), -(-length // page)
    col = torch.arange(rows.shape[1], device="cuda")
    drop = col >= new[:, None]
    last = col == (new - 1)[:, None]
    shared = st["refs"][rows.clamp(min=0).long()] > 1
    own_copy = last & shared & ((length < was) & (length % page != 0))[:, None]
    alloc = own_copy | ((col >= old[:, None]) & (col < new[:, None]))
    ok, lacking, copied = _take(st, seqs, rows, rows, drop, alloc,
                                torch.where(own_copy, rows, torch.full_like(rows, -1)))
    st["lens"][seqs] = torch.where(ok, length, was)
    _note(st, lacking, copied)


def _fork(st):
    src, dst, page = st["src"].long(), st["dst"].long(), st["case"]["page"]
    was, rows, old = st["lens"][src], st["table"][src], st["table"][dst]
    col = torch.arange(rows.shape[1], device="cuda")
    alloc = (col == (was // page)[:, None]) & (was % page != 0)[:, None]
    ok, lacking, copied = _take(st, dst, old, rows, rows < 0, alloc,
                                torch.where(alloc, rows, torch.full_like(rows, -1)))
    st["lens"][dst] = torch.where(ok, was, st["lens"][dst])
    _note(st, lacking, copied)


def _compact(st):
    live = st["refs"] > 0
    n = live.sum()
    page = torch.arange(live.numel(), device="cuda")
    holes = page[~live & (page < n)]
    movers = page[live & (page >= n)]
    st["data"][:, holes] = st["data"][:, movers]
    to = page.clone()
    to[movers] = holes
    st["refs"][holes] = st["refs"][movers]
    st["refs"][movers] = 0
    t = st["table"]
    t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()].int(), t))
    _note(st, 0, holes.numel())


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] not in ("attention", "append"):
        return _exact_pool(case, st)
    return (_exact_attention if case["kind"] == "attention" else _exact_append)(case, st)


def _rows_of(st, b, n, page):
    """Cache rows of the first n positions of sequence b: [2, hkv, n, dim] in 64 bits."""
    pages = st["table"][b, :-(-n // page)].long()
    x = st["cache"].index_select(0, pages).double()
    return x.movedim(0, 2).flatten(2, 3)[:, :, :n]


def _exact_attention(case, st):
    new, total = _lengths(case)
    dim, hq, hkv = case["dim"], case["hq"], case["hkv"]
    out = torch.zeros((sum(new), hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), hq), float("-inf"), dtype=torch.float64, device="cuda")
    start = 0
    for b, (n, m) in enumerate(zip(new, total)):
        if n == 0:
            continue
        k, v = _rows_of(st, b, m, case["page"])
        i = torch.arange(m - n, m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")[None]
        hidden = (j > i) | ((j <= i - case["window"]) if case["window"] else (j > i))
        q = st["q"][start:start + n].double().view(n, hq, dim)
        for h in range(hq):
            s = q[:, h] @ k[h * hkv // hq].T / dim ** 0.5
            s[hidden] = float("-inf")
            lse[start:start + n, h] = torch.logsumexp(s, 1)
            out[start:start + n, h] = torch.softmax(s, 1) @ v[h * hkv // hq]
        start += n
    return out.flatten(1), lse


def _exact_append(case, st):
    new, total = _lengths(case)
    dim, hq, hkv, half = case["dim"], case["hq"], case["hkv"], case["rot"] // 2
    tokens = sum(new)
    x = st["qkv"].double().view(tokens, hq + 2 * hkv, dim)
    pos = torch.tensor([m - n + t for n, m in zip(new, total) for t in range(n)], device="cuda")
    seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device="cuda")
    qk = x[:, :hq + hkv].clone()
    if case["norm"]:
        w = torch.cat([st["wq"].double().expand(hq, dim), st["wk"].double().expand(hkv, dim)])
        qk *= w / (qk.pow(2).sum(-1, keepdim=True) / dim + 1e-6).sqrt()
    turn = torch.complex(st["rope"][pos, :half].double(), st["rope"][pos, half:].double())
    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    z = torch.complex(qk[..., first], qk[..., second]) * turn[:, None]
    qk[..., first], qk[..., second] = z.real, z.imag
    cache = st["cache"].double()
    page = st["table"][seq, pos // case["page"]].long()
    cache[page, 0, :, pos % case["page"]] = qk[:, hq:]
    cache[page, 1, :, pos % case["page"]] = x[:, hq + hkv:]
    return qk[:, :hq].flatten(1), cache


class _Pages:
    """The pages of a pool one by one, in host lists; page contents in 64 bits."""

    def __init__(self, case, st):
        self.page, self.data = case["page"], st["data"].double()
        self.refs, self.lens = st["refs"].tolist(), st["lens"].tolist()
        self.rows = [[p for p in row if p >= 0] for row in st["table"].tolist()]
        self.info = [0, 0, 0, 0]

    def call(self, wants):
        """One call: `wants` lists (sequence, kept pages, pages to add, page to copy first or
        None, length). Pages given back are not handed out again before the next call."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        lacking = sum(w[2] for w in wants) - len(free)
        copies = []
        for s, keep, add, model, length in wants if lacking <= 0 else []:
            fresh, free = free[:add], free[add:]
            for p in self.rows[s]:
                self.refs[p] -= 1
            self.rows[s], self.lens[s] = keep + fresh, length
            for p in self.rows[s]:
                self.refs[p] += 1
            copies += [(model, fresh[0])] if model is not None else []
        for a, b in copies:
            self.data[:, b] = self.data[:, a]
        self.info = [max(0, lacking), self.refs.count(0), len(copies), 0]

    def resize(self, seqs, length):
        wants = []
        for s, n in zip(seqs, length):
            have, blocks = self.rows[s], -(-n // self.page)
            keep, model = have[:blocks], None
            if n < self.lens[s] and n % self.page and self.refs[keep[-1]] > 1:
                keep, model = keep[:-1], keep[-1]
            wants.append((s, keep, blocks - len(keep), model, n))
        self.call(wants)

    def fork(self, src, dst):
        wants = []
        for a, b in zip(src, dst):
            n, have = self.lens[a], self.rows[a]
            full = n // self.page
            wants.append((b, have[:full], len(have) - full, have[full] if n % self.page else None, n))
        self.call(wants)

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r]
        to = dict(zip([p for p in live if p >= len(live)],
                      [p for p in range(len(live)) if not self.refs[p]]))
        for a, b in to.items():
            self.data[:, b] = self.data[:, a]
            self.refs[a], self.refs[b] = 0, self.refs[a]
        self.rows = [[to.get(p, p) for p in row] for row in self.rows]
        self.info = [0, self.refs.count(0), len(to), 0]


def _exact_pool(case, st):
    p = _Pages(case, st)
    if case["kind"] == "step":
        p.resize(st["seqs"].tolist(), st["back"].tolist())
        p.resize(st["seqs"].tolist(), st["ahead"].tolist())
    elif case["kind"] == "fork":
        p.resize(st["dst"].tolist(), [0] * case["n"])
        p.fork(st["src"].tolist(), st["dst"].tolist())
    elif case["kind"] == "copy":
        for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
            p.data[:, b] = p.data[:, a]
    else:
        p.compact()
    table = [row + [-1] * (case["width"] - len(row)) for row in p.rows]
    out = dict(data=p.data, table=_i32(table), refs=_i32(p.refs), lens=_i32(p.lens))
    if case["kind"] != "copy":
        out["info"] = _i32(p.info)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def _page_bytes(case):
    return 2 * case["hkv"] * case["page"] * case["dim"] * 2


def work(case):
    kind, dim, hq, hkv = case["kind"], case["dim"], case["hq"], case["hkv"]
    if kind == "attention":
        new, total = _lengths(case)
        keys = pairs = 0
        for n, m in zip(new, total):
            w = case["window"] or m
            keys += max(0, m - max(0, m - n - w + 1)) if n else 0
            pairs += sum(min(w, p + 1) for p in range(m - n, m))
        tokens = sum(new)
        return {"bytes": keys * hkv * dim * 4 + tokens * hq * (dim * 4 + 4), "flops": 4 * pairs * hq * dim}
    if kind == "append":
        new, total = _lengths(case)
        tokens = sum(new)
        heads = hq + 2 * hkv
        places = len({p for n, m in zip(new, total) for p in range(m - n, m)})
        return {"bytes": tokens * heads * dim * 4 + places * case["rot"] * 4,
                "flops": 8 * tokens * (hq + hkv) * dim}
    lens = _pool_lengths(case)
    ints = 4 * (case["pool"] + 2 * case["seqs"])
    first, _ = _parts(case)
    if kind == "step":
        entries = sum(-(-lens[s] // case["page"]) for s in first)
        return {"bytes": 2 * ints + 4 * entries, "flops": 0}
    if kind == "fork":
        left = case["seqs"] - case["n"]
        blocks = sum(-(-lens[s] // case["page"]) for s in range(left)) / left
        copied = case["n"] * (1 - 1 / case["page"]) * case["layers"] * _page_bytes(case)
        return {"bytes": int(2 * ints + 12 * case["n"] * blocks + 2 * copied), "flops": 0}
    if kind == "copy":
        return {"bytes": 2 * case["n"] * case["layers"] * _page_bytes(case) + 8 * case["n"],
                "flops": 0}
    live = sum(-(-n // case["page"]) - _shared(lens, s, case["page"]) for s, n in enumerate(lens))
    moved = live * (1 - live / case["pool"])
    return {"bytes": int(2 * moved * case["layers"] * _page_bytes(case) + 2 * ints
                         + 8 * case["seqs"] * case["width"]), "flops": 0}
