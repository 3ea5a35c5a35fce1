"""A paged cache for the tests, and what its calls compute in 64 bits.

Plain torch on the CPU in float64, one sequence and one token at a time; the
page calls are simulated page by page. Places of a cache that no sequence uses
hold NaN, so that a kernel that reads one shows it.
"""
from __future__ import annotations

import torch

BF = torch.bfloat16
U = 2.0 ** -8   # unit roundoff of bf16 (8 significant bits, nearest)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=g) * std).to(dtype)


class Batch:
    """A batch over a cache of one layer: new[b] new tokens, total[b] positions
    (the new tokens included), on the CPU; .cuda() gives the device tensors."""

    def __init__(self, new, total, hq, hkv, dim, page, seed=0, std=1.0, extra=3, pad=0, rows=None):
        g = gen(seed)
        self.new, self.total, self.hq, self.hkv, self.dim, self.page = new, total, hq, hkv, dim, page
        self.rows = list(range(len(new))) if rows is None else rows
        nrows = max(self.rows) + 1
        blocks = [-(-n // page) for n in total]
        self.pages = sum(blocks) + extra
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((nrows, max(blocks + [1]) + 1), -1, dtype=torch.int32)
        self.kv_len = torch.zeros(nrows, dtype=torch.int32)
        self.cache = torch.full((self.pages, 2, hkv, page, dim), float("nan"), dtype=BF)
        self.k, self.v = [], []
        for b, n in enumerate(total):
            mine = [order.pop() for _ in range(blocks[b])]
            self.table[self.rows[b], :blocks[b]] = torch.tensor(mine, dtype=torch.int32)
            self.kv_len[self.rows[b]] = n
            k, v = normal(g, hkv, n, dim, std=std), normal(g, hkv, n, dim)
            self.put(b, k, v)
            self.k.append(k)
            self.v.append(v)
        self.cu_q = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32)
        self.tokens = sum(new) + pad
        self.q = normal(g, max(self.tokens, 1), hq * dim, std=std)[:self.tokens]

    def put(self, b, k, v):
        for j in range(k.shape[1]):
            pg = int(self.table[self.rows[b], j // self.page])
            self.cache[pg, 0, :, j % self.page] = k[:, j]
            self.cache[pg, 1, :, j % self.page] = v[:, j]

    def device(self, dg, cache=None, max_q=0, **kw):
        cu = lambda t: t.cuda()  # noqa: E731
        rows = (None if self.rows == list(range(len(self.new)))
                else torch.tensor(self.rows, dtype=torch.int32).cuda())
        return dg.PagedKV(cu(self.cache) if cache is None else cache, cu(self.table), cu(self.cu_q),
                          cu(self.kv_len), rows=rows, max_q=max_q, **kw)


def attention(bt, window=0, scale=None):
    """(out, lse, absolute) in 64 bits: absolute = sum_j p_j |v_j|, the size that
    rounding the weights p can move an output by, in units of bf16's roundoff."""
    g = bt.hq // bt.hkv
    scale = bt.dim ** -0.5 if scale is None else scale
    out = torch.zeros(bt.tokens, bt.hq, bt.dim, dtype=torch.float64)
    lse = torch.full((bt.tokens, bt.hq), float("-inf"), dtype=torch.float64)
    ab = torch.zeros_like(out)
    at = 0
    for b, (n, m) in enumerate(zip(bt.new, bt.total)):
        k, v = bt.k[b].double(), bt.v[b].double()
        for t in range(n):
            pos = m - n + t
            lo = max(0, pos - window + 1) if window else 0
            if pos >= 0:
                q = bt.q[at].double().view(bt.hkv, g, bt.dim)
                s = torch.einsum("hgd,hkd->hgk", q, k[:, lo:pos + 1]) * scale
                p = torch.softmax(s, -1)
                out[at] = torch.einsum("hgk,hkd->hgd", p, v[:, lo:pos + 1]).reshape(bt.hq, bt.dim)
                ab[at] = torch.einsum("hgk,hkd->hgd", p,
                                      v[:, lo:pos + 1].abs()).reshape(bt.hq, bt.dim)
                lse[at] = torch.logsumexp(s, -1).reshape(-1)
            at += 1
    return out.reshape(bt.tokens, -1), lse, ab.reshape(bt.tokens, -1)


def check_attention(bt, out, lse, window=0, scale=None, what="", tokens=None):
    """out within the two bf16 roundings it has (the weights', then its own) and
    2^-12 of the weighted sum for the fp32 arithmetic before them (scores of up
    to a few tens carry a few 2^-24 of themselves, times dim sums); lse within
    2^-16 of its size."""
    ref, rl, ab = attention(bt, window, scale)
    n = bt.tokens if tokens is None else tokens
    ref, rl, ab = ref[:n], rl[:n], ab[:n]
    o, l = out.double().cpu()[:n], lse.double().cpu()[:n]
    err, bound = (o - ref).abs(), U * ref.abs() + (U + 2.0 ** -12) * ab
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d outputs off, worst %g over %g, at %s" % (
        what, int(bad.sum()), float(err[bad].max()), float(bound[bad].min()),
        bad.nonzero()[:4].tolist())
    empty = rl == float("-inf")
    assert torch.equal(l == float("-inf"), empty), what + ": empty rows"
    le = (l[~empty] - rl[~empty]).abs()
    assert bool((le <= 2.0 ** -16 * (1 + rl[~empty].abs())).all()), "%s: lse off by %g" % (
        what, float(le.max()))


def append(qkv, w, rope, pos, dim, hq, hkv, rot, interleaved, eps=1e-6):
    """Heads of qkv [T, (hq+2hkv)*dim] normed and rotated, in 64 bits:
    [T, hq+2hkv, dim]; w: (wq, wk) or None."""
    x = qkv.double().view(-1, hq + 2 * hkv, dim).clone()
    y = x[:, :hq + hkv]
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        y = torch.cat([y[:, :hq] * w[0].double(), y[:, hq:] * w[1].double()], 1)
    r = rope.double()[pos][:, None]
    c, s = r[..., :rot // 2], r[..., rot // 2:]
    out = y.clone()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    x[:, :hq + hkv] = out
    return x


class Pages:
    """The pages of a pool one by one, in host lists; contents are copied in `data`
    [layers, pages, ...]."""

    def __init__(self, data, refs, table, lens, page):
        self.data, self.page, self.width = data.clone(), page, table.shape[1]
        self.refs, self.lens = refs.tolist(), lens.tolist()
        self.rows = [[p for p in r if p >= 0] for r in table.tolist()]
        self.info = [0, 0, 0]

    def table(self):
        return torch.tensor([r + [-1] * (self.width - len(r)) for r in self.rows], dtype=torch.int32)

    def _call(self, wants):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        lacking = sum(w[2] for w in wants) - len(free)
        copies = []
        if lacking <= 0:
            for s, keep, add, model, length in wants:
                fresh, free = free[:add], free[add:]
                for p in self.rows[s]:
                    self.refs[p] -= 1
                self.rows[s], self.lens[s] = keep + fresh, length
                for p in self.rows[s]:
                    self.refs[p] += 1
                if model is not None:
                    copies.append((model, fresh[0]))
            for a, b in copies:
                self.data[:, b] = self.data[:, a]
        self.info = [max(0, lacking), self.refs.count(0), len(copies)]

    def resize(self, seqs, lens):
        wants = []
        for s, n in zip(seqs, lens):
            if not 0 <= s < len(self.rows) or not 0 <= n <= self.width * self.page:
                continue
            blocks = -(-n // self.page)
            keep, model = self.rows[s][:blocks], None
            if n < self.lens[s] and n % self.page and self.refs[keep[-1]] > 1:
                keep, model = keep[:-1], keep[-1]
            wants.append((s, keep, blocks - len(keep), model, n))
        self._call(wants)

    def fork(self, src, dst):
        wants = []
        for a, b in zip(src, dst):
            n, have = self.lens[a], self.rows[a]
            full = n // self.page
            wants.append((b, have[:full], len(have) - full,
                          have[full] if n % self.page else None, n))
        self._call(wants)

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r]
        to = dict(zip([p for p in live if p >= len(live)],
                      [p for p in range(len(live)) if not self.refs[p]]))
        for a, b in to.items():
            self.data[:, b] = self.data[:, a]
            self.refs[a], self.refs[b] = 0, self.refs[a]
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        self.info = [0, self.refs.count(0), len(to)]


def random_pool(seed, seqs, width, page, pages, layers=2, heads=1, dim=64, fill=0.6):
    """(data, refs, table, lens) of a pool in which some sequences share pages."""
    g = gen(seed)
    r = lambda n: int(torch.randint(0, n, (1,), generator=g))  # noqa: E731
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((seqs, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    lens = torch.zeros(seqs, dtype=torch.int32)
    used = 0
    for s in range(seqs):
        n = r(width * page + 1) if r(8) else 0
        blocks = -(-n // page)
        common = 0
        if s and r(2):
            common = min(n // page, int(lens[s - 1]) // page)
            common = r(common + 1)
        if used + blocks - common > fill * pages:
            continue
        table[s, :common] = table[s - 1, :common]
        table[s, common:blocks] = torch.tensor(order[used:used + blocks - common], dtype=torch.int32)
        used += blocks - common
        lens[s] = n
        for p in table[s, :blocks].tolist():
            refs[p] += 1
    data = normal(g, layers, pages, 2, heads, page, dim)
    return data, refs, table, lens
