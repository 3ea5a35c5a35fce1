"""The paged cache's calls on the GPU, against 64-bit plain forms (tests/_paged.py).

Tolerances: see _paged.check_attention for the attention; the append rounds
once, from fp32 sums of a few dozen roundings (U = 2^-8 relative, plus 2^-18 of
the head's largest element for cancellation in the rotation). Pages, tables and
counts are whole numbers and copies: equal.
"""
import pytest

import _paged as pg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_decode_gemm_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


import moe_decode_gemm_gb300 as dg  # noqa: E402

BF = torch.bfloat16


def run(bt, window=0, scale=None, max_q=0, kv=None, q=None):
    kv = bt.device(dg, max_q=max_q) if kv is None else kv
    lse = torch.full((bt.tokens, bt.hq), 7.0, device="cuda")
    out = dg.kv_attention(bt.q.cuda() if q is None else q, kv, lse=lse, window=window, scale=scale)
    assert dg.sync_check() == dg.DEC_OK
    return out, lse


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dim,page", [(128, 64), (128, 16), (64, 32), (64, 128), (128, 256)])
@pytest.mark.parametrize("hq,hkv", [(14, 1), (8, 8), (28, 2), (17, 1), (33, 1), (64, 1)])
def test_decode_lengths_around_page_and_tile_ends(dim, page, hq, hkv):
    total = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 300]
    bt = pg.Batch([1] * len(total), total, hq, hkv, dim, page, seed=1)
    pg.check_attention(bt, *run(bt, max_q=1), what="%s" % ((dim, page, hq, hkv),))


@pytest.mark.parametrize("max_q", [1, 3, 40])
@pytest.mark.parametrize("dim,page,hq,hkv", [(128, 16, 14, 1), (64, 64, 8, 2), (128, 32, 4, 4)])
def test_ragged_chunks_any_hint(dim, page, hq, hkv, max_q):
    new = [3, 0, 1, 40, 7, 0, 2, 33]
    total = [3, 0, 90, 41, 200, 64, 2, 500]
    bt = pg.Batch(new, total, hq, hkv, dim, page, seed=2)
    pg.check_attention(bt, *run(bt, max_q=max_q))


@pytest.mark.parametrize("window", [1, 2, 15, 64, 65, 1000])
@pytest.mark.parametrize("max_q", [1, 20])
def test_window(window, max_q):
    bt = pg.Batch([1, 5, 20, 1], [300, 131, 20, 1], 14, 1, 128, 16, seed=3)
    pg.check_attention(bt, *run(bt, window=window, max_q=max_q), window=window)


@pytest.mark.parametrize("max_q", [0, 1, 4, 30])
def test_rows_that_see_nothing(max_q):
    # fewer positions than new tokens: the first tokens' positions are negative
    bt = pg.Batch([4, 30, 1, 3], [0, 11, 0, 3], 8, 2, 64, 16, seed=4)
    out, lse = run(bt, max_q=max_q)
    pg.check_attention(bt, out, lse)
    assert torch.all(out[:4] == 0) and torch.all(lse[:4] == float("-inf"))


@pytest.mark.parametrize("dim,hq,hkv,q,total", [
    (128, 14, 1, 1, 9001), (64, 4, 4, 1, 7000), (128, 4, 1, 5, 4099), (128, 32, 1, 2, 3000),
    (128, 14, 1, 100, 2500), (64, 8, 1, 300, 1301), (128, 2, 2, 200, 700)])
def test_long_sequence_is_split_over_ctas(dim, hq, hkv, q, total):
    bt = pg.Batch([q], [total], hq, hkv, dim, 64, seed=5)
    kv = bt.device(dg, max_q=q)
    out, lse = run(bt, kv=kv)
    pg.check_attention(bt, out, lse)
    for _ in range(3):   # the same bits from run to run
        o2, l2 = run(bt, kv=kv)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_large_batch():
    n = 700
    new = [(b * 7) % 3 for b in range(n)]
    total = [new[b] + (b * 13) % 90 for b in range(n)]
    bt = pg.Batch(new, total, 4, 2, 64, 16, seed=6)
    pg.check_attention(bt, *run(bt, max_q=2))


@pytest.mark.parametrize("std,scale", [(8.0, None), (1.0, 30.0), (1.0, 0.0), (2.0, -1.0)])
@pytest.mark.parametrize("max_q", [3, 64])
def test_large_and_flat_scores(std, scale, max_q):
    # scores of several hundred: the fp32 score's own error, 2^-24 * dim-sum
    # terms of up to |q||k|, is still within the 2^-12 of check_attention
    bt = pg.Batch([3, 64], [200, 150], 4, 1, 64, 16, seed=7, std=std)
    pg.check_attention(bt, *run(bt, scale=scale, max_q=max_q), scale=scale)


@pytest.mark.parametrize("max_q", [1, 50])
def test_strides_and_row_numbers(max_q):
    # q and out are column slices of wider rows, pages are further apart than
    # their size, the batch's table rows are out of order
    bt = pg.Batch([1, 50, 2], [77, 60, 300], 14, 1, 128, 32, seed=8, rows=[5, 0, 3])
    wide = torch.full((bt.tokens, 14 * 128 + 256), float("nan"), dtype=BF, device="cuda")
    wide[:, 128:128 + 14 * 128] = bt.q.cuda()
    pool = torch.full((bt.pages, 3, 2, 1, 32, 128), float("nan"), dtype=BF, device="cuda")
    pool[:, 1] = bt.cache.cuda()
    kv = bt.device(dg, cache=pool[:, 1], max_q=max_q)
    res = torch.full((bt.tokens, 14 * 128 + 64), 3.0, dtype=BF, device="cuda")
    lse = torch.empty((bt.tokens, 14), device="cuda")
    out = dg.kv_attention(wide[:, 128:128 + 14 * 128], kv, out=res[:, :14 * 128], lse=lse)
    assert dg.sync_check() == dg.DEC_OK
    pg.check_attention(bt, out, lse)
    assert torch.all(res[:, 14 * 128:] == 3.0)


@pytest.mark.parametrize("dim,page,window", [(64, 32, 0), (128, 16, 0), (64, 128, 130)])
@pytest.mark.parametrize("many", [False, True])
def test_many_row_tiles(dim, page, window, many):
    # several times as many pairs of row tiles (4 tokens here) as SMs
    if many:
        new = [28 if b % 7 else 0 for b in range(45)]
        bt = pg.Batch(new, [28 + (b * 331) % 900 for b in range(45)], 128, 2, dim, page, seed=12)
    else:
        bt = pg.Batch([3, 500, 290, 201, 1], [3, 500, 320, 700, 64], 128, 2, dim, page, seed=13)
    kv = bt.device(dg, max_q=max(bt.new))
    out, lse = run(bt, window, kv=kv)
    assert dg.last_attention() == "tc"
    for _ in range(3):
        again, lse2 = run(bt, window, kv=kv)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    pg.check_attention(bt, out, lse, window)


def test_padded_batch_leaves_other_rows_alone():
    bt = pg.Batch([1, 2], [30, 40], 4, 2, 64, 16, seed=9, pad=5)
    kv = bt.device(dg)
    out = torch.full((bt.tokens, 4 * 64), 5.0, dtype=BF, device="cuda")
    lse = torch.full((bt.tokens, 4), 5.0, device="cuda")
    dg.kv_attention(bt.q.cuda(), kv, out=out, lse=lse)
    assert dg.sync_check() == dg.DEC_OK
    pg.check_attention(bt, out, lse, tokens=3)
    assert torch.all(out[3:] == 5.0) and torch.all(lse[3:] == 5.0)


@pytest.mark.parametrize("max_q", [2, 40])
def test_pages_and_rows_out_of_range_are_reported(max_q):
    bt = pg.Batch([2, 40], [100, 100], 4, 1, 64, 16, seed=10)
    bt.table[0, 2] = bt.pages + 5
    bt.table[1, 1] = -7
    kv = bt.device(dg, max_q=max_q)
    dg.kv_attention(bt.q.cuda(), kv)
    assert dg.sync_check() == dg.DEC_EBOUNDS
    assert dg.sync_check() == dg.DEC_OK
    bt = pg.Batch([2, 40], [100, 100], 4, 1, 64, 16, seed=10)
    bt.kv_len[1] = 100000
    kv = bt.device(dg, max_q=max_q)
    dg.kv_attention(bt.q.cuda(), kv)
    assert dg.sync_check() == dg.DEC_EBOUNDS


def test_two_streams_and_graph_follow_the_lengths():
    bt = pg.Batch([1] * 5, [70, 3, 200, 64, 129], 14, 1, 128, 16, seed=11)
    kv = bt.device(dg, max_q=1)
    q, lse = bt.q.cuda(), torch.empty((5, 14), device="cuda")
    out = torch.empty((5, 14 * 128), dtype=BF, device="cuda")
    dg.kv_attention(q, kv, out=out, lse=lse)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dg.kv_attention(q, kv, out=out, lse=lse)
    for cut in (0, 1, 2):
        total = [max(0, n - 17 * cut) for n in (70, 3, 200, 64, 129)]
        kv.kv_len.copy_(torch.tensor(total, dtype=torch.int32))
        bt.total = total
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert dg.sync_check() == dg.DEC_OK
        pg.check_attention(bt, out, lse, what="cut %d" % cut)
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    dg.kv_attention(q, kv, out=out, lse=lse, stream=s)
    s.synchronize()
    pg.check_attention(bt, out, lse)


@pytest.mark.parametrize("dim,hq,hkv,new,long", [
    (128, 14, 1, 40, 20000), (64, 8, 2, 60, 9000), (128, 4, 1, 1, 30000), (64, 8, 4, 5, 12000)])
def test_one_long_sequence_among_many_short_ones(dim, hq, hkv, new, long):
    # shared by many CTAs while the others' row tiles fit into one
    n = 44
    bt = pg.Batch([new] * n, [long if b == 17 else new + 3 * b for b in range(n)], hq, hkv, dim, 64,
                  seed=13)
    kv = bt.device(dg, max_q=new)
    out, lse = run(bt, kv=kv)
    pg.check_attention(bt, out, lse)
    o2, l2 = run(bt, kv=kv)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dim,hq,hkv,new,total", [(128, 14, 1, 20, 15000), (64, 16, 2, 70, 30000)])
def test_few_row_tiles_shared_by_all_sms(dim, hq, hkv, new, total):
    bt = pg.Batch([new], [total], hq, hkv, dim, 128, seed=14)
    kv = bt.device(dg, max_q=new)
    out, lse = run(bt, kv=kv)
    pg.check_attention(bt, out, lse)
    o2, l2 = run(bt, kv=kv)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


# ------------------------------------------------------------------ append
def _append(bt, rot, interleaved, norm, positions=None, seed=0, alias=False):
    g = pg.gen(seed)
    hq, hkv, dim = bt.hq, bt.hkv, bt.dim
    qkv = pg.normal(g, bt.tokens, (hq + 2 * hkv) * dim, std=0.8)
    w = (pg.normal(g, dim), pg.normal(g, dim)) if norm else None
    length = max(bt.total + [1]) + 7
    ang = torch.rand(length, rot // 2, generator=g, dtype=torch.float64) * 6.3
    rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    kv = bt.device(dg)
    x = qkv.cuda()
    q = dg.kv_append(x, kv, rope.cuda(), *([t.cuda() for t in w] if w else [None, None]),
                     q=x[:, :hq * dim] if alias else None, interleaved=interleaved,
                     positions=None if positions is None else positions.cuda())
    assert dg.sync_check() == dg.DEC_OK
    pos, seq = [], []
    for b, (n, m) in enumerate(zip(bt.new, bt.total)):
        pos += [m - n + t for t in range(n)]
        seq += [b] * n
    n = len(pos)
    rp = torch.tensor(pos) if positions is None else positions.long()[:n]
    ref = pg.append(qkv[:n], w, rope, rp, dim, hq, hkv, rot, interleaved)
    big = ref.abs().amax(-1, keepdim=True)
    near = lambda y, r, m: bool(((y - r).abs() <= pg.U * r.abs() + 2.0 ** -18 * m).all())  # noqa: E731
    assert near(q.double().cpu().view(-1, hq, dim)[:n], ref[:, :hq], big[:, :hq])
    want = bt.cache.clone()
    cache = kv.cache.cpu()
    for t in range(n):
        page, at = int(bt.table[bt.rows[seq[t]], pos[t] // bt.page]), pos[t] % bt.page
        got = cache[page, :, :, at].double()
        assert near(got[0], ref[t, hq:hq + hkv], big[t, hq:hq + hkv])
        assert torch.equal(got[1], ref[t, hq + hkv:])
        want[page, :, :, at] = cache[page, :, :, at]
    # nothing else has changed
    assert torch.equal(cache.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (128, 16), (64, 64), (64, 32), (64, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,page", [(14, 1, 16), (3, 3, 64)])
def test_append(dim, rot, interleaved, hq, hkv, page):
    bt = pg.Batch([1, 0, 5, 33, 1], [1, 9, 70, 33, 129], hq, hkv, dim, page, seed=20)
    _append(bt, rot, interleaved, norm=True, seed=21)


@pytest.mark.parametrize("tokens", [1, 2, 64, 1000])
def test_append_token_counts(tokens):
    bt = pg.Batch([tokens], [tokens + 3], 56, 4, 128, 64, seed=22)
    _append(bt, 128, False, norm=tokens != 2, seed=23, alias=tokens == 64)


def test_append_positions_rows_and_padding():
    bt = pg.Batch([2, 3], [20, 40], 4, 2, 64, 16, seed=24, pad=4, rows=[2, 0])
    _append(bt, 64, False, True, positions=torch.tensor([5, 0, 7, 7, 39, 1, 1, 1, 1],
                                                        dtype=torch.int32))


def test_append_out_of_range_is_reported():
    bt = pg.Batch([2, 3], [20, 40], 4, 2, 64, 16, seed=25)
    bt.table[0, 1] = -1
    kv = bt.device(dg)
    qkv = pg.normal(pg.gen(1), 5, 8 * 64).cuda()
    rope = torch.zeros(64, 64, device="cuda")
    dg.kv_append(qkv, kv, rope)
    assert dg.sync_check() == dg.DEC_EBOUNDS
    kv = pg.Batch([2, 3], [20, 40], 4, 2, 64, 16, seed=25).device(dg)
    dg.kv_append(qkv, kv, rope[:30])      # a position past the angles
    assert dg.sync_check() == dg.DEC_EBOUNDS
    dg.kv_append(qkv, kv, rope)
    assert dg.sync_check() == dg.DEC_OK


def test_token_ranges_that_do_not_rise_are_reported():
    # some tokens lie past the end of the sequence that the offsets point to
    for max_q in (1, 40):
        bt = pg.Batch([9, 2, 2, 15], [80] * 4, 4, 2, 64, 16, seed=26)
        bt.cu_q = torch.tensor([0, 9, 3, 5, 28], dtype=torch.int32)
        kv = bt.device(dg, max_q=max_q)
        dg.kv_append(pg.normal(pg.gen(1), 28, 8 * 64).cuda(), kv, torch.zeros(128, 64, device="cuda"))
        assert dg.sync_check() == dg.DEC_EBOUNDS
        dg.kv_attention(bt.q.cuda(), kv)
        assert dg.sync_check() == dg.DEC_EBOUNDS
        assert dg.sync_check() == dg.DEC_OK


# ------------------------------------------------------------------ pages
def _pool(seed, **kw):
    data, refs, table, lens = pg.random_pool(seed, **kw)
    info = torch.full((3,), 9, dtype=torch.int32, device="cuda")
    pool = dg.KVPool(data.cuda(), refs.cuda(), table.cuda(), lens.cuda(), info)
    return pool, pg.Pages(data, refs, table, lens, data.shape[-2])


def _same(pool, ref, info=True):
    assert dg.sync_check() == dg.DEC_OK
    assert pool.refs.tolist() == ref.refs
    assert pool.lens.tolist() == ref.lens
    assert torch.equal(pool.table.cpu(), ref.table())
    assert torch.equal(pool.data.cpu(), ref.data)
    if info:
        assert pool.info.tolist() == ref.info


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


SIZES = [dict(seqs=6, width=5, page=16, pages=40), dict(seqs=40, width=9, page=32, pages=200),
         dict(seqs=3, width=2, page=64, pages=7), dict(seqs=200, width=12, page=16, pages=9001, dim=64),
         dict(seqs=1, width=1, page=16, pages=1)]


@pytest.mark.parametrize("size", SIZES)
def test_resize_steps(size):
    pool, ref = _pool(30, **size)
    g = pg.gen(31)
    for step in range(8):
        n = int(torch.randint(1, size["seqs"] + 1, (1,), generator=g))
        seqs = torch.randperm(size["seqs"], generator=g)[:n].tolist()
        most = size["width"] * size["page"]
        lens = [max(0, min(most, ref.lens[s] + int(torch.randint(-40, 41, (1,), generator=g))))
                if step % 3 else int(torch.randint(0, most + 1, (1,), generator=g)) for s in seqs]
        dg.kv_resize(pool, _i32(seqs), _i32(lens))
        ref.resize(seqs, lens)
        _same(pool, ref)


@pytest.mark.parametrize("size", SIZES[:4])
def test_fork_free_compact(size):
    pool, ref = _pool(32, **size)
    g = pg.gen(33)
    for step in range(6):
        order = torch.randperm(size["seqs"], generator=g).tolist()
        n = max(1, size["seqs"] // 2)
        dst = order[:n]
        src = [order[n:][int(torch.randint(0, size["seqs"] - n, (1,), generator=g))] for _ in dst]
        dg.kv_fork(pool, _i32(src), _i32(dst))
        ref.fork(src, dst)
        _same(pool, ref)
        gone = order[n // 2:n // 2 + 1 + n // 3]
        dg.kv_free(pool, _i32(gone))
        ref.resize(gone, [0] * len(gone))
        _same(pool, ref)
        dg.kv_compact(pool)
        ref.compact()
        _same(pool, ref)
        grown = [min(size["width"] * size["page"], n + 5) for n in ref.lens]
        dg.kv_resize(pool, _i32(list(range(size["seqs"]))), _i32(grown))
        ref.resize(range(size["seqs"]), grown)
        _same(pool, ref)


def test_lacking_pages_change_nothing():
    pool, ref = _pool(34, seqs=6, width=8, page=16, pages=20, fill=1.0)
    dg.kv_resize(pool, _i32([0, 1, 2]), _i32([128, 128, 128]))
    ref.resize([0, 1, 2], [128, 128, 128])
    assert ref.info[0] > 0
    _same(pool, ref)


def test_full_and_empty_pools_compact():
    for refs in ([1] * 9, [0] * 9):
        table = torch.arange(9, dtype=torch.int32)[None] if refs[0] else torch.full((1, 9), -1,
                                                                                    dtype=torch.int32)
        data = pg.normal(pg.gen(35), 2, 9, 2, 1, 16, 64)
        lens = torch.tensor([144 if refs[0] else 0], dtype=torch.int32)
        r = torch.tensor(refs, dtype=torch.int32)
        info = torch.zeros(3, dtype=torch.int32, device="cuda")
        pool = dg.KVPool(data.cuda(), r.cuda(), table.cuda(), lens.cuda(), info)
        ref = pg.Pages(data, r, table, lens, 16)
        dg.kv_compact(pool)
        ref.compact()
        _same(pool, ref)


def test_requests_out_of_range_are_left_out_and_reported():
    pool, ref = _pool(36, seqs=6, width=5, page=16, pages=60)
    dg.kv_resize(pool, _i32([0, 6, 2, -1, 3]), _i32([17, 16, 81, 16, 33]))
    assert dg.sync_check() == dg.DEC_EBOUNDS
    ref.resize([0, 3], [17, 33])
    _same(pool, ref)
    dg.kv_copy(pool, _i32([0, 60]), _i32([-1, 3]))
    assert dg.sync_check() == dg.DEC_EBOUNDS
    _same(pool, ref)


@pytest.mark.parametrize("layers_inside", [False, True])
def test_copy_any_layout(layers_inside):
    # pages of 3 layers, layer by layer or all layers of a page together
    base = pg.normal(pg.gen(37), *((50, 3) if layers_inside else (3, 50)), 2, 3, 16, 64).cuda()
    data = base.transpose(0, 1) if layers_inside else base
    pool = dg.KVPool(data, *(torch.zeros(s, dtype=torch.int32, device="cuda")
                             for s in ((50,), (2, 4), (2,))))
    order = torch.randperm(50, generator=pg.gen(38)).int()
    want = data.clone()
    want[:, order[25:].long().cuda()] = want[:, order[:25].long().cuda()]
    dg.kv_copy(pool, order[:25].cuda(), order[25:].cuda())
    assert dg.sync_check() == dg.DEC_OK
    assert torch.equal(data, want)


def test_a_pools_layer_is_attended():
    """Room, append and attention over one layer of a pool, then a fork that goes its own way."""
    hq, hkv, dim, page, layers = 8, 2, 64, 16, 3
    data = torch.full((layers, 30, 2, hkv, page, dim), float("nan"), dtype=BF, device="cuda")
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = dg.KVPool(data, z(30), torch.full((4, 6), -1, dtype=torch.int32, device="cuda"), z(4))
    ang = torch.zeros(200, dim // 2)
    rope = torch.cat([ang.cos(), ang.sin()], 1).cuda()
    g = pg.gen(40)
    past = [[None, None] for _ in range(4)]

    def step(rows, new):
        lens = [0 if past[r][0] is None else past[r][0].shape[1] for r in rows]
        dg.kv_resize(pool, _i32(rows), _i32([a + b for a, b in zip(lens, new)]))
        cu = _i32([0] + torch.tensor(new).cumsum(0).tolist())
        for l in (1, 2):
            kv = pool.layer(l, cu, rows=_i32(rows), max_q=max(new))
            qkv = pg.normal(g, sum(new), (hq + 2 * hkv) * dim)
            q = dg.kv_append(qkv.cuda(), kv, rope)
            lse = torch.empty((sum(new), hq), device="cuda")
            out = dg.kv_attention(q, kv, lse=lse)
            if l == 2:
                at = 0
                for r, n in zip(rows, new):
                    x = qkv[at:at + n].view(n, hq + 2 * hkv, dim).transpose(0, 1)
                    k, v = x[hq:hq + hkv], x[hq + hkv:]
                    past[r] = [k, v] if past[r][0] is None else [torch.cat([past[r][0], k], 1),
                                                                 torch.cat([past[r][1], v], 1)]
                    at += n
                bt = pg.Batch(new, [past[r][0].shape[1] for r in rows], hq, hkv, dim, page)
                bt.k, bt.v = [past[r][0] for r in rows], [past[r][1] for r in rows]
                bt.q = qkv[:, :hq * dim]
                assert dg.sync_check() == dg.DEC_OK
                pg.check_attention(bt, out, lse)

    step([2, 0], [37, 5])
    step([0, 2], [1, 1])
    dg.kv_fork(pool, _i32([2, 2]), _i32([1, 3]))
    past[1], past[3] = list(past[2]), list(past[2])
    step([0, 1, 2, 3], [1, 2, 1, 3])
    dg.kv_free(pool, _i32([0]))
    past[0] = [None, None]
    dg.kv_compact(pool)
    step([3, 1, 2, 0], [1, 20, 1, 40])


# ------------------------------------------------------------------ non-finite values
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("new,total,window,max_q", [
    ([6], [200], 0, 6), ([6], [130], 40, 6), ([40], [300], 0, 40), ([40], [40], 0, 40),
    ([90], [400], 64, 90), ([200], [1000], 0, 200), ([1, 3], [66, 67], 0, 3)])
def test_non_finite_values_reach_only_the_rows_that_see_them(bad, new, total, window, max_q):
    bt = pg.Batch(new, total, 14, 1, 128, 16, seed=50)
    g = pg.gen(51)
    for b, (n, m) in enumerate(zip(new, total)):
        k, v = bt.k[b], bt.v[b]
        for _ in range(4):  # among the new tokens, and where windows end
            j = m - 1 - int(torch.randint(0, min(m, n + window), (1,), generator=g))
            v[0, j, int(torch.randint(0, 128, (1,), generator=g))] = bad
        v[0, m - 1, 5] = bad
        bt.put(b, k, v)
    out, lse = run(bt, window=window, max_q=max_q)
    ref, rl, ab = pg.attention(bt, window)
    o = out.double().cpu()
    fine = ref.isfinite()
    assert torch.equal(o.isfinite(), fine)
    assert torch.equal(o.isnan(), ref.isnan())
    assert torch.equal(o[~fine & ~ref.isnan()], ref[~fine & ~ref.isnan()])
    err = (o - ref)[fine].abs()
    assert bool((err <= (pg.U * ref.abs() + (pg.U + 2.0 ** -12) * ab)[fine]).all())
    assert bool(((lse.double().cpu() - rl).abs() <= 2.0 ** -16 * (1 + rl.abs())).all())


@pytest.mark.parametrize("max_q", [5, 100])
def test_non_finite_keys_reach_only_the_rows_that_see_them(max_q):
    bt = pg.Batch([5, 100], [90, 333], 14, 1, 128, 16, seed=52)
    for b, j in ((0, 87), (1, 300)):
        bt.k[b][0, j, 3] = float("nan")
        bt.put(b, bt.k[b], bt.v[b])
    out, lse = run(bt, max_q=max_q)
    ref, rl, ab = pg.attention(bt)
    o = out.double().cpu()
    assert torch.equal(o.isnan(), ref.isnan()) and torch.equal(lse.cpu().isnan(), rl.isnan())
    fine = ref.isfinite()
    assert bool(((o - ref)[fine].abs()
                 <= (pg.U * ref.abs() + (pg.U + 2.0 ** -12) * ab)[fine]).all())


def test_regimes_and_forced_regimes(monkeypatch):
    bt = pg.Batch([3, 70], [100, 300], 14, 1, 128, 64, seed=53)
    res = {}
    for force in ("", "mma", "tc"):
        monkeypatch.setenv("DEC_FORCE", force)
        for max_q in (1, 70):
            res[force, max_q] = run(bt, max_q=max_q)
            pg.check_attention(bt, *res[force, max_q], what="%s %d" % (force, max_q))
            assert dg.last_attention() == (force or ("mma" if max_q == 1 else "tc"))


@pytest.mark.parametrize("force", ["", "mma", "tc"])
@pytest.mark.parametrize("dim,hq,hkv,page,new,total,window", [
    (128, 14, 1, 16, [3, 4, 1, 0], [3, 300, 129, 40], 0),
    (128, 24, 8, 64, [12, 20, 7], [500, 20, 135], 40),
    (64, 8, 2, 32, [8, 16, 31, 1], [130, 16, 700, 257], 100),
    (64, 17, 1, 128, [2, 5, 7], [128, 1000, 7], 0),
    (64, 4, 4, 256, [100, 33], [100, 290], 9)])
def test_some_tens_of_rows(monkeypatch, force, dim, hq, hkv, page, new, total, window):
    # where either kernel may be chosen, and each when it is forced
    monkeypatch.setenv("DEC_FORCE", force)
    bt = pg.Batch(new, total, hq, hkv, dim, page, seed=54)
    pg.check_attention(bt, *run(bt, window, max_q=max(new)), window)
    assert dg.last_attention() in ([force] if force else ["mma", "tc"])


# ------------------------------------------------------------------ the rest
def test_index_checks_find_nothing():
    """The index-checking build of the library over shapes that split and join."""
    old = dg.use_library(dg.DEBUG_LIB_PATH)
    try:
        assert dg.lib().dec_debug_build() == 1
        for new, total, max_q in (([1], [5000], 1), ([1] * 9, list(range(30, 1200, 130)), 1),
                                  ([70, 3], [2000, 40], 70), ([40] * 20, [40 + 60 * i for i in range(20)], 40)):
            bt = pg.Batch(new, total, 14, 1, 128, 32, seed=70)
            pg.check_attention(bt, *run(bt, max_q=max_q))
        _append(pg.Batch([1, 0, 5, 33, 1], [1, 9, 70, 33, 129], 14, 1, 128, 16, seed=71), 64, True,
                norm=True)
    finally:
        dg.use_library(old)


def test_calls_after_shutdown():
    bt = pg.Batch([1, 70], [300, 200], 14, 1, 128, 64, seed=72)
    for _ in range(2):
        for max_q in (1, 70):
            pg.check_attention(bt, *run(bt, max_q=max_q))
        torch.cuda.synchronize()
        dg.shutdown()


def test_binding_refuses():
    bt = pg.Batch([1, 2], [30, 40], 4, 2, 64, 16, seed=73)
    kv = bt.device(dg)
    q, f32 = bt.q.cuda(), dict(dtype=torch.float32, device="cuda")
    rope = torch.zeros(64, 64, device="cuda")
    qkv = torch.zeros(3, 8 * 64, dtype=BF, device="cuda")
    w = torch.zeros(64, dtype=BF, device="cuda")
    i3 = _i32([0, 1, 2])
    for exc, msg, call in (
            (TypeError, "q: expected torch.bfloat16", lambda: dg.kv_attention(q.float(), kv)),
            (TypeError, "q: expected a torch tensor", lambda: dg.kv_attention(None, kv)),
            (ValueError, "q: expected a CUDA tensor", lambda: dg.kv_attention(bt.q, kv)),
            (ValueError, "q: expected 2 dimensions", lambda: dg.kv_attention(q[0], kv)),
            (ValueError, "unit column stride", lambda: dg.kv_attention(q.t().contiguous().t(), kv)),
            (ValueError, "q: expected [T, Hq*64]", lambda: dg.kv_attention(q[:, :192], kv)),
            (ValueError, "out: expected shape", lambda: dg.kv_attention(q, kv, out=q[:2])),
            (ValueError, "lse: expected", lambda: dg.kv_attention(q, kv, lse=torch.zeros(3, 5, **f32))),
            (TypeError, "lse: expected torch.float32", lambda: dg.kv_attention(q, kv, lse=q)),
            (ValueError, "qkv: expected [T, (Hq + 4)*64]", lambda: dg.kv_append(qkv[:, :256], kv, rope)),
            (TypeError, "rope: expected torch.float32", lambda: dg.kv_append(qkv, kv, rope.bfloat16())),
            (ValueError, "rope: must be contiguous", lambda: dg.kv_append(qkv, kv, rope[:, :32])),
            (ValueError, "give both or neither", lambda: dg.kv_append(qkv, kv, rope, w)),
            (ValueError, "wk: expected shape", lambda: dg.kv_append(qkv, kv, rope, w, w[:32])),
            (ValueError, "positions: expected shape", lambda: dg.kv_append(qkv, kv, rope, positions=i3[:2])),
            (ValueError, "q: expected shape", lambda: dg.kv_append(qkv, kv, rope, q=q[:2])),
            (dg.DecError, "kv_append failed", lambda: dg.kv_append(qkv, kv, rope[:, :8].contiguous())),
            (ValueError, "kv_len: expected shape",
             lambda: dg.PagedKV(kv.cache, kv.table, kv.cu_q, kv.kv_len[:1])),
            (ValueError, "table: 2 rows for a batch of 4",
             lambda: dg.PagedKV(kv.cache, kv.table, _i32([0] * 5), kv.kv_len)),
            (TypeError, "table: expected torch.int32",
             lambda: dg.PagedKV(kv.cache, kv.table.long(), kv.cu_q, kv.kv_len))):
        with pytest.raises(exc) as e:
            call()
        assert msg in str(e.value), (msg, str(e.value))
    pool, _ = _pool(74, seqs=3, width=4, page=16, pages=20)
    for exc, msg, call in (
            (TypeError, "seqs: expected torch.int32", lambda: dg.kv_free(pool, i3.long())),
            (ValueError, "lens: expected shape", lambda: dg.kv_resize(pool, i3, i3[:2])),
            (ValueError, "dst: expected shape", lambda: dg.kv_fork(pool, i3, i3[:1])),
            (ValueError, "src: expected a CUDA tensor", lambda: dg.kv_copy(pool, i3.cpu(), i3)),
            (ValueError, "seqs: must be contiguous", lambda: dg.kv_free(pool, _i32([0, 1, 2, 0])[::2])),
            (ValueError, "refs: expected shape",
             lambda: dg.KVPool(pool.data, pool.refs[:5], pool.table, pool.lens))):
        with pytest.raises(exc) as e:
            call()
        assert msg in str(e.value), (msg, str(e.value))
    # nothing to do is no error
    assert dg.kv_attention(q[:0], kv).shape == (0, 256)
    dg.kv_free(pool, i3[:0])
    assert dg.sync_check() == dg.DEC_OK
