"""The paged cache's calls without a GPU: the C ABI refuses bad arguments with the
documented codes before it touches CUDA, the binding refuses tensors the ABI
would misread, and both agree on the structures."""
import ctypes
import os
import shutil
import subprocess

import pytest

import moe_decode_gemm_gb300 as dg
from conftest import ROOT
from moe_decode_gemm_gb300 import paged

A = 1 << 20          # an aligned fake pointer: never dereferenced
OK, EINVAL, EUNS = dg.DEC_OK, dg.DEC_EINVAL, dg.DEC_EUNSUPPORTED


@pytest.fixture(scope="module")
def L():
    from moe_decode_gemm_gb300 import build
    build.build()
    return dg.lib()


def view(**kw):
    a = dict(cache=A, page_stride=2 * 4 * 64 * 128, pages=10, heads=4, page_size=64, dim=128, table=A,
             table_stride=8, width=8, table_rows=3, rows=None, cu_q=A, kv_len=A, batch=3, max_q=1)
    a.update(kw)
    return paged._View(**a)


def attention(L, v, **kw):
    a = dict(q=A, ldq=56 * 128, out=A, ldo=56 * 128, lse=None, tokens=3, heads=56, scale=0.1, window=0)
    a.update(kw)
    return L.kv_attention(None if v is None else ctypes.byref(v), a["q"], a["ldq"], a["out"],
                          a["ldo"], a["lse"], a["tokens"], a["heads"], a["scale"], a["window"], None)


def append(L, v, **kw):
    a = dict(qkv=A, ld=64 * 128, wq=A, wk=A, eps=1e-6, rope=A, n=100, rot=128, il=0, pos=None, q=A,
             ldq=56 * 128, tokens=3, heads=56)
    a.update(kw)
    return L.kv_append(None if v is None else ctypes.byref(v), a["qkv"], a["ld"], a["wq"], a["wk"],
                       a["eps"], a["rope"], a["n"], a["rot"], a["il"], a["pos"], a["q"], a["ldq"],
                       a["tokens"], a["heads"], None)


VIEWS = [
    (dict(cache=None), EINVAL), (dict(cache=A + 8), EINVAL), (dict(table=None), EINVAL),
    (dict(cu_q=None), EINVAL), (dict(kv_len=None), EINVAL), (dict(kv_len=A + 2), EINVAL),
    (dict(pages=0), EINVAL), (dict(heads=0), EINVAL), (dict(batch=0), EINVAL),
    (dict(width=0), EINVAL), (dict(table_rows=0), EINVAL), (dict(table_rows=2), EINVAL),
    (dict(max_q=-1), EINVAL), (dict(table_stride=7), EINVAL),
    (dict(page_stride=2 * 4 * 64 * 128 - 8), EINVAL), (dict(page_stride=2 * 4 * 64 * 128 + 4), EINVAL),
    (dict(page_size=48, page_stride=1 << 20), EINVAL),
    (dict(page_size=8, page_stride=1 << 20), EUNS), (dict(page_size=512, page_stride=1 << 20), EUNS),
    (dict(dim=96, page_stride=1 << 20), EUNS), (dict(batch=1025, table_rows=2000), EUNS),
    (dict(width=1 << 26, table_stride=1 << 26), EUNS),
]


@pytest.mark.parametrize("kw,code", VIEWS)
def test_views_are_checked(L, kw, code):
    assert attention(L, view(**kw)) == code
    assert append(L, view(**kw)) == code


def test_no_view(L):
    assert attention(L, None) == EINVAL and append(L, None) == EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(q=A + 8), EINVAL), (dict(lse=A + 2), EINVAL),
    (dict(tokens=0), EINVAL), (dict(heads=0), EINVAL), (dict(heads=57, ldq=8000), EINVAL),
    (dict(ldq=55 * 128), EINVAL), (dict(ldq=56 * 128 + 4), EINVAL), (dict(ldo=100), EINVAL),
    (dict(window=-1), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(heads=4 * 65, ldq=4 * 65 * 128, ldo=4 * 65 * 128), EUNS),
])
def test_attention_refuses(L, kw, code):
    assert attention(L, view(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(qkv=None), EINVAL), (dict(q=None), EINVAL), (dict(rope=None), EINVAL), (dict(rope=A + 4), EINVAL),
    (dict(wq=None), EINVAL), (dict(wk=None), EINVAL), (dict(wq=A + 2), EINVAL), (dict(tokens=0), EINVAL),
    (dict(heads=0), EINVAL), (dict(n=0), EINVAL), (dict(rot=8), EINVAL), (dict(rot=24), EINVAL),
    (dict(rot=144), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(ld=63 * 128), EINVAL), (dict(ld=64 * 128 + 4), EINVAL), (dict(ldq=55 * 128), EINVAL),
    (dict(pos=A + 1), EINVAL), (dict(heads=32761, ld=1 << 23, ldq=1 << 23), EUNS),
])
def test_append_refuses(L, kw, code):
    assert append(L, view(), **kw) == code


def pool(**kw):
    a = dict(data=A, layer_stride=1 << 24, page_stride=1 << 16, page_bytes=1 << 16, layers=4,
             pages=100, page_size=64, refs=A, table=A, table_stride=8, width=8, lens=A, seqs=5,
             info=None)
    a.update(kw)
    return paged._Pool(**a)


POOLS = [
    (dict(data=None), EINVAL), (dict(data=A + 8), EINVAL), (dict(refs=None), EINVAL),
    (dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(info=A + 2), EINVAL),
    (dict(layers=0), EINVAL), (dict(pages=0), EINVAL), (dict(seqs=0), EINVAL), (dict(width=0), EINVAL),
    (dict(page_size=48), EINVAL), (dict(page_bytes=8), EINVAL), (dict(page_bytes=24), EINVAL),
    (dict(page_stride=1 << 15), EINVAL), (dict(layer_stride=16), EINVAL), (dict(table_stride=7), EINVAL),
    (dict(pages=(1 << 19) + 1), EUNS),
]


@pytest.mark.parametrize("kw,code", POOLS)
def test_pools_are_checked(L, kw, code):
    p = ctypes.byref(pool(**kw))
    assert L.kv_resize(p, A, A, 3, None) == code
    assert L.kv_free(p, A, 3, None) == code
    assert L.kv_fork(p, A, A, 3, None) == code
    assert L.kv_copy(p, A, A, 3, None) == code
    assert L.kv_compact(p, None) == code


def test_page_calls_refuse(L):
    p = ctypes.byref(pool())
    for f, lists in ((L.kv_resize, 2), (L.kv_fork, 2), (L.kv_copy, 2), (L.kv_free, 1)):
        full = [A] * lists
        assert f(p, *full, 0, None) == EINVAL
        assert f(None, *full, 3, None) == EINVAL
        for i in range(lists):
            for bad in (None, A + 2):
                assert f(p, *(bad if k == i else A for k in range(lists)), 3, None) == EINVAL
        if f is not L.kv_copy:
            assert f(p, *full, 1025, None) == EUNS
    assert L.kv_compact(None, None) == EINVAL


def test_last_attention_before_any_call(L):
    import threading
    out = []
    t = threading.Thread(target=lambda: out.append(L.kv_last_attention()))
    t.start()
    t.join()
    assert out == [dg.REGIME_NONE]


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
@pytest.mark.parametrize("name,struct", [("dec_kv_view", paged._View), ("dec_kv_pool", paged._Pool)])
def test_structures_match_the_header(tmp_path, name, struct):
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "decgemm.h"\nint main(void) {\n'
                   + "".join('  printf("%%zu\\n", offsetof(%s, %s));\n' % (name, f) for f in fields)
                   + '  printf("%%zu\\n", sizeof(%s));\n  return 0;\n}\n' % name)
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], check=True, capture_output=True).stdout.split()]
    assert got == [getattr(struct, f).offset for f in fields] + [ctypes.sizeof(struct)]


# ------------------------------------------------------------------ binding
torch = pytest.importorskip("torch")


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _kv(**kw):
    a = dict(cache=torch.zeros(10, 2, 1, 16, 64, dtype=torch.bfloat16), table=_i(3, 4), cu_q=_i(4),
             kv_len=_i(3))
    a.update(kw)
    return dg.PagedKV(**a)


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(cache=None), TypeError, "cache: expected a torch tensor"),
    (dict(cache=torch.zeros(10, 1, 16, 64)), ValueError, "cache: expected [pages, 2,"),
    (dict(cache=torch.zeros(10, 2, 16, 2, 64, dtype=torch.bfloat16).transpose(2, 3)), ValueError,
     "a page must be contiguous"),
    (dict(cache=torch.zeros(10, 2, 1, 16, 64)), TypeError, "cache: expected torch.bfloat16"),
    (dict(), ValueError, "cache: expected a CUDA tensor"),
])
def test_paged_kv_refuses(kw, exc, msg):
    with pytest.raises(exc) as e:
        _kv(**kw)
    assert msg in str(e.value)


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(data=3), TypeError, "data: expected a torch tensor"),
    (dict(data=torch.zeros(4, 5)), ValueError, "data: expected [layers, pages, ...]"),
    (dict(data=torch.zeros(0, 5, 16)), ValueError, "data: expected [layers, pages, ...]"),
    (dict(), ValueError, "data: expected a CUDA tensor"),
])
def test_pool_refuses(kw, exc, msg):
    a = dict(data=torch.zeros(2, 5, 16, 8), refs=_i(5), table=_i(3, 4), lens=_i(3))
    a.update(kw)
    with pytest.raises(exc) as e:
        dg.KVPool(**a)
    assert msg in str(e.value)
