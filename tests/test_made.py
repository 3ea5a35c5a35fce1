"""Where a call's own tensors come from, without a GPU: the stream that the call is
given, not the current one, whose freed memory may still be in use there."""
from types import SimpleNamespace

import pytest

import moe_decode_gemm_gb300 as dg

torch = pytest.importorskip("torch")

CUDA = torch.device("cuda", 0)


class Streams:
    """torch's current stream, as far as _made asks for it."""

    def __init__(self, monkeypatch):
        self.main, self.side = SimpleNamespace(cuda_stream=0), SimpleNamespace(cuda_stream=7)
        self.now = self.main
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(torch.cuda, "stream", self._on)

    def _on(self, stream):
        outer = self

        class On:
            def __enter__(self):
                self.before, outer.now = outer.now, stream

            def __exit__(self, *exc):
                outer.now = self.before

        return On()

    def make(self, *shape, device, dtype):
        t = SimpleNamespace(shape=shape, dtype=dtype, device=device, of=self.now, recorded=[])
        t.record_stream = t.recorded.append
        return t


@pytest.mark.parametrize("given,of,recorded", [
    (None, "main", []), ("main", "main", []), ("side", "side", ["main"])])
def test_tensors_are_of_the_calls_stream(monkeypatch, given, of, recorded):
    s = Streams(monkeypatch)
    t = dg._made(given and getattr(s, given), CUDA, s.make, 2, 3, dtype=torch.bfloat16)
    assert t.of is getattr(s, of) and t.shape == (2, 3) and t.device == CUDA
    assert t.recorded == [getattr(s, r) for r in recorded]
    assert s.now is s.main


def test_a_work_space_is_the_calls_alone(monkeypatch):
    s = Streams(monkeypatch)
    t = dg._made(s.side, CUDA, s.make, 9, dtype=torch.uint8, seen=False)
    assert t.of is s.side and t.recorded == []


def _fake(shape, dtype, strides=None):
    """A CUDA tensor as far as the calls look at it before they launch."""
    t = SimpleNamespace(shape=torch.Size(shape), dtype=dtype, device=CUDA)
    strides = strides or (shape[1], 1)
    t.stride = lambda i=None: strides if i is None else strides[i]
    t.get_device, t.data_ptr, t.is_contiguous = lambda: 0, lambda: 1 << 20, lambda: True
    return t


@pytest.mark.parametrize("call", ["norm", "norm of a slice", "norm_mx", "linear", "linear with work space", "quant"])
def test_the_norm_and_the_projections_make_theirs_there(monkeypatch, call):
    from moe_decode_gemm_gb300 import w4

    s = Streams(monkeypatch)
    made = []

    def empty(shape, dtype, device):
        assert s.now is s.side
        t = _fake(shape if isinstance(shape, (tuple, torch.Size)) else (1, shape), dtype)
        t.record_stream = lambda stream: None
        made.append(t)
        return t

    def like(x):
        raise AssertionError("made on the current stream")

    bf = torch.bfloat16
    h = SimpleNamespace(device=CUDA, _index=0, _bf16=bf, _f8=torch.float8_e4m3fn, _e8=torch.float8_e8m0fnu,
                        _u8=torch.uint8, _empty=empty, _like=like, _getdev=lambda: 0, _current=lambda i: 0,
                        _stream=lambda stream: stream.cuda_stream)
    monkeypatch.setitem(w4._handles, 0, h)
    launched = []

    def fn(*args):
        launched.append(args[-1])
        return 0

    monkeypatch.setattr(w4, "lib", lambda: SimpleNamespace(
        dec_rmsnorm=fn, dec_rmsnorm_mx=fn, dec_linear_w4=fn, dec_quant_w4=fn, dec_linear_w4_work=lambda m, k: 4096))
    x, w = _fake((20, 64), bf), _fake((64,), bf, (1,))
    W = w4.W4.__new__(w4.W4)._set(_fake((1, 1), torch.uint8), _fake((1, 1), torch.uint8), 16, 64)
    if call == "norm":
        w4.dec_rmsnorm(x, w, _fake((20, 64), bf), stream=s.side)
    elif call == "norm of a slice":
        w4.dec_rmsnorm(_fake((20, 64), bf, (128, 1)), w, _fake((20, 64), bf), stream=s.side)
    elif call == "norm_mx":
        w4.dec_rmsnorm_mx(x, w, _fake((20, 64), bf), stream=s.side)
    elif call == "linear":
        w4.dec_linear_w4(_fake((3, 64), bf), W, stream=s.side)
    elif call == "linear with work space":
        w4.dec_linear_w4(x, W, stream=s.side)
    else:
        w4.dec_quant_w4(x, stream=s.side)
    assert launched == [7] and s.now is s.main
    assert len(made) == {"norm_mx": 3, "linear": 1}.get(call, 2)


def _operand(shape, dtype, strides=None):
    t = _fake(shape, dtype, strides)
    t.dim = lambda: len(shape)
    t.numel = lambda: int(torch.Size(shape).numel())
    return t


@pytest.mark.parametrize("call", ["linear", "splitk", "moe", "latent", "add", "append", "attention"])
def test_the_other_calls_make_theirs_there(monkeypatch, call):
    from moe_decode_gemm_gb300 import paged

    s = Streams(monkeypatch)
    bf, f32, made, launched = torch.bfloat16, torch.float32, [], []

    def empty(shape, dtype=None, device=None):
        assert s.now is s.side
        t = _operand(shape if isinstance(shape, (tuple, torch.Size)) else shape.shape, dtype or bf)
        t.record_stream = made.append
        return t

    class Lib:
        def __getattr__(self, name):
            return lambda *args: launched.append(name) or 0

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", empty)
    monkeypatch.setattr(dg, "_need", lambda t, *a, **k: t)
    for module in (dg, paged):
        monkeypatch.setattr(module, "lib", lambda: Lib())
    x, W = _operand((4, 64), bf), _operand((16, 64), bf)
    if call == "linear":
        dg.dec_linear(x, W, stream=s.side)
    elif call == "splitk":
        dg.dec_linear_splitk(x, W, 1, stream=s.side)
    elif call == "moe":
        dg.moe_decode(x, _operand((8, 64), bf), _operand((8, 32, 64), bf, (2048, 64, 1)),
                      _operand((8, 64, 16), bf, (1024, 16, 1)), None, None, 2, stream=s.side)
    elif call == "latent":
        dg.moe_decode_latent(x, _operand((40, 64), bf), _operand((8, 32, 32), bf, (1024, 32, 1)),
                             _operand((8, 32, 16), bf, (512, 16, 1)), _operand((64, 32), bf), None, None, 2,
                             stream=s.side)
    elif call == "add":
        dg.dec_add(x, x, stream=s.side)
    else:
        kv = paged._Handle()
        kv.device, kv._index, kv._bf16, kv._f32, kv._empty = CUDA, 0, bf, f32, empty
        kv.dim, kv.heads, kv._ref = 16, 1, None
        if call == "append":
            dg.kv_append(x, kv, _operand((9, 16), f32), stream=s.side)
        else:
            dg.kv_attention(x, kv, stream=s.side)
    assert len(launched) == 1 and made == [s.main] and s.now is s.main
