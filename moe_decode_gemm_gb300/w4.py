"""The residual stream's norm, and projections with 4-bit weights.

What a decode layer does around its attention and its experts:

  dec_rmsnorm      the residual's addition and the root-mean-square norm, in bf16
  dec_rmsnorm_mx   the same with an output in 8 bits (MX8) for the next projection
  dec_linear_w4    y = x·Wᵀ (+ residual), W in 4 bits (W4), x bf16 or MX8
  dec_quant_w4     bf16 weights as W4, once, when a model is loaded

W4 and MX8 hold blocks of 32 numbers with a shared power of two (the OCP
microscaling formats MXFP4 and MXFP8). They check their tensors once, keep them
alive and do not change them for others; a tensor that was given other memory
(``t.data = ...``) is looked over anew by the next call.
"""
from __future__ import annotations

import operator

from . import _check, _made, lib
from .paged import _Handle, _int32

_handles = {}


def _bound(index):
    """What calls on CUDA device ``index`` use of torch."""
    h = _handles.get(index)
    if h is None:
        import torch

        h = _Handle()
        h._bind(torch.device("cuda", index))
        h._f8, h._e8, h._u8 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8
        h._like = torch.empty_like
        h._getdev, h._guard = torch._C._cuda_getDevice, torch.cuda.device
        _handles[index] = h
    return h


def _elsewhere(h, fn, args, stream):
    """One C call on a device that is not the current one."""
    with h._guard(h._index):
        return fn(*args, h._stream(stream))


def _is_matrix(t, dtype, index, rows, width):
    """Rows of unit column stride on the device: the row stride, or 0 if it is no such matrix."""
    try:
        if t.dtype is not dtype or t.get_device() != index or t.shape != (rows, width):
            return 0
        ld, one = t.stride()
    except (AttributeError, ValueError):
        return 0
    if one != 1 and width > 1:
        return 0
    return ld if rows > 1 else width  # a single row's stride says nothing


def _explain(what, t, dtype, shape, align):
    """Raise what is wrong with a matrix (its device last)."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch tensor, got %s" % (what, type(t).__name__))
    if t.dtype is not dtype:
        raise TypeError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError("%s: expected shape [%s], got %s"
                         % (what, ", ".join("any" if n is None else str(n) for n in shape),
                            tuple(t.shape)))
    for n in t.shape:
        if n >> 31:
            raise ValueError("%s: %d does not fit 32 bits" % (what, n))
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("%s: needs unit column stride" % what)
    if t.dim() == 2 and t.shape[0] > 1:
        if t.stride(0) < t.shape[1]:
            raise ValueError("%s: its rows overlap" % what)
        if t.stride(0) % align:
            raise ValueError("%s: needs a row stride that is a multiple of %d" % (what, align))


def _wrong(device, *operands):
    """No operand was fit for the C ABI as it is: say which and why. operands:
    (name, tensor or None, dtype, shape, row stride's alignment)."""
    for what, t, dtype, shape, align in operands:
        if t is not None:
            _explain(what, t, dtype, shape, align)
    for what, t, _, _, _ in operands:
        if t is not None and t.device.type != "cuda":
            raise ValueError("%s: expected a CUDA tensor, got one on %s" % (what, t.device))
    for what, t, _, _, _ in operands:
        if t is not None and device is not None and t.device != device:
            raise ValueError("%s: on %s, the other operands on %s" % (what, t.device, device))
    raise ValueError("the operands are not fit for this call")


class MX8:
    """Activations in 8 bits: x[t][j] = q[t][j] * 2^(s[t][j/32] - 127).

    q [T, H] torch.float8_e4m3fn, rows any multiple of 16 apart; s [T, H/32] scale
    bytes, torch.float8_e8m0fnu or torch.uint8 (255: NaN). H a multiple of 32.
    """

    def __init__(self, q, s):
        import torch

        if isinstance(s, torch.Tensor) and s.dtype is torch.uint8:
            s = s.view(torch.float8_e8m0fnu)
        f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
        _explain("q", q, f8, (None, None), 16)
        T, H = q.shape
        if H % 32 or not H:
            raise ValueError("q: expected [T, H] with H a multiple of 32, got shape %s"
                             % (tuple(q.shape),))
        _explain("s", s, e8, (T, H // 32), 1)
        if q.device != s.device:
            raise ValueError("s: on %s, the other operands on %s" % (s.device, q.device))
        self._set(q, s, q.shape, q.get_device(), q.stride(0) if T > 1 else H, s.stride(0) if T > 1 else H // 32)

    def _set(self, q, s, shape, index, ldq, lds):
        self._q, self._s, self._shape, self._index = q, s, shape, index
        self._args = (q.data_ptr(), ldq, s.data_ptr(), lds)
        return self

    q, s, shape = (property(operator.attrgetter(name)) for name in ("_q", "_s", "_shape"))

    def _at(self):
        """What the C ABI is given of it."""
        a = self._args
        if self._q.data_ptr() != a[0] or self._s.data_ptr() != a[2]:
            self.__init__(self._q, self._s)
        return self._args


class W4:
    """Weights of N outputs and K inputs in 4 bits, as dec_linear_w4 reads them.

    W[n][k] = code * 2^(b - 127), b the scale byte of its 32 k: a code has its
    sign in bit 3 and stands for 0, .5, 1, 1.5, 2, 3, 4 or 6.
    q [ceil(N/128), ceil(K/128), 128, 64] uint8: row n % 128, element 2i of its 128
    k in the low half of byte i. s [ceil(N/128), ceil(K/128), 32, 4, 4] uint8: scale
    of row n at [n % 32, n % 128 // 32, k % 128 // 32]. What lies past N has no effect,
    past K only a scale of 255. dec_quant_w4 makes them from bf16 weights, `pack` from
    codes.
    """

    def __init__(self, q, s, n, k):
        import torch

        n, k = _int32("n", int(n)), _int32("k", int(k))
        if n < 1 or k < 8 or k % 8:
            raise ValueError("W4: expected n >= 1 and k a multiple of 8, got %d, %d" % (n, k))
        nt, kc = -(-n // 128), -(-k // 128)
        for what, t, shape in (("q", q, (nt, kc, 128, 64)), ("s", s, (nt, kc, 32, 4, 4))):
            _explain(what, t, torch.uint8, shape, 1)
            if not t.is_contiguous():
                raise ValueError("%s: must be contiguous" % what)
        if q.device != s.device:
            raise ValueError("s: on %s, the other operands on %s" % (s.device, q.device))
        self._set(q, s, n, k)

    def _set(self, q, s, n, k):
        self._q, self._s, self._n, self._k = q, s, n, k
        self._index = q.get_device()
        self._args = (q.data_ptr(), s.data_ptr())
        return self

    q, s, n, k = (property(operator.attrgetter(name)) for name in ("_q", "_s", "_n", "_k"))

    def _at(self):
        """What the C ABI is given of it."""
        a = self._args
        if self._q.data_ptr() != a[0] or self._s.data_ptr() != a[1]:
            self.__init__(self._q, self._s, self._n, self._k)
        return self._args

    @staticmethod
    def empty(n, k, device="cuda"):
        """Room for the weights, not initialised."""
        import torch

        nt, kc = -(-n // 128), -(-k // 128)
        return W4(torch.empty((nt, kc, 128, 64), dtype=torch.uint8, device=device),
                  torch.empty((nt, kc, 32, 4, 4), dtype=torch.uint8, device=device), n, k)

    @staticmethod
    def pack(codes, scales):
        """Codes [N, K] uint8 (0..15) and scale bytes [N, ceil(K/32)] uint8 of weights
        that are in 4 bits already, put in order (torch, on any device)."""
        import torch

        _explain("codes", codes, torch.uint8, (None, None), 1)
        n, k = codes.shape
        if codes.numel() and int(codes.max()) > 15:
            raise ValueError("codes: expected 0 to 15, got %d" % int(codes.max()))
        _explain("scales", scales, torch.uint8, (n, -(-k // 32)), 1)
        nt, kc = -(-n // 128), -(-k // 128)
        c = codes.new_zeros((nt * 128, kc * 128))
        c[:n, :k] = codes
        c = c.view(nt, 128, kc, 64, 2)
        b = scales.new_zeros((nt * 128, kc * 4))
        b[:n, :scales.shape[1]] = scales
        return W4((c[..., 0] | c[..., 1] << 4).transpose(1, 2).contiguous(),
                  b.view(nt, 4, 32, kc, 4).permute(0, 3, 2, 1, 4).contiguous(), n, k)


# ---------------------------------------------------------------- the calls
# (The calls of a decode step are short: what they pass is looked over in few steps,
# and _wrong says what is the matter.)
def _new(b, shape, dtype, stream, seen=True):
    """A tensor for a call on ``stream``."""
    if stream is None:
        return b._empty(shape, dtype=dtype, device=b.device)
    return _made(stream, b.device, b._empty, shape, dtype=dtype, seen=seen)


def _rows_of(b, x, ldx, stream):
    """A matrix of x's shape for a call on ``stream``."""
    return b._like(x) if stream is None and ldx == x.shape[1] else _new(b, x.shape, b._bf16, stream)


def _norm(what, mx, x, w, residual, h, out, eps, stream):
    try:
        T, H = shape = x.shape
        ldx, one = x.stride()
        index = x.get_device()
        b = _handles.get(index) or _bound(index) if index >= 0 else None
        bf = b._bf16
        if T < 2:
            ldx = H  # a single row's stride says nothing
        ok = (x.dtype is bf and one == 1 and ldx % 8 == 0 and ldx >= H and not (T | H) >> 31 and w.dtype is bf
              and w.get_device() == index and w.shape == (H,) and w.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        ok = False
    ldr = ldh = ldo = 0
    rp = hp = None
    if residual is not None:
        if ok:
            ldr = _is_matrix(residual, bf, index, T, H)
            if h is None:
                h = _rows_of(b, x, ldx, stream)
                ldh = H
            else:
                ldh = _is_matrix(h, bf, index, T, H)
            ok = ldr and ldr % 8 == 0 and ldh and ldh % 8 == 0
            if ok:
                rp, hp = residual.data_ptr(), h.data_ptr()
    elif h is not None:
        raise ValueError("h: given without a residual")
    if ok and out is not None:
        if mx:
            if type(out) is not MX8:
                raise TypeError("out: expected an MX8, got %s" % type(out).__name__)
            at = out._at()
            if out._index != index or out._shape != shape:
                raise ValueError("out: expected shape %s on %s, got %s on %s"
                                 % ((T, H), x.device, tuple(out.shape), out.q.device))
        else:
            ldo = _is_matrix(out, bf, index, T, H)
            ok = ldo and ldo % 8 == 0
    if not ok:
        import torch

        bf = torch.bfloat16
        _explain("x", x, bf, (None, None), 8)
        _wrong(x.device, ("x", x, bf, (None, None), 8), ("w", w, bf, (x.shape[1],), 1),
               ("residual", residual, bf, tuple(x.shape), 8), ("h", h, bf, tuple(x.shape), 8),
               ("y", None if mx else out, bf, tuple(x.shape), 8))
    if mx:
        if H % 32 or not H:
            raise ValueError("x: an 8-bit output needs a width that is a multiple of 32, got %d" % H)
        if out is None:
            q = _new(b, (T, H), b._f8, stream)
            s = _new(b, (T, H // 32), b._e8, stream)
            out = MX8.__new__(MX8)._set(q, s, x.shape, index, H, H // 32)
            at = out._args
        fn = lib().dec_rmsnorm_mx
        args = (x.data_ptr(), ldx, rp, ldr, w.data_ptr(), eps, hp, ldh, *at, T, H)
    else:
        if out is None:
            out = _rows_of(b, x, ldx, stream)
            ldo = H
        fn = lib().dec_rmsnorm
        args = (x.data_ptr(), ldx, rp, ldr, w.data_ptr(), eps, hp, ldh, out.data_ptr(), ldo, T, H)
    if T:
        if b._getdev() == index:
            rc = fn(*args, b._current(index) if stream is None else stream.cuda_stream)
        else:
            rc = _elsewhere(b, fn, args, stream)
        if rc:
            _check(rc, what)
    return out if residual is None else (out, h)


def dec_rmsnorm(x, w, residual=None, h=None, y=None, eps=1e-6, stream=None):
    """y = h * rsqrt(mean(h^2) + eps) * w with h = bf16(x + residual), or h = x.

    x [T, H] bf16, H a multiple of 8 up to 65536; w [H] bf16; residual [T, H]
    bf16. Rows of x, residual, h and y may be further apart than H (a multiple of
    8 elements). h may be x or residual, y may be x or residual (not h). Returns
    y, or (y, h) with a residual (both new tensors unless given).
    """
    return _norm("dec_rmsnorm", False, x, w, residual, h, y, eps, stream)


def dec_rmsnorm_mx(x, w, residual=None, h=None, out=None, eps=1e-6, stream=None):
    """dec_rmsnorm with an output in 8 bits: returns an MX8, or (MX8, h) with a
    residual. H a multiple of 32. For each 32 values the scale is the least power
    of two that brings the largest to 448 or less; a group with a value that is
    not finite gets the scale NaN."""
    return _norm("dec_rmsnorm_mx", True, x, w, residual, h, out, eps, stream)


def dec_linear_w4(x, W, y=None, residual=None, stream=None):
    """y = x·Wᵀ in bf16 with 4-bit weights, or residual + x·Wᵀ.

    x: [M, K] bf16 (rows may be further apart than K, a multiple of 8 elements)
    or MX8, M <= 64. W: W4. y, residual: [M, N] bf16 contiguous; y may be residual,
    not x. fp32 sums, one rounding. bf16 tokens are taken as two 8-bit numbers
    each: exact for values down to 2^-13.8 of the largest of their 32 (aligned) k,
    off by at most 2^-21.8 of the largest below. A token with a value that is not
    finite gives NaN in all its outputs. More than 16 bf16 tokens take a work space
    from torch's allocator for the call.
    """
    if not isinstance(W, W4):
        raise TypeError("W: expected a W4, got %s" % type(W).__name__)
    wat = W._at()
    index, N, K = W._index, W._n, W._k
    mx = type(x) is MX8
    ok = index >= 0
    if ok:
        b = _handles.get(index) or _bound(index)
        bf = b._bf16
        if mx:
            xat = x._at()
            M, k = x._shape
            ok = x._index == index and k == K and not M >> 31
        else:
            try:
                M, k = x.shape
                ld, one = x.stride()
                if M < 2:
                    ld = K  # a single row's stride says nothing
                ok = (k == K and x.dtype is bf and x.get_device() == index and one == 1 and ld % 8 == 0
                      and ld >= K and not M >> 31)
            except (AttributeError, ValueError):
                ok = False
    if ok and y is not None:
        ok = _is_matrix(y, bf, index, M, N) and y.is_contiguous()
    if ok and residual is not None:
        ok = _is_matrix(residual, bf, index, M, N) and residual.is_contiguous()
    if not ok:
        import torch

        bf = torch.bfloat16
        if mx:
            if x.shape[1] != K:
                raise ValueError("x: expected shape [any, %d], got %s" % (K, tuple(x.shape)))
            _int32("x", x.shape[0])
            xt, dt, al = x.q, torch.float8_e4m3fn, 16
        else:
            _explain("x", x, bf, (None, K), 8)
            xt, dt, al = x, bf, 8
        shape = (x.shape[0], N)
        for what, t in (("y", y), ("residual", residual)):
            if t is not None:
                _explain(what, t, bf, shape, 1)
                if not t.is_contiguous():
                    raise ValueError("%s: must be contiguous (row-major)" % what)
        _wrong(W.q.device, ("x", xt, dt, (None, K), al), ("y", y, bf, shape, 1),
               ("residual", residual, bf, shape, 1), ("W", W.q, torch.uint8, tuple(W.q.shape), 1))
    if y is None:
        y = _new(b, (M, N), bf, stream)
    if M:
        L = lib()
        rp = None if residual is None else residual.data_ptr()
        if mx:
            fn, args = L.dec_linear_w4_mx, (*xat, *wat, rp, y.data_ptr(), M, N, K)
        else:
            wp = None
            if M > 16:
                n = L.dec_linear_w4_work(M, K)
                if n:
                    work = _new(b, n, b._u8, stream, seen=False)
                    wp = work.data_ptr()
            fn, args = L.dec_linear_w4, (x.data_ptr(), ld, *wat, rp, y.data_ptr(), M, N, K, wp)
        if b._getdev() == index:
            rc = fn(*args, b._current(index) if stream is None else stream.cuda_stream)
        else:
            rc = _elsewhere(b, fn, args, stream)
        if rc:
            _check(rc, "dec_linear_w4")
    return y


def dec_quant_w4(W, out=None, stream=None):
    """bf16 weights [N, K] (K a multiple of 8; rows may be further apart) as a W4.

    For each 32 weights of a row (groups start at multiples of 32) the scale is the
    least power of two that brings the largest to 6 or less; codes are the nearest,
    ties to the even one. A group with a value that is not finite gets the scale NaN.
    """
    try:
        N, K = W.shape
        index = W.get_device()
        b = _handles.get(index) or _bound(index) if index >= 0 else None
        ld = _is_matrix(W, b._bf16, index, N, K)
        ok = ld and ld % 8 == 0 and N >= 1 and K >= 8 and K % 8 == 0 and not (N | K) >> 31
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        import torch

        _explain("W", W, torch.bfloat16, (None, None), 8)
        N, K = W.shape
        if N < 1 or K < 8 or K % 8:
            raise ValueError("W: expected [N, K] with K a multiple of 8, got shape %s" % (tuple(W.shape),))
        _wrong(None, ("W", W, torch.bfloat16, (None, None), 8))
    if out is None:
        nt, kc = -(-N // 128), -(-K // 128)
        out = W4.__new__(W4)._set(_new(b, (nt, kc, 128, 64), b._u8, stream),
                                  _new(b, (nt, kc, 32, 4, 4), b._u8, stream), N, K)
    elif type(out) is not W4:
        raise TypeError("out: expected a W4, got %s" % type(out).__name__)
    elif out._at() and (out.n, out.k) != (N, K):
        raise ValueError("out: expected a W4 of %d x %d, got %d x %d" % (N, K, out.n, out.k))
    elif out._index != index:
        raise ValueError("out: on %s, the other operands on %s" % (out.q.device, W.device))
    fn, args = lib().dec_quant_w4, (W.data_ptr(), ld, *out._args, N, K)
    rc = (fn(*args, b._stream(stream)) if b._getdev() == index else
          _elsewhere(b, fn, args, stream))
    if rc:
        _check(rc, "dec_quant_w4")
    return out
