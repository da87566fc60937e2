"""Rows before and after the experts as calls on tensors, on top of the C ABI.

The norm in front of the layer, with the residual's addition and an output in FP8
or MXFP4 for the products (``products.py``), and its gradient; tokens' rows to the
sorted order of their pairs and back with the router's weights, and the gradient.

Checks, streams and outputs are those of ``products.py``: every call checks its
tensors, allocates what it is not given, and enqueues on the current stream of the
tensors' device or on ``stream``; nothing is computed by PyTorch, and nothing is
recorded for autograd (inputs that require grad are refused where gradients are
enabled; the gradients are calls of their own). Rows are bf16, contiguous, start at
a multiple of 16 bytes and have a multiple of 8 columns; sums are fp32, and each
output is rounded once.

A pair is (token t, one of its k experts j). ``pair_row`` (int32 [T, k], as
``moe_permute`` writes it) is the row that the pair has in sorted order; a pair
whose row is outside the sorted rows (-1, say) takes no part.
"""
from __future__ import annotations

import torch

from . import _lib, products as P
from .products import _BF16, _F32, _FP8, _I32, _fail, _int, _matrix, _need, _no_history, _output, _run

_U8 = (torch.uint8,)
_OUT = (torch.bfloat16, torch.float32)


def _vector(t, name, n, dev):
    if _need(t, name, _BF16, dev).shape != (n,):
        _fail(f"{name}: {tuple(t.shape)}, [{n}] is needed")
    return t.data_ptr()


def _like(t, name, shape, dtypes, dev):
    """Address of t, which may be None."""
    if t is None:
        return None
    if _need(t, name, dtypes, dev).shape != shape:
        _fail(f"{name}: {tuple(t.shape)}, {list(shape)} is needed")
    return t.data_ptr()


def _given(t, name, shape, dtypes, dev, stream):
    t = _output(t, name, shape, dtypes, dev, stream)
    if t.shape != shape:
        _fail(f"{name}: {tuple(t.shape)}, {list(shape)} is needed")
    return t


def _norm(x, weight, eps, residual, out, total, quant, q, s, stream):
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x, weight, residual)
    R, H = x.shape
    pw, pr = _vector(weight, "weight", H, dev), _like(residual, "residual", x.shape, _BF16, dev)
    if residual is not None:
        total = _given(total, "total", x.shape, _BF16, dev, stream)
    elif total is not None:
        _fail("total: given without a residual")
    _run("moe_rms_norm", dev, stream, x.data_ptr(), pr, pw, eps, R, H,
         None if total is None else total.data_ptr(), _like(out, "out", x.shape, _BF16, dev), quant,
         None if q is None else q.data_ptr(), None if s is None else s.data_ptr())
    return total


def rms_norm(x, weight, eps=1e-6, residual=None, *, out=None, total=None, stream=None):
    """y = t / sqrt(mean(t^2) + eps) * weight of rows t = x [R, H], or with
    ``residual`` [R, H] t = bf16(x + residual): y bf16, or (y, t). ``total``, where t
    goes, may be x or residual."""
    dev = _matrix(x, "x", _BF16).get_device()
    out = _given(out, "out", x.shape, _BF16, dev, stream)
    total = _norm(x, weight, eps, residual, out, total, _lib.MOE_QUANT_NONE, None, None, stream)
    return out if total is None else (out, total)


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, *, out=None, total=None, q=None, s=None,
                 stream=None):
    """``rms_norm`` with y as ``products.quant_fp8`` has it, of the unrounded values:
    (codes [R, H], scales [R, ceil(H/128)]), with ``residual`` followed by t. ``out``
    (bf16 [R, H], optional) receives y itself as well, for the router."""
    dev = _matrix(x, "x", _BF16).get_device()
    R, H = x.shape
    q = _given(q, "q", (R, H), _FP8, dev, stream)
    s = _given(s, "s", (R, -(-H // 128)), _F32, dev, stream)
    total = _norm(x, weight, eps, residual, out, total, _lib.MOE_QUANT_FP8, q, s, stream)
    return (q, s) if total is None else (q, s, total)


def rms_norm_mxfp4(x, weight, eps=1e-6, residual=None, *, out=None, total=None, q=None, s=None,
                   stream=None):
    """``rms_norm`` with y as ``products.quant_mxfp4`` has it, of the unrounded values:
    (codes [R, H/2], scales [R, H/32]), with ``residual`` followed by t. ``out`` as for
    ``rms_norm_fp8``. H is a multiple of 32."""
    dev = _matrix(x, "x", _BF16).get_device()
    R, H = x.shape
    if H % 32:
        _fail(f"x: {H} columns, a multiple of 32 is needed")
    q = _given(q, "q", (R, H // 2), _U8, dev, stream)
    s = _given(s, "s", (R, H // 32), P._E8M0, dev, stream)
    total = _norm(x, weight, eps, residual, out, total, _lib.MOE_QUANT_MXFP4, q, s, stream)
    return (q, s) if total is None else (q, s, total)


_sizes = {}      # workspace bytes by (R, H, GPU)


def _grad_workspace(R, H, dev, stream, ws):
    if ws is not None:
        return _need(ws, "ws", _U8, dev)
    n = _sizes.get((R, H, dev))
    if n is None:
        if len(_sizes) > 4096:
            _sizes.clear()
        with torch.cuda.device(dev):
            n = _sizes[R, H, dev] = _lib.moe_rms_norm_grad_workspace(R, H)
    return _output(None, "ws", (n,), _U8, dev, stream)


def rms_norm_grad(x, weight, dy, eps=1e-6, dtotal=None, *, dx=None, dw=None, accumulate=False,
                  ws=None, stream=None):
    """Gradients of y = x / sqrt(mean(x^2) + eps) * weight for dy [R, H]: (dx bf16, dw
    fp32 [H]). ``dtotal`` (bf16 [R, H], optional; dx may be the same tensor) is the
    gradient that comes to x past the norm and is added to dx; with x the rows t of
    ``rms_norm``, dx is the gradient of x and of residual alike. ``accumulate`` adds to
    ``dw``. H is at most 16384. ``ws`` (uint8): as ``products.py`` has it, of
    ``_lib.moe_rms_norm_grad_workspace``'s bytes; needed with a stream handle."""
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x, weight, dy, dtotal)
    R, H = x.shape
    pw = _vector(weight, "weight", H, dev)
    if _matrix(dy, "dy", _BF16, dev).shape != x.shape:
        _fail(f"dy: {tuple(dy.shape)}, {list(x.shape)} is needed")
    pt = _like(dtotal, "dtotal", x.shape, _BF16, dev)
    if accumulate and dw is None:
        _fail("dw: needed to accumulate into")
    dx = _given(dx, "dx", x.shape, _BF16, dev, stream)
    dw = _given(dw, "dw", (H,), _F32, dev, stream)
    ws = _grad_workspace(R, H, dev, stream, ws)
    _run("moe_rms_norm_grad", dev, stream, x.data_ptr(), pw, dy.data_ptr(), pt, eps, R, H, dx.data_ptr(),
         dw.data_ptr(), int(bool(accumulate)), ws.data_ptr(), ws.numel())
    return dx, dw


def _pairs(pair_row, T, dev):
    """(address, k)"""
    _need(pair_row, "pair_row", _I32, dev)
    if pair_row.dim() != 2 or pair_row.shape[0] != T or pair_row.shape[1] < 1:
        _fail(f"pair_row: {tuple(pair_row.shape)}, [{T}, k] is needed")
    _int(pair_row.numel(), "pair_row")
    return pair_row.data_ptr(), pair_row.shape[1]


def dispatch(x, pair_row, *, out=None, stream=None):
    """Tokens to sorted order: out[pair_row[t, j]] = x[t] of x bf16 [T, H]. ``out``
    [n, H] ([T * k, H] where it is not given) keeps the rows that no pair has; the rows
    of the pairs are distinct. The gradient is ``combine`` without weights."""
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x)
    T, H = x.shape
    pr, k = _pairs(pair_row, T, dev)
    out = _output(out, "out", (T * k, H), _BF16, dev, stream)
    if out.dim() != 2 or out.shape[1] != H:
        _fail(f"out: {tuple(out.shape)}, [n, {H}] is needed")
    _run("moe_dispatch", dev, stream, x.data_ptr(), pr, T, k, H, out.data_ptr(), _int(out.shape[0], "out"))
    return out


def combine(y, pair_row, w=None, add=None, *, out=None, stream=None):
    """Sorted rows back to their tokens: out[t] = sum_j w[t, j] y[pair_row[t, j]] +
    add[t], bf16 [T, H], of y bf16 or fp32 [n, H], w fp32 [T, k] (1 without) and add
    bf16 [T, H] (the always-on expert's rows, or a residual)."""
    dev = _matrix(y, "y", _OUT).get_device()
    _no_history(y, w, add)
    if not isinstance(pair_row, torch.Tensor) or pair_row.dim() != 2:
        _fail("pair_row: an int32 tensor [T, k] is needed")
    T, H = pair_row.shape[0], y.shape[1]
    pr, k = _pairs(pair_row, T, dev)
    pw, pa = _like(w, "w", (T, k), _F32, dev), _like(add, "add", (T, H), _BF16, dev)
    out = _given(out, "out", (T, H), _BF16, dev, stream)
    _run("moe_combine_rows", dev, stream, y.data_ptr(), int(y.dtype is torch.float32), y.shape[0], pr, pw, pa,
         T, k, H, out.data_ptr())
    return out


def combine_grad(dout, y, pair_row, w, *, dy=None, dw=None, stream=None):
    """Gradients of ``combine`` for dout bf16 [T, H]: (dy bf16 of y's shape, dw fp32
    [T, k]): dy[pair_row[t, j]] = w[t, j] dout[t], and the rows that no pair has are
    left as they are (anything, in a dy that is not given); dw[t, j] = <dout[t],
    y[pair_row[t, j]]>, 0 for a pair without a row. y is bf16, the pairs' rows are
    distinct. add's gradient is dout."""
    dev = _matrix(dout, "dout", _BF16).get_device()
    _no_history(dout, y, w)
    T, H = dout.shape
    if _matrix(y, "y", _BF16, dev).shape[1] != H:
        _fail(f"y: {y.shape[1]} columns, dout has {H}")
    pr, k = _pairs(pair_row, T, dev)
    if w is None:
        _fail("w: needed (without weights, dispatch gives dy)")
    pw = _like(w, "w", (T, k), _F32, dev)
    dy = _given(dy, "dy", y.shape, _BF16, dev, stream)
    dw = _given(dw, "dw", (T, k), _F32, dev, stream)
    _run("moe_combine_rows_grad", dev, stream, dout.data_ptr(), y.data_ptr(), y.shape[0], pr, pw, T, k, H,
         dy.data_ptr(), dw.data_ptr())
    return dy, dw
