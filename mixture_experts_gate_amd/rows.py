"""Rows before and after the experts as calls on tensors, on top of the C ABI.

The norm in front of the layer, with the residual's addition and an output in FP8
or MXFP4 for the products (``products.py``), and its gradient; tokens' rows to the
sorted order of their pairs and back with the router's weights, and the gradient.

Checks, streams and outputs are those of ``products.py``: every call checks its
tensors, allocates what it is not given, and enqueues on the current stream of the
tensors' device or on ``stream``; nothing is computed by PyTorch, and nothing is
recorded for autograd (inputs that require grad are refused where gradients are
enabled; the gradients are calls of their own). Rows are bf16, contiguous, start at
a multiple of 16 bytes and have a multiple of 8 columns; sums are fp32 (64 bits for a
row of the norm or its gradient whose sums leave fp32's range), and each output is
rounded once.

A pair is (token t, one of its k experts j). ``pair_row`` (int32 [T, k], as
``moe_permute`` writes it) is the row that the pair has in sorted order; a pair
whose row is outside the sorted rows (-1, say) takes no part.
"""
from __future__ import annotations

import torch

from . import _lib, products as P
from .products import (_BF16, _F32, _FP8, _I32, _OUT, _U8, _at, _fail, _int, _matrix, _need, _no_history, _output,
                       _run)


def _given(t, name, shape, dtypes, dev, stream):
    """(t, its address); a new tensor where t is None."""
    if t is None:
        t = _output(None, name, shape, dtypes, dev, stream)
        return t, t.data_ptr()
    return t, _at(t, name, dtypes, shape, dev)


def _norm(x, weight, eps, residual, out, total, quant, q, s, stream):
    """The norm's call: (y, q, s, total), what is asked for of them."""
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x, weight, residual)
    shape = x.shape
    R, H = shape
    pw = _at(weight, "weight", _BF16, (H,), dev)
    pr = pt = py = pq = ps = None
    if residual is not None:
        pr = _at(residual, "residual", _BF16, shape, dev)
        total, pt = _given(total, "total", shape, _BF16, dev, stream)
    elif total is not None:
        _fail("total: given without a residual")
    if out is not None or quant == _lib.MOE_QUANT_NONE:
        out, py = _given(out, "out", shape, _BF16, dev, stream)
    if quant == _lib.MOE_QUANT_FP8:
        q, pq = _given(q, "q", shape, _FP8, dev, stream)
        s, ps = _given(s, "s", (R, -(-H // 128)), _F32, dev, stream)
    elif quant == _lib.MOE_QUANT_MXFP4:
        if H % 32:
            _fail(f"x: {H} columns, a multiple of 32 is needed")
        q, pq = _given(q, "q", (R, H // 2), _U8, dev, stream)
        s, ps = _given(s, "s", (R, H // 32), P._E8M0, dev, stream)
    _run("moe_rms_norm", dev, stream, x.data_ptr(), pr, pw, eps, R, H, pt, py, quant, pq, ps)
    return out, q, s, total


def rms_norm(x, weight, eps=1e-6, residual=None, *, out=None, total=None, stream=None):
    """y = t / sqrt(mean(t^2) + eps) * weight of rows t = x [R, H], or with
    ``residual`` [R, H] t = bf16(x + residual): y bf16, or (y, t). ``total``, where t
    goes, may be x or residual."""
    y, _, _, t = _norm(x, weight, eps, residual, out, total, _lib.MOE_QUANT_NONE, None, None, stream)
    return y if residual is None else (y, t)


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, *, out=None, total=None, q=None, s=None,
                 stream=None):
    """``rms_norm`` with y as ``products.quant_fp8`` has it, of the unrounded values:
    (codes [R, H], scales [R, ceil(H/128)]), with ``residual`` followed by t. ``out``
    (bf16 [R, H], optional) receives y itself as well, for the router."""
    _, q, s, t = _norm(x, weight, eps, residual, out, total, _lib.MOE_QUANT_FP8, q, s, stream)
    return (q, s) if residual is None else (q, s, t)


def rms_norm_mxfp4(x, weight, eps=1e-6, residual=None, *, out=None, total=None, q=None, s=None,
                   stream=None):
    """``rms_norm`` with y as ``products.quant_mxfp4`` has it, of the unrounded values:
    (codes [R, H/2], scales [R, H/32]), with ``residual`` followed by t. ``out`` as for
    ``rms_norm_fp8``. H is a multiple of 32."""
    _, q, s, t = _norm(x, weight, eps, residual, out, total, _lib.MOE_QUANT_MXFP4, q, s, stream)
    return (q, s) if residual is None else (q, s, t)


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
    fp32 [H]). ``dtotal`` (bf16 [R, H], optional) is the gradient that comes
    to x past the norm and is added to dx, which may be dy or dtotal itself; with x the rows t of
    ``rms_norm``, dx is the gradient of x and of residual alike. ``accumulate`` adds to
    ``dw``. H is at most 16384. ``ws`` (uint8): as ``products.py`` has it, of
    ``_lib.moe_rms_norm_grad_workspace``'s bytes; needed with a stream handle."""
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x, weight, dy, dtotal)
    shape = x.shape
    R, H = shape
    pw = _at(weight, "weight", _BF16, (H,), dev)
    pdy = _at(dy, "dy", _BF16, shape, dev)
    pt = None if dtotal is None else _at(dtotal, "dtotal", _BF16, shape, dev)
    if accumulate and dw is None:
        _fail("dw: needed to accumulate into")
    dx, pdx = _given(dx, "dx", shape, _BF16, dev, stream)
    dw, pdw = _given(dw, "dw", (H,), _F32, dev, stream)
    ws = _grad_workspace(R, H, dev, stream, ws)
    _run("moe_rms_norm_grad", dev, stream, x.data_ptr(), pw, pdy, pt, eps, R, H, pdx, pdw,
         int(bool(accumulate)), ws.data_ptr(), ws.numel())
    return dx, dw


def _pairs(pair_row, dev):
    """(address, T, k)"""
    _need(pair_row, "pair_row", _I32, dev)
    if pair_row.dim() != 2:
        _fail(f"pair_row: {tuple(pair_row.shape)}, [T, k] is needed")
    T, k = pair_row.shape
    if k < 1 or T * k > 0x7FFFFFFF:
        _fail(f"pair_row: {T} x {k} pairs")
    return pair_row.data_ptr(), T, k


def dispatch(x, pair_row, *, out=None, stream=None):
    """Tokens to sorted order: out[pair_row[t, j]] = x[t] of x bf16 [T, H]. Rows of
    ``out`` [n, H] that no pair has are left as they are (anything, in an out that is
    not given, [T * k, H]); the rows of the pairs are distinct. The gradient is
    ``combine`` without weights."""
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x)
    pr, T, k = _pairs(pair_row, dev)
    if x.shape[0] != T:
        _fail(f"x: {x.shape[0]} rows, pair_row has {T}")
    H = x.shape[1]
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
    pr, T, k = _pairs(pair_row, dev)
    n, H = y.shape
    pw = None if w is None else _at(w, "w", _F32, (T, k), dev)
    pa = None if add is None else _at(add, "add", _BF16, (T, H), dev)
    out, po = _given(out, "out", (T, H), _BF16, dev, stream)
    _run("moe_combine_rows", dev, stream, y.data_ptr(), int(y.dtype is torch.float32), n, pr, pw, pa, T, k, H, po)
    return out


def combine_grad(dout, y, pair_row, w, *, dy=None, dw=None, stream=None):
    """Gradients of ``combine`` for dout bf16 [T, H]: (dy bf16 of y's shape, dw fp32
    [T, k]): dy[pair_row[t, j]] = w[t, j] dout[t], and the rows that no pair has are
    left as they are (anything, in a dy that is not given); dw[t, j] = <dout[t],
    y[pair_row[t, j]]>, 0 for a pair without a row. y is bf16, the pairs' rows are
    distinct. add's gradient is dout."""
    dev = _matrix(dout, "dout", _BF16).get_device()
    _no_history(dout, y, w)
    shape = _matrix(y, "y", _BF16, dev).shape
    n, H = shape
    pr, T, k = _pairs(pair_row, dev)
    if dout.shape != (T, H):
        _fail(f"dout: {tuple(dout.shape)}, [{T}, {H}] is needed")
    if w is None:
        _fail("w: needed (without weights, dispatch gives dy)")
    pw = _at(w, "w", _F32, (T, k), dev)
    dy, pdy = _given(dy, "dy", shape, _BF16, dev, stream)
    dw, pdw = _given(dw, "dw", (T, k), _F32, dev, stream)
    _run("moe_combine_rows_grad", dev, stream, dout.data_ptr(), y.data_ptr(), n, pr, pw, T, k, H, pdy, pdw)
    return dy, dw
