"""The expert products as calls on tensors, on top of the C ABI.

For experts whose matrices are bf16 (with both gradients, for training), FP8
with a scale per 128 x 128 block or MXFP4 (E2M1 codes with an E8M0 scale per 32
columns): the products grouped by expert, the gated activation between them with
its gradient, and rows to FP8 and MXFP4. Every call checks
its tensors (types, shapes, contiguity, one device), allocates what it is not
given, and enqueues one kernel of ``libmoe.so`` on the current stream of the
tensors' device, or on ``stream`` (a torch stream or the handle of one). Nothing
is computed by PyTorch, but for the zeros of a ``dw`` that ``swiglu_grad`` makes.

A product with few output tiles and a long sum cuts it into parts, which a
second kernel adds up, where it has a workspace (``ws``, uint8; the bytes are
``_lib.moe_grouped_gemm_workspace``'s, at most ``workspace_bound``'s). One that
is not given is allocated, except with a stream handle, with which nothing is:
without ``ws``, or with a smaller one, the sum runs whole, which takes longer and
rounds in another order. Calls that may overlap need workspaces of their own.

Rows are in *sorted order*: grouped by expert, expert e owning rows
``offsets[e]`` .. ``offsets[e+1] - 1`` (``offsets`` int32 [E+1] on the device,
as ``moe_permute`` writes it; ``None`` means one group of all rows). An input
read through ``rows`` (int32 [R]) gives sorted row i its row ``rows[i] // div``:
``rows=sorted_pair, div=k`` reads each pair's token. An output written through
``out_rows`` takes sorted row i at its row ``out_rows[i]`` (distinct):
``out_rows=sorted_pair`` writes pair order. Rows at and past ``offsets[E]`` and
rows with an index outside their matrix are left as they are in the output.
Outputs must not overlap inputs.

The calls record nothing for autograd: where gradients are enabled, an input that
requires one is refused, since its gradient would be lost without a word. Call
them under ``torch.no_grad()`` or from a ``torch.autograd.Function`` (the
gradients are calls of their own).

Matrices ``w`` are a tensor [E, N, K] (or [N, K] for one group), or
``TableMatrices`` for those a device table of ``moe_expert_w`` points to (an
expert cache's, or ``expert_table``'s).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib

_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_FP8 = (torch.float8_e4m3fn, torch.uint8)
_OUT = (torch.bfloat16, torch.float32)
_U8, _E8M0 = (torch.uint8,), (torch.uint8, torch.float8_e8m0fnu)


class TableMatrices(NamedTuple):
    """W13 (``mat=MOE_MAT_W13``) or W2 of the experts of a device table of
    moe_expert_w (int64 tensor [E, 4], or its address as an expert cache's
    prefetch returns it); N x K row-major each."""
    table: object
    mat: int
    E: int
    N: int
    K: int


def _fail(what):
    raise ValueError(what)


def _need(t, name, dtypes, dev=None):
    """t is a contiguous tensor of one of `dtypes` on a GPU (number `dev`).
    (One line where it is: a call's checks cost as much as a small kernel.)"""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous()
            and (dev is None or t.get_device() == dev)):
        return t
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _fail(f"{name}: a tensor on the GPU is needed")
    if t.dtype not in dtypes:
        _fail(f"{name}: {t.dtype}, {' or '.join(map(str, dtypes))} is needed")
    if not t.is_contiguous():
        _fail(f"{name}: must be contiguous")
    _fail(f"{name}: on GPU {t.get_device()}, the others are on {dev}")


def _at(t, name, dtypes, shape, dev):
    """Address of t: contiguous, one of `dtypes`, of this shape, on GPU `dev`. (A small
    call's time is its checks: one line where all is well.)"""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    _need(t, name, dtypes, dev)
    _fail(f"{name}: {tuple(t.shape)}, {list(shape)} is needed")


def _int(n, name):
    """n, as the library's 32-bit int takes it (ctypes would cut it to that)."""
    if not -0x80000000 <= n <= 0x7FFFFFFF:
        _fail(f"{name}: {n} is past 32 bits")
    return n


def _no_history(*inputs):
    """Refuses inputs whose gradient autograd would be expected to find."""
    for t in inputs:
        if getattr(t, "requires_grad", False) and torch.is_grad_enabled():
            _fail("an input requires grad, and the result carries no history for autograd: "
                  "call under torch.no_grad() (the gradients are calls of their own)")


def _matrix(t, name, dtype, dev=None):
    shape = _need(t, name, dtype, dev).shape
    if len(shape) != 2:
        _fail(f"{name}: two dimensions are needed, got {tuple(shape)}")
    if shape[0] > 0x7FFFFFFF or shape[1] > 0x7FFFFFFF:
        _int(max(shape), name)
    return t


def _weights(w, ws, dtype, dev):
    """(w address, scale address, table address, mat, E, N, K)"""
    if isinstance(w, TableMatrices):
        if w.mat not in (_lib.MOE_MAT_W13, _lib.MOE_MAT_W2):
            _fail(f"w.mat: {w.mat}")
        for n, name in zip(w[2:], ("w.E", "w.N", "w.K")):
            _int(n, name)
        if ws is not None:
            _fail("w_scale: the table of w has the scales")
        if isinstance(w.table, torch.Tensor):
            _need(w.table, "w.table", (torch.int64,), dev)
            if w.table.numel() < 4 * w.E:
                _fail("w.table: fewer than E entries")
        return None, None, _lib._ptr(w.table), w.mat, w.E, w.N, w.K
    _need(w, "w", dtype, dev)
    if w.dim() not in (2, 3):
        _fail(f"w: [E, N, K] or [N, K] is needed, got {tuple(w.shape)}")
    E, N, K = (1, *w.shape) if w.dim() == 2 else w.shape
    _int(max(w.shape), "w")
    if dtype is _BF16:
        return w.data_ptr(), None, None, 0, E, N, K
    _need(ws, "w_scale", _F32, dev)
    want = (-(-N // 128), -(-K // 128))
    if ws.shape[-2:] != want or ws.numel() != E * want[0] * want[1]:
        _fail(f"w_scale: {tuple(ws.shape)}, [E, {want[0]}, {want[1]}] is needed")
    return w.data_ptr(), ws.data_ptr(), None, 0, E, N, K


def _offsets(offsets, E, dev):
    if offsets is None:
        if E != 1:
            _fail(f"offsets: needed for {E} groups")
        return None
    _need(offsets, "offsets", _I32, dev)
    if offsets.numel() != E + 1:
        _fail(f"offsets: {offsets.numel()} values, E + 1 = {E + 1} are needed")
    return offsets.data_ptr()


def _index(rows, name, R, dev):
    if rows is None:
        return None
    _need(rows, name, _I32, dev)
    if rows.numel() != R:
        _fail(f"{name}: {rows.numel()} values for {R} rows")
    return rows.data_ptr()


def _count(x, rows, name):
    """Sorted rows: the index's, or all rows of x."""
    if rows is None:
        return x.shape[0]
    if not isinstance(rows, torch.Tensor):
        _fail(f"{name}: an int32 tensor is needed")
    return _int(rows.numel(), name)


def _output(out, name, shape, dtypes, dev, stream):
    """`out`, checked, or a new tensor (made on the stream that writes it)."""
    if out is None:
        if stream is None:
            return torch.empty(shape, dtype=dtypes[0], device=torch.device("cuda", dev))
        if isinstance(stream, int):
            _fail(f"{name}: a stream handle needs the output given")
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtypes[0], device=torch.device("cuda", dev))
    _need(out, name, dtypes, dev)
    return out


def _rows_output(out, name, R, n, out_rows, dtypes, dev, stream):
    out = _output(out, name, (R, n), dtypes, dev, stream)
    shape = out.shape
    if len(shape) != 2 or shape[1] != n or (out_rows is None and shape[0] < R):
        _fail(f"{name}: {tuple(shape)}, [{R}, {n}] is needed")
    if shape[0] > 0x7FFFFFFF:
        _int(shape[0], name)
    return out


_calls = {}      # the library's functions, once looked up
_current_device = getattr(torch._C, "_cuda_getDevice", None)             # (none in a build without GPUs)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_sizes = {}      # workspace bytes by (kind, R, N, K, E, GPU)


def workspace_bound(R, N, K, E, device="cuda"):
    """Bytes of workspace that suffice for every product of at most R rows with
    matrices [E, N, K], gradients among them: sums are cut into at most 16
    parts, and their tiles of 128 x 128 fp32 are at most two a compute unit."""
    device = torch.device(device)
    cu = torch.cuda.get_device_properties(device).multi_processor_count if device.type == "cuda" else 256
    return min(16 * 4 * max(R * max(N, K), E * N * K), 2 * cu * 128 * 128 * 4)


def _workspace(kind, R, N, K, E, dev, stream, ws):
    """(tensor or None, address, bytes) of the workspace the product can use."""
    if ws is not None:
        _need(ws, "ws", (torch.uint8,), dev)
        return ws, ws.data_ptr(), ws.numel()
    key = (kind, R, N, K, E, dev)
    n = _sizes.get(key)
    if n is None:
        if len(_sizes) > 4096:
            _sizes.clear()
        if torch._C._cuda_getDevice() != dev:
            with torch.cuda.device(dev):
                n = _lib.moe_grouped_gemm_workspace(kind, R, N, K, E)
        else:
            n = _lib.moe_grouped_gemm_workspace(kind, R, N, K, E)
        _sizes[key] = n
    if n == 0 or isinstance(stream, int):
        return None, None, 0
    ws = _output(None, "workspace", (n,), (torch.uint8,), dev, stream)
    return ws, ws.data_ptr(), n


def _run(fn, dev, stream, *args):
    """Enqueue on the current stream of GPU `dev`, or on `stream`."""
    call = _calls.get(fn)
    if call is None:
        call = _calls[fn] = getattr(_lib.load(), fn)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return _run(fn, dev, stream, *args)
    if stream is None:
        stream = _current_stream(dev)
    elif not isinstance(stream, int):
        if stream.device_index != dev:
            _fail(f"stream: of GPU {stream.device_index}, the tensors are on {dev}")
        stream = stream.cuda_stream
    rc = call(*args, stream)
    if rc < 0:
        _lib._check(fn, rc)


def grouped_matmul(x, w, offsets=None, *, rows=None, div=1, out_rows=None, out=None, ws=None,
                   stream=None):
    """y[i] = W_e x[i] over sorted rows: x bf16 [n, K], w bf16 -> [R, N] (``out``
    may be bf16, the default, or fp32). N and K are multiples of 8."""
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x, w)
    pw, _, tab, mat, E, N, K = _weights(w, None, _BF16, dev)
    if x.shape[1] != K:
        _fail(f"x: {x.shape[1]} columns, w has {K}")
    R = _count(x, rows, "rows")
    out = _rows_output(out, "out", R, N, out_rows, _OUT, dev, stream)
    ws, pws, nws = _workspace(_lib.MOE_GEMM_BF16, R, N, K, E, dev, stream, ws)
    _run("moe_grouped_gemm", dev, stream, x.data_ptr(), _index(rows, "rows", R, dev), _int(div, "div"),
         x.shape[0], _offsets(offsets, E, dev), pw, tab, mat, R, N, K, E, out.data_ptr(),
         _index(out_rows, "out_rows", R, dev), out.shape[0],
         int(out.dtype is torch.float32), pws, nws)
    return out


def grouped_matmul_fp8(x, x_scale, w, w_scale=None, offsets=None, *, rows=None, div=1,
                       out_rows=None, out=None, ws=None, stream=None):
    """y[i] = W_e x[i] over sorted rows from block-scaled FP8: x E4M3 [n, K]
    (float8_e4m3fn or uint8 codes) with fp32 scales [n, ceil(K/128)] (from
    ``quant_fp8``), w E4M3 with fp32 scales [E, ceil(N/128), ceil(K/128)] ->
    [R, N] bf16 or fp32. N is a multiple of 8, K of 16."""
    dev = _matrix(x, "x", _FP8).get_device()
    _no_history(x, x_scale, w, w_scale)
    pw, ps, tab, mat, E, N, K = _weights(w, w_scale, _FP8, dev)
    if x.shape[1] != K:
        _fail(f"x: {x.shape[1]} columns, w has {K}")
    if _matrix(x_scale, "x_scale", _F32, dev).shape != (x.shape[0], -(-K // 128)):
        _fail(f"x_scale: {tuple(x_scale.shape)}, [{x.shape[0]}, {-(-K // 128)}] is needed")
    R = _count(x, rows, "rows")
    out = _rows_output(out, "out", R, N, out_rows, _OUT, dev, stream)
    ws, pws, nws = _workspace(_lib.MOE_GEMM_FP8, R, N, K, E, dev, stream, ws)
    _run("moe_grouped_gemm_fp8", dev, stream, x.data_ptr(), x_scale.data_ptr(),
         _index(rows, "rows", R, dev), _int(div, "div"), x.shape[0], _offsets(offsets, E, dev), pw, ps, tab,
         mat, R, N, K, E, out.data_ptr(), _index(out_rows, "out_rows", R, dev), out.shape[0],
         int(out.dtype is torch.float32), pws, nws)
    return out


def grouped_matmul_mxfp4(x, x_scale, w, w_scale=None, offsets=None, *, rows=None, div=1,
                         out_rows=None, out=None, ws=None, stream=None):
    """y[i] = W_e x[i] over sorted rows from MXFP4: x E2M1 codes [n, K/2] (uint8) with
    E8M0 scales [n, K/32] (from ``quant_mxfp4``), w in the kernel layout, codes [E, N,
    K/2] with scales [E, N, K/32] (from ``quant_mxfp4_matrices``) or the
    ``TableMatrices`` of packed "mxfp4" blobs -> [R, N] bf16 or fp32. N is a multiple
    of 16, K of 128."""
    dev = _matrix(x, "x", _U8).get_device()
    _no_history(x_scale, w_scale)
    n, half = x.shape
    if isinstance(w, TableMatrices):
        pw, ps, tab, mat, E, N, K = _weights(w, w_scale, _U8, dev)
    else:
        if _need(w, "w", _U8, dev).dim() not in (2, 3):
            _fail(f"w: [E, N, K/2] or [N, K/2] is needed, got {tuple(w.shape)}")
        shape = w.shape
        E, N = shape[:2] if len(shape) == 3 else (1, shape[0])
        K = 2 * shape[-1]
        pw, ps, tab, mat = w.data_ptr(), _at(w_scale, "w_scale", _E8M0, (*shape[:-1], K // 32), dev), None, 0
    if 2 * half != K:
        _fail(f"x: {2 * half} columns, w has {K}")
    pxs = _at(x_scale, "x_scale", _E8M0, (n, K // 32), dev)
    _int(max(E, N, K), "w")
    pr = po = None
    R = n
    if rows is not None:
        R = _int(_need(rows, "rows", _I32, dev).numel(), "rows")
        pr = rows.data_ptr()
    if out_rows is not None:
        po = _index(out_rows, "out_rows", R, dev)
    out = _rows_output(out, "out", R, N, out_rows, _OUT, dev, stream)
    ws, pws, nws = _workspace(_lib.MOE_GEMM_MXFP4, R, N, K, E, dev, stream, ws)
    _run("moe_grouped_gemm_mxfp4", dev, stream, x.data_ptr(), pxs, pr, _int(div, "div"), n,
         _offsets(offsets, E, dev), pw, ps, tab, mat, R, N, K, E, out.data_ptr(), po, out.shape[0],
         int(out.dtype is torch.float32), pws, nws)
    return out


def grouped_matmul_dx(dy, w, offsets=None, *, rows=None, div=1, out_rows=None, out=None,
                      ws=None, stream=None):
    """dx[i] = W_e^T dy[i] over sorted rows: dy bf16 [n, N], w bf16 -> [R, K]
    bf16 or fp32; ``rows``/``div`` index dy, ``out_rows`` dx."""
    dev = _matrix(dy, "dy", _BF16).get_device()
    _no_history(dy, w)
    pw, _, tab, mat, E, N, K = _weights(w, None, _BF16, dev)
    if dy.shape[1] != N:
        _fail(f"dy: {dy.shape[1]} columns, w has {N} rows")
    R = _count(dy, rows, "rows")
    out = _rows_output(out, "out", R, K, out_rows, _OUT, dev, stream)
    ws, pws, nws = _workspace(_lib.MOE_GEMM_DX, R, N, K, E, dev, stream, ws)
    _run("moe_grouped_gemm_dx", dev, stream, dy.data_ptr(), _index(rows, "rows", R, dev), _int(div, "div"),
         dy.shape[0], _offsets(offsets, E, dev), pw, tab, mat, R, N, K, E, out.data_ptr(),
         _index(out_rows, "out_rows", R, dev), out.shape[0],
         int(out.dtype is torch.float32), pws, nws)
    return out


def grouped_matmul_dw(dy, x, offsets=None, *, dy_rows=None, dy_div=1, x_rows=None, x_div=1,
                      out=None, accumulate=False, ws=None, stream=None):
    """dW_e = sum over the expert's sorted rows i of dy[i] x[i]^T: dy bf16
    [n, N], x bf16 [m, K] -> [E, N, K] fp32 (or bf16, given as ``out``); zeros
    for an expert without rows. ``accumulate`` adds to fp32 ``out``."""
    dev = _matrix(dy, "dy", _BF16).get_device()
    _matrix(x, "x", _BF16, dev)
    _no_history(dy, x)
    N, K = dy.shape[1], x.shape[1]
    R = _count(dy, dy_rows, "dy_rows")
    if _count(x, x_rows, "x_rows") != R:
        _fail(f"dy and x: {R} and {_count(x, x_rows, 'x_rows')} rows")
    E = 1 if offsets is None else _need(offsets, "offsets", _I32, dev).numel() - 1
    if accumulate and out is None:
        _fail("out: needed to accumulate into")
    out = _output(out, "out", (E, N, K), (torch.float32, torch.bfloat16), dev, stream)
    if out.shape[-2:] != (N, K) or out.numel() != E * N * K:
        _fail(f"out: {tuple(out.shape)}, [{E}, {N}, {K}] is needed")
    ws, pws, nws = _workspace(_lib.MOE_GEMM_DW, R, N, K, E, dev, stream, ws)
    _run("moe_grouped_gemm_dw", dev, stream, dy.data_ptr(), _index(dy_rows, "dy_rows", R, dev),
         _int(dy_div, "dy_div"), dy.shape[0], x.data_ptr(), _index(x_rows, "x_rows", R, dev),
         _int(x_div, "x_div"), x.shape[0], _offsets(offsets, E, dev), R, N, K, E, out.data_ptr(), int(out.dtype is torch.float32),
         int(bool(accumulate)), pws, nws)
    return out


def _row_weights(w, w_rows, R, dev):
    if w is None:
        if w_rows is not None:
            _fail("w_rows: given without w")
        return None, None, 0
    _need(w, "w", _F32, dev)
    if w_rows is None and w.numel() < R:
        _fail(f"w: {w.numel()} weights for {R} rows")
    return w.data_ptr(), _index(w_rows, "w_rows", R, dev), _int(w.numel(), "w")


def _limit(n_rows, dev):
    if n_rows is None:
        return None
    if _need(n_rows, "n_rows", _I32, dev).numel() != 1:
        _fail("n_rows: one value is needed")
    return n_rows.data_ptr()


def _halves(h):
    if _matrix(h, "h", _BF16).shape[1] % 2:
        _fail(f"h: an even number of columns is needed, got {h.shape[1]}")
    return h.shape[0], h.shape[1] // 2, h.get_device()


def swiglu(h, w=None, w_rows=None, n_rows=None, out=None, stream=None):
    """a[r] = w_r silu(g) u of rows h [R, 2I] = [g | u], bf16 [R, I]; w fp32:
    the row's weight ``w[w_rows[r]]`` (``w[r]`` without ``w_rows``, 1 without
    ``w``). ``n_rows`` (int32 [1] on the device, e.g. ``offsets[E:]``): only the
    rows below it. I is a multiple of 8."""
    R, I, dev = _halves(h)
    _no_history(h, w)
    pw, pr, wn = _row_weights(w, w_rows, R, dev)
    out = _rows_output(out, "out", R, I, None, _BF16, dev, stream)
    _run("moe_swiglu", dev, stream, h.data_ptr(), pw, pr, wn, _limit(n_rows, dev), R, I,
         out.data_ptr())
    return out


def swiglu_grad(h, da, w=None, w_rows=None, n_rows=None, dh=None, dw=None, a=None, stream=None):
    """Gradients of ``swiglu`` for da [R, I]: (dh [R, 2I] bf16, dw fp32 of w's
    shape, or None without w). dw is written at the rows' indices, which must be
    distinct; a ``dw`` that is not given is zero elsewhere. ``a`` (bf16 [R, I],
    optional) receives swiglu's result again."""
    R, I, dev = _halves(h)
    if _matrix(da, "da", _BF16, dev).shape != (R, I):
        _fail(f"da: {tuple(da.shape)}, [{R}, {I}] is needed")
    _no_history(h, da, w)
    pw, pr, wn = _row_weights(w, w_rows, R, dev)
    dh = _rows_output(dh, "dh", R, 2 * I, None, _BF16, dev, stream)
    if w is not None:
        if dw is None:
            dw = _output(dw, "dw", w.shape, _F32, dev, stream)
            with torch.cuda.stream(stream):
                dw.zero_()
        elif _need(dw, "dw", _F32, dev).numel() != wn:
            _fail(f"dw: {tuple(dw.shape)}, {tuple(w.shape)} is needed")
    elif dw is not None:
        _fail("dw: given without w")
    if a is not None and _matrix(a, "a", _BF16, dev).shape != (R, I):
        _fail(f"a: {tuple(a.shape)}, [{R}, {I}] is needed")
    _run("moe_swiglu_grad", dev, stream, h.data_ptr(), da.data_ptr(), pw, pr, wn,
         _limit(n_rows, dev), R, I, dh.data_ptr(), None if dw is None else dw.data_ptr(),
         None if a is None else a.data_ptr())
    return dh, dw


def _to_fp8(fn, x, R, K, n_rows, q, s, dev, stream):
    q = _output(q, "q", (R, K), _FP8, dev, stream)
    s = _output(s, "s", (R, -(-K // 128)), _F32, dev, stream)
    if q.shape != (R, K) or s.shape != (R, -(-K // 128)):
        _fail(f"q, s: {tuple(q.shape)}, {tuple(s.shape)} for {R} rows of {K}")
    _run(fn, dev, stream, x.data_ptr(), _limit(n_rows, dev), R, K, q.data_ptr(), s.data_ptr())
    return q, s


def quant_fp8(x, n_rows=None, q=None, s=None, stream=None):
    """Rows x bf16 [R, K] as (E4M3 codes [R, K], fp32 scales [R, ceil(K/128)]):
    scale = max(amax, 2^-100) / 448 over 128 columns of a row, code = x / scale
    to the nearest E4M3. K is a multiple of 8."""
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x)
    return _to_fp8("moe_quant_fp8", x, x.shape[0], x.shape[1], n_rows, q, s, dev, stream)


def swiglu_quant_fp8(h, n_rows=None, q=None, s=None, stream=None):
    """``quant_fp8`` of the fp32 values silu(g) u of rows h [R, 2I] = [g | u]."""
    R, I, dev = _halves(h)
    _no_history(h)
    return _to_fp8("moe_swiglu_quant_fp8", h, R, I, n_rows, q, s, dev, stream)


def _to_mxfp4(fn, x, R, K, n_rows, q, s, dev, stream):
    if K % 32:
        _fail(f"{K} columns, a multiple of 32 is needed")
    if q is None:
        q = _output(None, "q", (R, K // 2), _U8, dev, stream)
    if s is None:
        s = _output(None, "s", (R, K // 32), _E8M0, dev, stream)
    _run(fn, dev, stream, x.data_ptr(), _limit(n_rows, dev), R, K, _at(q, "q", _U8, (R, K // 2), dev),
         _at(s, "s", _E8M0, (R, K // 32), dev))
    return q, s


def quant_mxfp4(x, n_rows=None, q=None, s=None, stream=None):
    """Rows x bf16 [R, K] in MXFP4: (E2M1 codes uint8 [R, K/2], the even column in the
    low half, E8M0 scales uint8 [R, K/32]): scale = 2^(floor(log2 amax) - 2), at least
    2^-127, over 32 columns of a row, code = x / scale to the nearest of 0, 0.5, 1, 1.5,
    2, 3, 4, 6 (ties to the even code). An infinity or NaN makes its block's scale NaN.
    ``n_rows`` as for ``swiglu``. K is a multiple of 32."""
    dev = _matrix(x, "x", _BF16).get_device()
    _no_history(x)
    return _to_mxfp4("moe_quant_mxfp4", x, x.shape[0], x.shape[1], n_rows, q, s, dev, stream)


def swiglu_quant_mxfp4(h, n_rows=None, q=None, s=None, stream=None):
    """``quant_mxfp4`` of the fp32 values silu(g) u of rows h [R, 2I] = [g | u]."""
    R, I, dev = _halves(h)
    _no_history(h)
    return _to_mxfp4("moe_swiglu_quant_mxfp4", h, R, I, n_rows, q, s, dev, stream)


def quant_mxfp4_matrices(w, q=None, s=None, stream=None):
    """Matrices w bf16 [E, N, K] (or [N, K]) in MXFP4, their rows as ``quant_mxfp4``
    has them, in the kernel layout that ``grouped_matmul_mxfp4`` reads (blocks of 16
    rows x 128 columns, include/moe.h): (codes [E, N, K/2], scales [E, N, K/32]). N is a
    multiple of 16, K of 128."""
    dev = _need(w, "w", _BF16).get_device()
    _no_history(w)
    if w.dim() not in (2, 3):
        _fail(f"w: [E, N, K] or [N, K] is needed, got {tuple(w.shape)}")
    E, N, K = (1, *w.shape) if w.dim() == 2 else w.shape
    if N % 16 or K % 128:
        _fail(f"w: {N} x {K}, multiples of 16 and 128 are needed")
    _int(max(E, N, K), "w")
    lead = w.shape[:-1]
    q = _output(q, "q", (*lead, K // 2), _U8, dev, stream)
    s = _output(s, "s", (*lead, K // 32), _E8M0, dev, stream)
    if q.shape != (*lead, K // 2) or s.shape != (*lead, K // 32):
        _fail(f"q, s: {tuple(q.shape)}, {tuple(s.shape)} for {tuple(w.shape)}")
    _run("moe_quant_mxfp4_matrices", dev, stream, w.data_ptr(), E, N, K, q.data_ptr(), s.data_ptr())
    return q, s
