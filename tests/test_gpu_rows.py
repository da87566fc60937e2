"""The norm with its outputs in bf16, FP8 and MXFP4 and its gradient, and the moves
between tokens and sorted order with theirs, against plain 64-bit forms.

Tolerances, by arithmetic. A sum of squares over H columns is made of chains of at
most H/64 additions a lane, six steps between lanes and three between wavefronts, all
of one sign: off by at most (H/64 + 10) 2^-24 of itself, its root's inverse by half of
that and three roundings. y has two more factors: y is within N = (H/64 + 16) 2^-24 of
its value before the rounding to bf16, 2^-8. FP8 and MXFP4 codes round values that are
that near: half a step of E4M3 (2^-4 of the value, 2^-10 of the scale at least) on
top, and MXFP4 codes between those of y (1 - N) and y (1 + N).
The gradient's row sum <g, x> has H terms of either sign: off by at most (H/64 + 12)
2^-24 of the sum of their magnitudes.
dw's sum over R rows: chains of R/slots rows a slot, slots/16 parts, 16 groups, at
most (R + 64) 2^-24 of the magnitudes, the terms themselves N off.
Moves: k products and sums in fp32, k 2^-23 of the magnitudes; a dot product of H
terms in chains of H/64 and six steps, (H/64 + 8) 2^-24 of them.
"""
import numpy as np
import pytest
import torch

from mixture_experts_gate_amd import _lib, products as P, rows as W

from test_gpu_mxfp4 import _gen, _randn, _within, _codes

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, EPS = 2.0 ** -8, 1e-6


def _near(H):
    return (H / 64 + 16) * 2.0 ** -24


def _stream_rows(g, R, H):
    """Rows of sizes far apart, as a residual stream has them."""
    size = torch.exp(2 * torch.randn(R, 1, device=DEV, generator=g))
    return (size * torch.randn(R, H, device=DEV, generator=g)).to(torch.bfloat16)


def _norm_ref(t, w, eps=EPS):
    t = t.double()
    return t / torch.sqrt((t * t).mean(1, keepdim=True) + eps) * w.double()


# rows, columns: a wavefront a row (up to 1024 columns) and a workgroup a row, in
# registers (up to 8192) and past them; ends inside a block of 128
NORMS = [(1, 8), (3, 64), (5, 512), (4, 520), (33, 1024), (2, 1032), (7, 2048), (300, 1096), (1, 4096), (9, 4104),
         (3, 8192), (2, 8200), (3, 20000), (1, 65536)]


@pytest.mark.parametrize("residual", ["none", "new", "over x", "over residual"])
@pytest.mark.parametrize("R,H", NORMS)
def test_norm(R, H, residual):
    g = _gen(R * H)
    x, w = _stream_rows(g, R, H), _randn(g, H)
    r = total = None
    t = x
    if residual != "none":
        r = _stream_rows(g, R, H)
        t = (x.float() + r.float()).to(torch.bfloat16)
        total = {"new": None, "over x": x, "over residual": r}[residual]
    out = W.rms_norm(x, w, EPS, r, total=total)
    y = out if r is None else out[0]
    if r is not None:
        assert torch.equal(out[1], t) and (total is None or out[1] is total)
    ref = _norm_ref(t, w)
    b = _near(H) * ref.abs()
    _within(y, ref, b + (ref.abs() + b) * BF16, "y")


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("R,H", NORMS)
def test_norm_fp8(R, H, residual):
    g = _gen(R + H)
    x, w = _stream_rows(g, R, H), _randn(g, H)
    r = _stream_rows(g, R, H) if residual else None
    plain = W.rms_norm(x, w, EPS, r)
    y = torch.empty_like(x)
    got = W.rms_norm_fp8(x, w, EPS, r, out=y)
    t = x
    if residual:
        t = plain[1]
        assert torch.equal(got[2], t)
        plain = plain[0]
    assert torch.equal(y, plain)
    q, s = got[:2]
    ref = _norm_ref(t, w)
    pad = torch.nn.functional.pad(ref, (0, -H % 128)).view(R, -1, 128)
    scale = pad.abs().amax(2).clamp(min=2.0 ** -100) / 448
    _within(s, scale, (_near(H) + 2 ** -22) * scale, "scale")
    each = s.double().repeat_interleave(128, 1)[:, :H]
    _within(q.double() * each, ref, _near(H) * ref.abs() + torch.maximum(2 ** -4 * ref.abs() * (1 + _near(H)), 2 ** -10 * each) * (1 + 2 ** -20), "q")
    # without y, and by the converter from y itself but for the rounding between
    q2, s2 = W.rms_norm_fp8(x, w, EPS, r)[:2]
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("R,H", [n for n in NORMS if n[1] % 32 == 0])
def test_norm_mxfp4(R, H):
    g = _gen(R + 2 * H)
    x, w, r = _stream_rows(g, R, H), _randn(g, H), _stream_rows(g, R, H)
    y = torch.empty_like(x)
    q, s, t = W.rms_norm_mxfp4(x, w, EPS, r, out=y)
    plain, total = W.rms_norm(x, w, EPS, r)
    assert torch.equal(y, plain) and torch.equal(t, total)
    ref, near = _norm_ref(t, w), _near(H)
    blocks = ref.abs().view(R, -1, 32).amax(-1)
    lo, hi = ((torch.frexp(blocks * f).exponent - 3).clamp(min=-127) + 127 for f in (1 - near, 1 + near))
    lo, hi = (torch.where(blocks > 0, b, 0) for b in (lo, hi))
    s = s.long()
    assert bool(((s >= lo) & (s <= hi)).all())
    both = torch.stack((q & 15, q >> 4), -1).reshape(R, H).long()
    c = torch.where(both >= 8, -(both & 7), both)
    a, b = _codes(ref * (1 - near), s), _codes(ref * (1 + near), s)
    assert bool(((c >= torch.minimum(a, b)) & (c <= torch.maximum(a, b))).all())
    q2, s2 = W.rms_norm_mxfp4(t, w, EPS)             # of the same rows, no residual
    assert torch.equal(q2, q) and torch.equal(s2.long(), s)


def test_norm_of_rows_at_the_edges():
    """Zero rows (with eps their norm is 0, without NaN), infinities and NaN stay in
    their rows, and values whose squares come near fp32's range."""
    H = 256
    x = _randn(_gen(1), 6, H)
    w = torch.ones(H, device=DEV, dtype=torch.bfloat16)
    x[1] = 0
    x[2, 7], x[3, 9] = float("inf"), float("nan")
    x[4] = 2.0 ** 58
    y = W.rms_norm(x, w, EPS)
    ref = _norm_ref(x, w)
    for i in (0, 1, 4, 5):
        _within(y[i], ref[i], (_near(H) + BF16 * (1 + _near(H))) * ref[i].abs(), f"row {i}")
    assert bool((y[1] == 0).all()) and bool(torch.isnan(y[3]).all())
    assert bool(torch.isnan(y[2, 7])) and bool((y[2, :7] == 0).all())
    assert bool(torch.isnan(W.rms_norm(x[1:2], w, 0.0)).all())
    q, s = W.rms_norm_fp8(x, w, EPS)
    assert bool(torch.isnan(s[3]).all()) and bool(torch.isfinite(s[[0, 1, 4, 5]]).all())
    q, s = W.rms_norm_mxfp4(x, w, EPS)
    assert bool((s[3] == 255).all()) and bool((s[[0, 1, 4, 5]] < 255).all())


# --------------------------------------------------------------- gradient --

def _grad_ref(x, w, dy, dt, eps=EPS):
    """(dx, dw, bounds of both before the rounding to bf16)"""
    x, w, dy = x.double(), w.double(), dy.double()
    R, H = x.shape
    inv = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    n, g = x * inv, dy * w
    mean, size = (g * n).mean(1, keepdim=True), (g * n).abs().mean(1, keepdim=True)
    dx = inv * (g - n * mean)
    near = _near(H)
    bound = 2 * near * inv * (g.abs() + n.abs() * (mean.abs() + size))
    if dt is not None:
        dx = dx + dt.double()
        bound = bound + 2.0 ** -23 * (dx.abs() + dt.double().abs())
    dw, mag = (dy * n).sum(0), (dy * n).abs().sum(0)
    return dx, dw, bound, ((R + 64) * 2.0 ** -24 + near) * mag


GRADS = [(1, 8), (3, 64), (5, 512), (2100, 72), (33, 1024), (2, 1032), (301, 2048), (700, 1096), (1, 4096), (520, 4104),
         (3, 8192), (2, 8200), (3, 16384), (5000, 128)]


@pytest.mark.parametrize("dtotal", [False, True])
@pytest.mark.parametrize("R,H", GRADS)
def test_norm_gradient(R, H, dtotal):
    g = _gen(R + H)
    x, w, dy = _stream_rows(g, R, H), _randn(g, H), _randn(g, R, H)
    dt = _randn(g, R, H) if dtotal else None
    ref, refw, b, bw = _grad_ref(x, w, dy, dt)
    dx, dw = W.rms_norm_grad(x, w, dy, EPS, dt)
    _within(dx, ref, b + (ref.abs() + b) * BF16, "dx")
    _within(dw, refw, bw, "dw")
    # accumulated, into dtotal's own rows, by the same bits
    held = torch.randn(H, device=DEV, generator=g)
    dw2 = held.clone()
    into = dt.clone() if dtotal else None
    dx2, _ = W.rms_norm_grad(x, w, dy, EPS, into, dx=into, dw=dw2, accumulate=True)
    assert torch.equal(dx2, dx) and torch.equal(dw2, held + dw)


def test_norm_gradient_against_differences():
    """<dx, v> and <dw, u> against central differences of the 64-bit norm. The
    difference quotient is off by its third derivative, h^2 / 6 of it, below 1e-9 of the
    value here; dx by its rounding, 2^-8 of each term, and the bound of the sums."""
    R, H = 4, 264
    g = _gen(9)
    x, w, dy = _randn(g, R, H), _randn(g, H), _randn(g, R, H)
    dx, dw = W.rms_norm_grad(x, w, dy, EPS)
    v = torch.randn(R, H, device=DEV, dtype=torch.float64, generator=g)
    u = torch.randn(H, device=DEV, dtype=torch.float64, generator=g)
    h = 1e-5

    def f(a, b):
        return float((_norm_ref(x.double() + a * v, w.double() + b * u) * dy.double()).sum())

    ref, refw, b, bw = _grad_ref(x, w, dy, None)
    for num, got, size in ((f(h, 0) - f(-h, 0), dx, (b + (ref.abs() + b) * BF16) * v.abs()),
                           (f(0, h) - f(0, -h), dw, bw * u.abs())):
        along = v if got is dx else u
        assert abs(num / (2 * h) - float((got.double() * along).sum())) <= float(size.sum()) + 1e-5


def test_norm_gradient_of_no_rows():
    x = torch.empty(0, 64, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(64, device=DEV, dtype=torch.bfloat16)
    dw = torch.full((64,), 3.0, device=DEV)
    W.rms_norm_grad(x, w, x, dw=dw, accumulate=True)
    assert bool((dw == 3).all())
    dx, dw = W.rms_norm_grad(x, w, x, dw=dw)
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    assert W.rms_norm(x, w).shape == (0, 64) and W.rms_norm_fp8(x, w)[0].shape == (0, 64)


def test_norm_gradient_same_bits_by_handle_and_graph():
    R, H = 700, 2048
    g = _gen(3)
    x, w, dy, dt = _randn(g, R, H), _randn(g, H), _randn(g, R, H), _randn(g, R, H)
    want = W.rms_norm_grad(x, w, dy, EPS, dt)
    ws = torch.empty(_lib.moe_rms_norm_grad_workspace(R, H), dtype=torch.uint8, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty(H, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with pytest.raises(ValueError):
        W.rms_norm_grad(x, w, dy, EPS, dt, dx=dx, dw=dw, stream=side.cuda_stream)
    W.rms_norm_grad(x, w, dy, EPS, dt, dx=dx, dw=dw, ws=ws, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.rms_norm_grad(x, w, dy, EPS, dt, dx=dx, dw=dw, ws=ws)
    for seed in range(3):
        x.copy_(_randn(_gen(seed), R, H))
        graph.replay()
        want = W.rms_norm_grad(x, w, dy, EPS, dt)
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    with pytest.raises(_lib.MoeError):
        W.rms_norm_grad(x, w, dy, EPS, dt, ws=ws[:-16])


# ------------------------------------------------------------------ moves --

def _pair_rows(g, T, k, n, dropped=0.0):
    """Distinct rows of n for T x k pairs; some of them none (-1, or past the end)."""
    rows = torch.randperm(n, generator=g, device=DEV)[:T * k].view(T, k)
    gone = torch.rand(T, k, device=DEV, generator=g) < dropped
    rows = torch.where(gone, torch.where(rows % 2 == 0, -1, n + rows), rows)
    return rows.to(torch.int32).contiguous(), ~gone


MOVES = [(1, 1, 8), (1, 8, 2048), (3, 2, 72), (7, 6, 4096), (64, 6, 520), (301, 3, 1032), (130, 9, 256), (40, 17, 2056),
         (2, 8, 20000)]


@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("T,k,H", MOVES)
def test_moves(T, k, H, dropped):
    g = _gen(T * k + H)
    n = T * k + 5
    rows, live = _pair_rows(g, T, k, n, dropped)
    at = rows[live].long()
    # dispatch
    x = _randn(g, T, H)
    out = torch.full((n, H), 7.0, device=DEV, dtype=torch.bfloat16)
    assert W.dispatch(x, rows, out=out) is out
    want = torch.full_like(out, 7.0)
    want[at] = x.repeat_interleave(k, 0).view(T, k, H)[live]
    assert torch.equal(out, want)
    # combine, with and without weights and the added rows, bf16 and fp32
    y, w, add = _randn(g, n, H), torch.randn(T, k, device=DEV, generator=g), _randn(g, T, H)
    picked = torch.where(live[:, :, None], y.double()[rows.long().clamp(0, n - 1)], 0.0)
    for wt in (w, None):
        terms = picked if wt is None else picked * wt.double()[:, :, None]
        for a in (add, None):
            ref = terms.sum(1) + (0 if a is None else a.double())
            mag = terms.abs().sum(1) + (0 if a is None else a.double().abs())
            b = (k + 1) * 2.0 ** -23 * mag
            for yy in (y, y.float()):
                _within(W.combine(yy, rows, wt, a), ref, b + (ref.abs() + b) * BF16, "out")
    # gradient of the combine
    dout = _randn(g, T, H)
    dy = torch.full((n, H), 7.0, device=DEV, dtype=torch.bfloat16)
    dy, dw = W.combine_grad(dout, y, rows, w, dy=dy)
    want = torch.full((n, H), 7.0, device=DEV, dtype=torch.float64)
    want[at] = (w.double()[:, :, None] * dout.double()[:, None, :])[live]
    left = torch.ones(n, dtype=torch.bool, device=DEV)
    left[at] = False
    assert bool((dy[left] == 7).all())
    _within(dy, want, (2.0 ** -24 + BF16 * (1 + 2.0 ** -24)) * want.abs(), "dy")
    terms = picked * dout.double()[:, None, :]
    _within(dw, terms.sum(2), (H / 64 + 8) * 2.0 ** -24 * terms.abs().sum(2), "dw")
    assert bool((dw[~live] == 0).all())
    # gradient of the dispatch: the rows of a token, added
    dx = W.combine(dy, rows)
    terms = torch.where(live[:, :, None], dy.double()[rows.long().clamp(0, n - 1)], 0.0)
    b = k * 2.0 ** -23 * terms.abs().sum(1)
    _within(dx, terms.sum(1), b + (terms.sum(1).abs() + b) * BF16, "dx")


def test_a_row_that_is_not_read_may_hold_anything():
    """Rows of no pair, and pairs without a row beside ones that have theirs, bring no
    NaN in; a weight of 0 does not hide one, as the formula has it."""
    T, k, H = 6, 3, 264
    g = _gen(5)
    n = T * k + 4
    rows, live = _pair_rows(g, T, k, n, 0.4)
    y = torch.full((n, H), float("nan"), device=DEV, dtype=torch.bfloat16)
    y[rows[live].long()] = _randn(g, int(live.sum()), H)
    w, dout = torch.rand(T, k, device=DEV, generator=g), _randn(g, T, H)
    w[~live] = float("nan")
    assert bool(torch.isfinite(W.combine(y, rows, w)).all())
    dy, dw = W.combine_grad(dout, y, rows, w, dy=torch.zeros_like(y))
    assert bool(torch.isfinite(dy).all()) and bool(torch.isfinite(dw).all())
    t, j = live.nonzero()[0].tolist()
    w[t, j] = 0.0
    y[rows[t, j].long()] = float("nan")
    assert bool(torch.isnan(W.combine(y, rows, w)[t]).all())


def test_one_row_for_several_pairs():
    """Reading allows it: the combine adds the row for each, also within a token."""
    g = _gen(6)
    y, w = _randn(g, 3, 64), torch.rand(4, 5, device=DEV, generator=g)
    rows = torch.randint(0, 3, (4, 5), device=DEV, generator=g, dtype=torch.int32)
    terms = y.double()[rows.long()] * w.double()[:, :, None]
    b = 6 * 2.0 ** -23 * terms.abs().sum(1)
    _within(W.combine(y, rows, w), terms.sum(1), b + (terms.sum(1).abs() + b) * BF16, "out")


def test_moves_beyond_4_gib():
    """Sorted rows past 4 GiB and past 2^31 values."""
    H, T, k = 4096, 9, 2
    n = (1 << 32) // (2 * H) + 40
    g = _gen(8)
    rows = (n - 1 - torch.randperm(30, generator=g, device=DEV)[:T * k]).view(T, k).to(torch.int32)
    x = _randn(g, T, H)
    y = torch.zeros(n, H, device=DEV, dtype=torch.bfloat16)
    W.dispatch(x, rows, out=y)
    assert torch.equal(y[rows.long()], x[:, None].expand(T, k, H))
    assert int((y != 0).any(1).sum()) == T * k
    assert torch.equal(W.combine(y, rows), 2 * x)
    w = torch.rand(T, k, device=DEV, generator=g)
    dy, dw = W.combine_grad(x, y, rows, w, dy=torch.empty_like(y))
    assert torch.equal(dy[rows.long()], (w[:, :, None] * x.float()[:, None]).to(torch.bfloat16))


def test_moves_without_sorted_rows():
    """No sorted rows at all: every pair's row is outside them."""
    g = _gen(14)
    T, k, H = 5, 3, 72
    rows = torch.randint(-1, 40, (T, k), device=DEV, generator=g, dtype=torch.int32)
    x, w = _randn(g, T, H), torch.rand(T, k, device=DEV, generator=g)
    none = torch.empty(0, H, device=DEV, dtype=torch.bfloat16)
    assert W.dispatch(x, rows, out=none) is none
    assert not bool(W.combine(none, rows, w).any())
    assert torch.equal(W.combine(none.float(), rows, w, x), x)
    dy, dw = W.combine_grad(x, none, rows, w, dw=torch.ones(T, k, device=DEV))
    assert dy.shape == (0, H) and not bool(dw.any())


@pytest.mark.parametrize("R,H", [((1 << 25) + 9, 8), ((1 << 20) + 3, 4104)])
def test_norm_and_gradient_over_many_rows(R, H):
    """More workgroups than a launch has along x, and values past 2^32."""
    g = _gen(15)
    x, w = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16), _randn(g, H)
    last, dlast = _stream_rows(g, 70, H), _randn(g, 70, H)
    x[-70:] = last
    y = W.rms_norm(x, w, EPS)
    assert torch.equal(y[-70:], W.rms_norm(last, w, EPS)) and not bool(y[-200:-70].any())
    del y
    q, s = W.rms_norm_fp8(x, w, EPS)
    q2, s2 = W.rms_norm_fp8(last, w, EPS)
    assert torch.equal(q[-70:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-70:], s2)
    del q, s
    dy = torch.zeros_like(x)
    dy[-70:] = dlast
    dx, dw = W.rms_norm_grad(x, w, dy, EPS, dx=dy)
    dx2, _ = W.rms_norm_grad(last, w, dlast, EPS)
    assert torch.equal(dx[-70:], dx2) and not bool(dx[-200:-70].any())
    n = last.double() / torch.sqrt((last.double() ** 2).mean(1, keepdim=True) + EPS)
    terms = dlast.double() * n
    b = (_near(H) + (70 + 64) * 2.0 ** -24) * terms.abs().sum(0)      # (the other rows add zeros)
    _within(dw, terms.sum(0), b, "dw")


def test_moves_of_many_pairs():
    """Units past 2^31: 34 GB of tokens, whose pairs have the few rows there are."""
    T, H = (1 << 28) + 3, 64
    g = _gen(16)
    rows = torch.full((T, 1), -1, device=DEV, dtype=torch.int32)
    at = torch.tensor([0, 1, (1 << 28) - 1, 1 << 28, T - 1], device=DEV)
    rows[at, 0] = torch.arange(5, device=DEV, dtype=torch.int32)
    y = _randn(g, 5, H)
    out = W.combine(y, rows)
    assert torch.equal(out[at], y)
    assert not bool(out[2:2000].any()) and not bool(out[-2000:-4].any())
    back = W.dispatch(out, rows, out=torch.zeros_like(y))
    assert torch.equal(back, y)
    w = torch.full((T, 1), 2.0, device=DEV)
    dy, dw = W.combine_grad(out, y, rows, w, dy=torch.zeros_like(y))
    assert torch.equal(dy, 2 * y)
    ref = (y.double() ** 2).sum(1)
    _within(dw[at, 0], ref, (H / 64 + 8) * 2.0 ** -24 * ref, "dw")
    assert not bool(dw[-2000:-4].any())


def test_two_calls_at_once():
    """On two streams, each call with workspaces of its own: each has its bits."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = []
    for i in range(2):
        g = _gen(17 + i)
        rows, _ = _pair_rows(g, 300, 8, 2400)
        sets.append((_stream_rows(g, 300, 2048), _randn(g, 2048), _randn(g, 300, 2048), rows,
                     torch.rand(300, 8, device=DEV, generator=g)))

    def run(i, stream):
        x, w, dy, rows, f = sets[i]
        y = W.rms_norm(x, w, EPS, stream=stream)
        out = W.combine(W.dispatch(y, rows, stream=stream), rows, f, x, stream=stream)
        return (y, out, *W.rms_norm_grad(x, w, dy, EPS, out, stream=stream))

    want = [run(i, None) for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(run(i, sides[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[i]))


def test_moves_in_a_graph_and_on_a_stream():
    T, k, H = 50, 4, 1024
    g = _gen(11)
    rows, _ = _pair_rows(g, T, k, T * k)
    x, w = _randn(g, T, H), torch.rand(T, k, device=DEV, generator=g)
    out, back = torch.empty(T * k, H, device=DEV, dtype=torch.bfloat16), torch.empty_like(x)
    dy, dw = torch.empty_like(out), torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.dispatch(x, rows, out=out)
        W.combine(out, rows, w, x, out=back)
        W.combine_grad(back, out, rows, w, dy=dy, dw=dw)
    side = torch.cuda.Stream()
    for seed in range(3):
        x.copy_(_randn(_gen(seed), T, H))
        w.copy_(torch.rand(T, k, device=DEV, generator=g))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        o2 = W.dispatch(x, rows, stream=side)
        b2 = W.combine(o2, rows, w, x, stream=side)
        d2, e2 = W.combine_grad(b2, o2, rows, w, stream=side)
        torch.cuda.synchronize()
        for got, want in ((out, o2), (back, b2), (dy, d2), (dw, e2)):
            assert torch.equal(got, want)


def test_refusals():
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, device=DEV, dtype=bf), torch.zeros(64, device=DEV, dtype=bf)
    rows, f = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    y = torch.zeros(8, 64, device=DEV, dtype=bf)
    grad = torch.zeros(4, 64, device=DEV, dtype=bf, requires_grad=True)
    bad = [
        lambda: W.rms_norm(x.float(), w), lambda: W.rms_norm(x[:, ::2], w), lambda: W.rms_norm(x, w[:32]),
        lambda: W.rms_norm(x, w.float()), lambda: W.rms_norm(x, w, residual=x[:3]), lambda: W.rms_norm(x, w, total=x),
        lambda: W.rms_norm(grad, w), lambda: W.rms_norm(x, w.cpu()), lambda: W.rms_norm(x, w, out=y),
        lambda: W.rms_norm_mxfp4(torch.zeros(4, 72, device=DEV, dtype=bf), w),
        lambda: W.rms_norm_fp8(x, w, q=torch.zeros(4, 32, device=DEV, dtype=torch.uint8)),
        lambda: W.rms_norm_grad(x, w, x[:3]), lambda: W.rms_norm_grad(x, w, x, dtotal=y),
        lambda: W.rms_norm_grad(x, w, x, accumulate=True), lambda: W.rms_norm_grad(x, w, grad),
        lambda: W.dispatch(x, rows[:3].contiguous()), lambda: W.dispatch(x, rows.long()), lambda: W.dispatch(x, rows.view(-1)),
        lambda: W.dispatch(x, rows, out=y[:, :32]), lambda: W.combine(y, rows, f.view(-1)), lambda: W.combine(y, rows, f, y),
        lambda: W.combine(y, rows, f.double()), lambda: W.combine(y, rows.cpu()), lambda: W.combine(y, None),
        lambda: W.combine_grad(x, y, rows, None), lambda: W.combine_grad(x, y.float(), rows, f),
        lambda: W.combine_grad(x, y, rows, f, dy=x), lambda: W.combine(grad, rows),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    odd = torch.zeros(4 * 60, device=DEV, dtype=bf).view(4, 60)
    off = torch.zeros(4 * 64 + 4, device=DEV, dtype=bf)[4:].view(4, 64)
    wide = torch.zeros(1, 16392, device=DEV, dtype=bf)
    for call in (lambda: W.rms_norm(odd, w[:60].contiguous()), lambda: W.rms_norm(off, w), lambda: W.rms_norm(x, w, -1.0),
                 lambda: W.rms_norm(x, w, float("nan")), lambda: W.dispatch(off, rows), lambda: W.dispatch(odd, rows),
                 lambda: W.rms_norm_grad(wide, wide[0], wide), lambda: W.combine(off, rows)):
        with pytest.raises(_lib.MoeError):
            call()
