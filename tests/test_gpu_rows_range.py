"""The norm and its gradient on rows whose squares, or whose products dy w x, lie
outside fp32's range: every finite row has its norm.

Tolerances are those of test_gpu_rows.py: these rows' sums are made in 64 bits, whose
errors are far below the fp32 ones that the bounds count, and results are rounded to
fp32 and then to the output as elsewhere. The sizes are chosen so that results
are normal bf16 numbers."""
import pytest
import torch

from mixture_experts_gate_amd import products as P, rows as W

from test_gpu_mxfp4 import _codes, _gen, _randn, _within
from test_gpu_rows import _grad_ref, _near, _norm_ref

pytestmark = pytest.mark.gpu
DEV, BF16 = "cuda", 2.0 ** -8

# around the borders of the squares' sum (2^128 and 2^-149, and inside them), and far past them
SIZES = (-120, -100, -76, -70, -60, -50, -45, -40, 0, 1, 40, 50, 54, 57, 58, 59, 60, 61, 62, 63, 64, 65, 90, 120)
HS = [8, 64, 520, 1024, 1096, 2048, 4104, 8192, 8200, 20000]


def _rows(g, sizes, H):
    """A row of each size, its values within a factor of about a hundred."""
    v = torch.rand(len(sizes), H, device=DEV, generator=g) + 0.01
    sign = torch.where(torch.rand(len(sizes), H, device=DEV, generator=g) < 0.5, -1.0, 1.0)
    scale = torch.exp2(torch.tensor(sizes, dtype=torch.float64, device=DEV))[:, None]
    return (v * sign).double().mul(scale).to(torch.bfloat16)


def _y_bound(ref, H):
    b = _near(H) * ref.abs()
    return b + (ref.abs() + b) * BF16


@pytest.mark.parametrize("H", HS)
def test_norm_of_rows_of_any_size(H):
    g = _gen(H)
    x, w = _rows(g, SIZES, H), _randn(g, H)
    ref = _norm_ref(x, w, 0.0)
    _within(W.rms_norm(x, w, 0.0), ref, _y_bound(ref, H), "y")
    # with eps the smallest rows are not stretched to 1; they stay normal numbers
    ref = _norm_ref(x, w, 1e-6)
    _within(W.rms_norm(x, w, 1e-6), ref, _y_bound(ref, H) + 2.0 ** -134, "y with eps")
    # the largest eps there may be
    ref = _norm_ref(x, w, float(torch.tensor(3e38)))
    _within(W.rms_norm(x, w, 3e38), ref, _y_bound(ref, H) + 2.0 ** -134, "y with the largest eps")


@pytest.mark.parametrize("H", HS)
@pytest.mark.parametrize("residual", ["new", "over x", "over residual"])
def test_residual_of_rows_of_any_size(H, residual):
    g = _gen(H + 1)
    x, r, w = _rows(g, SIZES, H), _rows(g, SIZES, H), _randn(g, H)
    t = (x.double() + r.double()).to(torch.float32).to(torch.bfloat16)
    total = {"new": None, "over x": x, "over residual": r}[residual]
    y, got = W.rms_norm(x, w, 0.0, r, total=total)
    assert torch.equal(got, t)
    ref = _norm_ref(t, w, 0.0)
    _within(y, ref, _y_bound(ref, H), "y")


@pytest.mark.parametrize("H", HS)
def test_codes_of_rows_of_any_size(H):
    g = _gen(H + 2)
    x, w = _rows(g, SIZES, H), _randn(g, H)
    R, near = x.shape[0], _near(H)
    y = torch.empty_like(x)
    q, s = W.rms_norm_fp8(x, w, 0.0, out=y)
    ref = _norm_ref(x, w, 0.0)
    _within(y, ref, _y_bound(ref, H), "y")
    pad = torch.nn.functional.pad(ref, (0, -H % 128)).view(R, -1, 128)
    scale = pad.abs().amax(2) / 448
    _within(s, scale, (near + 2 ** -22) * scale, "scale")
    each = s.double().repeat_interleave(128, 1)[:, :H]
    _within(q.double() * each, ref,
            near * ref.abs() + torch.maximum(2 ** -4 * ref.abs() * (1 + near), 2 ** -10 * each) * (1 + 2 ** -20), "q")
    if H % 32:
        return
    q, s = W.rms_norm_mxfp4(x, w, 0.0)
    blocks = ref.abs().view(R, -1, 32).amax(-1)
    lo, hi = (torch.frexp(blocks * f).exponent - 3 + 127 for f in (1 - near, 1 + near))
    s = s.long()
    assert bool(((s >= lo) & (s <= hi)).all())
    both = torch.stack((q & 15, q >> 4), -1).reshape(R, H).long()
    c = torch.where(both >= 8, -(both & 7), both)
    a, b = _codes(ref * (1 - near), s), _codes(ref * (1 + near), s)
    assert bool(((c >= torch.minimum(a, b)) & (c <= torch.maximum(a, b))).all())


# x, dy and w of 2^a, 2^b and 2^c; every result is a normal bf16 number
GRAD_SIZES = [(0, 0), (60, 60), (64, 90), (38, 50), (100, 20), (120, 110), (58, -20), (1, 90), (-70, -40), (-76, -60),
              (-110, -50), (-45, 0), (-40, 60), (0, -60)]


@pytest.mark.parametrize("dtotal", [False, True])
@pytest.mark.parametrize("wsize", [0, 38])
@pytest.mark.parametrize("R,H", [(14, 8), (14, 520), (4200, 72), (28, 1024), (1150, 1032), (1040, 2056), (28, 4104),
                                 (600, 4104), (14, 8200), (28, 16384)])
def test_norm_gradient_of_rows_of_any_size(R, H, wsize, dtotal):
    """Several rows a slot among them, far ones beside near ones."""
    g = _gen(R + H)
    pick = torch.randint(0, len(GRAD_SIZES), (R,), generator=torch.Generator().manual_seed(R)).tolist()
    if R < 100:
        pick = [i % len(GRAD_SIZES) for i in range(R)]
    x, dy = (_rows(g, [GRAD_SIZES[i][j] - (wsize if j else 0) for i in pick], H) for j in (0, 1))
    w = (_randn(g, H).double() * 2.0 ** wsize).to(torch.bfloat16)
    dt = _rows(g, [GRAD_SIZES[i][1] - GRAD_SIZES[i][0] for i in pick], H) if dtotal else None
    ref, refw, b, bw = _grad_ref(x, w, dy, dt, 0.0)
    dx, dw = W.rms_norm_grad(x, w, dy, 0.0, dt)
    _within(dx, ref, b + (ref.abs() + b) * BF16, "dx")
    _within(dw, refw, bw, "dw")
    # over dy's own rows, the same bits
    dx2, dw2 = W.rms_norm_grad(x, w, dy, 0.0, dt, dx=dy)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_far_rows_that_are_not_finite():
    """Infinities and NaN stay in their rows, also in one whose other values are far."""
    H = 2048
    g = _gen(3)
    x, w, dy = _rows(g, [100, 100, 100, -100], H), _randn(g, H), _rows(g, [0, 0, 0, -60], H)
    x[1, 5], x[2, 6] = float("inf"), float("nan")
    y = W.rms_norm(x, w, 0.0)
    assert bool(torch.isnan(y[1, 5])) and not bool(y[1, :5].any()) and bool(torch.isnan(y[2]).all())
    ref = _norm_ref(x, w, 0.0)
    for i in (0, 3):
        _within(y[i], ref[i], _y_bound(ref[i], H), f"row {i}")
    dx, _ = W.rms_norm_grad(x, w, dy, 0.0)
    assert bool(torch.isnan(dx[1:3]).all())
    ref, _, b, _ = _grad_ref(x[[0, 3]], w, dy[[0, 3]], None, 0.0)
    _within(dx[[0, 3]], ref, b + (ref.abs() + b) * BF16, "dx")
    # rows of zeros: NaN without eps, as the formula has it, and 0 with it
    x.zero_()
    assert bool(torch.isnan(W.rms_norm(x, w, 0.0)).all()) and not bool(W.rms_norm(x, w, 1e-6).any())
    assert bool(torch.isnan(W.rms_norm_grad(x, w, dy, 0.0)[0]).all())


def test_far_rows_in_a_graph_give_the_calls_bits():
    H = 4096
    g = _gen(4)
    x, w, dy = _rows(g, SIZES, H), _randn(g, H), _rows(g, [0] * len(SIZES), H)
    y, t, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(H, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.rms_norm(x, w, 0.0, dy, out=y, total=t)
        W.rms_norm_grad(t, w, dy, 0.0, dx=dx, dw=dw)
    for seed in range(3):
        x.copy_(_rows(_gen(10 + seed), SIZES[::-1] if seed % 2 else SIZES, H))
        graph.replay()
        want_y, want_t = W.rms_norm(x, w, 0.0, dy)
        want_dx, want_dw = W.rms_norm_grad(want_t, w, dy, 0.0)
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(t, want_t)
        assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)


@pytest.mark.parametrize("R,H", [((1 << 23) + 70, 8), ((1 << 20) + 600, 1032)])
def test_far_rows_among_many(R, H):
    """Two thousand and more rows a slot: far rows at the first and last places of the
    kernel's turns of 2048, and neighbours of ordinary ones. (The other rows add zeros.)"""
    g = _gen(R)
    slots = (8 if H <= 1024 else 2) * torch.cuda.get_device_properties(0).multi_processor_count
    assert R > 2048 * slots
    at = [0, 1, slots - 1, 63 * slots, 64 * slots + 3, 65 * slots + 3, 2047 * slots + 5, 2048 * slots, 2048 * slots + 7, R - 1]
    far = [0, 5, 1, 8, 2, 3, 10, 4, 6, 7]
    x, dy = (torch.zeros(R, H, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    x[:] = 1.0
    xs, ds = (_rows(g, [GRAD_SIZES[i][j] for i in far], H) for j in (0, 1))
    x[at], dy[at] = xs, ds
    w = _randn(g, H)
    ref, refw, b, bw = _grad_ref(xs, w, ds, None, 0.0)
    dx, dw = W.rms_norm_grad(x, w, dy, 0.0, dx=dy)
    _within(dx[at], ref, b + (ref.abs() + b) * BF16, "dx")
    _within(dw, refw, bw, "dw")
    dx[at] = 0
    assert not bool(dx.any())
