"""Rows and matrices to MXFP4 and the product of MXFP4 rows with MXFP4 matrices,
against plain 64-bit forms.

Rows of bf16 quantise exactly: the scale is a power of two and the rounding has one
result, so codes and scales are compared as whole numbers (with the numpy encoder).
Quantised activations silu(g) u are computed in fp32 first, to within D = 2^-20 of
their value (sigmoid's few units of 2^-24 and three roundings): a code has to lie
between those of v (1 - D) and v (1 + D), a scale likewise.

The product. The matrix core's instruction adds at most 128 exact products (E2M1 x
E2M1 x powers of two) and the sum so far; over 3e6 random operands with scales up to
2^60 apart the result was off by at most 3.7 2^-24 of the sum of their magnitudes,
and 2^-22 is what the header promises. K/64 instructions at most make |error| <= K/64
2^-22 sum |x||w|; 16 parts of a cut sum add 16 roundings, 2^-20 of it. A bf16 result
adds its rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from mixture_experts_gate_amd import _lib, layer as LY, products as P, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, D = 2.0 ** -8, 2.0 ** -20


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def _within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst "
        f"{float((err / bound.clamp(min=1e-300)).max()):.3g} of the bound")


_GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
GRID = torch.cat([_GRID, -_GRID])


def decode(q, s):
    """float64 values of codes [.., K/2] and scales [.., K/32]."""
    q, s = q.view(torch.uint8).cpu(), s.view(torch.uint8).cpu()
    both = torch.stack((q & 15, q >> 4), -1).long()
    v = GRID[both].reshape(*s.shape, 32)
    scale = torch.where(s == 255, torch.tensor(float("nan"), dtype=torch.float64), torch.exp2(s.double() - 127))
    return (v * scale[..., None]).reshape(*s.shape[:-1], -1).to(DEV)


def kernel_order(q, s):
    """Row-major codes [E, N, K/2] and scales in blocks of 16 rows x 128 columns."""
    E, N, h = q.shape
    return (q.view(E, N // 16, 16, h // 64, 4, 16).permute(0, 1, 3, 4, 2, 5).reshape(E, N, h).contiguous(),
            s.view(E, N // 16, 16, h // 64, 4).permute(0, 1, 3, 4, 2).reshape(E, N, h // 16).contiguous())


def _encode(x):
    """The numpy encoder on rows of any float tensor, on the device."""
    q, s = synth.encode_mxfp4(x.float().cpu().numpy())
    return torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)


# ------------------------------------------------------------ quantisation --

@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (17, 160), (1, 4096), (130, 2048), (257, 8160)])
def test_rows_to_mxfp4_are_the_encoders(R, K):
    g = _gen(R * K)
    x = torch.randn(R, K, device=DEV, generator=g)
    x *= torch.exp2(torch.randint(-30, 30, (R, K // 32), device=DEV, generator=g).float()).repeat_interleave(32, 1)
    x[torch.rand(R, K, device=DEV, generator=g) < 0.05] = 0.0
    x = x.to(torch.bfloat16)
    q, s = P.quant_mxfp4(x)
    eq, es = _encode(x)
    assert q.dtype == s.dtype == torch.uint8
    assert torch.equal(s, es) and torch.equal(q, eq)


def test_every_bf16_value_to_mxfp4():
    """Every finite bf16, alone in its block beside one value 1 to 256 times as large
    (the block's scale), and next to nothing."""
    bits = torch.arange(65536, dtype=torch.int32)
    v = (bits << 16).view(torch.float32)
    v = v[torch.isfinite(v)]
    rows = []
    for factor in (0.0, 1.0, 1.99, 4.0, 13.0, 256.0):
        block = torch.zeros(v.numel(), 32)
        block[:, 5] = v
        block[:, 17] = (v * factor).clamp(-3e38, 3e38)
        rows.append(block)
    x = torch.cat(rows).to(torch.bfloat16).to(DEV)
    x[~torch.isfinite(x)] = 0
    q, s = P.quant_mxfp4(x)
    eq, es = _encode(x)
    assert torch.equal(s, es) and torch.equal(q, eq)


def test_rows_that_are_not_finite():
    x = _randn(_gen(1), 4, 128)
    x[0, 40], x[1, 3], x[2, 127] = float("inf"), float("nan"), float("-inf")
    q, s = P.quant_mxfp4(x)
    bad = torch.zeros(4, 4, dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[1, 0] = bad[2, 3] = True
    assert bool((s[bad] == 255).all()) and bool((s[~bad] < 255).all())
    assert not bool(q.view(4, 4, 16)[bad].any())
    eq, es = _encode(torch.where(torch.isfinite(x), x, torch.zeros_like(x)))
    assert torch.equal(q.view(4, 4, 16)[~bad], eq.view(4, 4, 16)[~bad])
    h = torch.zeros(1, 128, device=DEV, dtype=torch.bfloat16)
    h[0, 0] = h[0, 64] = 3e38                        # silu(g) u passes fp32
    q, s = P.swiglu_quant_mxfp4(h)
    assert s.tolist() == [[255, 0]] and not bool(q.any())


def _codes(v, s):
    """Codes (as signed whole numbers along the grid) of float64 v at scale bytes s."""
    a = (v / torch.exp2(s.double() - 127).repeat_interleave(32, -1)).abs()
    m = torch.where(a < 2, torch.round(2 * a), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    return torch.where(v < 0, -1, 1) * m.clamp(max=7)


def between(q, s, v):
    """Codes and scales are those of values within D of v."""
    blocks = v.abs().view(*v.shape[:-1], -1, 32).amax(-1)
    lo, hi = ((torch.frexp(blocks * f).exponent - 3).clamp(min=-127) + 127 for f in (1 - D, 1 + D))
    lo, hi = (torch.where(blocks > 0, b, 0) for b in (lo, hi))
    s = s.long()
    assert bool(((s >= lo) & (s <= hi)).all())
    both = torch.stack((q & 15, q >> 4), -1).reshape(v.shape).long()
    c = torch.where(both >= 8, -(both & 7), both)
    a, b = _codes(v * (1 - D), s), _codes(v * (1 + D), s)
    assert bool(((c >= torch.minimum(a, b)) & (c <= torch.maximum(a, b))).all())


@pytest.mark.parametrize("R,I", [(1, 32), (5, 96), (33, 2048), (300, 768)])
def test_activation_to_mxfp4(R, I):
    g = _gen(R + I)
    h = (3 * torch.randn(R, 2 * I, device=DEV, generator=g)).to(torch.bfloat16)
    q, s = P.swiglu_quant_mxfp4(h)
    a, u = h.double().chunk(2, 1)
    between(q, s, a * torch.sigmoid(a) * u)


def test_row_limit_leaves_the_rest():
    x, h = _randn(_gen(2), 9, 64), _randn(_gen(3), 9, 128)
    for n in (0, 4, 9, 100, -3):
        lim = torch.tensor([n], dtype=torch.int32, device=DEV)
        for call, arg in ((P.quant_mxfp4, x), (P.swiglu_quant_mxfp4, h)):
            q = torch.full((9, 32), 77, device=DEV, dtype=torch.uint8)
            s = torch.full((9, 2), 77, device=DEV, dtype=torch.uint8)
            call(arg, n_rows=lim, q=q, s=s)
            fq, fs = call(arg)
            m = min(max(n, 0), 9)
            assert torch.equal(q[:m], fq[:m]) and torch.equal(s[:m], fs[:m])
            assert bool((q[m:] == 77).all()) and bool((s[m:] == 77).all())


@pytest.mark.parametrize("E,N,K", [(1, 16, 128), (3, 48, 384), (2, 256, 1024)])
def test_matrices_to_mxfp4(E, N, K):
    w = (0.02 * torch.randn(E, N, K, device=DEV, generator=_gen(N))).to(torch.bfloat16)
    q, s = P.quant_mxfp4_matrices(w)
    eq, es = _encode(w.view(E * N, K))
    eq, es = kernel_order(eq.view(E, N, K // 2), es.view(E, N, K // 32))
    assert torch.equal(q, eq) and torch.equal(s, es)
    q1, s1 = P.quant_mxfp4_matrices(w[0])
    assert torch.equal(q1, q[0]) and torch.equal(s1, s[0])


# ---------------------------------------------------------------- product --

# counts per expert, N, K: the streaming kernel (up to 16 rows per expert), tiles,
# tiles whose sum is cut
SHAPES = [
    ([1], 16, 128),
    ([1, 0, 1, 0], 64, 128),
    ([3, 0, 17, 5], 48, 256),
    ([16, 15, 1, 0, 16], 272, 1152),
    ([0, 40, 1, 16, 17, 0, 3] + [0] * 9, 144, 4736),
    ([2] * 100 + [0] * 50, 128, 384),
    ([0] * 499 + [37], 32, 640),
    ([0, 0, 130], 256, 256),
    ([33, 64, 65, 0, 1, 127, 128, 129], 272, 128),
    ([257, 1, 255, 256, 300], 528, 384),
    ([17], 16, 128),
    ([700], 144, 512),
    ([261, 130], 112, 3712),
    ([2500], 144, 1024),
    ([40], 256, 4096),
    ([100, 0, 31], 48, 2176),
    ([150, 61, 0, 97] * 14, 768, 768),
    ([1300, 513, 1, 900, 1255], 2064, 1152),
    # large tiles, several a workgroup; K of an odd number of slabs
    ([300, 259, 0, 1, 700, 257] * 8, 2064, 768),
    ([130] * 50 + [0] * 3 + [700], 3856, 1024),
    ([2000, 2049, 31], 4112, 1280),
    ([513] * 16, 2048, 1792),
    ([300] * 24, 1040, 1664),
]


def _case(counts, N, K, seed, spread=6):
    """Random codes (all sixteen) and scales: (x codes, scales, w codes, scales, as
    row-major; w in the kernel layout)."""
    g = _gen(seed)

    def byte(*shape):
        return torch.randint(0, 256, shape, device=DEV, generator=g).to(torch.uint8)

    def scale(*shape):
        return (120 + torch.randint(-spread, spread + 1, shape, device=DEV, generator=g)).to(torch.uint8)

    E, R = len(counts), sum(counts)
    return g, byte, scale, (byte(E, N, K // 2), scale(E, N, K // 32))


def _ref(xd, wd, counts, idx):
    R = sum(counts)
    y = torch.zeros(R, wd.shape[1], dtype=torch.float64, device=DEV)
    m, lo = torch.zeros_like(y), 0
    for e, n in enumerate(counts):
        if n:
            a, b = xd[idx[lo:lo + n]], wd[e].t().contiguous()
            y[lo:lo + n], m[lo:lo + n] = a @ b, a.abs() @ b.abs()
        lo += n
    return y, m


def _bound(ref, mag, K, dtype):
    b = (K / 64 + 4) * 2.0 ** -22 * mag
    return b + (ref.abs() + b) * BF16 if dtype == torch.bfloat16 else b


@pytest.mark.parametrize("indexing", ["plain", "gather", "scatter"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_product(shape, dtype, indexing):
    counts, N, K = SHAPES[shape]
    R = sum(counts)
    g, byte, scale, (wq, ws) = _case(counts, N, K, shape)
    rows = out_rows = None
    n, div, idx = R, 1, torch.arange(R, device=DEV)
    if indexing == "gather":
        n, div = max(1, R // 2), 3
        rows = torch.randint(0, n * div, (R,), generator=g, device=DEV, dtype=torch.int32)
        idx = (rows // div).long()
    if indexing == "scatter":
        out_rows = torch.randperm(R, generator=g, device=DEV).to(torch.int32)
    x, xs = byte(n, K // 2), scale(n, K // 32)
    kq, ks = kernel_order(wq, ws)
    ref, mag = _ref(decode(x, xs), decode(wq, ws), counts, idx)
    out = torch.full((R, N), 7.0, device=DEV, dtype=dtype)
    y = P.grouped_matmul_mxfp4(x, xs, kq, ks, _offsets(counts), rows=rows, div=div, out_rows=out_rows, out=out)
    assert y is out
    _within(y if out_rows is None else y[out_rows.long()], ref, _bound(ref, mag, K, dtype), "y")


@pytest.mark.parametrize("shape", [3, 9, 12])
def test_product_with_far_scales(shape):
    """Scales 2^-30 to 2^30 apart inside a row."""
    counts, N, K = SHAPES[shape]
    _, byte, scale, (wq, ws) = _case(counts, N, K, 50 + shape, spread=30)
    R = sum(counts)
    x, xs = byte(R, K // 2), scale(R, K // 32)
    ref, mag = _ref(decode(x, xs), decode(wq, ws), counts, torch.arange(R, device=DEV))
    y = P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), _offsets(counts),
                               out=torch.empty(R, N, device=DEV))
    _within(y, ref, _bound(ref, mag, K, torch.float32), "y")


@pytest.mark.parametrize("shape", [3, 9, 12])
def test_nan_scales_reach_their_rows_and_columns_alone(shape):
    counts, N, K = SHAPES[shape]
    _, byte, scale, (wq, ws) = _case(counts, N, K, 60 + shape)
    R, E = sum(counts), len(counts)
    x, xs = byte(R, K // 2), scale(R, K // 32)
    off = _offsets(counts)
    clean = P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), off)
    xs[R - 1, 1] = 255
    last = max(e for e in range(E) if counts[e])
    ws[last, 5, K // 32 - 1] = 255
    y = P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), off)
    nan = torch.zeros(R, N, dtype=torch.bool, device=DEV)
    nan[R - 1] = True
    nan[R - counts[last]:, 5] = True
    assert torch.equal(torch.isnan(y), nan)
    assert torch.equal(y[~nan], clean[~nan])


def test_product_from_packed_blobs():
    """TableMatrices of packed "mxfp4" blobs give the tensors' bits, W13 and W2."""
    H, I, E = 256, 128, 5
    rng = np.random.default_rng(3)
    blobs = np.stack([synth._gauss_mxfp4_blob(rng, H, I, 0.05) for _ in range(E)])
    lay = synth.blob_layout(H, I, "mxfp4")
    ex = LY.DeviceExperts(blobs, lay)
    counts = [3, 0, 50, 1, 30]
    off, g = _offsets(counts), _gen(4)
    host = torch.from_numpy(blobs).to(DEV)
    for mat, N, K, oc, os_ in ((_lib.MOE_MAT_W13, 2 * I, H, lay.w13, lay.s13), (_lib.MOE_MAT_W2, H, I, lay.w2, lay.s2)):
        x, xs = P.quant_mxfp4(_randn(g, sum(counts), K))
        wq = host[:, oc:oc + N * K // 2].reshape(E, N, K // 2).contiguous()
        ws = host[:, os_:os_ + N * K // 32].reshape(E, N, K // 32).contiguous()
        want = P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), off)
        got = P.grouped_matmul_mxfp4(x, xs, P.TableMatrices(ex.table, mat, E, N, K), None, off)
        assert torch.equal(got, want)
        ref, mag = _ref(decode(x, xs), decode(wq, ws), counts, torch.arange(sum(counts), device=DEV))
        _within(got, ref, _bound(ref, mag, K, torch.bfloat16), "y")


# the streaming kernel, tiles, tiles with a cut sum, large tiles
PATHS = {"stream": ([5, 0, 9, 3], 64, 512), "tiles": ([300, 0, 140, 77] * 8, 1040, 256), "cut": ([60, 0, 31], 64, 2048),
         "large": ([300, 0, 140, 77] * 8, 2064, 768)}


@pytest.mark.parametrize("path", list(PATHS))
def test_rows_that_are_left(path):
    """Rows past offsets[E] and rows whose index is out of range, on either side."""
    counts, N, K = PATHS[path]
    _, byte, scale, (wq, ws) = _case(counts, N, K, 70)
    R, E, extra = sum(counts), len(counts), 13
    n = R + extra
    x, xs = byte(n, K // 2), scale(n, K // 32)
    kq, ks = kernel_order(wq, ws)
    want = P.grouped_matmul_mxfp4(x, xs, kq, ks, _offsets(counts), out=torch.empty(n, N, device=DEV))
    assert (P._workspace(_lib.MOE_GEMM_MXFP4, n, N, K, E, 0, None, None)[2] > 0) == (path == "cut")
    rows = torch.arange(n, dtype=torch.int32, device=DEV)
    rows[2], rows[R - 1] = -1, n
    to = torch.arange(n, dtype=torch.int32, device=DEV)
    to[4], to[6] = -5, n + 3
    out = torch.full((n, N), 7.0, device=DEV)
    P.grouped_matmul_mxfp4(x, xs, kq, ks, _offsets(counts), rows=rows, out_rows=to, out=out)
    left = torch.zeros(n, dtype=torch.bool, device=DEV)
    left[[2, R - 1, 4, 6]] = True
    left[R:] = True
    assert bool((out[left] == 7.0).all())
    assert torch.equal(out[~left], want[~left])


@pytest.mark.parametrize("path", list(PATHS))
def test_offsets_that_do_not_ascend_stay_inside(path):
    counts, N, K = PATHS[path]
    _, byte, scale, (wq, ws) = _case(counts, N, K, 80)
    R, E = sum(counts), len(counts)
    x, xs = byte(R, K // 2), scale(R, K // 32)
    kq, ks = kernel_order(wq, ws)
    g = torch.Generator().manual_seed(1)
    for trial in range(4):
        off = torch.randint(-R, 2 * R, (E + 1,), generator=g).to(torch.int32)
        if trial == 0:
            off = torch.tensor([0, R] * E, dtype=torch.int32)[:E + 1]
        buf = torch.full((R + 64, N), 7.0, device=DEV)
        P.grouped_matmul_mxfp4(x, xs, kq, ks, off.to(DEV), out=buf[:R])
        torch.cuda.synchronize()
        assert bool((buf[R:] == 7.0).all())


@pytest.mark.parametrize("path", list(PATHS))
def test_same_bits_by_handle_stream_and_graph(path):
    """A stream handle (nothing is allocated), another stream, and a captured call
    replayed with other inputs between give the call's bits."""
    counts, N, K = PATHS[path]
    _, byte, scale, (wq, ws) = _case(counts, N, K, 90)
    R, E = sum(counts), len(counts)
    x, xs = byte(R, K // 2), scale(R, K // 32)
    kq, ks = kernel_order(wq, ws)
    off, dev = _offsets(counts), 0
    size = P._workspace(_lib.MOE_GEMM_MXFP4, R, N, K, E, dev, None, None)[2]
    want = P.grouped_matmul_mxfp4(x, xs, kq, ks, off)
    space = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    out = torch.empty(R, N, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    P.grouped_matmul_mxfp4(x, xs, kq, ks, off, out=out, ws=space, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want)
    got = P.grouped_matmul_mxfp4(x, xs, kq, ks, off, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        P.grouped_matmul_mxfp4(x, xs, kq, ks, off, stream=side.cuda_stream)
    xb = torch.randn(R, K, device=DEV, generator=_gen(91)).to(torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.quant_mxfp4(xb, q=x, s=xs)
        P.grouped_matmul_mxfp4(x, xs, kq, ks, off, out=out, ws=space)
    for seed in range(3):
        xb.copy_(torch.randn(R, K, device=DEV, generator=_gen(92 + seed)))
        graph.replay()
        q2, s2 = P.quant_mxfp4(xb)
        eager = P.grouped_matmul_mxfp4(q2, s2, kq, ks, off)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("path", list(PATHS))
def test_two_products_at_once(path):
    """On two streams, the sums' workspaces their own: each has its bits."""
    counts, N, K = PATHS[path]
    R, off = sum(counts), _offsets(counts)
    sides, sets = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(2):
        _, byte, scale, w = _case(counts, N, K, 96 + i)
        sets.append((byte(R, K // 2), scale(R, K // 32), *kernel_order(*w), off))
    want = [P.grouped_matmul_mxfp4(*s) for s in sets]
    torch.cuda.synchronize()
    got = [[P.grouped_matmul_mxfp4(*sets[i], stream=sides[i]) for i in range(2)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


def test_cut_sum_without_its_workspace_runs_whole():
    counts, N, K = PATHS["cut"]
    _, byte, scale, (wq, ws) = _case(counts, N, K, 95)
    R, E = sum(counts), len(counts)
    x, xs = byte(R, K // 2), scale(R, K // 32)
    kq, ks = kernel_order(wq, ws)
    ref, mag = _ref(decode(x, xs), decode(wq, ws), counts, torch.arange(R, device=DEV))
    y = P.grouped_matmul_mxfp4(x, xs, kq, ks, _offsets(counts), out=torch.empty(R, N, device=DEV),
                               ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    _within(y, ref, _bound(ref, mag, K, torch.float32), "y")


def test_product_beyond_4_gib():
    """Rows of x, of the matrices and of the result past 4 GiB."""
    K, N, n = 4096, 64, (1 << 32) // 2048 + 300
    g = _gen(7)
    x = torch.zeros(n, K // 2, dtype=torch.uint8, device=DEV)
    xs = torch.full((n, K // 32), 127, dtype=torch.uint8, device=DEV)
    x[-300:] = torch.randint(0, 256, (300, K // 2), device=DEV, generator=g).to(torch.uint8)
    wq = torch.randint(0, 256, (1, N, K // 2), device=DEV, generator=g).to(torch.uint8)
    ws = torch.full((1, N, K // 32), 120, dtype=torch.uint8, device=DEV)
    rows = torch.arange(n - 300, n, dtype=torch.int32, device=DEV)
    kq, ks = kernel_order(wq, ws)
    for take in (300, 9):
        idx = rows[-take:].contiguous()
        ref, mag = _ref(decode(x[-take:], xs[-take:]), decode(wq, ws), [take], torch.arange(take, device=DEV))
        y = P.grouped_matmul_mxfp4(x, xs, kq, ks, rows=idx)
        _within(y, ref, _bound(ref, mag, K, torch.bfloat16), "y")


def test_more_tiles_a_workgroup_than_are_looked_up_at_a_time():
    """512 experts of a row or two, 33 columns of tiles each: 66 tiles a compute unit."""
    E, N, K = 512, 8448, 768
    counts = [1 + (e % 5 == 0) for e in range(E)]
    R, g = sum(counts), _gen(12)
    x = torch.randint(0, 256, (R, K // 2), device=DEV, generator=g, dtype=torch.uint8)
    xs = (120 + torch.randint(-6, 7, (R, K // 32), device=DEV, generator=g)).to(torch.uint8)
    wq = torch.randint(0, 256, (E, N, K // 2), device=DEV, generator=g, dtype=torch.uint8)
    ws = (120 + torch.randint(-6, 7, (E, N, K // 32), device=DEV, generator=g)).to(torch.uint8)
    y = P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), _offsets(counts), out=torch.empty(R, N, device=DEV))
    xd, first = decode(x, xs), np.concatenate([[0], np.cumsum(counts)])
    for e in list(range(0, E, 23)) + [1, 255, 256, 510, 511]:
        lo, hi = int(first[e]), int(first[e + 1])
        ref, mag = _ref(xd[lo:hi], decode(wq[e], ws[e])[None], [hi - lo], torch.arange(hi - lo, device=DEV))
        _within(y[lo:hi], ref, _bound(ref, mag, K, torch.float32), f"expert {e}")


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.uint8, device=DEV)
    xs = torch.zeros(4, 4, dtype=torch.uint8, device=DEV)
    w = torch.zeros(2, 16, 64, dtype=torch.uint8, device=DEV)
    ws = torch.zeros(2, 16, 4, dtype=torch.uint8, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    P.grouped_matmul_mxfp4(x, xs, w, ws, off)
    P.grouped_matmul_mxfp4(x, xs.view(torch.float8_e8m0fnu), w, ws.view(torch.float8_e8m0fnu), off)
    bad = [
        lambda: P.grouped_matmul_mxfp4(x.float(), xs, w, ws, off),
        lambda: P.grouped_matmul_mxfp4(x[:, :32], xs, w, ws, off),
        lambda: P.grouped_matmul_mxfp4(x, xs[:3].contiguous(), w, ws, off),
        lambda: P.grouped_matmul_mxfp4(x, xs, w, None, off),
        lambda: P.grouped_matmul_mxfp4(x, xs, w, ws[:, :8].contiguous(), off),
        lambda: P.grouped_matmul_mxfp4(x, xs, w, ws),
        lambda: P.grouped_matmul_mxfp4(x, xs, w, ws, off[:2].contiguous()),
        lambda: P.grouped_matmul_mxfp4(x, xs, w.cpu(), ws, off),
        lambda: P.grouped_matmul_mxfp4(x, xs, w, ws, off, out=torch.empty(3, 16, device=DEV)),
        lambda: P.quant_mxfp4(torch.zeros(4, 40, dtype=torch.bfloat16, device=DEV)),
        lambda: P.quant_mxfp4(torch.zeros(4, 64, device=DEV)),
        lambda: P.quant_mxfp4(torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV, requires_grad=True)),
        lambda: P.swiglu_quant_mxfp4(torch.zeros(4, 80, dtype=torch.bfloat16, device=DEV)),
        lambda: P.quant_mxfp4_matrices(torch.zeros(2, 24, 128, dtype=torch.bfloat16, device=DEV)),
        lambda: P.quant_mxfp4_matrices(torch.zeros(2, 16, 64, dtype=torch.bfloat16, device=DEV)),
        lambda: P.quant_mxfp4(torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV), q=x),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    # an N that is no multiple of 16, rows that start off a multiple of 16
    with pytest.raises(_lib.MoeError):
        P.grouped_matmul_mxfp4(x, xs, w[:, :8].contiguous(), ws[:, :8].contiguous(), off)
    flat = torch.zeros(4 * 64 + 8, dtype=torch.uint8, device=DEV)
    with pytest.raises(_lib.MoeError):
        P.grouped_matmul_mxfp4(flat[8:].view(4, 64), xs, w, ws, off)
