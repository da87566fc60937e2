"""The expert products at the edges of what their calls allow: rows whose index
is outside its matrix next to values that are not finite.

Tolerance of a sum of n products of bf16 values in fp32: every addition is off
by at most one unit in the last place of a result that is at most the sum of the
terms' magnitudes, |error| <= n 2^-23 sum |a||b|.
"""
import numpy as np
import pytest
import torch

from mixture_experts_gate_amd import _lib, products as P, synth
from mixture_experts_gate_amd.layer import DeviceExperts, Fp8BlockLayer
from mixture_experts_gate_amd.train import TrainExperts

pytestmark = pytest.mark.gpu
DEV = "cuda"
SUM = 2.0 ** -23


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


# counts per expert, N, K and what the sizes select: 128 x 128 tiles, those with
# the sum cut into parts, 256 x 256 tiles (more than half of 256 compute units)
DW_PATHS = {
    "small": ([40, 0, 90, 700], 72, 80),
    "parts": ([1500], 256, 136),
    "large": ([700, 0, 1, 130, 64], 1544, 1288),
}


@pytest.mark.parametrize("side", ["x", "dy", "both", "x_of_indexed", "dy_of_indexed"])
@pytest.mark.parametrize("path", list(DW_PATHS))
def test_dw_row_without_a_partner_adds_nothing(path, side):
    """A sorted row whose index is outside one matrix adds nothing to dw, also
    where its row of the other matrix holds NaN or an infinity; every step of
    64 rows has such rows but one."""
    counts, N, K = DW_PATHS[path]
    g = _gen(sum(map(ord, path + side)))
    R, E, div = sum(counts), len(counts), 3
    parts = _lib.moe_grouped_gemm_workspace(_lib.MOE_GEMM_DW, R, N, K, E) > 0
    assert parts == (path == "parts")
    dy, x = _randn(g, R, N), _randn(g, R, K)
    pos = torch.arange(R, device=DEV)
    bad_x, bad_y = (pos * 7 % 61 == 3) & (pos // 64 != 2), (pos * 5 % 83 == 9) & (pos // 64 != 2)
    if side.startswith("x"):
        bad_y[:] = False
    if side.startswith("dy"):
        bad_x[:] = False
    bad = bad_x | bad_y
    assert bool(bad.any())
    # the row's place in each matrix: through an index or its own
    index_x, index_y = side != "dy", side != "x"
    at_x = torch.randperm(R, generator=g, device=DEV) if index_x else pos
    at_y = torch.randperm(R, generator=g, device=DEV) if index_y else pos
    dy[at_y[bad]] = float("nan")
    x[at_x[bad], ::2] = float("inf")
    kw = {}
    outside = torch.tensor([-1, R * div, -2 ** 31, 2 ** 31 - 1], device=DEV)
    if index_x:
        rows = at_x * div + pos % div
        rows[bad_x] = outside[pos[bad_x] % 4]
        kw.update(x_rows=rows.to(torch.int32), x_div=div)
    if index_y:
        rows = at_y * div + pos % div
        rows[bad_y] = outside[pos[bad_y] % 4]
        kw.update(dy_rows=rows.to(torch.int32), dy_div=div)
    yd, xd = dy.double()[at_y], x.double()[at_x]
    yd[bad], xd[bad] = 0, 0
    dw = P.grouped_matmul_dw(dy, x, _offsets(counts), **kw)
    lo = 0
    for e, n in enumerate(counts):
        a, b = yd[lo:lo + n].t().contiguous(), xd[lo:lo + n]
        lo += n
        err, bound = (dw[e].double() - a @ b).abs(), n * SUM * (a.abs() @ b.abs())
        assert bool((err <= bound).all()), f"expert {e}: {int((~(err <= bound)).sum())} values off"


def _same_rows(got, want, rows, what):
    for g, w in zip(got, want):
        assert torch.equal(g[rows], w), what


@pytest.mark.parametrize("call", ["swiglu", "swiglu_grad", "quant_fp8", "swiglu_quant_fp8"])
def test_rows_whose_threads_pass_32_bits(call):
    """More than 2^32 threads: the first rows, those around the 2^32nd thread and
    the last ones have the bits that a call on these rows alone gives."""
    # threads a row: I / 8 (swiglu), 64 (its gradient), 16 a block of 128 (FP8);
    # bytes of tensors for each of a row's I values
    R, I, per, size = {"swiglu": ((1 << 20) + 3, 32768, 4096, 6),
                       "swiglu_grad": ((1 << 26) + 5, 8, 64, 11),
                       "quant_fp8": ((1 << 28) + 77, 8, 16, 3.5),
                       "swiglu_quant_fp8": ((1 << 28) + 77, 8, 16, 5.5)}[call]
    assert R * per > 1 << 32
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < R * I * size + (1 << 30):
        pytest.skip("not enough free memory")
    g, edge = _gen(3), (1 << 32) // per
    rows = torch.tensor(sorted({0, 1, edge // 2, edge - 1, edge, edge + 1, R - 2, R - 1}), device=DEV)
    width = I if call == "quant_fp8" else 2 * I
    small = _randn(g, len(rows), width)
    h = torch.empty(R, width, device=DEV, dtype=torch.bfloat16)
    h[rows] = small
    if call == "swiglu":
        _same_rows([P.swiglu(h)], [P.swiglu(small)], rows, call)
    elif call == "swiglu_grad":
        dsmall = _randn(g, len(rows), I)
        da = torch.empty(R, I, device=DEV, dtype=torch.bfloat16)
        da[rows] = dsmall
        w = torch.rand(len(rows), generator=g, device=DEV)
        wide = torch.empty(R, device=DEV)
        wide[rows] = w
        _same_rows(P.swiglu_grad(h, da, wide), P.swiglu_grad(small, dsmall, w), rows, call)
    else:
        fn = getattr(P, call)
        (q, s), (qs, ss) = fn(h), fn(small)
        _same_rows([q.view(torch.uint8), s], [qs.view(torch.uint8), ss], rows, call)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["product", "dx", "fp8"])
def test_products_of_nearly_the_most_rows(kind):
    """One expert of 1.8e9 rows: the first, a middle and the last rows. Small
    whole numbers, whose sums (at most 16 * 9) are exact in bf16."""
    R, n = 1800 * 10 ** 6, 16
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < R * n * 4.5 + (1 << 30):
        pytest.skip("not enough free memory")
    g = _gen(4)
    at = torch.tensor([0, 1, R // 3, R - 300, R - 2, R - 1], device=DEV)
    few = torch.randint(-3, 4, (len(at), n), generator=g, device=DEV)
    w = torch.randint(-3, 4, (1, n, n), generator=g, device=DEV)
    ref = few.double() @ (w[0] if kind == "dx" else w[0].t().contiguous()).double()
    out = torch.zeros(R, n, device=DEV, dtype=torch.bfloat16)
    if kind == "fp8":
        e4m3 = torch.float8_e4m3fn
        x = torch.zeros(R, n, device=DEV, dtype=torch.uint8)
        x[at] = few.to(torch.float32).to(e4m3).view(torch.uint8)
        P.grouped_matmul_fp8(x, torch.ones(R, 1, device=DEV), w.to(torch.float32).to(e4m3),
                             torch.ones(1, 1, 1, device=DEV), out=out)
    else:
        x = torch.zeros(R, n, device=DEV, dtype=torch.bfloat16)
        x[at] = few.to(torch.bfloat16)
        (P.grouped_matmul if kind == "product" else P.grouped_matmul_dx)(
            x, w.to(torch.bfloat16), out=out)
    assert torch.equal(out[at].double(), ref)
    del x, out
    torch.cuda.empty_cache()


def _guarded(rows, n, dtype):
    """(a tensor [rows, n] of ones inside a larger one, a check that the rest is as it was)"""
    big = torch.ones(rows + 600, n, device=DEV, dtype=dtype)

    def rest():
        return bool((big[:300] == 1).all()) and bool((big[300 + rows:] == 1).all())
    return big[300:300 + rows], rest


# R, E, N, K: the streaming kernel (K held in registers, copied), 128 x 128 tiles,
# those in parts, 256 x 256 tiles
ROW_PATHS = {"stream": (150, 16, 64, 256), "stream_long": (150, 16, 64, 4672),
             "small": (400, 6, 136, 144), "parts": (261, 2, 112, 3648),
             "large": (4000, 5, 2056, 2064)}


@pytest.mark.parametrize("kind", ["product", "dx", "fp8", "dw"])
@pytest.mark.parametrize("path", list(ROW_PATHS))
def test_offsets_that_do_not_ascend_stay_inside(path, kind):
    R, E, N, K = ROW_PATHS[path]
    g = _gen(len(path))
    dy, x, w = _randn(g, R, N), _randn(g, R, K), _randn(g, E, N, K)
    for seed in range(4):
        h = torch.randint(-R, 2 * R, (E + 1,), generator=g, device=DEV).to(torch.int32)
        if seed == 3:
            h[0::2], h[1::2] = 0, R
        if kind == "dw":
            out, rest = _guarded(E * N, K, torch.float32)
            P.grouped_matmul_dw(dy, x, h, out=out.view(E, N, K))
        else:
            out, rest = _guarded(R, K if kind == "dx" else N, torch.bfloat16)
            if kind == "fp8":
                x8, s8 = P.quant_fp8(x)
                w8 = w.view(torch.uint8)[:, :, ::2].contiguous() & 0x3F
                P.grouped_matmul_fp8(x8, s8, w8, torch.ones(E, -(-N // 128), -(-K // 128), device=DEV),
                                     h, out=out)
            else:
                (P.grouped_matmul if kind == "product" else P.grouped_matmul_dx)(
                    x if kind == "product" else dy, w, h, out=out)
        assert rest(), (seed, h.tolist())


def test_offsets_whose_tiles_pass_32_bits():
    """256 of 512 experts that claim all of 2^29 rows: 2^29 tiles of 256 rows, and
    their total is cut to what ascending offsets can give."""
    R, E, n = 1 << 29, 512, 8
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < R * n * 5:
        pytest.skip("not enough free memory")
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1::2] = R
    x = torch.ones(R, n, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(E, n, n, device=DEV, dtype=torch.bfloat16)
    out, rest = _guarded(R, n, torch.bfloat16)
    for fn in (P.grouped_matmul, P.grouped_matmul_dx):
        out.fill_(1)
        fn(x, w, off, out=out)
        # (the first expert's rows are all of them: every row is computed)
        assert rest() and bool((out == 8).all())
    del x, out, rest
    torch.cuda.empty_cache()


def test_whole_numbers_past_32_bits_are_refused():
    """Divisors and sizes of a table's matrices that an int would cut to a valid one."""
    x, w = _randn(_gen(1), 4, 16), _randn(_gen(2), 1, 8, 16)
    rows = torch.arange(4, dtype=torch.int32, device=DEV)
    dy, big = _randn(_gen(3), 4, 8), 2 ** 32
    tab = torch.tensor([w.data_ptr(), 0, 0, 0], dtype=torch.int64, device=DEV)
    ok = P.TableMatrices(tab, _lib.MOE_MAT_W13, 1, 8, 16)
    assert torch.equal(P.grouped_matmul(x, ok), P.grouped_matmul(x, w))
    for div in (big + 1, 1 - big):
        for bad in (lambda: P.grouped_matmul(x, w, rows=rows, div=div),
                    lambda: P.grouped_matmul_dx(dy, w, rows=rows, div=div),
                    lambda: P.grouped_matmul_dw(dy, x, dy_rows=rows, dy_div=div),
                    lambda: P.grouped_matmul_dw(dy, x, x_rows=rows, x_div=div),
                    lambda: P.grouped_matmul_fp8(*P.quant_fp8(x), w.view(torch.uint8)[:, :, ::2].contiguous(),
                                                 torch.ones(1, 1, 1, device=DEV), rows=rows, div=div)):
            with pytest.raises(ValueError):
                bad()
    for bad in (ok._replace(E=big + 1), ok._replace(N=big + 8), ok._replace(K=big + 16)):
        with pytest.raises(ValueError):
            P.grouped_matmul(x, bad)
        with pytest.raises(ValueError):
            P._weights(bad, None, P._BF16, 0)


# ------------------------------------------------------------------ autograd --

def test_inputs_that_require_grad_are_refused():
    """Where gradients are enabled, by every call and for every input that has
    one; under no_grad the results are those of the plain tensors."""
    g = _gen(12)
    x, w, dy = _randn(g, 6, 32), _randn(g, 2, 16, 32), _randn(g, 6, 16)
    off, wt = _offsets([2, 4]), torch.rand(6, generator=g, device=DEV)
    w8, ws = w.view(torch.uint8)[:, :, ::2].contiguous(), torch.ones(2, 1, 1, device=DEV)
    x8, xs = P.quant_fp8(x)
    da = _randn(g, 6, 16)
    calls = [(lambda a, b: P.grouped_matmul(a, b, off), (x, w)),
             (lambda a, b: P.grouped_matmul_dx(a, b, off), (dy, w)),
             (lambda a, b: P.grouped_matmul_dw(a, b, off), (dy, x)),
             (lambda a, b: P.grouped_matmul_fp8(x8, a, w8, b, off), (xs, ws)),
             (lambda a, b: P.swiglu(a, b), (x, wt)),
             (lambda a, b, c: P.swiglu_grad(a, b, c), (x, da, wt)),
             (lambda a: P.quant_fp8(a), (x,)), (lambda a: P.swiglu_quant_fp8(a), (x,))]
    for call, inputs in calls:
        want = call(*inputs)
        for i in range(len(inputs)):
            leaf = [t.detach().requires_grad_(j == i) for j, t in enumerate(inputs)]
            with pytest.raises(ValueError, match="grad"):
                call(*leaf)
            with torch.no_grad():
                got = call(*leaf)
            for a, b in zip(*((r if isinstance(r, tuple) else (r,)) for r in (got, want))):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_product_inside_an_autograd_function():
    """The calls as forward and backward of a Function give autograd the product's
    gradients."""
    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, off):
            ctx.save_for_backward(x, w, off)
            return P.grouped_matmul(x, w, off)

        @staticmethod
        def backward(ctx, dy):
            x, w, off = ctx.saved_tensors
            dw = torch.empty_like(w)
            return (P.grouped_matmul_dx(dy, w, off), P.grouped_matmul_dw(dy, x, off, out=dw), None)

    g = _gen(13)
    x, w, dy = _randn(g, 40, 32), _randn(g, 2, 16, 32), _randn(g, 40, 16)
    off = _offsets([15, 25])
    x.requires_grad_(), w.requires_grad_()
    Product.apply(x, w, off).backward(dy)
    with torch.no_grad():
        assert torch.equal(x.grad, P.grouped_matmul_dx(dy, w, off))
        out = torch.empty_like(w)
        assert torch.equal(w.grad, P.grouped_matmul_dw(dy, x, off, out=out))


def test_layers_refuse_inputs_that_require_grad():
    g = _gen(14)
    T, E, k, H, I = 5, 4, 2, 64, 32
    x, wg = _randn(g, T, H), _randn(g, E, H)
    w13, w2 = _randn(g, E, 2 * I, H), _randn(g, E, H, I)
    ids = torch.tensor([[0, 1], [2, 3], [1, 2], [3, 0], [0, 2]], dtype=torch.int32, device=DEV)
    w, dout = torch.rand(T, k, generator=g, device=DEV), _randn(g, T, H)
    m = TrainExperts(H, E, k, I, T)
    want = m.forward(x, ids, w, w13, w2).clone()
    grads = [t.clone() for t in m.backward(dout)]
    for i in range(4):
        args = [t.detach().requires_grad_(j == i) for j, t in enumerate((x, w, w13, w2))]
        with pytest.raises(ValueError, match="grad"):
            m.forward(args[0], ids, *args[1:])
        with torch.no_grad():
            assert torch.equal(m.forward(args[0], ids, *args[1:]), want)
        # (backward's results are the gradients: it runs where gradients are enabled)
        assert all(torch.equal(a, b) for a, b in zip(m.backward(dout), grads))
    layer = Fp8BlockLayer(H, E, k, I, T)
    zeros = torch.zeros(2 * I * H, dtype=torch.uint8, device=DEV)      # codes and scales of all
    table = torch.full((E, 4), zeros.data_ptr(), dtype=torch.int64, device=DEV)
    for kw in (dict(x=x.detach().requires_grad_(), wg=wg), dict(x=x, wg=wg.detach().requires_grad_())):
        with pytest.raises(ValueError, match="grad"):
            layer.forward(T, table=table, **kw)


# ---------------------------------------------------- workspaces and streams --

# kind, R, N, K, E of products whose sums are cut
CUT = {"product": (_lib.MOE_GEMM_BF16, 261, 112, 3648, 1), "dx": (_lib.MOE_GEMM_DX, 300, 2048, 64, 2),
       "fp8": (_lib.MOE_GEMM_FP8, 261, 112, 3648, 1), "dw": (_lib.MOE_GEMM_DW, 1500, 256, 136, 1)}


@pytest.mark.parametrize("kind", list(CUT))
def test_stream_handle_and_given_workspace(kind):
    """A call with a workspace has the same bits on a stream, through its handle
    and with the workspace given; without one the sum runs whole: the same value
    within the two orders' errors. Nothing is written past the workspace."""
    gemm, R, N, K, E = CUT[kind]
    size = _lib.moe_grouped_gemm_workspace(gemm, R, N, K, E)
    assert 0 < size <= P.workspace_bound(R, N, K, E)
    g = _gen(31)
    x, w, dy = _randn(g, R, K), _randn(g, E, N, K), _randn(g, R, N)
    off = _offsets([R // E] * E)
    x8, xs = P.quant_fp8(x)
    w8, ws8 = P.quant_fp8(w.view(E * N, K))
    ws8 = torch.rand(E, -(-N // 128), -(-K // 128), generator=g, device=DEV)
    shape = {"product": (R, N), "fp8": (R, N), "dx": (R, K), "dw": (E, N, K)}[kind]

    def call(**kw):
        out = torch.zeros(shape, device=DEV)
        torch.cuda.synchronize()
        if kind == "product":
            P.grouped_matmul(x, w, off, out=out, **kw)
        elif kind == "dx":
            P.grouped_matmul_dx(dy, w, off, out=out, **kw)
        elif kind == "dw":
            P.grouped_matmul_dw(dy, x, off, out=out, **kw)
        else:
            P.grouped_matmul_fp8(x8, xs, w8.view(E, N, K), ws8, off, out=out, **kw)
        torch.cuda.synchronize()
        return out

    want, side = call(), torch.cuda.Stream()
    big = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    ws = big[256:256 + size]
    assert torch.equal(call(stream=side), want)
    assert torch.equal(call(ws=ws), want)
    assert torch.equal(call(ws=ws, stream=side.cuda_stream), want)
    assert bool((big[:256] == 0x5A).all()) and bool((big[256 + size:] == 0x5A).all())
    whole = call(stream=side.cuda_stream)
    assert torch.equal(call(ws=ws[:size - 16]), whole)
    # each order's additions (one a term): n 2^-23 of the magnitudes, and for FP8 the
    # scaled sums' 3 2^-24 a term (the instruction's own sums are the same)
    if kind == "dw":
        mag, n = dy.double().abs().t().contiguous() @ x.double().abs(), R
    elif kind == "fp8":
        a = x8.float().double().abs() * xs.double().repeat_interleave(128, 1)[:, :K]
        b = w8.float().double().abs() * ws8[0].double().repeat_interleave(128, 0)[:N].repeat_interleave(
            128, 1)[:, :K]
        mag, n = a @ b.t().contiguous(), K + 3
    else:
        parts = []
        for e in range(E):
            a = (x if kind == "product" else dy).double().abs()[e * (R // E):(e + 1) * (R // E)]
            b = w[e].double().abs()
            parts.append(a @ (b.t().contiguous() if kind == "product" else b))
        mag, n = torch.cat(parts), K if kind == "product" else N
    assert bool(((whole.double() - want.double()).abs() <= 2 * n * SUM * mag).all())
    for bad in (ws.view(torch.float32), ws[::2], ws.cpu()):
        with pytest.raises(ValueError):
            call(ws=bad)
    with pytest.raises(_lib.MoeError):
        call(ws=big[8:8 + size])


def _allocations():
    return torch.cuda.memory_stats()["allocation.all.allocated"]


def test_training_layer_allocates_nothing():
    """Also at sizes whose sums are cut, forward and backward."""
    T, E, k, H, I = 260, 1, 1, 2048, 128
    for gemm, N, K in ((_lib.MOE_GEMM_BF16, 2 * I, H), (_lib.MOE_GEMM_DX, H, I)):
        assert _lib.moe_grouped_gemm_workspace(gemm, T * k, N, K, E) > 0
    g = _gen(41)
    x, dout = _randn(g, T, H), _randn(g, T, H)
    w13, w2 = _randn(g, E, 2 * I, H), _randn(g, E, H, I)
    ids = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    w = torch.rand(T, k, generator=g, device=DEV)
    m = TrainExperts(H, E, k, I, T)
    before = _allocations()
    out = m.forward(x, ids, w, w13, w2)
    m.backward(dout)
    assert _allocations() == before
    # the products one by one, with workspaces of their own
    h = P.grouped_matmul(x, w13)
    y = P.grouped_matmul(P.swiglu(h, w.view(-1)), w2)
    assert torch.equal(out, y)
    da = P.grouped_matmul_dx(dout, w2)
    dh, dw = P.swiglu_grad(h, da, w.view(-1))
    assert torch.equal(m.dx, P.grouped_matmul_dx(dh, w13)) and torch.equal(m.dtopk_w.view(-1), dw)
    assert torch.equal(m.dw13, P.grouped_matmul_dw(dh, x))


def test_fp8_block_layer_allocates_nothing_and_is_the_same_by_handle():
    T, E, k, H, I = 260, 1, 1, 2048, 128
    assert _lib.moe_grouped_gemm_workspace(_lib.MOE_GEMM_FP8, T * k, 2 * I, H, E) > 0
    rng = np.random.default_rng(42)
    lay = synth.blob_layout(H, I, "fp8_block")
    ex = DeviceExperts(np.stack([synth._gauss_fp8_block_blob(rng, H, I, 0.05) for _ in range(2)]), lay)
    g = _gen(43)
    x, logits = _randn(g, T, H), _randn(g, T, E, dtype=torch.float32)
    layer = Fp8BlockLayer(H, E, k, I, T, shared=True)
    kw = dict(logits=logits, shared_table=ex.table[1:])
    before = _allocations()
    out = layer.forward(T, x, ex.table, **kw)
    assert _allocations() == before
    want = out.clone()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        layer.out.zero_()
        torch.cuda.synchronize()
        layer.forward(T, x, ex.table, stream=stream, **kw)
        torch.cuda.synchronize()
        assert torch.equal(layer.out, want)


def test_training_layer_checks_everything_before_the_first_launch():
    g = _gen(51)
    T, E, k, H, I = 6, 4, 2, 64, 32
    x, dout = _randn(g, T, H), _randn(g, T, H)
    w13, w2 = _randn(g, E, 2 * I, H), _randn(g, E, H, I)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV).to(torch.int32)
    w = torch.rand(T, k, generator=g, device=DEV)
    m = TrainExperts(H, E, k, I, T)
    buffers = [m.offsets, m.sorted_pair, m.h, m.a, m.y, m.out, m.da, m.dh, m.dx, m.dtopk_w, m.dw13, m.dw2]

    def untouched(call, error=ValueError):
        for b in buffers:
            b.fill_(77)
        with pytest.raises(error):
            call()
        assert all(bool((b == 77).all()) for b in buffers)

    off = torch.zeros(T * H + 4, device=DEV, dtype=torch.bfloat16)[4:].view(T, H)      # 8 bytes on
    good = dict(x=x, topk_ids=ids, topk_w=w, w13=w13, w2=w2)
    for name, t in (("x", x.float()), ("x", x.t().contiguous().t()), ("x", x[0]), ("x", off), ("x", x.cpu()),
                    ("x", torch.cat([x, x])), ("x", None), ("topk_ids", ids.long()), ("topk_ids", ids[:3]),
                    ("topk_w", w.double()), ("topk_w", w.t().contiguous().t()), ("w13", w13.float()),
                    ("w13", w13.cpu()), ("w13", w13.transpose(1, 2)), ("w13", w13[:, :I]),
                    ("w2", w2.half()), ("w2", w2.cpu()), ("w2", w2.transpose(1, 2).contiguous().transpose(1, 2)),
                    ("w2", None)):
        untouched(lambda: m.forward(**{**good, name: t}))
        untouched(lambda: m.backward(dout), RuntimeError)     # no forward to belong to
    # (an index or weights from any address)
    w_off = torch.zeros(T * k + 1, device=DEV)[1:].view(T, k).copy_(w)
    want = m.forward(**good).clone()
    assert torch.equal(m.forward(**{**good, "topk_w": w_off}), want)
    m.forward(**good)
    buffers = [m.da, m.dh, m.dx, m.dtopk_w, m.dw13, m.dw2]
    for t in (dout.float(), dout[:3], dout.t().contiguous().t(), off, dout.cpu(), None):
        untouched(lambda: m.backward(t))
    m.backward(dout)
    for H_, I_, E_ in ((60, 32, 4), (64, 36, 4), (64, 32, 513)):
        with pytest.raises(ValueError):
            TrainExperts(H_, E_, 2, I_, 4)


def test_fp8_block_layer_checks_everything_before_the_first_launch():
    T, E, k, H, I = 4, 4, 2, 64, 32
    rng, g = np.random.default_rng(61), _gen(61)
    lay = synth.blob_layout(H, I, "fp8_block")
    ex = DeviceExperts(np.stack([synth._gauss_fp8_block_blob(rng, H, I, 0.05) for _ in range(E)]), lay)
    x, logits = _randn(g, T, H), _randn(g, T, E, dtype=torch.float32)
    layer = Fp8BlockLayer(H, E, k, I, T)
    buffers = [layer.topk_ids, layer.topk_w, layer.offsets, layer.sorted_pair, layer.xq, layer.xs, layer.h,
               layer.aq, layer.y, layer.out]
    off = torch.zeros(T * H + 4, device=DEV, dtype=torch.bfloat16)[4:].view(T, H)      # 8 bytes on
    tab = ex.table
    good = dict(T=T, x=x, table=tab, logits=logits)
    for kw in (dict(shared_table=tab[:1]), dict(table=None), dict(table=0), dict(table=tab[:3]),
               dict(table=tab.to(torch.int32)), dict(table=tab.cpu()), dict(table=tab.t()), dict(x=off),
               dict(logits=None)):
        for b in buffers:
            b.fill_(77)
        with pytest.raises(ValueError):
            layer.forward(**{**good, **kw})
        if "logits" not in kw:
            with pytest.raises((ValueError, _lib.MoeError)):
                layer.ffn(T, kw.get("x", x), kw.get("table", tab), kw.get("shared_table"))
        assert all(bool((b == 77).all()) for b in buffers), kw
    assert layer.forward(0, x, None, logits=logits).shape == (0, H)
    with pytest.raises(ValueError):
        Fp8BlockLayer(H, 513, k, I, T)
    a = layer.forward(**good).clone()
    assert torch.equal(layer.forward(**{**good, "table": tab.data_ptr()}), a)


# --------------------------------------------- rows that are left, on each path --
#
# Whole numbers up to 3: products up to 9 and sums up to 9 * 4672 < 2^24 are exact in
# fp32 in any order, and the FP8 instruction drops nothing above 2^-13 of 9.

def _whole(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device=DEV)


def _e4m3(t):
    return t.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def _forward(kind, x, w, off, **kw):
    """The call of `kind` on whole numbers x (99 stands for NaN) and w."""
    if kind == "fp8":
        codes = torch.where(x == 99, torch.tensor(0x7F, dtype=torch.uint8, device=DEV), _e4m3(x.clamp(-3, 3)))
        E, N, K = w.shape
        return P.grouped_matmul_fp8(codes, torch.ones(x.shape[0], -(-K // 128), device=DEV), _e4m3(w),
                                    torch.ones(E, -(-N // 128), -(-K // 128), device=DEV), off, **kw)
    xb = torch.where(x == 99, torch.tensor(float("nan"), device=DEV), x.float()).to(torch.bfloat16)
    return (P.grouped_matmul if kind == "product" else P.grouped_matmul_dx)(xb, w.to(torch.bfloat16), off, **kw)


@pytest.mark.parametrize("kind", ["product", "dx", "fp8"])
@pytest.mark.parametrize("path", list(ROW_PATHS))
def test_rows_that_are_left_on_each_path(path, kind):
    """Rows before offsets[0] and behind offsets[E], rows whose index is outside x
    and rows whose place is outside the output are left as they are; the others
    are right, with NaN in every row of x that none of them reads."""
    R, E, N, K = ROW_PATHS[path]
    g = _gen(71 + len(path))
    gemm = {"product": _lib.MOE_GEMM_BF16, "dx": _lib.MOE_GEMM_DX, "fp8": _lib.MOE_GEMM_FP8}[kind]
    cut = _lib.moe_grouped_gemm_workspace(gemm, R, N, K, E) > 0
    assert cut == (path == "parts" and kind != "dx")     # (dx sums over N, which is short there)
    C, Q = (N, K) if kind == "dx" else (K, N)
    lo, hi, n, div = 5, R - R // 8, R // 2 + 1, 2
    # ascending offsets from lo to hi, some experts without rows
    inner = torch.sort(torch.randint(lo, hi + 1, (E - 1,), generator=g, device=DEV)).values
    if E > 3:
        inner[1] = inner[0]
    off = torch.cat([torch.tensor([lo], device=DEV), inner, torch.tensor([hi], device=DEV)]).to(torch.int32)
    pos = torch.arange(R, device=DEV)
    rows = torch.randint(0, n * div, (R,), generator=g, device=DEV)
    bad = pos % 17 == 7
    rows[bad] = torch.tensor([-1, n * div, -2 ** 31, 2 ** 31 - 1], device=DEV)[pos[bad] % 4]
    place = torch.randperm(R, generator=g, device=DEV)
    lost = pos % 23 == 11
    target = place.clone()
    target[lost] = torch.tensor([-1, R, 2 ** 31 - 1], device=DEV)[pos[lost] % 3]
    live = (pos >= lo) & (pos < hi) & ~bad & ~lost
    x, w = _whole(g, n, C), _whole(g, E, N, K)
    used = torch.zeros(n, dtype=torch.bool, device=DEV)
    used[(rows[live] // div)] = True
    x[~used] = 99
    out = torch.full((R, Q), 5.0, device=DEV)
    _forward(kind, x, w, off, rows=rows.to(torch.int32), div=div, out_rows=target.to(torch.int32), out=out)
    expert = torch.searchsorted(off[1:].contiguous().long(), pos, right=True).clamp(max=E - 1)
    wd = w.double()
    want = torch.full((R, Q), 5.0, dtype=torch.float64, device=DEV)
    for e in range(E):
        at = pos[live & (expert == e)]
        a = x[rows[at] // div].double()
        want[place[at]] = a @ (wd[e] if kind == "dx" else wd[e].t().contiguous())
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("kind", ["product", "fp8"])
@pytest.mark.parametrize("K", [64, 4672])
@pytest.mark.parametrize("where", ["first", "last", "spread"])
def test_streaming_kernel_with_all_rows_on_few_experts(kind, K, where):
    """16 rows per expert on average, the most that this kernel takes, on one
    expert of 512 or with a row on each of the others: an entry list near its
    capacity."""
    E, N = 512, 24
    counts = [0] * E
    if where == "spread":
        counts = [1] * E
        counts[300] = 16 * E - (E - 1)
    else:
        counts[0 if where == "first" else E - 1] = 16 * E
    g = _gen(81)
    x, w = _whole(g, 16 * E, K), _whole(g, E, N, K)
    out = torch.zeros(16 * E, N, device=DEV)
    _forward(kind, x, w, _offsets(counts), out=out)
    e = max(range(E), key=lambda i: counts[i])
    xd, lo = x.double(), sum(counts[:e])
    want = torch.zeros(16 * E, N, dtype=torch.float64, device=DEV)
    want[lo:lo + counts[e]] = xd[lo:lo + counts[e]] @ w[e].double().t().contiguous()
    at = 0
    for i in range(E):
        if i != e and counts[i]:
            want[at] = w[i].double() @ xd[at]
        at += counts[i]
    assert torch.equal(out.double(), want)


def test_activation_between_roundings_is_held_in_fp32():
    """The values that are not rounded to bf16 on the way out: the scale of a row
    with one gate (silu(g) u / 448) and the weight's gradient (da silu(g) u).

    In units of 2^-24: e^-|g| 3 (the exponential instruction's one unit in the last
    place, and one rounding), 1 + e^-|g| another 1, its reciprocal 1, their product
    1, times g 1; u and da are 1. The scale adds 1. The errors of e^-|g| in the
    numerator and in 1 + e^-|g| have opposite signs and count once: 7, 8."""
    unit = 2.0 ** -24
    gate = torch.cat([torch.arange(-70 * 32, 70 * 32 + 1) / 32, torch.randn(4000) * 3]).to(torch.bfloat16)
    gate = gate[gate != 0].to(DEV)
    h = torch.zeros(len(gate), 16, device=DEV, dtype=torch.bfloat16)
    h[:, 3], h[:, 8 + 3] = gate, 1
    g = gate.double()
    ref = g * torch.sigmoid(g)
    _, s = P.swiglu_quant_fp8(h)
    # (against 2^-100 / 448, the smallest scale)
    want = (ref.abs() / 448).clamp(min=2.0 ** -100 / 448)
    err = ((s[:, 0].double() - want).abs() / want / unit)
    assert float(err.max()) <= 8, f"scale: {float(err.max()):.3g} units"
    _, dw = P.swiglu_grad(h, torch.ones(len(gate), 8, device=DEV, dtype=torch.bfloat16),
                          torch.ones(len(gate), device=DEV))
    err = ((dw.double() - ref).abs() / ref.abs() / unit)
    assert float(err.max()) <= 7, f"dw: {float(err.max()):.3g} units"


def test_activation_of_the_largest_gates():
    """Finite gates of any size: silu(g) u and its gradients without NaN, the
    derivative 1 and 0 far out; NaN stays in its element's outputs."""
    top = torch.finfo(torch.bfloat16).max
    gate = torch.tensor([-top, -1e30, -1e4, -129, -128, -100, -88, 88, 100, 128, 129, 1e4, 1e30, top], device=DEV)
    h = torch.ones(1, 2 * 16, device=DEV, dtype=torch.bfloat16)
    h[0, :14] = gate.to(torch.bfloat16)
    a = P.swiglu(h)[0, :14]
    assert bool((a[:7].abs() <= 1e-36).all()) and torch.equal(a[7:], h[0, 7:14])
    da = torch.ones(1, 16, device=DEV, dtype=torch.bfloat16)
    dh, _ = P.swiglu_grad(h, da)
    assert bool((dh[0, :7].abs() <= 1e-36).all()) and bool((dh[0, 7:14] == 1).all())
    assert torch.equal(dh[0, 16:30], a)
    h[0, 3] = float("nan")
    a, (dh, _) = P.swiglu(h), P.swiglu_grad(h, da)
    assert a.isnan().sum() == 1 and bool(a[0, 3].isnan())
    assert dh.isnan().sum() == 2 and bool(dh[0, 3].isnan()) and bool(dh[0, 19].isnan())
