"""Runs of the norm, the moves and the MXFP4 product as they are used together: a
layer served from MXFP4 experts with MXFP4 rows (resident, and through the expert
cache), both coded layers with the norm in front, and the experts of a training step
with their rows in sorted order.

The served layer is checked stage by stage on what the stage before it left, with each
operator's own bounds (the codes' rounding is too coarse for a bound on the whole)."""
import numpy as np
import pytest
import torch

from mixture_experts_gate_amd import _lib, layer as LY, products as P, rows as W, synth

from test_gpu_mxfp4 import _bound, _encode, _gen, _randn, _ref, _within, between, decode
from test_gpu_rows import _near, _norm_ref

pytestmark = pytest.mark.gpu
DEV, BF16 = "cuda", 2.0 ** -8


def _blobs(seed, n, H, I):
    rng = np.random.default_rng(seed)
    return np.stack([synth._gauss_mxfp4_blob(rng, H, I, 0.05) for _ in range(n)])


def _matrices(blobs, H, I):
    """([n, 2I, H], [n, H, I]) in float64."""
    lay, host = synth.blob_layout(H, I, "mxfp4"), torch.from_numpy(blobs)
    out = []
    for r, c, oc, os_ in ((2 * I, H, lay.w13, lay.s13), (H, I, lay.w2, lay.s2)):
        out.append(decode(host[:, oc:oc + r * c // 2].reshape(-1, r, c // 2), host[:, os_:os_ + r * c // 32].reshape(-1, r, c // 32)))
    return out


def _check_stages(layer, T, x, w13, w2, shared, out):
    """Every stage of the last forward of T tokens with input rows x (bf16)."""
    k, E, n = layer.k, layer.E, T * layer.k
    ids = layer.topk_ids[:T].long().reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E).tolist()
    pair = layer.sorted_pair[:n].long()
    assert torch.equal(pair, order)
    xd = decode(layer.xq[:T], layer.xs[:T])
    ref, mag = _ref(xd, w13, counts, pair // k)
    _within(layer.h[:n], ref, _bound(ref, mag, layer.H, torch.bfloat16), "h")
    g, u = layer.h[:n].double().chunk(2, 1)
    between(layer.aq[:n], layer.a_s[:n], g * torch.sigmoid(g) * u)
    ad = decode(layer.aq[:n], layer.a_s[:n])
    ref, mag = _ref(ad, w2, counts, torch.arange(n, device=DEV))
    _within(layer.y[:n][pair], ref, _bound(ref, mag, layer.I, torch.bfloat16), "y")
    terms = layer.y[:n].double().view(T, k, -1) * layer.topk_w[:T].double()[:, :, None]
    ref, mag = terms.sum(1), terms.abs().sum(1)
    if shared is not None:
        s13, s2 = shared
        r13, m13 = _ref(xd, s13, [T], torch.arange(T, device=DEV))
        _within(layer.h_sh[:T], r13, _bound(r13, m13, layer.H, torch.bfloat16), "h_sh")
        g, u = layer.h_sh[:T].double().chunk(2, 1)
        between(layer.aq_sh[:T], layer.as_sh[:T], g * torch.sigmoid(g) * u)
        r2, m2 = _ref(decode(layer.aq_sh[:T], layer.as_sh[:T]), s2, [T], torch.arange(T, device=DEV))
        _within(layer.y_sh[:T], r2, _bound(r2, m2, layer.I, torch.bfloat16), "y_sh")
        ref, mag = ref + layer.y_sh[:T].double(), mag + layer.y_sh[:T].double().abs()
    b = (k + 1) * 2.0 ** -23 * mag
    _within(out, ref, b + (ref.abs() + b) * BF16, "out")


@pytest.mark.parametrize("norm", ["none", "norm", "residual"])
@pytest.mark.parametrize("T,E,k,H,I,shared", [(1, 8, 2, 256, 128, False), (5, 8, 2, 128, 384, True),
                                              (33, 16, 4, 256, 256, True), (200, 4, 2, 384, 128, False),
                                              (1500, 8, 3, 768, 1024, True)])
def test_mxfp4_layer(T, E, k, H, I, shared, norm):
    blobs, sh = _blobs(T, E, H, I), _blobs(1000 + T, 1, H, I)
    lay = synth.blob_layout(H, I, "mxfp4")
    ex, exs = LY.DeviceExperts(blobs, lay), LY.DeviceExperts(sh, lay)
    g = _gen(T)
    x, wg = _randn(g, T + 2, H), _randn(g, E, H)
    layer = LY.Mxfp4Layer(H, E, k, I, T + 3, shared=shared, norm=True)
    kw, rows = {}, x[:T]
    if norm != "none":
        w, r = _randn(g, H), _randn(g, T, H) if norm == "residual" else None
        kw = {"norm_w": w, "residual": r}
        y = W.rms_norm(x[:T].contiguous(), w, 1e-6, r)
        if r is not None:
            rows, t = y
        else:
            rows = y
    out = layer.forward(T, x, ex.table, wg=wg, shared_table=exs.table if shared else None, **kw)
    if norm == "none":
        q, s = _encode(rows)
    else:
        q, s = W.rms_norm_mxfp4(x[:T].contiguous(), w, 1e-6, r)[:2]
        assert torch.equal(layer.xn[:T], rows)
        assert r is None or torch.equal(layer.total[:T], t)
    assert torch.equal(layer.xq[:T], q) and torch.equal(layer.xs[:T], s)
    ids = torch.topk(layer.logits[:T], k, dim=1).indices            # (the router reads the normed rows)
    assert torch.equal(ids.to(torch.int32).sort(1).values, layer.topk_ids[:T].sort(1).values)
    ref = rows.double() @ wg.double().t().contiguous()
    mag = rows.double().abs() @ wg.double().abs().t().contiguous()
    _within(layer.logits[:T], ref, (H / 64 + 14) * 2.0 ** -24 * mag, "logits")
    w13, w2 = _matrices(blobs, H, I)
    _check_stages(layer, T, rows, w13, w2, _matrices(sh, H, I) if shared else None, out)
    # another call leaves no trace of this one
    again = layer.forward(T, x, ex.table, wg=wg, shared_table=exs.table if shared else None, **kw).clone()
    layer.forward(min(T, 3), x, ex.table, wg=wg)
    assert torch.equal(layer.forward(T, x, ex.table, wg=wg, shared_table=exs.table if shared else None, **kw), again)


def test_mxfp4_layer_through_the_expert_cache():
    """Experts in the kernel layout streamed through the cache give the resident bits."""
    T, E, k, H, I = 9, 8, 2, 256, 128
    blobs = _blobs(7, E, H, I)
    lay = synth.blob_layout(H, I, "mxfp4")
    ex = LY.DeviceExperts(blobs, lay)
    store = LY.HostExperts([blobs], lay)
    cache = LY.ExpertCache(store, 1, E, (E + 1) * ((lay.nbytes + 255) // 256 * 256))
    g = _gen(3)
    x, logits = _randn(g, T, H), torch.randn(T, E, device=DEV, generator=g)
    layer = LY.Mxfp4Layer(H, E, k, I, T)
    want = layer.forward(T, x, ex.table, logits=logits).clone()
    table = cache.prefetch(0, None, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(layer.forward(T, x, table, logits=logits), want)
    torch.cuda.synchronize()
    cache.close()


def test_fp8_layer_with_the_norm():
    """The norm's codes are what the experts read, its bf16 rows what the router reads."""
    T, E, k, H, I = 17, 8, 2, 256, 128
    rng = np.random.default_rng(5)
    blobs = np.stack([synth._gauss_fp8_block_blob(rng, H, I, 0.05) for _ in range(E)])
    ex = LY.DeviceExperts(blobs, synth.blob_layout(H, I, "fp8_block"))
    g = _gen(6)
    x, r, w, wg = _randn(g, T, H), _randn(g, T, H), _randn(g, H), _randn(g, E, H)
    layer, plain = LY.Fp8BlockLayer(H, E, k, I, T, norm=True), LY.Fp8BlockLayer(H, E, k, I, T)
    out = layer.forward(T, x, ex.table, wg=wg, norm_w=w, residual=r).clone()
    y, t = W.rms_norm(x, w, 1e-6, r)
    q, s, _ = W.rms_norm_fp8(x, w, 1e-6, r)
    assert torch.equal(layer.total, t) and torch.equal(layer.xn, y)
    assert torch.equal(layer.xq, q.view(torch.uint8)) and torch.equal(layer.xs, s)
    # the layer without a norm, its rows replaced by the norm's codes
    plain.forward(T, y, ex.table, wg=wg)
    assert torch.equal(plain.topk_ids, layer.topk_ids)
    plain.xq.copy_(layer.xq), plain.xs.copy_(layer.xs)
    ys, _ = plain._experts(T, ex.table, None, None)
    _lib.moe_combine(ys, False, plain.topk_w, None, T, k, H, plain.out)
    assert torch.equal(plain.out, out)


def test_coded_layers_refuse_before_the_first_launch():
    H, E, k, I, T = 256, 4, 2, 128, 3
    ex = LY.DeviceExperts(_blobs(1, E, H, I), synth.blob_layout(H, I, "mxfp4"))
    g = _gen(1)
    x, w, lg = _randn(g, T, H), _randn(g, H), torch.randn(T, E, device=DEV, generator=g)
    layer = LY.Mxfp4Layer(H, E, k, I, T, norm=True)
    for b in (layer.out, layer.xq, layer.xn, layer.topk_ids):
        b.fill_(7)
    bad = [dict(residual=x), dict(norm_w=w[:128].contiguous()), dict(norm_w=w.float()), dict(norm_w=w.cpu()),
           dict(norm_w=w, residual=x[:2]), dict(norm_w=w, residual=x.float()), dict(norm_w=w, eps=-1.0),
           dict(norm_w=w, eps=float("nan")), dict(norm_w=w.clone().requires_grad_()), dict(shared_table=ex.table)]
    for kw in bad:
        with pytest.raises(ValueError):
            layer.forward(T, x, ex.table, logits=lg, **kw)
            pytest.fail(str(kw))
    with pytest.raises(ValueError):
        LY.Mxfp4Layer(H, E, k, I, T).forward(T, x, ex.table, logits=lg, norm_w=w)
    for args in ((192, E, k, I, T), (H, E, k, 96, T), (H, 513, k, I, T)):
        with pytest.raises(ValueError):
            LY.Mxfp4Layer(*args)
    torch.cuda.synchronize()
    for b in (layer.out, layer.xq, layer.xn, layer.topk_ids):
        assert bool((b == 7).all())


def test_mxfp4_layer_in_a_graph_allocates_nothing():
    T, E, k, H, I = 65, 8, 2, 256, 384
    ex = LY.DeviceExperts(_blobs(2, E, H, I), synth.blob_layout(H, I, "mxfp4"))
    g = _gen(2)
    x, r, w, wg = _randn(g, T, H), _randn(g, T, H), _randn(g, H), _randn(g, E, H)
    layer = LY.Mxfp4Layer(H, E, k, I, T, norm=True)
    call = lambda: layer.forward(T, x, ex.table, wg=wg, norm_w=w, residual=r)      # noqa: E731
    call()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    call()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(3):
        x.copy_(_randn(_gen(20 + seed), T, H))
        graph.replay()
        got, t = layer.out.clone(), layer.total.clone()
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(t, layer.total)


# A training step of a block, its rows in sorted order: norm, gate, dispatch, experts,
# combine with the router's weights and the residual. Each bf16 rounding is within 2^-8
# of its value; forward (t, y, x rows, h, a, expert rows, out) makes 7 of them and a
# gradient's path (the forward values it uses and dout's way back: dy, da, dh, dx rows,
# their sum, dx) 7 + 6, each of them independent from value to value: the relative L2
# error stays below 13 2^-8 = 0.051 even if all of them were half a step off and added up.
STEP_L2 = 13 * 2.0 ** -8


@pytest.mark.parametrize("T,E,k,H,I", [(24, 4, 2, 128, 64), (150, 8, 3, 256, 96)])
def test_training_step_of_a_block(T, E, k, H, I):
    g = _gen(T)
    x, r = _randn(g, T, H), _randn(g, T, H)
    w = (1 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(torch.bfloat16)
    wg = (torch.randn(E, H, device=DEV, generator=g) * H ** -0.5).to(torch.bfloat16)
    w13 = (torch.randn(E, 2 * I, H, device=DEV, generator=g) * H ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(E, H, I, device=DEV, generator=g) * I ** -0.5).to(torch.bfloat16)
    dout = _randn(g, T, H)
    n = T * k
    i32 = torch.int32

    # forward
    y, t = W.rms_norm(x, w, 1e-6, r)
    topk_ids, topk_w = torch.empty(T, k, device=DEV, dtype=i32), torch.empty(T, k, device=DEV)
    logits = torch.empty(T, E, device=DEV)
    _lib.moe_route(y, wg, None, logits, T, H, E, k, True, topk_ids, topk_w)
    off, pair, row = torch.empty(E + 1, device=DEV, dtype=i32), torch.empty(n, device=DEV, dtype=i32), torch.empty(n, device=DEV, dtype=i32)
    nws = max(_lib.moe_workspace_size(T, k, H, I, E)[0], 256)
    _lib.moe_permute(topk_ids, T, k, E, off, pair, row, torch.empty(nws, device=DEV, dtype=torch.uint8), nws)
    at = row.view(T, k)
    xr = W.dispatch(y, at)
    h = P.grouped_matmul(xr, w13, off)
    a = P.swiglu(h)
    e = P.grouped_matmul(a, w2, off)
    out = W.combine(e, at, topk_w, t)
    # backward
    de, dtopk = W.combine_grad(dout, e, at, topk_w)
    da = P.grouped_matmul_dx(de, w2, off)
    dw2 = P.grouped_matmul_dw(de, a, off)
    dh, _ = P.swiglu_grad(h, da)
    dxr = P.grouped_matmul_dx(dh, w13, off)
    dw13 = P.grouped_matmul_dw(dh, xr, off)
    dy = W.combine(dxr, at)
    dt, dw = W.rms_norm_grad(t, w, dy, 1e-6, dout)

    # the same in 64 bits, by autograd (the router's choice as it was made, its weights
    # as inputs)
    d = lambda v: v.double().requires_grad_()                                     # noqa: E731
    X, Rr, Wn, W13, W2, TW = d(x), d(r), d(w), d(w13), d(w2), d(topk_w)
    tt = X + Rr
    yy = tt / torch.sqrt((tt * tt).mean(1, keepdim=True) + 1e-6) * Wn
    res = tt
    for j in range(k):
        for ee in range(E):
            m = (topk_ids[:, j] == ee).nonzero().reshape(-1)
            if m.numel():
                gg, uu = (yy[m] @ W13[ee].t()).chunk(2, 1)
                res = res.index_add(0, m, TW[m, j:j + 1] * ((gg * torch.sigmoid(gg) * uu) @ W2[ee].t()))
    res.backward(dout.double())
    for name, got, ref in (("out", out, res), ("dx", dt, X.grad), ("dresidual", dt, Rr.grad), ("dweight", dw, Wn.grad),
                           ("dw13", dw13, W13.grad), ("dw2", dw2, W2.grad), ("dtopk", dtopk, TW.grad)):
        err = float((got.double() - ref.detach()).norm() / ref.detach().norm())
        assert err <= STEP_L2, (name, err)
