"""Runs of the expert products as they are used together: a layer served from
block-scaled FP8 experts (resident, and through the expert cache), and the
experts' forward and backward in training."""
import numpy as np
import pytest
import torch

from mixture_experts_gate_amd import _lib, layer as LY, products as P, synth
from mixture_experts_gate_amd.train import TrainExperts

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _blobs(seed, n, H, I):
    rng = np.random.default_rng(seed)
    return np.stack([synth._gauss_fp8_block_blob(rng, H, I, 0.05) for _ in range(n)])


def _matrices(blob, H, I):
    """(W13, W2) of one blob in float64."""
    lay = synth.blob_layout(H, I, "fp8_block")
    out = []
    for rows, cols, oc, os_ in ((2 * I, H, lay.w13, lay.s13), (H, I, lay.w2, lay.s2)):
        q = torch.from_numpy(blob[oc:oc + rows * cols].copy()).view(torch.float8_e4m3fn).double()
        nr, nk = -(-rows // 128), -(-cols // 128)
        s = torch.from_numpy(blob[os_:os_ + 4 * nr * nk].copy().view(np.float32)).double()
        s = s.view(nr, nk).repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
        out.append(q.view(rows, cols) * s)
    return out


def _expert(x, w13, w2):
    g, u = (x @ w13.t()).chunk(2, 1)
    return (g * torch.sigmoid(g) * u) @ w2.t()


def _layer_ref(x, blobs, ids, w, H, I, shared=None):
    mats = [_matrices(b, H, I) for b in blobs]
    out = torch.zeros(x.shape[0], H, dtype=torch.float64)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t].tolist()):
            out[t] += float(w[t, j]) * _expert(x[t:t + 1], *mats[e])[0]
    if shared is not None:
        out += _expert(x, *_matrices(shared, H, I))
    return out


# A token's FP8 rounding is at most 2^-4 of each value (and independent from
# value to value), twice (x, then the activation); the sums over K of such errors
# grow as its root while the sums themselves do too, so the relative L2 error of
# the output stays below sqrt(2) 2^-4 = 0.088 (the rounding's rms is about half of its bound).
FP8_L2 = 0.088


def _l2(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


@pytest.mark.parametrize("T,E,k,H,I,shared", [(1, 8, 2, 256, 128, False), (5, 8, 2, 160, 96, True),
                                              (33, 16, 4, 256, 320, True), (200, 4, 2, 384, 128, False)])
def test_fp8_block_layer(T, E, k, H, I, shared):
    blobs, sh = _blobs(T, E, H, I), _blobs(1000 + T, 1, H, I)
    lay = synth.blob_layout(H, I, "fp8_block")
    ex, exs = LY.DeviceExperts(blobs, lay), LY.DeviceExperts(sh, lay)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g)
    layer = LY.Fp8BlockLayer(H, E, k, I, T + 3, shared=shared)
    out = layer.forward(T, x.to(DEV), ex.table, logits=logits.to(DEV),
                        shared_table=exs.table if shared else None)
    ids, w = layer.topk_ids[:T].cpu(), layer.topk_w[:T].cpu()
    ref = _layer_ref(x.double(), blobs, ids, w, H, I, sh[0] if shared else None)
    assert _l2(out, ref) <= FP8_L2
    # the same from the rows as the layer quantised them: only its activation's
    # rounding and bf16 are left
    xq = layer.xq[:T].cpu().view(torch.float8_e4m3fn).double()
    xq = xq * layer.xs[:T].cpu().double().repeat_interleave(128, 1)[:, :H]
    ref = _layer_ref(xq, blobs, ids, w, H, I, None)
    if not shared:
        assert _l2(out, ref) <= 2.0 ** -4


def test_fp8_block_layer_through_the_cache():
    """Experts streamed through the cache give the resident experts' bits."""
    H, I, E, k, T, layers = 256, 128, 8, 2, 24, 3
    lay = synth.blob_layout(H, I, "fp8_block")
    blobs = [_blobs(50 + l, E, H, I) for l in range(layers)]
    resident = [LY.DeviceExperts(b, lay) for b in blobs]
    store = LY.HostExperts(blobs, lay)
    slot = (lay.nbytes + 255) // 256 * 256
    cache = LY.ExpertCache(store, layers, E, slot * (E + 4))
    layer = LY.Fp8BlockLayer(H, E, k, I, T)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    for rep in range(2):
        for l in range(layers):
            logits = torch.randn(T, E, generator=g).to(DEV)
            want = layer.forward(T, x, resident[l].table, logits=logits).clone()
            tab = cache.prefetch(l, None)
            got = layer.forward(T, x, tab, logits=logits)
            assert torch.equal(got, want), (rep, l)
    cache.close()


def _train_ref(x, ids, w, w13, w2, dout):
    """Outputs and gradients in float64 by autograd."""
    x, w, w13, w2 = (t.double().cpu().requires_grad_(True) for t in (x, w, w13, w2))
    out = []
    for t in range(x.shape[0]):
        acc = 0
        for j, e in enumerate(ids[t].tolist()):
            acc = acc + w[t, j] * _expert(x[t:t + 1], w13[e], w2[e])
        out.append(acc)
    out = torch.cat(out)
    out.backward(dout.double().cpu())
    return out.detach(), x.grad, w.grad, w13.grad, w2.grad


# bf16 roundings on the way, each at most 2^-8 of what it rounds: h, a, y, out
# forward; h, a, da, dh, the pairs' dx and dx backward. Their relative L2 errors
# add up to at most 6 2^-8 where the products between keep relative sizes
# (random matrices do), and 2^-8 is twice the mean.
TRAIN_L2 = 6 * 2.0 ** -8


def _train_case(T, E, k, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    w13 = (torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(E, H, I, generator=g) * I ** -0.5).to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    dout = torch.randn(T, H, generator=g).to(torch.bfloat16)
    return [t.to(DEV) for t in (x, ids, w, w13, w2, dout)]


@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 64, 32), (7, 8, 2, 72, 40), (65, 6, 3, 128, 96),
                                       (150, 2, 1, 96, 64)])
def test_training_gradients(T, E, k, H, I):
    x, ids, w, w13, w2, dout = _train_case(T, E, k, H, I, 7 * T + E)
    m = TrainExperts(H, E, k, I, T + 2)
    out = m.forward(x, ids, w, w13, w2).clone()
    got = (out, *m.backward(dout))
    for name, a, r in zip(("out", "dx", "dtopk_w", "dw13", "dw2"), got,
                          _train_ref(x, ids.cpu(), w, w13, w2, dout)):
        err = float((a.double().cpu() - r).norm() / r.norm())
        assert err <= TRAIN_L2, f"{name}: {err:.3g}"
    # gradients of a second batch are added
    first = [t.clone() for t in got[3:]]
    m.forward(x, ids, w, w13, w2)
    m.backward(dout, accumulate=True)
    for a, b in zip(first, (m.dw13, m.dw2)):
        assert torch.allclose(b, 2 * a, rtol=2.0 ** -20, atol=1e-6)


def test_training_gradients_against_differences():
    """<dout, out> moves with a matrix as the matrix's gradient says, to first
    order."""
    x, ids, w, w13, w2, dout = _train_case(40, 4, 2, 128, 64, 5)
    m = TrainExperts(128, 4, 2, 64, 40)
    base = m.forward(x, ids, w, w13, w2).double()
    _, _, dw13, dw2 = m.backward(dout)
    for mat, grad in ((w13, dw13.clone()), (w2, dw2.clone())):
        # a step large against bf16's of the weights, small against the curvature
        step = (0.05 * float(mat.float().norm()) / float(grad.norm())) * grad
        moved = (mat.float() + step).to(torch.bfloat16)
        new = m.forward(x, ids, w, moved if mat is w13 else w13, moved if mat is w2 else w2).double()
        gain = float(((new - base) * dout.double()).sum())
        expect = float((grad.double() * (moved.double() - mat.double())).sum())
        # second order: 0.05 of the first; roundings of out: 2^-8 |out| |dout| in
        # the worst, its root of the number of values on average
        slack = 0.15 * abs(expect) + 2.0 ** -8 * float(base.norm()) * 3
        assert abs(gain - expect) <= slack, (gain, expect)


def test_training_step_in_a_graph():
    """Captured and replayed with new inputs: the eager step's bits."""
    x, ids, w, w13, w2, dout = _train_case(50, 4, 2, 128, 64, 9)
    eager, cap = TrainExperts(128, 4, 2, 64, 50), TrainExperts(128, 4, 2, 64, 50)
    cap.forward(x, ids, w, w13, w2), cap.backward(dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap.forward(x, ids, w, w13, w2)
        cap.backward(dout)
    for k in range(4):
        nx, nids, nw, _, _, nd = _train_case(50, 4, 2, 128, 64, 100 + k)
        x.copy_(nx), ids.copy_(nids), w.copy_(nw), dout.copy_(nd)
        graph.replay()
        torch.cuda.synchronize()
        eager.forward(x, ids, w, w13, w2)
        eager.backward(dout)
        torch.cuda.synchronize()
        for a, b in ((eager.out, cap.out), (eager.dx, cap.dx), (eager.dtopk_w, cap.dtopk_w),
                     (eager.dw13, cap.dw13), (eager.dw2, cap.dw2)):
            assert torch.equal(a, b), k


def test_fp8_block_layer_refuses_its_inputs():
    """Tokens, logits and gate matrices of other shapes or types, before the
    router reads them."""
    layer = LY.Fp8BlockLayer(64, 4, 2, 64, 4)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    logits = torch.zeros(4, 4, device=DEV)
    wg = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(x=x[:3], logits=logits), dict(x=x[:, :32], logits=logits),
               dict(x=x.float(), logits=logits), dict(x=x, logits=logits[:2]),
               dict(x=x, logits=logits.double()), dict(x=x, logits=logits.cpu()),
               dict(x=x, wg=wg[:3]), dict(x=x, wg=wg.t())):
        with pytest.raises(ValueError):
            layer.forward(4, table=None, **kw)


def test_refusals():
    x, ids, w, w13, w2, dout = _train_case(4, 4, 2, 64, 32, 1)
    m = TrainExperts(64, 4, 2, 32, 4)
    with pytest.raises(RuntimeError):
        m.backward(dout)
    for bad in (lambda: m.forward(torch.cat([x, x]), ids, w, w13, w2),
                lambda: m.forward(x, ids.long(), w, w13, w2),
                lambda: m.forward(x, ids, w[:2], w13, w2),
                lambda: m.forward(x, ids, w, w2, w13)):
        with pytest.raises(ValueError):
            bad()
    m.forward(x, ids, w, w13, w2)
    with pytest.raises(ValueError):
        m.backward(dout[:2])
    with pytest.raises(ValueError):
        LY.Fp8BlockLayer(40, 4, 2, 64, 4)
    layer = LY.Fp8BlockLayer(64, 4, 2, 64, 4)
    with pytest.raises(ValueError):
        layer.forward(5, x, None)
    _, _ = P, _lib
