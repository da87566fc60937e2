"""Host-side checks of the norm, the moves and the MXFP4 calls: bad arguments are
refused before anything touches a device."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_gate_amd import _lib
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_gate_amd import build
        build.build()
    return _lib


D = 0x1000          # never dereferenced: validation fails first


def test_mxfp4_calls_reject_bad_arguments(lib):
    L, bad = lib.load(), lib.MOE_EINVAL
    for fn in (L.moe_quant_mxfp4, L.moe_swiglu_quant_mxfp4):
        for args in ((D, None, 4, 40, D, D), (None, None, 4, 64, D, D), (D, None, 4, 64, None, D), (D, None, 4, 64, D, None),
                     (D, None, 4, 64, D + 8, D), (D + 2, None, 4, 64, D, D), (D, None, -1, 64, D, D),
                     (D, None, 2 ** 31 - 1, 64, D, D), (D, None, 4, 0, D, D), (D, None, 4, (1 << 24) + 32, D, D)):
            assert fn(*args, None) == bad, args
        assert fn(None, None, 0, 64, None, None, None) == lib.MOE_OK
    for args in ((D, 2, 24, 128, D, D), (D, 2, 16, 64, D, D), (D, -1, 16, 128, D, D), (None, 2, 16, 128, D, D),
                 (D, 2, 16, 128, D + 4, D), (D, 2, 16, 128, D, None), (D, 2, 1 << 21, 128, D, D)):
        assert L.moe_quant_mxfp4_matrices(*args, None) == bad, args
    assert L.moe_quant_mxfp4_matrices(None, 0, 16, 128, None, None, None) == lib.MOE_OK

    def gemm(x=D, xs=D, rows=None, div=1, n=8, off=D, w=D, ws=D, tab=None, mat=0, R=8, N=16, K=128, E=2, y=D,
             y_rows=None, y_n=8, space=None):
        return L.moe_grouped_gemm_mxfp4(x, xs, rows, div, n, off, w, ws, tab, mat, R, N, K, E, y, y_rows, y_n, 0,
                                        space, 0, None)

    for kw in (dict(x=None), dict(x=D + 8), dict(xs=None), dict(xs=D + 2), dict(w=None), dict(ws=None), dict(tab=D),
               dict(w=D + 8), dict(ws=D + 8), dict(N=24), dict(N=8), dict(K=64), dict(K=192), dict(R=-1), dict(R=2 ** 31 - 1),
               dict(E=0), dict(E=513), dict(off=None), dict(mat=2), dict(y=None), dict(y=D + 8), dict(n=7),
               dict(rows=D, n=0), dict(rows=D, div=0), dict(y_n=7), dict(y_rows=D, y_n=0), dict(space=D + 4),
               dict(N=1 << 20, K=1 << 20, E=4)):
        assert gemm(**kw) == bad, kw
    assert gemm(R=0, x=None, y=None) == lib.MOE_OK


def test_mxfp4_workspace(lib):
    from mixture_experts_gate_amd import products as P
    import random
    ws = lambda *a: lib.moe_grouped_gemm_workspace(lib.MOE_GEMM_MXFP4, *a)      # noqa: E731
    assert ws(40, 256, 4096, 1) >= 2 * 40 * 256 * 4          # one tile over 32 slabs
    assert ws(16, 256, 4096, 1) == 0                         # the streaming kernel
    assert ws(65536, 1536, 2048, 128) == 0 and ws(0, 16, 128, 1) == 0
    rng, cut = random.Random(6), 0
    for _ in range(4000):
        R, E = int(2 ** rng.uniform(0, 15)), rng.choice((1, 1, 2, 8, 64, 300))
        N, K = 16 * int(2 ** rng.uniform(0, 9)), 128 * int(2 ** rng.uniform(0, 6))
        size = ws(R, N, K, E)
        assert size <= P.workspace_bound(R, N, K, E, "cpu"), (R, N, K, E)
        cut += size > 0
    assert cut > 100
    for args in ((8, 24, 128, 1), (8, 16, 64, 1), (-1, 16, 128, 1), (8, 16, 128, 513)):
        with pytest.raises(lib.MoeError):
            ws(*args)


def test_norm_rejects_bad_arguments(lib):
    L, bad = lib.load(), lib.MOE_EINVAL

    def norm(x=D, res=None, w=D, eps=1e-6, R=4, H=64, total=None, y=D, quant=0, q=None, s=None):
        return L.moe_rms_norm(x, res, w, eps, R, H, total, y, quant, q, s, None)

    for kw in (dict(x=None), dict(x=D + 8), dict(w=None), dict(w=D + 2), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(R=-1), dict(R=2 ** 31 - 1), dict(H=60), dict(H=0), dict(H=1 << 25), dict(total=D),
               dict(res=D + 4), dict(res=D, total=D + 4), dict(y=None), dict(y=D + 8), dict(quant=3), dict(quant=-1),
               dict(quant=1), dict(quant=1, q=D), dict(quant=1, q=D + 8, s=D), dict(quant=1, q=D, s=D + 2),
               dict(quant=2, q=D, s=D, H=72), dict(quant=2, q=D), dict(quant=2, s=D)):
        assert norm(**kw) == bad, kw
    assert norm(R=0, x=None, w=None, y=None) == lib.MOE_OK

    def grad(x=D, w=D, dy=D, dt=None, eps=1e-6, R=4, H=64, dx=D, dw=D, acc=0, ws=D, n=1 << 30):
        return L.moe_rms_norm_grad(x, w, dy, dt, eps, R, H, dx, dw, acc, ws, n, None)

    for kw in (dict(x=None), dict(w=None), dict(dy=None), dict(dx=None), dict(dx=D + 2), dict(dt=D + 8), dict(dw=D + 4),
               dict(ws=None), dict(ws=D + 8), dict(n=4 * 64 * 4 - 1), dict(H=16392), dict(H=60), dict(eps=-1.0), dict(R=-1)):
        assert grad(**kw) == bad, kw
    assert lib.moe_rms_norm_grad_workspace(4, 64) == 4 * 64 * 4
    assert lib.moe_rms_norm_grad_workspace(0, 64) == 0
    for args in ((4, 60), (-1, 64), (4, 16392)):
        with pytest.raises(lib.MoeError):
            lib.moe_rms_norm_grad_workspace(*args)


def test_moves_reject_bad_arguments(lib):
    L, bad, ok = lib.load(), lib.MOE_EINVAL, lib.MOE_OK

    def dispatch(x=D, rows=D, T=4, k=2, H=64, out=D, n=8):
        return L.moe_dispatch(x, rows, T, k, H, out, n, None)

    for kw in (dict(x=None), dict(x=D + 8), dict(rows=None), dict(out=None), dict(out=D + 2), dict(T=-1), dict(k=0),
               dict(H=60), dict(n=-1), dict(T=2 ** 30, k=2), dict(H=0)):
        assert dispatch(**kw) == bad, kw
    assert dispatch(T=0, x=None, out=None) == ok
    assert dispatch(out=None, n=0) == ok             # (nothing to write)

    def combine(y=D, f32=0, n=8, rows=D, w=D, add=None, T=4, k=2, H=64, out=D):
        return L.moe_combine_rows(y, f32, n, rows, w, add, T, k, H, out, None)

    for kw in (dict(y=None), dict(y=D + 8), dict(rows=None), dict(add=D + 8), dict(out=None), dict(T=-1), dict(k=0),
               dict(H=60), dict(n=-1), dict(T=2 ** 30, k=2)):
        assert combine(**kw) == bad, kw
    assert combine(T=0, y=None, out=None) == ok
    assert combine(y=None, n=0, out=None) == bad

    def grad(dout=D, y=D, n=8, rows=D, w=D, T=4, k=2, H=64, dy=D, dw=D):
        return L.moe_combine_rows_grad(dout, y, n, rows, w, T, k, H, dy, dw, None)

    for kw in (dict(dout=None), dict(y=None), dict(rows=None), dict(dy=None, dw=None), dict(dy=D + 8), dict(T=-1),
               dict(k=0), dict(H=60), dict(n=-1)):
        assert grad(**kw) == bad, kw
    assert grad(T=0, dout=None) == ok


def test_calls_need_device_tensors():
    import torch
    from mixture_experts_gate_amd import products as P, rows as W
    x, w = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(128, dtype=torch.bfloat16)
    r, f = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    u = torch.zeros(4, 64, dtype=torch.uint8)
    for call in (lambda: W.rms_norm(x, w), lambda: W.rms_norm_fp8(x, w), lambda: W.rms_norm_mxfp4(x, w),
                 lambda: W.rms_norm_grad(x, w, x), lambda: W.dispatch(x, r), lambda: W.combine(x, r, f),
                 lambda: W.combine_grad(x, x, r, f), lambda: P.quant_mxfp4(x), lambda: P.swiglu_quant_mxfp4(x),
                 lambda: P.quant_mxfp4_matrices(x), lambda: P.grouped_matmul_mxfp4(u, u, u)):
        with pytest.raises(ValueError):
            call()
