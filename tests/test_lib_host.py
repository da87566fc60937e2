"""Host-side checks of the HIP library (no GPU needed): it loads, exports every
symbol the header declares, and rejects bad arguments before touching the
device."""
import ctypes as C
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe.h")


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_gate_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_gate_amd import build
        build.build()
    return _lib


def _declared_functions():
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"\b(moe_\w+|expert_cache_\w+)\s*\(", src)
    return sorted(set(names))


def test_header_declares_binding_exports(lib):
    assert _declared_functions() == sorted(lib.EXPORTS)


def test_library_exports_every_symbol(lib):
    L = C.CDLL(lib.LIB_PATH)
    for name in _declared_functions():
        assert hasattr(L, name), name


def test_strerror_and_options(lib):
    L = lib.load()
    assert L.moe_strerror(0) == b"ok"
    assert L.moe_strerror(lib.MOE_EINVAL) == b"invalid argument"
    assert L.moe_strerror(-99) == b"unknown error"
    assert L.moe_get_option(lib.MOE_OPT_FFN_PATH) == 0
    assert L.moe_set_option(lib.MOE_OPT_FFN_PATH, 3) == lib.MOE_EINVAL
    assert L.moe_set_option(99, 0) == lib.MOE_EINVAL


def test_workspace_sizes(lib):
    pb, fb = lib.moe_workspace_size(64, 8, 2048, 768, 128)
    assert pb == 0                      # one-workgroup permutation needs no workspace
    assert fb >= 64 * 8 * 768 * 2
    pb, fb = lib.moe_workspace_size(8192, 8, 2048, 768, 128)
    assert pb >= (64 * 128 + 65536) * 4
    assert fb >= 65536 * 768 * 2
    # tiled path: two FP8 terms + block scales of the activation and of x, and
    # the token-tile map (at most n_pairs / 128 + E tiles)
    assert fb >= (2 * 65536 * 768 + 65536 * 768 // 32 + 2 * 8192 * 2048 + 8192 * 2048 // 32
                  + (65536 // 128 + 128 + 1) * 4)
    with pytest.raises(lib.MoeError):
        lib.moe_workspace_size(-1, 8, 2048, 768, 128)


def test_argument_errors_before_any_device_work(lib):
    L = lib.load()
    dummy = 0x1000  # never dereferenced: validation fails first
    # k > E
    assert L.moe_route(None, None, dummy, None, 4, 64, 8, 9, 1, dummy, dummy, None) == lib.MOE_EINVAL
    # gate needs H % 8 == 0
    assert L.moe_route(dummy, dummy, None, None, 4, 12, 8, 2, 1, dummy, dummy, None) == lib.MOE_EINVAL
    # E above the permutation's limit
    assert L.moe_permute(dummy, 4, 2, 513, dummy, dummy, dummy, None, 0, None) == lib.MOE_EINVAL
    # H not a multiple of 32
    assert L.moe_expert_ffn(dummy, dummy, dummy, dummy, 1, 4, 2, 48, 64, 8, dummy, 0, dummy,
                            1 << 20, None) == lib.MOE_EINVAL
    # workspace too small
    assert L.moe_expert_ffn(dummy, dummy, dummy, dummy, 1, 4, 2, 64, 64, 8, dummy, 0, dummy,
                            16, None) == lib.MOE_EINVAL
    # more experts than the FFN supports
    assert L.moe_expert_ffn(dummy, dummy, dummy, dummy, 1, 4, 2, 128, 128, 513, dummy, 0, dummy,
                            1 << 30, None) == lib.MOE_EINVAL
    # packing: unknown format, K not a multiple of 128, null pointers
    assert L.moe_pack_weights(0, dummy, dummy, 1, 1 << 20, 1 << 20, 256, 256, 0, 0, 0, 0,
                              None) == lib.MOE_EINVAL
    assert L.moe_pack_weights(2, dummy, dummy, 1, 1 << 20, 1 << 20, 256, 192, 0, 0, 0, 0,
                              None) == lib.MOE_EINVAL
    assert L.moe_pack_weights(3, None, dummy, 1, 1 << 20, 1 << 20, 256, 256, 0, 0, 0, 0,
                              None) == lib.MOE_EINVAL
    assert L.moe_pack_weights(3, None, None, 0, 0, 0, 256, 256, 0, 0, 0, 0, None) == lib.MOE_OK
    # NVFP4 / FP8 FFN calls need H, I multiples of 128
    assert L.moe_expert_ffn(dummy, dummy, dummy, dummy, 2, 4, 2, 192, 128, 8, dummy, 0, dummy,
                            1 << 30, None) == lib.MOE_EINVAL
    # bad weight format
    assert L.moe_expert_ffn(dummy, dummy, dummy, dummy, 7, 4, 2, 64, 64, 8, dummy, 0, dummy,
                            1 << 20, None) == lib.MOE_EINVAL
    # combine: H % 8
    assert L.moe_combine(dummy, 0, dummy, None, 4, 2, 12, dummy, None) == lib.MOE_EINVAL
    # T == 0 is a no-op that succeeds
    assert L.moe_combine(None, 0, None, None, 0, 2, 64, None, None) == lib.MOE_OK
    assert L.moe_route(None, None, None, None, 0, 64, 8, 2, 1, None, None, None) == lib.MOE_OK


def test_ffn_shared_argument_errors(lib):
    """moe_expert_ffn_shared: a missing shared expert, a workspace sized for the
    routed rows only and too many experts are refused before device work."""
    L = lib.load()
    dummy = 0x1000  # never dereferenced: validation fails first
    T, k, H, I, E = 8, 4, 256, 128, 16
    _, fb_k = lib.moe_workspace_size(T, k, H, I, E)
    _, fb_k1 = lib.moe_workspace_size(T, k + 1, H, I, E)
    assert fb_k1 > fb_k
    assert L.moe_expert_ffn_shared(dummy, dummy, dummy, dummy, None, 1, T, k, H, I, E, dummy, 0,
                                   dummy, fb_k1, None) == lib.MOE_EINVAL
    assert L.moe_expert_ffn_shared(dummy, dummy, dummy, dummy, dummy, 1, T, k, H, I, E, dummy, 0,
                                   dummy, fb_k, None) == lib.MOE_EINVAL
    assert L.moe_expert_ffn_shared(dummy, dummy, dummy, dummy, dummy, 1, T, k, H, I, 513, dummy,
                                   0, dummy, 1 << 30, None) == lib.MOE_EINVAL
    assert L.moe_expert_ffn_shared(None, None, None, None, None, 1, 0, k, H, I, E, None, 0, None,
                                   0, None) == lib.MOE_OK


def test_ffn_combine_argument_errors(lib):
    """moe_expert_ffn_combine: missing router weights or outputs, a workspace
    sized without the shared expert's rows and a bad format are refused
    before device work; T == 0 succeeds."""
    L = lib.load()
    dummy = 0x1000  # never dereferenced: validation fails first
    T, k, H, I, E = 4, 4, 256, 128, 16
    _, fb_k = lib.moe_workspace_size(T, k, H, I, E)
    _, fb_k1 = lib.moe_workspace_size(T, k + 1, H, I, E)
    args = lambda shared, fmt, tw, y, out, wsb: (dummy, dummy, dummy, dummy, shared, fmt, T, k, H,
                                                 I, E, tw, y, out, dummy, wsb, None)
    assert L.moe_expert_ffn_combine(*args(None, 1, None, dummy, dummy, fb_k)) == lib.MOE_EINVAL
    assert L.moe_expert_ffn_combine(*args(None, 1, dummy, None, dummy, fb_k)) == lib.MOE_EINVAL
    assert L.moe_expert_ffn_combine(*args(None, 1, dummy, dummy, None, fb_k)) == lib.MOE_EINVAL
    assert L.moe_expert_ffn_combine(*args(dummy, 1, dummy, dummy, dummy, fb_k)) == lib.MOE_EINVAL
    assert L.moe_expert_ffn_combine(*args(None, 9, dummy, dummy, dummy, fb_k1)) == lib.MOE_EINVAL
    assert L.moe_expert_ffn_combine(None, None, None, None, None, 1, 0, k, H, I, E, None, None,
                                    None, None, 0, None) == lib.MOE_OK


def test_permute_ffn_combine_argument_errors(lib):
    """moe_permute_ffn_combine: missing offsets, ids, permutation outputs or
    router weights, a workspace sized without the shared expert's rows, too
    many experts and a bad format are refused before device work."""
    L = lib.load()
    dummy = 0x1000  # never dereferenced: validation fails first
    T, k, H, I, E = 8, 4, 256, 128, 16
    _, fb_k = lib.moe_workspace_size(T, k, H, I, E)
    _, fb_k1 = lib.moe_workspace_size(T, k + 1, H, I, E)

    def call(ids=dummy, tw=dummy, shared=None, fmt=1, E_=E, off=dummy, sp=dummy, pr=dummy,
             wsb=fb_k):
        return L.moe_permute_ffn_combine(dummy, ids, tw, dummy, shared, fmt, T, k, H, I, E_, off,
                                         sp, pr, dummy, dummy, dummy, wsb, None)
    assert call(off=None) == lib.MOE_EINVAL
    assert call(ids=None) == lib.MOE_EINVAL
    assert call(tw=None) == lib.MOE_EINVAL
    assert call(sp=None) == lib.MOE_EINVAL
    assert call(pr=None) == lib.MOE_EINVAL
    assert call(shared=dummy) == lib.MOE_EINVAL          # workspace without the shared rows
    assert call(fmt=9, wsb=fb_k1) == lib.MOE_EINVAL
    assert call(E_=513, wsb=1 << 30) == lib.MOE_EINVAL


def test_layer_fused_argument_errors(lib):
    """moe_layer_fused: missing logits, outputs or sync buffer, a misaligned
    sync buffer, a workspace too small or T = 0 are refused (MOE_EINVAL), and
    batches outside the one-launch sizes are declined (MOE_EUNSUPPORTED), both
    before any device work."""
    L = lib.load()
    dummy = 0x1000  # never dereferenced: validation fails first
    T, k, H, I, E = 1, 8, 2048, 768, 128
    _, fb = lib.moe_workspace_size(T, k, H, I, E)

    def call(T_=T, k_=k, H_=H, I_=I, E_=E, fmt=1, lg=dummy, out=dummy, sync=dummy, wsb=fb,
             shared=None):
        return L.moe_layer_fused(dummy, lg, dummy, shared, fmt, T_, k_, H_, I_, E_, 1, dummy,
                                 dummy, dummy, dummy, dummy, dummy, out, dummy, wsb, sync, None)
    assert call(lg=None) == lib.MOE_EINVAL
    assert call(out=None) == lib.MOE_EINVAL
    assert call(sync=None) == lib.MOE_EINVAL
    assert call(sync=dummy + 4) == lib.MOE_EINVAL            # not 8-byte aligned
    assert call(wsb=fb - 1) == lib.MOE_EINVAL
    assert call(T_=0) == lib.MOE_EINVAL
    assert call(k_=200) == lib.MOE_EINVAL                    # k > E
    big = 1 << 30
    assert call(T_=4, wsb=big) == lib.MOE_EUNSUPPORTED       # 32 rows
    assert call(T_=9, k_=1, wsb=big) == lib.MOE_EUNSUPPORTED  # more tokens than wavefronts
    assert call(E_=300, wsb=big) == lib.MOE_EUNSUPPORTED     # ids past 8 bits
    assert call(fmt=0, wsb=big) == lib.MOE_EUNSUPPORTED      # bf16 weights
    assert call(H_=1536, wsb=big) == lib.MOE_EUNSUPPORTED    # 12 slabs of gate/up
    assert call(I_=1024, wsb=big) == lib.MOE_EUNSUPPORTED    # 8 slabs of down
    assert call(shared=dummy, k_=7, T_=4, wsb=big) == lib.MOE_EUNSUPPORTED  # 32 rows


def test_cache_reserve_argument_errors(lib):
    L = lib.load()
    h = C.c_void_p(0)
    src = (C.c_void_p * 2)(0x1000, 0x2000)
    # pool too small for one layer of experts
    assert L.expert_cache_reserve(C.byref(h), 0x1000, 1024, 1024, 1, 2, src, 0, 0, 0, 0,
                                  None) == lib.MOE_ENOMEM
    # null host source
    src0 = (C.c_void_p * 2)(0x1000, None)
    assert L.expert_cache_reserve(C.byref(h), 0x1000, 1 << 20, 1024, 1, 2, src0, 0, 0, 0, 0,
                                  None) == lib.MOE_EINVAL
    assert L.expert_cache_destroy(None) == lib.MOE_EINVAL
    assert L.expert_cache_slots(None) == lib.MOE_EINVAL
    assert L.expert_cache_resize(None, 0x1000, 1 << 20, None, None) == lib.MOE_EINVAL


def test_products_reject_bad_arguments(lib):
    """The expert products and their companions: sizes, null pointers,
    alignment, contradictory matrices (before any device work)."""
    L, d, bad = lib.load(), 0x1000, lib.MOE_EINVAL

    def gemm(fn, x=d, rows=None, div=1, n=8, off=d, w=d, tab=None, mat=0, R=8, N=16, K=16, E=2,
             y=d, y_rows=None, y_n=8, ws=None):
        return fn(x, rows, div, n, off, w, tab, mat, R, N, K, E, y, y_rows, y_n, 0, ws, 0, None)

    for fn in (L.moe_grouped_gemm, L.moe_grouped_gemm_dx):
        for kw in (dict(R=-1), dict(E=0), dict(E=513), dict(N=12), dict(K=12), dict(N=0), dict(N=1 << 21), dict(N=1 << 20, K=1 << 20, E=4),
                   dict(off=None), dict(w=None), dict(tab=d), dict(mat=2), dict(y=None),
                   dict(y=d + 8), dict(x=None), dict(x=d + 2), dict(n=7), dict(rows=d, n=0),
                   dict(rows=d, div=0), dict(y_n=7), dict(y_rows=d, y_n=0), dict(ws=d + 4)):
            assert gemm(fn, **kw) == bad, kw
        assert gemm(fn, R=0, x=None, y=None) == lib.MOE_OK

    def fp8(x=d, xs=d, n=8, w=d, ws=d, tab=None, K=16, N=16, y=d):
        return L.moe_grouped_gemm_fp8(x, xs, None, 1, n, d, w, ws, tab, 0, 8, N, K, 2, y, None, 8,
                                      0, None, 0, None)

    for kw in (dict(x=None), dict(xs=None), dict(ws=None), dict(w=None), dict(tab=d), dict(K=24),
               dict(K=8), dict(N=12), dict(y=None), dict(n=3), dict(x=d + 8)):
        assert fp8(**kw) == bad, kw

    def dw(dy=d, n=8, x=d, m=8, off=d, R=8, N=16, K=16, E=2, out=d, f32=1, acc=0):
        return L.moe_grouped_gemm_dw(dy, None, 1, n, x, None, 1, m, off, R, N, K, E, out, f32, acc,
                                     None, 0, None)

    for kw in (dict(dy=None), dict(x=None), dict(n=7), dict(m=7), dict(off=None), dict(out=None),
               dict(f32=0, acc=1), dict(N=4), dict(K=20), dict(out=d + 4), dict(E=600)):
        assert dw(**kw) == bad, kw

    def act(h=d, w=None, rows=None, wn=0, R=4, I=16, a=d):
        return L.moe_swiglu(h, w, rows, wn, None, R, I, a, None)

    for kw in (dict(h=None), dict(a=None), dict(I=12), dict(R=-1), dict(rows=d), dict(w=d, wn=3),
               dict(w=d, rows=d, wn=0), dict(h=d + 4)):
        assert act(**kw) == bad, kw
    assert L.moe_swiglu_grad(d, d, None, None, 0, None, 4, 16, d, d, None, None) == bad  # dw, no w
    assert L.moe_swiglu_grad(d, None, None, None, 0, None, 4, 16, d, None, None, None) == bad
    assert L.moe_swiglu_grad(d, d, None, None, 0, None, 4, 16, d, None, d + 2, None) == bad
    for fn in (L.moe_quant_fp8, L.moe_swiglu_quant_fp8):
        assert fn(d, None, 4, 12, d, d, None) == bad
        assert fn(None, None, 4, 16, d, d, None) == bad
        assert fn(d, None, 4, 16, d, None, None) == bad
        assert fn(d, None, 4, 16, d + 4, d, None) == bad
        assert fn(d, None, 0, 16, None, None, None) == lib.MOE_OK


def test_product_workspace_sizes(lib):
    ws = lib.moe_grouped_gemm_workspace
    # 3 x 1 tiles of 128 x 128 over K = 3648: at least two parts of [261][112] fp32
    assert ws(lib.MOE_GEMM_BF16, 261, 112, 3648, 1) >= 2 * 261 * 112 * 4
    assert ws(lib.MOE_GEMM_DW, 6546, 3320, 280, 1) % (3320 * 280 * 4) == 0
    # many tiles, few steps, a handful of rows, none: whole
    assert ws(lib.MOE_GEMM_BF16, 65536, 1536, 2048, 128) == 0
    assert ws(lib.MOE_GEMM_DX, 300, 64, 256, 1) == 0
    assert ws(lib.MOE_GEMM_BF16, 8, 1536, 2048, 128) == 0
    assert ws(lib.MOE_GEMM_DW, 0, 64, 64, 4) == 0
    for bad in ((4, 8, 64, 64, 1), (0, -1, 64, 64, 1), (0, 8, 60, 64, 1), (1, 8, 64, 24, 1),
                (0, 8, 64, 64, 513)):
        with pytest.raises(lib.MoeError):
            ws(*bad)


def test_products_module_needs_device_tensors():
    import torch
    from mixture_experts_gate_amd import products as P
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    w = torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    for call in (lambda: P.grouped_matmul(x, w), lambda: P.grouped_matmul_dx(x, w),
                 lambda: P.grouped_matmul_dw(x, x), lambda: P.swiglu(x), lambda: P.quant_fp8(x),
                 lambda: P.swiglu_grad(x, x), lambda: P.swiglu_quant_fp8(x),
                 lambda: P.grouped_matmul_fp8(x, x, w)):
        with pytest.raises(ValueError):
            call()


def test_products_reject_rows_past_32_bits(lib):
    """The threads of a last workgroup and the rows of a last tile have to fit
    an int: R = 2^31 - 1 is refused by every entry point."""
    L, d, R = lib.load(), 0x1000, 2 ** 31 - 1
    for fn in (L.moe_grouped_gemm, L.moe_grouped_gemm_dx):
        assert fn(d, None, 1, R, None, d, None, 0, R, 16, 16, 1, d, None, R, 0, None, 0,
                  None) == lib.MOE_EINVAL
    assert L.moe_grouped_gemm_fp8(d, d, None, 1, R, None, d, d, None, 0, R, 16, 16, 1, d, None, R,
                                  0, None, 0, None) == lib.MOE_EINVAL
    assert L.moe_grouped_gemm_dw(d, None, 1, R, d, None, 1, R, None, R, 16, 16, 1, d, 1, 0, None,
                                 0, None) == lib.MOE_EINVAL
    assert L.moe_swiglu(d, None, None, 0, None, R, 8, d, None) == lib.MOE_EINVAL
    assert L.moe_swiglu_grad(d, d, None, None, 0, None, R, 8, d, None, None, None) == lib.MOE_EINVAL
    for fn in (L.moe_quant_fp8, L.moe_swiglu_quant_fp8):
        assert fn(d, None, R, 8, d, d, None) == lib.MOE_EINVAL
    with pytest.raises(lib.MoeError):
        lib.moe_grouped_gemm_workspace(lib.MOE_GEMM_BF16, R, 16, 16, 1)


def test_product_layers_need_device_tensors():
    """Host tensors are refused before anything is enqueued, and a refused
    forward leaves no state for a backward."""
    import torch
    from mixture_experts_gate_amd.layer import Fp8BlockLayer
    from mixture_experts_gate_amd.train import TrainExperts
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    m = TrainExperts(64, 4, 2, 32, 4, device="cpu")
    with pytest.raises(ValueError):
        m.forward(x, ids, w, torch.zeros(4, 64, 64, dtype=torch.bfloat16),
                  torch.zeros(4, 64, 32, dtype=torch.bfloat16))
    with pytest.raises(RuntimeError):
        m.backward(x)
    layer = Fp8BlockLayer(64, 4, 2, 32, 4, device="cpu")
    with pytest.raises(ValueError):
        layer.forward(4, x, None, logits=torch.zeros(4, 4))


def test_product_workspaces_are_within_their_bound(lib):
    """workspace_bound(R, ...) suffices for every product of at most R rows."""
    import random
    from mixture_experts_gate_amd import products as P
    rng, cut = random.Random(5), 0
    for _ in range(4000):
        R, E = int(2 ** rng.uniform(0, 15)), rng.choice((1, 1, 2, 8, 64, 300))
        N, K = 16 * int(2 ** rng.uniform(0, 9)), 16 * int(2 ** rng.uniform(0, 9))
        for kind in (lib.MOE_GEMM_BF16, lib.MOE_GEMM_FP8, lib.MOE_GEMM_DX, lib.MOE_GEMM_DW):
            size = lib.moe_grouped_gemm_workspace(kind, R, N, K, E)
            assert size <= P.workspace_bound(R, N, K, E, "cpu"), (kind, R, N, K, E)
            cut += size > 0
    assert cut > 100
    # sums that are cut: 2 x 3 tiles over 6546 rows of one expert
    assert lib.moe_grouped_gemm_workspace(lib.MOE_GEMM_DW, 6546, 3320, 280, 1) >= 2 * 3320 * 280 * 4
