"""The MXFP4 product at its edges: inputs that it refuses, which kernel a size takes,
and scales at the ends of their range. Bounds are those of test_gpu_mxfp4.py."""
import pytest
import torch

from mixture_experts_gate_amd import _lib, products as P

from test_gpu_mxfp4 import PATHS, _bound, _case, _offsets, _ref, _within, decode, kernel_order

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_scales_that_require_grad_are_refused():
    """E8M0 scales are a floating-point type, whose gradient would be lost."""
    e8 = torch.float8_e8m0fnu
    x, w = torch.zeros(4, 64, dtype=torch.uint8, device=DEV), torch.zeros(16, 64, dtype=torch.uint8, device=DEV)
    xs, ws = torch.zeros(4, 4, dtype=torch.uint8, device=DEV).view(e8), torch.zeros(16, 4, dtype=torch.uint8, device=DEV).view(e8)
    for a, b in ((xs.detach().requires_grad_(), ws), (xs, ws.detach().requires_grad_())):
        with pytest.raises(ValueError):
            P.grouped_matmul_mxfp4(x, a, w, b)
        with torch.no_grad():
            P.grouped_matmul_mxfp4(x, a, w, b)


# ------------------------------------------------------- which kernel ran --

# what a call of each path launches
LAUNCHES = {"stream": ["product_mxfp4_stream"], "tiles": ["product_mxfp4"], "cut": ["product_join", "product_mxfp4"],
            "large": ["product_mxfp4_large"]}


def _launched(call):
    """(the call's result, the names of the kernels that it launched)"""
    torch.cuda.synchronize()
    _lib.moe_set_option(_lib.MOE_OPT_TIMING, 1)
    try:
        out = call()
        torch.cuda.synchronize()
        return out, sorted(_lib.timing_report())
    finally:
        _lib.moe_set_option(_lib.MOE_OPT_TIMING, 0)


def _takes(path, call):
    out, names = _launched(call)
    assert names == LAUNCHES[path], (path, names)
    return out


@pytest.mark.parametrize("path", list(PATHS))
def test_each_path_takes_its_kernel(path):
    """The sizes by which the other tests name a kernel run that kernel."""
    counts, N, K = PATHS[path]
    _, byte, scale, (wq, ws) = _case(counts, N, K, 20)
    R = sum(counts)
    args = (byte(R, K // 2), scale(R, K // 32), *kernel_order(wq, ws), _offsets(counts))
    out = torch.empty(R, N, dtype=torch.bfloat16, device=DEV)
    _takes(path, lambda: P.grouped_matmul_mxfp4(*args, out=out))
    rows = torch.arange(R, dtype=torch.int32, device=DEV)
    tall = torch.empty(R + 13, N, dtype=torch.float32, device=DEV)
    _takes(path, lambda: P.grouped_matmul_mxfp4(*args, rows=rows, out_rows=rows, out=tall))
    # 13 rows past the last expert's end, as the tests of rows that are left have them
    more = (byte(R + 13, K // 2), scale(R + 13, K // 32), *args[2:])
    _takes(path, lambda: P.grouped_matmul_mxfp4(*more, out=tall))
    if path == "cut":
        _takes("tiles", lambda: P.grouped_matmul_mxfp4(*args, out=out, ws=torch.empty(16, dtype=torch.uint8, device=DEV)))


# ------------------------------------------------------------ scale bytes --

@pytest.mark.parametrize("path", list(PATHS))
def test_scale_bytes_at_the_ends(path):
    """2^-127 (which a block of zeros or of tiny values has) to 2^127 on one side, as
    much the other way on the other: every block's products are of size 1."""
    counts, N, K = PATHS[path]
    g, byte, _, (wq, _) = _case(counts, N, K, 30)
    R, E, nb = sum(counts), len(counts), K // 32
    ends = torch.tensor([0, 254, 1, 253, 127], device=DEV)[torch.randint(0, 5, (nb,), generator=g, device=DEV)]
    ends[:4] = torch.tensor([0, 254, 1, 253], device=DEV)
    x, xs = byte(R, K // 2), ends.expand(R, nb).to(torch.uint8).contiguous()
    ws = (254 - ends).expand(E, N, nb).to(torch.uint8).contiguous()
    ref, mag = _ref(decode(x, xs), decode(wq, ws), counts, torch.arange(R, device=DEV))
    y = _takes(path, lambda: P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), _offsets(counts),
                                                    out=torch.empty(R, N, device=DEV)))
    _within(y, ref, _bound(ref, mag, K, torch.float32), "y")
