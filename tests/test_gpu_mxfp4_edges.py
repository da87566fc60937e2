"""The MXFP4 product at its edges: inputs that it refuses, which kernel a size takes,
scales at the ends of their range, and tensors past the widths of the kernels'
offsets. Bounds are those of test_gpu_mxfp4.py."""
import pytest
import torch

from mixture_experts_gate_amd import _lib, products as P

from test_gpu_mxfp4 import PATHS, _bound, _case, _gen, _offsets, _ref, _within, decode, kernel_order

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


# ---------------------------------------------------------- far addresses --

def _random(g, *shape):
    return torch.randint(0, 256, shape, device=DEV, generator=g, dtype=torch.uint8)


def _scales(g, *shape):
    return (120 + torch.randint(-6, 7, shape, device=DEV, generator=g)).to(torch.uint8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("path,R", [("stream", 9), ("tiles", 300), ("cut", 300)])
def test_result_beyond_4_gib(path, R, dtype):
    N, K, g = 64, 2176, _gen(40)
    n = (1 << 32) // (N * dtype.itemsize) + 1000
    x, xs, wq, ws = _random(g, R, K // 2), _scales(g, R, K // 32), _random(g, 1, N, K // 2), _scales(g, 1, N, K // 32)
    to = (n - 1 - torch.randperm(900, generator=g, device=DEV)[:R]).to(torch.int32)
    out = torch.full((n, N), 7.0, dtype=dtype, device=DEV)
    space = torch.empty(16, dtype=torch.uint8, device=DEV) if path == "tiles" else None
    _takes(path, lambda: P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), out_rows=to, out=out, ws=space))
    ref, mag = _ref(decode(x, xs), decode(wq, ws), [R], torch.arange(R, device=DEV))
    _within(out[to.long()], ref, _bound(ref, mag, K, dtype), "y")
    out[to.long()] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("over", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_result_at_the_large_tiles_limit(dtype, over):
    """2 GiB less 16 bytes of rows, the last of them written, N a part of a tile; a row
    more goes to the smaller tiles. Some rows have no place."""
    N, K, R, g = 2064, 768, 7424, _gen(41)
    n = 0x7FFFFFF0 // (N * dtype.itemsize) + over
    x, xs, wq, ws = _random(g, R, K // 2), _scales(g, R, K // 32), _random(g, 1, N, K // 2), _scales(g, 1, N, K // 32)
    to = n - 1 - torch.randperm(8000, generator=g, device=DEV)[:R]
    to[7], to[300], to[R - 1] = n - 1, -1, n
    to[8:][to[8:] == n - 1] = 0
    to = to.to(torch.int32)
    out = torch.full((n, N), 7.0, dtype=dtype, device=DEV)
    _takes("tiles" if over else "large",
           lambda: P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), out_rows=to, out=out))
    ref, mag = _ref(decode(x, xs), decode(wq, ws), [R], torch.arange(R, device=DEV))
    live = (to >= 0) & (to < n)
    _within(out[to[live].long()], ref[live], _bound(ref, mag, K, dtype)[live], "y")
    out[to[live].long()] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("over", [False, True])
def test_rows_at_the_large_tiles_limit(over):
    """Just under 4 GiB of x, its last rows read; two rows more go to the smaller tiles."""
    N, K, R, g = 2064, 1024, 7424, _gen(42)
    n = 0xFFFFFFFF // (K // 2) + 2 * over
    x, xs = torch.zeros(n, K // 2, dtype=torch.uint8, device=DEV), torch.full((n, K // 32), 127, dtype=torch.uint8, device=DEV)
    for part in (slice(0, 300), slice(n - 300, n)):
        x[part], xs[part] = _random(g, 300, K // 2), _scales(g, 300, K // 32)
    wq, ws = _random(g, 1, N, K // 2), _scales(g, 1, N, K // 32)
    pick = torch.randint(-300, 300, (R,), generator=g, device=DEV)
    pick[0], pick[R - 1] = -1, -300
    rows = torch.where(pick < 0, n + pick, pick).to(torch.int32)
    y = _takes("tiles" if over else "large", lambda: P.grouped_matmul_mxfp4(x, xs, *kernel_order(wq, ws), rows=rows))
    xd = torch.cat([decode(x[:300], xs[:300]), decode(x[-300:], xs[-300:])])
    ref, mag = _ref(xd, decode(wq, ws), [R], torch.where(pick < 0, 600 + pick, pick))
    _within(y, ref, _bound(ref, mag, K, torch.bfloat16), "y")


@pytest.mark.parametrize("path,K,counts", [("stream", 16384, (1, 2, 3)), ("tiles", 16512, (60, 1, 150)),
                                           ("large", 16384, (60, 1, 150))])
def test_matrices_beyond_4_gib(path, K, counts):
    """270 experts of 16 MiB, of which the first and the last two have rows."""
    E, N, g = 270, 2048, _gen(43)
    live, R = (0, E - 2, E - 1), sum(counts)
    kq, ks = torch.zeros(E, N, K // 2, dtype=torch.uint8, device=DEV), torch.full((E, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    wq, ws = _random(g, 3, N, K // 2), _scales(g, 3, N, K // 32)
    for i, e in enumerate(live):
        a, b = kernel_order(wq[i:i + 1], ws[i:i + 1])
        kq[e], ks[e] = a[0], b[0]
    assert kq[E - 1].data_ptr() - kq.data_ptr() > 1 << 32
    x, xs = _random(g, R, K // 2), _scales(g, R, K // 32)
    every = [0] * E
    for i, e in enumerate(live):
        every[e] = counts[i]
    y = _takes(path, lambda: P.grouped_matmul_mxfp4(x, xs, kq, ks, _offsets(every), out=torch.empty(R, N, device=DEV)))
    xd = decode(x, xs)
    for cols in (slice(0, 80), slice(N - 80, N)):
        ref, mag = _ref(xd, decode(wq[:, cols].contiguous(), ws[:, cols].contiguous()), counts, torch.arange(R, device=DEV))
        _within(y[:, cols], ref, _bound(ref, mag, K, torch.float32), "y")
