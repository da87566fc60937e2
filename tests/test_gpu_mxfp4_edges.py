"""The MXFP4 product at its edges: inputs that it refuses, which kernel a size takes,
scales at the ends of their range, and tensors past the widths of the kernels'
offsets. Bounds are those of test_gpu_mxfp4.py."""
import pytest
import torch

from mixture_experts_gate_amd import products as P

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
