"""The routed experts of a layer in training: forward and backward in bf16 with
fp32 sums, from the library's products.

With pairs p = (token t, choice j), expert e, router weight w_p:
  h_p = W13_e x_t = [g | u],  a_p = w_p silu(g) u,  out_t = sum_j W2_e a_p.
The weight sits in the activation, so that the tokens' sum and its gradient need
no weights: dy_p = dout_t, and dw_p = <da_p, silu(g) u> comes with the
activation's gradient.
"""
from __future__ import annotations

import torch

from . import _lib, products as P


class TrainExperts:
    """Buffers and call sequence for at most T_max tokens. ``forward`` keeps what
    ``backward`` needs: its inputs must be unchanged until then, and one
    backward belongs to the last forward. Both run on the current stream and
    allocate nothing, so a training step can be captured into a graph.

    Autograd is not involved: the gradients are ``backward``'s results, and
    ``forward`` refuses inputs that require grad where gradients are enabled
    (call it under ``torch.no_grad()``, or from a ``torch.autograd.Function``)."""

    def __init__(self, H, E, k, I, T_max, device="cuda"):
        if H % 8 or I % 8 or E > 512:
            raise ValueError("H and I must be multiples of 8, E at most 512")
        self.H, self.E, self.k, self.I, self.T_max = H, E, k, I, T_max
        n = max(T_max * k, 1)

        def buf(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=device)

        self.offsets = buf(E + 1, dtype=torch.int32)
        self.sorted_pair, self.pair_row = buf(n, dtype=torch.int32), buf(n, dtype=torch.int32)
        self.ws_bytes = max(_lib.moe_workspace_size(T_max, k, H, I, E)[0], 256)
        self.ws = buf(self.ws_bytes, dtype=torch.uint8)
        self.ws_sum = buf(max(P.workspace_bound(n, 2 * I, H, E, device),
                              P.workspace_bound(n, H, I, E, device)), dtype=torch.uint8)
        self.ones = torch.ones(T_max, k, dtype=torch.float32, device=device)
        self.h, self.a = buf(n, 2 * I), buf(n, I)
        self.y, self.out = buf(n, H), buf(T_max, H)
        self.da, self.dh, self.dx = buf(n, I), buf(n, 2 * I), buf(T_max, H)
        self.dtopk_w = buf(T_max, k, dtype=torch.float32)
        self.dw13 = buf(E, 2 * I, H, dtype=torch.float32)
        self.dw2 = buf(E, H, I, dtype=torch.float32)
        self._saved = None

    def _check(self, t, name, dtype, *shape):
        """Before the first launch: a refused call leaves every buffer as it was."""
        if (not isinstance(t, torch.Tensor) or t.device != self.out.device or t.dtype != dtype
                or tuple(t.shape) != shape or not t.is_contiguous()
                or (dtype is torch.bfloat16 and t.data_ptr() % 16)):
            got = (f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor)
                   else type(t).__name__)
            raise ValueError(f"{name}: {got}; contiguous {dtype} {list(shape)} on {self.out.device} is "
                             "needed (bf16: from an address that is a multiple of 16)")

    def forward(self, x, topk_ids, topk_w, w13, w2):
        """out [T, H] bf16 of x [T, H] bf16, the router's topk_ids [T, k] int32
        (distinct experts of a token, all of them in [0, E): the caller's to see
        to; a padding token has any of them, with weights 0) and topk_w [T, k]
        fp32, w13 [E, 2I, H] and w2 [E, H, I] bf16."""
        self._saved = None
        if not isinstance(x, torch.Tensor) or not x.is_cuda or x.device != self.out.device:
            raise ValueError(f"x: a tensor on {self.out.device}, where the buffers are, is needed")
        if x.get_device() != torch.cuda.current_device():
            with torch.cuda.device(x.device):
                return self.forward(x, topk_ids, topk_w, w13, w2)
        k, bf16 = self.k, torch.bfloat16
        T = min(x.shape[0], self.T_max) if x.dim() else 0       # (at most T_max)
        self._check(x, "x", bf16, T, self.H)
        self._check(topk_ids, "topk_ids", torch.int32, T, k)
        self._check(topk_w, "topk_w", torch.float32, T, k)
        self._check(w13, "w13", bf16, self.E, 2 * self.I, self.H)
        self._check(w2, "w2", bf16, self.E, self.H, self.I)
        P._no_history(x, topk_w, w13, w2)
        n = T * k
        if T == 0:
            self._saved = (x, topk_w, w13, w2)
            return self.out[:0]
        pair, off = self.sorted_pair[:n], self.offsets
        _lib.moe_permute(topk_ids, T, k, self.E, off, self.sorted_pair, self.pair_row, self.ws,
                         self.ws_bytes)
        P.grouped_matmul(x, w13, off, rows=pair, div=k, out=self.h[:n], ws=self.ws_sum)
        P.swiglu(self.h[:n], topk_w, pair, off[self.E:], out=self.a[:n])
        P.grouped_matmul(self.a[:n], w2, off, out_rows=pair, out=self.y[:n], ws=self.ws_sum)
        _lib.moe_combine(self.y, False, self.ones, None, T, k, self.H, self.out)
        self._saved = (x, topk_w, w13, w2)
        return self.out[:T]

    @torch.no_grad()
    def backward(self, dout, accumulate=False):
        """(dx [T, H] bf16, dtopk_w [T, k] fp32, dw13, dw2 fp32) of the last
        forward for dout [T, H] bf16; with ``accumulate`` the matrices' gradients
        are added to what dw13 and dw2 hold."""
        if self._saved is None:
            raise RuntimeError("backward without a forward")
        x, topk_w, w13, w2 = self._saved
        if x.get_device() != torch.cuda.current_device():
            with torch.cuda.device(x.device):
                return self.backward(dout, accumulate)
        T, k = x.shape[0], self.k
        self._check(dout, "dout", torch.bfloat16, T, self.H)
        n = T * k
        if T == 0:
            if not accumulate:
                self.dw13.zero_(), self.dw2.zero_()
            return self.dx[:0], self.dtopk_w[:0], self.dw13, self.dw2
        pair, off = self.sorted_pair[:n], self.offsets
        da, dh, dxp = self.da[:n], self.dh[:n], self.y[:n]
        P.grouped_matmul_dx(dout, w2, off, rows=pair, div=k, out=da, ws=self.ws_sum)
        P.grouped_matmul_dw(dout, self.a[:n], off, dy_rows=pair, dy_div=k, out=self.dw2,
                            accumulate=accumulate, ws=self.ws_sum)
        P.swiglu_grad(self.h[:n], da, topk_w.view(-1), pair, off[self.E:], dh=dh,
                      dw=self.dtopk_w[:T].view(-1))
        P.grouped_matmul_dx(dh, w13, off, out_rows=pair, out=dxp, ws=self.ws_sum)
        _lib.moe_combine(dxp, False, self.ones, None, T, k, self.H, self.dx)
        P.grouped_matmul_dw(dh, x, off, x_rows=pair, x_div=k, out=self.dw13, accumulate=accumulate,
                            ws=self.ws_sum)
        return self.dx[:T], self.dtopk_w[:T], self.dw13, self.dw2
