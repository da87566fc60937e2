"""The expert products and what goes with them, as cases to measure.

Four operators of the mixture-of-experts layer whose experts' weights are bf16
or block-scaled FP8 matrices:

  product      y = W_e x for rows grouped by expert (bf16), and "gradients":
               dx = W_e^T dy and dW_e = sum of dy x^T over the expert's rows
  gated        a = w silu(g) u of the halves [g | u] of a row with the router's
               weight w of the row, and "gated_gradients": d[g | u] and dw
  to_fp8       rows as E4M3 codes with one scale per 128 columns, and
               "gated_to_fp8": the same of silu(g) u
  product_fp8  y = W_e x from E4M3 codes with a scale per 128 columns of a row
               of x and per 128 x 128 block of W_e

A pair is (token, one of its k experts), numbered token * k + j. "sorted order"
is the pairs grouped by expert. side "in": the product reads token rows and
writes sorted order (the gate/up projection); side "out": it reads sorted order
and writes pair order (the down projection). The gradients mirror that.
"""
import math

import torch

own = False

_MIN_AMAX = 2.0 ** -100          # smallest block maximum a scale is made from
_KINDS_R = ("product", "gradients", "product_fp8")


# ------------------------------------------------------------------- cases --

def listed():
    def rows(name, kind, T, k, E, N, K, side, skew):
        return {"name": name, "kind": kind, "T": T, "k": k, "E": E, "N": N, "K": K, "side": side,
                "skew": skew}

    return [
        # one token's gate/up projection in a decode step: latency
        rows("gate/up of one token", "product", 1, 8, 128, 1536, 2048, "in", 0.0),
        # the gate/up projection of a prompt: the matrix cores
        rows("gate/up of 8192 tokens", "product", 8192, 8, 128, 1536, 2048, "in", 0.22),
        # one small training batch on a small layer, odd row counts
        rows("gradients of 301 tokens", "gradients", 301, 2, 8, 1024, 256, "in", 0.22),
        # a training batch's gradients of the down projection
        rows("gradients of 4096 tokens", "gradients", 4096, 8, 128, 2048, 768, "out", 0.22),
        # the activation of a decode step's 8 rows
        {"name": "activation of one token", "kind": "gated", "R": 8, "I": 768},
        # the activation's gradient in a training step
        {"name": "activation gradient, 32768 rows", "kind": "gated_gradients", "R": 32768, "I": 768},
        # a decode batch's rows to FP8
        {"name": "16 rows to FP8", "kind": "to_fp8", "R": 16, "K": 4096},
        # a prompt's activations to FP8, between the two projections
        {"name": "activation of 24576 rows to FP8", "kind": "gated_to_fp8", "R": 24576, "K": 2048},
        # one token's gate/up projection of a large sparse layer from FP8 weights
        rows("FP8 gate/up of one token", "product_fp8", 1, 6, 256, 4096, 4096, "in", 1.0),
        # a decode batch of 64 on the same layer: one to tens of rows an expert
        rows("FP8 gate/up of 64 tokens", "product_fp8", 64, 6, 256, 4096, 4096, "in", 1.0),
        # a prompt's down projection of the same layer
        rows("FP8 down of 4096 tokens", "product_fp8", 4096, 6, 256, 4096, 2048, "out", 0.22),
        # the always-on expert of the same layer: one group, an odd row count
        rows("FP8 gate/up, one expert", "product_fp8", 4001, 1, 1, 4096, 4096, "in", 0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("product", "product", "gradients", "gradients", "gated", "gated_gradients",
                       "to_fp8", "gated_to_fp8", "product_fp8", "product_fp8", "product_fp8"))
    if kind in ("gated", "gated_gradients"):
        return {"kind": kind, "R": _log_int(rng, 1, 32768), "I": 8 * _log_int(rng, 4, 256)}
    if kind in ("to_fp8", "gated_to_fp8"):
        return {"kind": kind, "R": _log_int(rng, 1, 32768), "K": 16 * _log_int(rng, 2, 128)}
    unit = 16 if kind == "product_fp8" else 8
    top = 400e9 if kind != "gradients" else 200e9
    while True:
        E = _log_int(rng, 1, 256)
        c = {"kind": kind, "T": _log_int(rng, 1, 8192), "k": rng.randint(1, min(E, 8)), "E": E,
             "N": unit * _log_int(rng, 64 // unit, 4096 // unit),
             "K": unit * _log_int(rng, 64 // unit, 4096 // unit),
             "side": rng.choice(("in", "out")), "skew": rng.choice((0.0, 0.22, 0.5))}
        if 2.0 * c["T"] * c["k"] * c["N"] * c["K"] <= top and E * c["N"] * c["K"] <= 1.0e9:
            return c


def work(case):
    kind = case["kind"]
    if kind in ("gated", "gated_gradients"):
        n = case["R"] * case["I"]
        if kind == "gated":
            return {"bytes": 6 * n + 8 * case["R"], "flops": 6 * n}
        return {"bytes": 10 * n + 12 * case["R"], "flops": 16 * n}
    if kind in ("to_fp8", "gated_to_fp8"):
        n, blocks = case["R"] * case["K"], case["R"] * -(-case["K"] // 128)
        return {"bytes": (5 if kind == "gated_to_fp8" else 3) * n + 4 * blocks, "flops": 4 * n}
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    R, live = T * k, E * (1.0 - (1.0 - k / E) ** T)
    n_in, n_out = (T, R) if case["side"] == "in" else (R, R)
    index = 8 * R + 4 * (E + 1)
    if kind == "product":
        return {"bytes": 2 * (live * N * K + n_in * K + n_out * N) + index, "flops": 2.0 * R * N * K}
    if kind == "product_fp8":
        blocks = -(-K // 128)
        return {"bytes": live * (N * K + 4 * -(-N // 128) * blocks) + n_in * (K + 4 * blocks)
                + 2 * n_out * N + index, "flops": 2.0 * R * N * K}
    n_dy, n_x = (R, T) if case["side"] == "in" else (T, R)
    return {"bytes": 2 * (live * N * K + n_dy * N + n_x * K + R * K) + 4 * E * N * K + index,
            "flops": 4.0 * R * N * K}


# ------------------------------------------------------------------ inputs --

def _routing(gen, T, k, E, skew):
    """k distinct experts for each token; experts differ in popularity by `skew`."""
    bias = skew * torch.randn(E, device="cuda", generator=gen)
    noise = torch.rand(T, E, device="cuda", generator=gen).clamp_(1e-9, 1 - 1e-7)
    return torch.topk(bias - torch.log(-torch.log(noise)), k, dim=1).indices


def _fp8_weights(gen, E, N, K):
    """Gaussian matrices as E4M3 codes with one scale per 128 x 128 block."""
    nb, kb = -(-N // 128), -(-K // 128)
    codes = torch.empty(E, N, K, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(E, nb, kb, device="cuda")
    step = max(1, (1 << 28) // (nb * kb * 16384))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.zeros(n, nb * 128, kb * 128, device="cuda")
        w[:, :N, :K] = 0.02 * torch.randn(n, N, K, device="cuda", generator=gen)
        w = w.view(n, nb, 128, kb, 128)
        s = w.abs().amax(dim=(2, 4)) / 448.0
        w = (w / s[:, :, None, :, None]).clamp_(-448, 448).view(n, nb * 128, kb * 128)
        codes[e:e + n] = w[:, :N, :K].to(torch.float8_e4m3fn)
        scales[e:e + n] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def bf16(*shape, sigma=1.0):
        x = torch.randn(*shape, device="cuda", dtype=torch.bfloat16, generator=gen)
        return x.mul_(sigma) if sigma != 1.0 else x

    kind = case["kind"]
    if kind in ("gated", "gated_gradients"):
        R, I = case["R"], case["I"]
        s = {"kind": kind, "h": bf16(R, 2 * I), "w": torch.rand(R, device="cuda", generator=gen),
             "w_rows": torch.randperm(R, device="cuda", generator=gen).to(torch.int32)}
        if kind == "gated":
            s["out"] = torch.empty(R, I, device="cuda", dtype=torch.bfloat16)
        else:
            s["da"] = bf16(R, I, sigma=0.1)
            s["dh"] = torch.empty(R, 2 * I, device="cuda", dtype=torch.bfloat16)
            s["dw"] = torch.empty(R, device="cuda")
        return s
    if kind in ("to_fp8", "gated_to_fp8"):
        R, K = case["R"], case["K"]
        return {"kind": kind, "x": bf16(R, K if kind == "to_fp8" else 2 * K),
                "q": torch.empty(R, K, device="cuda", dtype=torch.float8_e4m3fn),
                "s": torch.empty(R, -(-K // 128), device="cuda")}

    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    R, side = T * k, case["side"]
    ids = _routing(gen, T, k, E, case["skew"])
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    # the plan of the plain form: the experts with rows, and each row's place
    # in a batch of as many rows for each of them
    live = counts.nonzero().reshape(-1)
    cap = int(counts.max())
    number = torch.zeros(E, dtype=torch.int64, device="cuda")
    number[live] = torch.arange(live.numel(), device="cuda")
    by_row = flat[order]
    slot = number[by_row] * cap + torch.arange(R, device="cuda") - offsets[by_row]
    s = {"kind": kind, "k": k, "R": R, "side": side, "ids": ids, "order": order, "live": live,
         "cap": cap, "slot": slot, "offsets": offsets.to(torch.int32),
         "pair": order.to(torch.int32)}
    if kind == "product_fp8":
        s["w"], s["ws"] = _fp8_weights(gen, E, N, K)
        kb = -(-K // 128)
        x = torch.zeros(T if side == "in" else R, kb * 128, device="cuda")
        x[:, :K] = torch.randn(x.shape[0], K, device="cuda", generator=gen)
        x = x.view(-1, kb, 128)
        s["xs"] = (x.abs().amax(dim=2) / 448.0).contiguous()
        x = (x / s["xs"][:, :, None]).clamp_(-448, 448).view(-1, kb * 128)
        s["x"] = x[:, :K].to(torch.float8_e4m3fn).contiguous()
    else:
        s["w"] = bf16(E, N, K, sigma=0.02)
        s["x"] = bf16(T if side == "in" else R, K)
    if kind == "gradients":
        s["dy"] = bf16(R if side == "in" else T, N, sigma=0.1)
        s["dx"] = torch.empty(R, K, device="cuda", dtype=torch.bfloat16)
        s["dw"] = torch.empty(E, N, K, device="cuda")
    else:
        s["y"] = torch.empty(R, N, device="cuda", dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------ plain form ----

def _batched(s, rows):
    """Sorted rows [R, n] in a batch [experts with rows, cap, n], zeros behind each."""
    b = torch.zeros(s["live"].numel() * s["cap"], rows.shape[1], device=rows.device)
    b[s["slot"]] = rows
    return b.view(s["live"].numel(), s["cap"], rows.shape[1])


def _flat(s, batch):
    return batch.reshape(-1, batch.shape[2])[s["slot"]]


def _pair_order(s, rows):
    out = torch.empty_like(rows)
    out[s["order"]] = rows
    return out


def _per_128(scale, n, dim):
    return scale.repeat_interleave(128, dim).narrow(dim, 0, n)


def _plain_product(s):
    token = s["order"] // s["k"]
    if s["kind"] == "product_fp8":
        x = s["x"].float() * _per_128(s["xs"], s["x"].shape[1], 1)
        w = s["w"][s["live"]].float()
        ws = _per_128(s["ws"][s["live"]], w.shape[1], 1)
        w = w * _per_128(ws, w.shape[2], 2)
    else:
        x, w = s["x"].float(), s["w"][s["live"]].float()
    x = x[token] if s["side"] == "in" else x
    y = torch.bmm(w, _batched(s, x).transpose(1, 2).contiguous()).transpose(1, 2)
    y = _flat(s, y)
    return (y if s["side"] == "in" else _pair_order(s, y)).to(torch.bfloat16)


def _plain_gradients(s):
    token = s["order"] // s["k"]
    x, dy = s["x"].float(), s["dy"].float()
    x, dy = (x[token], dy) if s["side"] == "in" else (x, dy[token])
    dyb, xb = _batched(s, dy), _batched(s, x)
    dx = _flat(s, torch.bmm(dyb, s["w"][s["live"]].float()))
    dx = _pair_order(s, dx) if s["side"] == "in" else dx
    dw = torch.zeros(s["w"].shape, device=x.device)
    dw[s["live"]] = torch.bmm(dyb.transpose(1, 2).contiguous(), xb)
    return dx.to(torch.bfloat16), dw


def _plain_gated(s):
    g, u = s["h"].float().chunk(2, dim=1)
    w = s["w"][s["w_rows"].long()][:, None]
    sig = 1.0 / (1.0 + torch.exp(-g))
    if s["kind"] == "gated":
        return (w * (g * sig * u)).to(torch.bfloat16)
    da = s["da"].float()
    dg = w * da * u * (sig * (1.0 + g * (1.0 - sig)))
    du = w * da * (g * sig)
    dw = torch.empty_like(s["w"])
    dw[s["w_rows"].long()] = (da * (g * sig * u)).sum(1)
    return torch.cat((dg, du), 1).to(torch.bfloat16), dw


def _plain_to_fp8(s):
    x = s["x"].float()
    if s["kind"] == "gated_to_fp8":
        g, u = x.chunk(2, dim=1)
        x = g / (1.0 + torch.exp(-g)) * u
    R, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 128)).view(R, -1, 128)
    scale = x.abs().amax(2).clamp(min=_MIN_AMAX) / 448.0
    q = (x / scale[:, :, None]).clamp(-448, 448).view(R, -1)[:, :K]
    return q.to(torch.float8_e4m3fn), scale


# ------------------------------------------------------------ the kernels ---

def _own(s):
    from mixture_experts_gate_amd import products as P

    kind = s["kind"]
    if kind == "gated":
        return P.swiglu(s["h"], w=s["w"], w_rows=s["w_rows"], out=s["out"])
    if kind == "gated_gradients":
        return P.swiglu_grad(s["h"], s["da"], w=s["w"], w_rows=s["w_rows"], dh=s["dh"], dw=s["dw"])
    if kind == "to_fp8":
        return P.quant_fp8(s["x"], q=s["q"], s=s["s"])
    if kind == "gated_to_fp8":
        return P.swiglu_quant_fp8(s["x"], q=s["q"], s=s["s"])
    pair, k, inner = s["pair"], s["k"], s["side"] == "in"
    if kind == "gradients":
        dy_rows, dy_div, x_rows, x_div = (None, 1, pair, k) if inner else (pair, k, None, 1)
        P.grouped_matmul_dx(s["dy"], s["w"], s["offsets"], rows=dy_rows, div=dy_div,
                            out_rows=pair if inner else None, out=s["dx"])
        P.grouped_matmul_dw(s["dy"], s["x"], s["offsets"], dy_rows=dy_rows, dy_div=dy_div,
                            x_rows=x_rows, x_div=x_div, out=s["dw"])
        return s["dx"], s["dw"]
    at = {"rows": pair, "div": k} if inner else {"out_rows": pair}
    if kind == "product_fp8":
        return P.grouped_matmul_fp8(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], out=s["y"], **at)
    return P.grouped_matmul(s["x"], s["w"], s["offsets"], out=s["y"], **at)


def run(state):
    if own:
        return _own(state)
    kind = state["kind"]
    if kind in ("gated", "gated_gradients"):
        return _plain_gated(state)
    if kind in ("to_fp8", "gated_to_fp8"):
        return _plain_to_fp8(state)
    return _plain_gradients(state) if kind == "gradients" else _plain_product(state)


# --------------------------------------------------------- 64-bit values ----

def _e4m3(v):
    """float64 values rounded to E4M3: 3 mantissa bits, half to even, from 2^-9 up to 448."""
    e = torch.frexp(v).exponent - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind in ("gated", "gated_gradients"):
        I = s["h"].shape[1] // 2
        g, u = s["h"][:, :I].double(), s["h"][:, I:].double()
        at = s["w_rows"].long()
        w = s["w"].double()[at].unsqueeze(1)
        act = torch.sigmoid(g) * g
        if kind == "gated":
            return w * act * u
        da = s["da"].double()
        p = torch.sigmoid(g)
        dh = torch.cat((da * w * u * (p + act * (1 - p)), da * w * act), 1)
        dw = torch.zeros(w.shape[0], dtype=torch.float64, device=w.device)
        return dh, dw.index_copy(0, at, (da * act * u).sum(1))
    if kind in ("to_fp8", "gated_to_fp8"):
        x = s["x"].double()
        if kind == "gated_to_fp8":
            K = x.shape[1] // 2
            x = torch.sigmoid(x[:, :K]) * x[:, :K] * x[:, K:]
        q, scale = torch.empty_like(x), []
        for c in range(0, x.shape[1], 128):
            b = x[:, c:c + 128]
            top = torch.clamp(b.abs().max(dim=1, keepdim=True).values, min=_MIN_AMAX) / 448
            q[:, c:c + 128] = _e4m3(b / top)
            scale.append(top)
        return q, torch.cat(scale, 1)
    flat = s["ids"].reshape(-1)
    R, k, side = flat.numel(), s["k"], s["side"]
    E, N, K = s["w"].shape
    pairs = [(flat == e).nonzero().reshape(-1) for e in range(E)]
    dx_or_y = torch.zeros(R, K if kind == "gradients" else N, dtype=torch.float64, device="cuda")
    dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda") if kind == "gradients" else None
    first = 0
    for e in range(E):
        p, n = pairs[e], pairs[e].numel()
        if n == 0:
            continue
        here = torch.arange(first, first + n, device="cuda")      # sorted order
        first += n
        w = s["w"][e].double()
        x = s["x"][p // k if side == "in" else here].double()
        if kind == "product_fp8":
            xs = s["xs"][p // k if side == "in" else here].double()
            y = torch.zeros(n, N, dtype=torch.float64, device="cuda")
            for b in range(xs.shape[1]):
                cols = slice(128 * b, min(128 * b + 128, K))
                part = x[:, cols] @ w[:, cols].t().contiguous()
                scale = s["ws"][e, :, b].double().repeat_interleave(128)[:N]
                y += part * xs[:, b:b + 1] * scale
            dx_or_y[here if side == "in" else p] = y
        elif kind == "product":
            dx_or_y[here if side == "in" else p] = x @ w.t().contiguous()
        else:
            dy = s["dy"][here if side == "in" else p // k].double()
            dx_or_y[p if side == "in" else here] = dy @ w
            dw[e] = dy.t().contiguous() @ x
    return (dx_or_y, dw) if kind == "gradients" else dx_or_y
