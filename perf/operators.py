"""Cases of the norm operators and of the 8-bit block-scaled product: their inputs, their plain
forms in elementary torch operations, their definitions in 64 bits, and the calls a user makes.

Operators (``case["op"]``):

* ``norm_forward``   y = ((x - mu) * r) * w + b per row, RMS (mu = 0) or layer kind
* ``norm_backward``  dx, dw, db of the same, the statistics taken from x again
* ``quantize``       e4m3 codes with one fp32 scale per 128 elements of a row (``act``), per 128
                     elements of a column with the codes transposed (``act_both`` does both), or
                     per 128 x 128 block with the transposed codes beside them (``weights``)
* ``product``        y = x w^T from codes (1 x 128 scales for x, 128 x 128 for w)
* ``grad_input``     dx = dy w,      ``grad_weight``  dw = dy^T x, from codes as well

Code matrices have their rows padded with zeros to a multiple of 16 bytes; scales of rows are kept
as [groups, rows], scales of blocks as [row blocks, column blocks].
"""
import math

import torch

own = False

TOP = 448.0  # largest finite e4m3 value


def listed():
    return [
        # decode step of the 3B-shaped layer: 16 tokens in front of the projections (latency)
        {"name": "rms forward, 16 tokens", "op": "norm_forward", "M": 16, "K": 3200, "kind": "rms", "bias": False, "x": "bf16", "y": "bf16"},
        # prefill of the 70B-shaped layer, layer norm with a bias
        {"name": "layer forward, prefill", "op": "norm_forward", "M": 8192, "K": 8192, "kind": "layer", "bias": True, "x": "bf16", "y": "bf16"},
        # fp32 training of a small model with a ragged width
        {"name": "layer backward, ragged fp32", "op": "norm_backward", "M": 2049, "K": 1537, "kind": "layer", "bias": True, "x": "f32", "dy": "f32", "dx": "f32"},
        # norm in front of the 3B-shaped down projection: bf16 activations, fp32 gradient of the product
        {"name": "rms backward, training", "op": "norm_backward", "M": 8192, "K": 8640, "kind": "rms", "bias": False, "x": "bf16", "dy": "f32", "dx": "f32"},
        # activations of one decode step (latency)
        {"name": "quantise tokens, decode", "op": "quantize", "what": "act", "M": 16, "K": 8192, "x": "bf16"},
        # fp32 gradient quantised along both axes for the two gradient products
        {"name": "quantise gradient, both ways", "op": "quantize", "what": "act_both", "M": 8192, "K": 3200, "x": "f32"},
        # the largest projection of the 70B-shaped layer, prepared for training
        {"name": "quantise weights, 70B up", "op": "quantize", "what": "weights", "M": 28672, "K": 8192, "x": "f32"},
        # one token through that projection (bound by the weights' bytes)
        {"name": "product, one token", "op": "product", "M": 1, "N": 28672, "K": 8192, "y": "bf16"},
        # a small ragged batch through a ragged head
        {"name": "product, ragged batch", "op": "product", "M": 77, "N": 4099, "K": 1543, "y": "f32"},
        # prefill of the 3B-shaped up projection (bound by the tensor cores)
        {"name": "product, prefill", "op": "product", "M": 8192, "N": 8640, "K": 3200, "y": "bf16"},
        # training of the 700M-shaped up projection, 4096 tokens, its two gradients
        {"name": "input gradient", "op": "grad_input", "M": 4096, "N": 4096, "K": 1536, "y": "f32"},
        {"name": "weight gradient", "op": "grad_weight", "M": 4096, "N": 4096, "K": 1536, "y": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A size over the logarithm of the range: a multiple of 64, of 8, or any."""
    n = _log(rng, lo, hi)
    step = rng.choice([64, 8, 1])
    return max(lo, n // step * step)


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "quantize", "product", "grad_input", "grad_weight"])
    t = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op in ("norm_forward", "norm_backward"):
        K = _width(rng, 256, 16384)
        M = _log(rng, 1, min(8192, 67_000_000 // K))
        c = {"op": op, "M": M, "K": K, "kind": rng.choice(["rms", "layer"]), "bias": rng.random() < 0.5, "x": t()}
        return {**c, "y": t()} if op == "norm_forward" else {**c, "dy": t(), "dx": t()}
    if op == "quantize":
        what = rng.choice(["act", "act_both", "weights"])
        K = _width(rng, 256, 28672)
        M = _log(rng, 1, min(8192, 134_000_000 // K)) if what != "weights" else _width(rng, 256, min(28672, 234_000_000 // K))
        return {"op": op, "what": what, "M": M, "K": K, "x": t()}
    N, K = _width(rng, 256, 28672), _width(rng, 256, 8192)
    M = _log(rng, 1, min(8192, 220_000_000_000 // (N * K)))
    return {"op": op, "M": M, "N": N, "K": K, "y": t()}


_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_B = {"bf16": 2, "f32": 4}


def _up(n, to):
    return -(-n // to) * to


def _groups(n):
    return -(-n // 128)


# ------------------------------------------------------------------------------- inputs --

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _acts(gen, M, K):
    """Activations with outlier channels: N(0, 1), 1% of the channels times 20."""
    x = _normal(gen, M, K)
    out = torch.rand(K, generator=gen, device="cuda") < 0.01
    return x * torch.where(out, 20.0, 1.0)


def _grads(gen, M, K):
    """Output gradients: small, with rows of very different sizes."""
    return _normal(gen, M, K) * (1e-3 * torch.exp(_normal(gen, M, 1)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    s = {"case": case}
    if op in ("norm_forward", "norm_backward"):
        s["x"] = _acts(gen, M, K).to(_T[case["x"]])
        s["w"] = 1.0 + 0.1 * _normal(gen, K)
        s["b"] = 0.1 * _normal(gen, K) if case["bias"] else None
        if op == "norm_backward":
            s["dy"] = _grads(gen, M, K).to(_T[case["dy"]])
    elif op == "quantize":
        x = 0.02 * _normal(gen, M, K) if case["what"] == "weights" else _grads(gen, M, K) if case["what"] == "act_both" else _acts(gen, M, K)
        s["x"] = x.to(_T[case["x"]])
    else:
        N = case["N"]
        if op == "product":
            s["a"], s["sa"] = _quant_rows(_acts(gen, M, K))
            s["b"], s["sb"], _ = _quant_blocks(0.02 * _normal(gen, N, K))
        elif op == "grad_input":
            s["a"], s["sa"] = _quant_rows(_grads(gen, M, N))
            _, s["sb"], s["b"] = _quant_blocks(0.02 * _normal(gen, N, K))
        else:
            s["a"], s["sa"] = _quant_rows(_grads(gen, M, N).t())
            s["b"], s["sb"] = _quant_rows(_acts(gen, M, K).t())
    return s


# --------------------------------------------------------------------------- plain forms --

_EPS = {"act": 1e-5, "act_both": 1e-12, "weights": 1e-5}


def _codes(x, ratio):
    """x * ratio in e4m3, its rows padded with zeros to a multiple of 16."""
    q = torch.zeros(x.shape[0], _up(x.shape[1], 16), device=x.device, dtype=torch.float32)
    q[:, :x.shape[1]] = x * ratio
    return q.to(torch.float8_e4m3fn)


def _quant_rows(x, eps=1e-12):
    """One scale per 128 elements of a row: codes [rows, padded], scales [groups, rows]."""
    x = x.float()
    R, C = x.shape
    G = _groups(C)
    a = torch.zeros(R, G * 128, device=x.device)
    a[:, :C] = x.abs()
    a = a.view(R, G, 128).amax(2).clamp(min=eps)
    return _codes(x, (TOP / a).repeat_interleave(128, 1)[:, :C]), (a / TOP).t().contiguous()


def _quant_blocks(w, eps=1e-5):
    """One scale per 128 x 128 block: codes, scales, and the codes transposed."""
    w = w.float()
    R, C = w.shape
    a = torch.zeros(_groups(R) * 128, _groups(C) * 128, device=w.device)
    a[:R, :C] = w.abs()
    a = a.view(_groups(R), 128, _groups(C), 128).amax((1, 3)).clamp(min=eps)
    ratio = (TOP / a).repeat_interleave(128, 0)[:R].repeat_interleave(128, 1)[:, :C]
    return _codes(w, ratio), a / TOP, _codes(w.t(), ratio.t())


def _real_rows(q, scales, n):
    return q[:, :n].float() * scales.t().repeat_interleave(128, 1)[:, :n]


def _real_blocks(q, scales, n):
    return q[:, :n].float() * scales.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :n]


def _plain_norm(s, eps=1e-5):
    x = s["x"].float()
    mu = x.mean(1, keepdim=True) if s["case"]["kind"] == "layer" else 0.0
    r = 1.0 / torch.sqrt((x - mu).square().mean(1, keepdim=True) + eps)
    return (x - mu) * r, r


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm_forward":
        y = _plain_norm(s)[0] * s["w"]
        return (y + s["b"] if c["bias"] else y).to(_T[c["y"]])
    if op == "norm_backward":
        xh, r = _plain_norm(s)
        dy = s["dy"].float()
        g = dy * s["w"]
        dx = g - xh * (g * xh).mean(1, keepdim=True)
        if c["kind"] == "layer":
            dx = dx - g.mean(1, keepdim=True)
        out = {"dx": (dx * r).to(_T[c["dx"]]), "dw": (dy * xh).sum(0)}
        return {**out, "db": dy.sum(0)} if c["bias"] else out
    if op == "quantize":
        eps = _EPS[c["what"]]
        if c["what"] == "weights":
            return _quant_blocks(s["x"], eps)
        rows = _quant_rows(s["x"], eps)
        return rows if c["what"] == "act" else rows + _quant_rows(s["x"].t(), eps)
    if op == "product":
        y = _real_rows(s["a"], s["sa"], c["K"]) @ _real_blocks(s["b"], s["sb"], c["K"]).t()
    elif op == "grad_input":
        y = _real_rows(s["a"], s["sa"], c["N"]) @ _real_blocks(s["b"], s["sb"].t(), c["N"]).t()
    else:
        y = _real_rows(s["a"], s["sa"], c["M"]) @ _real_rows(s["b"], s["sb"], c["M"]).t()
    return y.to(_T[c["y"]])


# ------------------------------------------------------------------- the framework's calls --

def _calls(s):
    import ternary_weight_bit_absmean_b200 as bl
    c = s["case"]
    op = c["op"]
    if op in ("norm_forward", "norm_backward"):
        kind = bl.BL_NORM_LAYER if c["kind"] == "layer" else bl.BL_NORM_RMS
        if op == "norm_forward":
            return bl.norm_forward(s["x"], s["w"], s["b"], kind=kind, out_dtype=_T[c["y"]])
        dx, dw, db = bl.norm_backward(s["dy"], s["x"], s["w"], kind=kind, bias=c["bias"], dx_dtype=_T[c["dx"]])
        return {"dx": dx, "dw": dw, "db": db} if c["bias"] else {"dx": dx, "dw": dw}
    if op == "quantize":
        eps = _EPS[c["what"]]
        if c["what"] == "weights":
            return bl.fp8_quantize_weights(s["x"], eps, transposed=True)
        return bl.fp8_quantize_act(s["x"], eps, transposed=c["what"] == "act_both")
    call = {"product": bl.fp8_forward, "grad_input": bl.fp8_backward_input, "grad_weight": bl.fp8_backward_weight}[op]
    return call(s["a"], s["sa"], s["b"], s["sb"], out_dtype=_T[c["y"]])


def run(state):
    if own:
        return _calls(state)
    return _plain(state)


# ---------------------------------------------------------------------------------- work --

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "norm_forward":
        return {"bytes": M * K * (_B[case["x"]] + _B[case["y"]]) + 4 * K * (1 + case["bias"]), "flops": 8 * M * K}
    if op == "norm_backward":
        return {"bytes": M * K * (_B[case["x"]] + _B[case["dy"]] + _B[case["dx"]]) + 4 * K * (2 + case["bias"]), "flops": 16 * M * K}
    if op == "quantize":
        w = case["what"]
        scales = _groups(M) * _groups(K) if w == "weights" else M * _groups(K) + (K * _groups(M) if w == "act_both" else 0)
        return {"bytes": M * K * (_B[case["x"]] + (1 if w == "act" else 2)) + 4 * scales, "flops": 3 * M * K}
    N = case["N"]
    ins = {"product": (M * K, N * K), "grad_input": (M * N, N * K), "grad_weight": (M * N, M * K)}[op]
    out = {"product": M * N, "grad_input": M * K, "grad_weight": N * K}[op]
    return {"bytes": sum(ins) * (1 + 1 / 32) + out * _B[case["y"]], "flops": 2 * M * N * K}


# ----------------------------------------------------------------- definitions in 64 bits --

def _e4m3(v):
    """The nearest e4m3 value, ties to the even one: three fraction bits, smallest exponent -6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _exact_quant(x, rows, cols, eps):
    """Codes and scales of blocks of rows x cols, block by block."""
    R, C = x.shape
    q = torch.zeros(R, _up(C, 16), dtype=torch.float64, device=x.device)
    d = torch.empty(-(-R // rows), -(-C // cols), dtype=torch.float64, device=x.device)
    for j in range(d.shape[1]):
        part = x[:, j * cols:(j + 1) * cols]
        top = part.abs().max(1).values
        if rows > 1:
            top = torch.nn.functional.pad(top, (0, d.shape[0] * rows - R)).view(-1, rows).max(1).values
        top = torch.where(top > eps, top, torch.full_like(top, eps))
        d[:, j] = top / TOP
        q[:, j * cols:j * cols + part.shape[1]] = _e4m3(part * (TOP / top).repeat_interleave(rows)[:R, None])
    return q, d


def _exact_product(a, sa, b, sb):
    """sum over groups g of sa[g, i] sb(g)[j] (a_g b_g^T), one group at a time."""
    y = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for g in range(sa.shape[0]):
        cols = slice(128 * g, 128 * g + 128)
        y += (a[:, cols].double() * sa[g, :, None].double()) @ (b[:, cols].double() * sb(g)[:, None].double()).t()
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm_forward", "norm_backward"):
        x, w = s["x"].double(), s["w"].double()
        K = x.shape[1]
        if case["kind"] == "layer":
            x = x - x.sum(1, keepdim=True) / K
        rstd = torch.rsqrt((x * x).sum(1, keepdim=True) / K + 1e-5)
        n = x * rstd
        if op == "norm_forward":
            return n * w + (s["b"].double() if case["bias"] else 0.0)
        dy = s["dy"].double()
        g = dy * w
        # the Jacobian of n = x rstd applied to g, row by row
        dx = rstd * g - rstd * n * ((g * n).sum(1, keepdim=True) / K)
        if case["kind"] == "layer":
            dx = dx - rstd * (g.sum(1, keepdim=True) / K)
        out = {"dx": dx, "dw": torch.einsum("mk,mk->k", dy, n)}
        return {**out, "db": torch.einsum("mk->k", dy)} if case["bias"] else out
    if op == "quantize":
        x, eps = s["x"].double(), _EPS[case["what"]]
        if case["what"] == "weights":
            q, d = _exact_quant(x, 128, 128, eps)
            t = torch.zeros(x.shape[1], _up(x.shape[0], 16), dtype=torch.float64, device=x.device)
            t[:, :x.shape[0]] = q[:, :x.shape[1]].t()
            return q, d, t
        q, d = _exact_quant(x, 1, 128, eps)
        if case["what"] == "act":
            return q, d.t().contiguous()
        q2, d2 = _exact_quant(x.t().contiguous(), 1, 128, eps)
        return q, d.t().contiguous(), q2, d2.t().contiguous()
    a, sa, b, sb = s["a"], s["sa"], s["b"], s["sb"]
    rows = b.shape[0]
    if op == "product":
        return _exact_product(a, sa, b, lambda g: sb[:, g].repeat_interleave(128)[:rows])
    if op == "grad_input":
        return _exact_product(a, sa, b, lambda g: sb[g].repeat_interleave(128)[:rows])
    return _exact_product(a, sa, b, lambda g: sb[g])
