"""The dense feed-forward operators, as a program calls them: per-row int8
quantisation, the int8 matrix product with token and channel scales, the gated
feed-forward block in int8 for serving, and the 16-bit gated block with its
backward pass for training.

Each case is one pass through one operator.  `run` computes it from elementary
torch operations, or, where `own` is true, through fp8_moe_layer_amd.  Layer
sizes are those of this repository's workloads: Mixtral-shaped (d 4096,
f 14336), Qwen3-shaped (2048, 768), DeepSeek-shaped (2048, 1408),
MoE-Prism-shaped (2048, 192) and the tiny layer (256, 512).
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}

# the largest pass, in multiply-add operations: the Mixtral-shaped training step
_MAX_FLOPS = 12 * 4096 * 4096 * 14336


def listed():
    return [
        # the rows of one decode step on their way into an int8 product
        dict(name="quantize_decode", op="quantize", T=9, d=4096, x="bf16"),
        # the intermediate rows of a ragged prefill batch, before the down projection
        dict(name="quantize_prefill", op="quantize", T=8191, d=14336, x="bf16"),
        # the fp32 activations that the layer itself works on
        dict(name="quantize_f32", op="quantize", T=4096, d=2048, x="f32"),
        # down projection of a single token
        dict(name="matmul_token", op="matmul", T=1, d=14336, n=4096, y="bf16", bias=False),
        # a ragged mixed batch into an odd number of outputs, with a bias
        dict(name="matmul_ragged", op="matmul", T=333, d=1408, n=2051, y="f32", bias=True),
        # down projection of a prefill batch
        dict(name="matmul_prefill", op="matmul", T=8192, d=14336, n=4096, y="bf16", bias=False),
        # both projections of a decode batch
        dict(name="gated_i8_decode", op="gated_i8", T=16, d=4096, f=14336, y="bf16"),
        # both projections of a ragged prefill batch of narrow layers
        dict(name="gated_i8_prefill", op="gated_i8", T=4099, d=2048, f=1408, y="f16"),
        # the unquantised block on a single token
        dict(name="gated_token", op="gated", T=1, d=2048, f=1408, x="f16"),
        # the unquantised block on a prefill batch
        dict(name="gated_prefill", op="gated", T=8192, d=4096, f=14336, x="bf16"),
        # a training step of a narrow layer, an odd number of tokens
        dict(name="train_narrow", op="train", T=2047, d=2048, f=768, x="f16"),
        # a training step of a wide layer
        dict(name="train_wide", op="train", T=4096, d=4096, f=14336, x="bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    while True:
        op = rng.choice(["quantize", "matmul", "matmul", "gated_i8", "gated", "train", "train"])
        case = dict(op=op, T=_log_int(rng, 1, 8192))
        if op == "quantize":
            case.update(d=_log_int(rng, 64, 16384, 16), x=rng.choice(["f32", "bf16", "f16"]))
        elif op == "matmul":
            case.update(d=_log_int(rng, 192, 16384, 16), n=_log_int(rng, 256, 16384),
                        y=rng.choice(["f32", "bf16", "f16"]), bias=rng.random() < 0.5)
        else:
            case.update(d=_log_int(rng, 256, 8192, 64), f=_log_int(rng, 192, 16384, 64))
            case.update({"gated_i8": dict(y=rng.choice(["f32", "bf16", "f16"]))}.get(
                op, dict(x=rng.choice(["bf16", "f16"]))))
        if work(case)["flops"] <= _MAX_FLOPS:
            return case


# ---------------------------------------------------------------------- inputs

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    x = torch.empty(shape, dtype=torch.float32, device=g.device)
    return x.normal_(0.0, std, generator=g).to(dtype)


def _tokens(g, T, d, dtype):
    """Hidden states: unit rows of uneven magnitude, a few large channels."""
    x = torch.empty((T, d), dtype=torch.float32, device=g.device).normal_(generator=g)
    row = torch.empty((T, 1), dtype=torch.float32, device=g.device).normal_(generator=g)
    x *= torch.exp(0.25 * row)
    x[:, ::max(1, d // 8)] *= 4.0
    return x.to(dtype)


def _codes(x):
    """Rows as a loaded checkpoint has them: int8 codes with a scale each."""
    s = x.abs().amax(1) / 127.0
    return torch.round(x / s[:, None]).to(torch.int8), s


def _inputs(case, seed):
    g = _gen(seed, torch.device("cuda", torch.cuda.current_device()))
    op, T, d = case["op"], case["T"], case["d"]
    if op == "quantize":
        return dict(x=_tokens(g, T, d, _DTYPES[case["x"]]))
    if op == "matmul":
        xq, sx = _codes(_tokens(g, T, d, torch.float32))
        wq, sw = _codes(_normal(g, (case["n"], d), d ** -0.5, torch.float32))
        bias = _normal(g, (case["n"],), 0.5, torch.float32) if case["bias"] else None
        return dict(xq=xq, sx=sx, wq=wq, sw=sw, bias=bias)
    f = case["f"]
    if op == "gated_i8":
        xq, sx = _codes(_tokens(g, T, d, torch.float32))
        wg, sg = _codes(_normal(g, (f, d), d ** -0.5, torch.float32))
        wu, su = _codes(_normal(g, (f, d), d ** -0.5, torch.float32))
        return dict(xq=xq, sx=sx, wg=wg, sg=sg, wu=wu, su=su)
    dtype = _DTYPES[case["x"]]
    out = dict(x=_tokens(g, T, d, dtype), wg=_normal(g, (f, d), d ** -0.5, dtype),
               wu=_normal(g, (f, d), d ** -0.5, dtype))
    if op == "train":
        out["dh"] = _normal(g, (T, f), 0.25, dtype)
    return out


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import fp8_moe_layer_amd
        state["lib"] = fp8_moe_layer_amd
    return state


# ---------------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    case, lib = s["case"], s["lib"]
    op = case["op"]
    if op == "quantize":
        q, scale = lib.quantize_rows_i8(s["x"])
        return q * scale[:, None], scale  # the values that the codes stand for
    if op == "matmul":
        return lib.matmul_i8(s["xq"], s["sx"], s["wq"], s["sw"], bias=s["bias"],
                             out_dtype=_DTYPES[case["y"]])
    if op == "gated_i8":
        return lib.gated_ffn_i8(s["xq"], s["sx"], s["wg"], s["sg"], s["wu"], s["su"],
                                out_dtype=_DTYPES[case["y"]])
    if op == "gated":
        return lib.gated_ffn(s["x"], s["wg"], s["wu"])
    h, g, u = lib.gated_ffn(s["x"], s["wg"], s["wu"], save=True)
    dx, dwg, dwu = lib.gated_ffn_backward(s["dh"], s["x"], s["wg"], s["wu"], g, u)
    return h, dx, dwg, dwu


def _product_i8(xq, sx, wq, sw):
    # the integer sums pass 24 bits: 64-bit floating point holds them
    acc = (xq.double() @ wq.double().t()).float()
    return acc * sx[:, None] * sw


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        x = s["x"].float()
        amax = x.abs().amax(1)
        m = amax.clamp_min(2.0 ** -100)
        top = torch.full_like(m, 127.0)  # both divided as tensors: a number's inverse is rounded first
        r = top / m
        scale = torch.where(amax == 0, torch.ones_like(amax), m / top)
        # rounded from the product in 64 bits: values next to a border between two codes
        q = torch.round(x.double() * r.double()[:, None]).float()
        return q * scale[:, None], scale
    if op == "matmul":
        y = _product_i8(s["xq"], s["sx"], s["wq"], s["sw"])
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(_DTYPES[case["y"]])
    if op == "gated_i8":
        g = _product_i8(s["xq"], s["sx"], s["wg"], s["sg"])
        u = _product_i8(s["xq"], s["sx"], s["wu"], s["su"])
        return (g / (1.0 + torch.exp(-g)) * u).to(_DTYPES[case["y"]])
    dtype = s["x"].dtype
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    sig = 1.0 / (1.0 + torch.exp(-g))
    h = (g * sig * u).to(dtype)
    if op == "gated":
        return h
    dh = s["dh"].float()
    dg = dh * u * sig * (1.0 + g * (1.0 - sig))
    du = dh * g * sig
    dx = dg @ wg + du @ wu
    return h, dx.to(dtype), (dg.t() @ x).to(dtype), (du.t() @ x).to(dtype)


# ---------------------------------------------------------------------- the definition, in 64 bits

def _silu64(g):
    return g * torch.sigmoid(g)


def exact(case, seed):
    s = {k: v for k, v in _inputs(case, seed).items() if v is not None}
    f64 = {k: v.to(torch.float64) for k, v in s.items()}
    op = case["op"]
    if op == "quantize":
        x = f64["x"]
        top = x.abs().max(dim=1, keepdim=True).values
        # the reciprocal scale is a 32-bit number by definition; the rest is not
        step = torch.maximum(top, torch.full_like(top, 2.0 ** -100))
        codes = torch.round(x * (127.0 / step).float().double())
        scale = torch.where(top == 0, torch.ones_like(top), step / 127.0)
        return codes * scale, scale[:, 0]
    if op == "matmul":
        y = torch.mm(f64["xq"] * f64["sx"].unsqueeze(1), (f64["wq"] * f64["sw"].unsqueeze(1)).T)
        return y + f64["bias"].unsqueeze(0) if "bias" in f64 else y
    if op == "gated_i8":
        x = f64["xq"] * f64["sx"].unsqueeze(1)
        g = torch.mm(x, (f64["wg"] * f64["sg"].unsqueeze(1)).T)
        return _silu64(g) * torch.mm(x, (f64["wu"] * f64["su"].unsqueeze(1)).T)
    x, wg, wu = f64["x"], f64["wg"], f64["wu"]
    g, u = torch.mm(x, wg.T), torch.mm(x, wu.T)
    h = _silu64(g) * u
    if op == "gated":
        return h
    p = torch.sigmoid(g)
    up_grad = f64["dh"] * _silu64(g)
    gate_grad = f64["dh"] * u * (p + _silu64(g) * (1.0 - p))
    dx = torch.mm(torch.cat([gate_grad, up_grad], 1), torch.cat([wg, wu], 0))
    return h, dx, torch.mm(gate_grad.T, x), torch.mm(up_grad.T, x)


# ---------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, T, d = case["op"], case["T"], case["d"]
    if op == "quantize":
        # the codes are one byte each; a few operations a value
        return dict(bytes=T * d * (_BYTES[case["x"]] + 1) + 4 * T, flops=4 * T * d)
    if op == "matmul":
        n = case["n"]
        return dict(bytes=T * d + n * d + 4 * (T + n) + (4 * n if case["bias"] else 0)
                    + T * n * _BYTES[case["y"]], flops=2 * T * d * n)
    f = case["f"]
    if op == "gated_i8":
        return dict(bytes=T * d + 2 * f * d + 4 * (T + 2 * f) + T * f * _BYTES[case["y"]],
                    flops=4 * T * d * f)
    forward = 2 * (T * d + 2 * f * d + T * f)
    if op == "gated":
        return dict(bytes=forward, flops=4 * T * d * f)
    # and dh in, dx and both weight gradients out
    return dict(bytes=forward + 2 * (T * f + T * d + 2 * f * d), flops=12 * T * d * f)
