"""What stands before, in and after a feed-forward block that is served in four
bits or trained in 16: the norms with gate and residual sum, forward and
backward; quantisation to groups of 32 e2m1 codes with a power-of-two scale; the
matrix product and the gated block on such weights; and a whole
mixture-of-experts layer of a few tokens with such experts.

Each case is one pass through one operator.  `run` computes it from elementary
torch operations, or, where `own` is true, through fp8_moe_layer_amd.  Layer
sizes are those of this repository's workloads: Mixtral-shaped (d 4096,
f 14336, 8 experts, 2 a token), Qwen3-shaped (2048, 768, 128, 8) and
DeepSeek-shaped (2048, 1408, 64, 6, two shared experts).
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-6
_GROUP = 32

# the largest passes: the gated block of a prefill batch, and the weights of the
# Mixtral-shaped layer
_MAX_FLOPS = 4 * 8192 * 4096 * 14336
_MAX_VALUES = 3 * 8 * 4096 * 14336


def listed():
    return [
        # between two blocks of one decode step: residual sum, then the next block's norm
        dict(name="norm_decode", op="residual", T=9, d=4096, x="bf16", w="bf16", post=False,
             gate="none", next=True),
        # norms on both sides of a block and a learned gate per channel, a ragged prefill batch
        dict(name="norm_prefill", op="residual", T=8191, d=4096, x="bf16", w="bf16", post=True,
             gate="channel", next=True),
        # a training step of a narrow layer: one gate row to each sequence of 9
        dict(name="norm_train_narrow", op="train", T=333, d=2048, x="f16", w="f32", post=True,
             gate="sequence", next=True),
        # a training step of a wide layer
        dict(name="norm_train_wide", op="train", T=4096, d=4096, x="bf16", w="bf16", post=True,
             gate="channel", next=True),
        # one expert's gate matrix, from the fp32 master weights and back
        dict(name="quantize_expert", op="quantize", rows=768, cols=2048, x="f32", y="f32"),
        # a wide layer's up projection, from a bf16 checkpoint and back
        dict(name="quantize_wide", op="quantize", rows=14336, cols=4096, x="bf16", y="bf16"),
        # down projection of a single token
        dict(name="matmul_token", op="matmul", T=1, d=14336, n=4096, x="bf16", y="bf16", bias=False),
        # a ragged mixed batch into an odd number of outputs, with a bias
        dict(name="matmul_ragged", op="matmul", T=333, d=1408, n=2051, x="f16", y="f32", bias=True),
        # both projections of a decode batch
        dict(name="gated_decode", op="gated", T=16, d=4096, f=14336, x="bf16"),
        # both projections of a prefill batch
        dict(name="gated_prefill", op="gated", T=8192, d=4096, f=14336, x="bf16"),
        # one token through the Qwen3-shaped layer
        dict(name="moe_token", op="moe", T=1, d=2048, f=768, E=128, k=8, shared=0, x="bf16"),
        # an odd decode batch through the DeepSeek-shaped layer
        dict(name="moe_batch", op="moe", T=13, d=2048, f=1408, E=64, k=6, shared=2, x="f16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    while True:
        op = rng.choice(["residual", "train", "train", "quantize", "matmul", "matmul", "gated", "moe",
                         "moe"])
        x = rng.choice(["bf16", "f16"])
        if op in ("residual", "train"):
            x = rng.choice(["f32", "bf16", "f16"])
            case = dict(op=op, T=_log_int(rng, 1, 8192), d=_log_int(rng, 64, 16384, 16), x=x,
                        w=rng.choice(["f32", x]), post=rng.random() < 0.7,
                        gate=rng.choice(["none", "channel", "sequence", "token"]),
                        next=rng.random() < 0.7)
        elif op == "quantize":
            case = dict(op=op, rows=_log_int(rng, 16, 16384), cols=_log_int(rng, 64, 16384, 32),
                        x=rng.choice(["f32", "bf16", "f16"]), y=rng.choice(["f32", "bf16"]))
        elif op == "matmul":
            case = dict(op=op, T=_log_int(rng, 1, 8192), d=_log_int(rng, 192, 16384, 32),
                        n=_log_int(rng, 256, 16384), x=x, y=rng.choice(["f32", x]),
                        bias=rng.random() < 0.5)
        elif op == "gated":
            case = dict(op=op, T=_log_int(rng, 1, 8192), d=_log_int(rng, 256, 8192, 32),
                        f=_log_int(rng, 192, 16384, 32), x=x)
        else:
            E = _log_int(rng, 8, 256)
            case = dict(op=op, T=_log_int(rng, 1, 32), d=_log_int(rng, 256, 4096, 32),
                        f=_log_int(rng, 192, 8192, 32), E=E, k=rng.randint(1, min(8, E)),
                        shared=rng.choice([0, 0, 1, 2]), x=x)
        values = 3 * (case["E"] + case["shared"]) * case["d"] * case["f"] if op == "moe" else 0
        if work(case)["flops"] <= _MAX_FLOPS and values <= _MAX_VALUES:
            return case


# ---------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=torch.device("cuda", torch.cuda.current_device()))
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype, mean=0.0):
    x = torch.empty(shape, dtype=torch.float32, device=g.device)
    return x.normal_(mean, std, generator=g).to(dtype)


def _tokens(g, T, d, dtype):
    """Hidden states: unit rows of uneven magnitude, a few large channels."""
    x = torch.empty((T, d), dtype=torch.float32, device=g.device).normal_(generator=g)
    row = torch.empty((T, 1), dtype=torch.float32, device=g.device).normal_(generator=g)
    x *= torch.exp(0.25 * row)
    x[:, ::max(1, d // 8)] *= 4.0
    return x.to(dtype)


def _checkpoint(g, shape):
    """A matrix as a 4-bit checkpoint has it: two codes a byte, the first in the
    low half, and a scale byte for each 32 of a row."""
    w = _normal(g, shape, shape[-1] ** -0.5, torch.float32).unflatten(-1, (-1, _GROUP))
    e = torch.ceil(torch.log2(w.abs().amax(-1, keepdim=True) / 7.0))
    a = w.abs() * torch.exp2(-e)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(a, borders).to(torch.uint8) | ((w < 0).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e[..., 0] + 127).to(torch.uint8)


def _gate_rows(case):
    T = case["T"]
    return {"none": 0, "channel": 1, "token": T,
            "sequence": next(n for n in range(max(1, T // 9), 0, -1) if T % n == 0)}[case["gate"]]


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("residual", "train"):
        T, d, dtype, wtype = case["T"], case["d"], _DTYPES[case["x"]], _DTYPES[case["w"]]
        rows = _gate_rows(case)
        s = dict(x=_tokens(g, T, d, dtype), y=_normal(g, (T, d), 0.7, dtype))
        s["w_post"] = _normal(g, (d,), 0.2, wtype, 1.0) if case["post"] else None
        s["gate"] = _normal(g, (rows, d), 0.3, wtype, 0.5) if rows else None
        s["w_next"] = _normal(g, (d,), 0.2, wtype, 1.0) if case["next"] else None
        if op == "train":
            s["dr"] = _normal(g, (T, d), 0.25, dtype)
            s["dn"] = _normal(g, (T, d), 0.25, dtype) if case["next"] else None
        return s
    if op == "quantize":
        return dict(x=_normal(g, (case["rows"], case["cols"]), case["cols"] ** -0.5,
                              _DTYPES[case["x"]]))
    T, d, dtype = case["T"], case["d"], _DTYPES[case["x"]]
    s = dict(x=_tokens(g, T, d, dtype))
    if op == "matmul":
        s["w"] = _checkpoint(g, (case["n"], d))
        s["bias"] = _normal(g, (case["n"],), 0.5, torch.float32) if case["bias"] else None
        return s
    f = case["f"]
    if op == "gated":
        s["wg"], s["wu"] = _checkpoint(g, (f, d)), _checkpoint(g, (f, d))
        return s
    s["w_router"] = _normal(g, (case["E"], d), d ** -0.5, torch.float32)
    n = case["E"] + case["shared"]  # the shared experts come last
    experts = [(_checkpoint(g, (f, d)), _checkpoint(g, (f, d)), _checkpoint(g, (d, f)))
               for _ in range(n)]
    for name, m in (("wg", 0), ("wu", 1), ("wd", 2)):
        s[name] = tuple(torch.stack([e[m][part] for e in experts]) for part in (0, 1))
    return s


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import fp8_moe_layer_amd as lib
        state["lib"] = lib
        # weights are laid out once, when they are loaded
        if case["op"] == "moe":
            E, n = case["E"], case["E"] + case["shared"]
            w = lib.Mx4Experts.empty(E, case["d"], case["f"], case["shared"])
            for e in range(n):
                for which, m in (("gate", "wg"), ("up", "wu"), ("down", "wd")):
                    codes, scales = state[m]
                    w.set_expert(which, e if e < E else e - E, codes[e], scales[e], shared=e >= E)
            state["layer"] = lib.Mx4MoELayer(w, state["w_router"], case["k"])
            state["ids"] = torch.empty((case["T"], case["k"]), dtype=torch.int32,
                                       device=state["x"].device)
            for m in ("wg", "wu", "wd"):
                del state[m]
        else:
            for m in ("w", "wg", "wu"):
                if m in state:
                    state[m] = lib.pack_mx4(*state[m])
    return state


# ---------------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    case, lib = s["case"], s["lib"]
    op = case["op"]
    if op == "residual":
        return lib.norm_residual(s["x"], s["y"], s["w_post"], s["gate"], s["w_next"], scale=0.5,
                                 eps=_EPS)
    if op == "train":
        r, n, rstd_y, rstd_r = lib.norm_residual(s["x"], s["y"], s["w_post"], s["gate"], s["w_next"],
                                                 scale=0.5, eps=_EPS, save=True)
        return (r, n) + lib.norm_residual_backward(
            s["dr"], s["dn"], s["x"], s["y"], rstd_y, rstd_r, s["w_post"], s["gate"], s["w_next"],
            scale=0.5)
    if op == "quantize":
        codes, scales = lib.quantize_rows_mx4(s["x"])
        # the values that the codes stand for
        return lib.dequantize_rows_mx4(codes, scales, _DTYPES[case["y"]]), scales
    if op == "matmul":
        return lib.matmul_mx4(s["x"], s["w"], bias=s["bias"], out_dtype=_DTYPES[case["y"]])
    if op == "gated":
        return lib.gated_ffn_mx4(s["x"], s["wg"], s["wu"])
    return s["layer"].forward(s["x"], topk_ids=s["ids"]), s["ids"]


def _values(w):
    """What the codes and scales of a checkpoint stand for."""
    codes, scales = w
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0,
                          -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    pairs = torch.stack([codes & 15, codes >> 4], -1).int()
    v = table[pairs].flatten(-2).unflatten(-1, (-1, _GROUP))
    return (v * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _plain_norm(x):
    rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + _EPS)
    return x * rstd, rstd


def _plain_residual(s):
    case = s["case"]
    dtype = s["x"].dtype
    f32 = {k: v.float() for k, v in s.items() if isinstance(v, torch.Tensor)}
    x, y = f32["x"], f32["y"]
    rep = case["T"] // s["gate"].shape[0] if s["gate"] is not None else 0
    gate = f32["gate"].repeat_interleave(rep, 0) if rep else 1.0
    yh, rstd_y = _plain_norm(y)
    z = yh * f32["w_post"] if case["post"] else y
    r = x + 0.5 * gate * z
    rh, rstd_r = _plain_norm(r)
    n = rh * f32["w_next"] if case["next"] else None
    out = r.to(dtype), None if n is None else n.to(dtype)
    if case["op"] == "residual":
        return out if case["next"] else out[0]
    total, dw_post, dgate, dw_next = f32["dr"], None, None, None
    if case["next"]:
        a = f32["dn"] * f32["w_next"]
        total = total + rstd_r * (a - rh * (a * rh).mean(1, keepdim=True))
        dw_next = (f32["dn"] * rh).sum(0).to(s["w_next"].dtype)
    e = 0.5 * total
    if rep:
        dgate = (e * z).unflatten(0, (-1, rep)).sum(1).to(s["gate"].dtype)
    c = e * gate
    dy = c
    if case["post"]:
        b = c * f32["w_post"]
        dy = rstd_y * (b - yh * (b * yh).mean(1, keepdim=True))
        dw_post = (c * yh).sum(0).to(s["w_post"].dtype)
    return out + (total.to(dtype), dy.to(dtype), dw_post, dgate, dw_next)


def _plain_quantize(x, dtype):
    v = x.float().unflatten(1, (-1, _GROUP))
    amax = v.abs().amax(2, keepdim=True)
    # the smallest power of two of which the largest value is at most seven
    e = torch.floor(torch.log2(amax.clamp_min(2.0 ** -120))) - 2.0
    e = torch.where(amax > 7.0 * torch.exp2(e), e + 1.0, e)
    e = torch.where(amax <= 3.5 * torch.exp2(e), e - 1.0, e)  # log2 rounded up
    e = torch.where(amax == 0, torch.zeros_like(e), e.clamp_min(-126.0))
    a = v.abs() * torch.exp2(-e)
    # e2m1 has steps of 1/2 up to 2, 1 up to 4, then 2; to nearest, ties to even
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp_max(6.0) * torch.sign(v)
    return (q * torch.exp2(e)).flatten(1).to(dtype), (e[..., 0] + 127.0).to(torch.uint8)


def _plain_moe(s):
    case = s["case"]
    T, E, k = case["T"], case["E"], case["k"]
    x = s["x"].float()
    # logits in 64 bits: two experts may be next to each other
    logits = (s["x"].double() @ s["w_router"].double().t()).float()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(1, keepdim=True)
    # every expert that has a token, or, where there are fewer picks than experts, every pick;
    # then the shared experts, which take every token
    token = torch.arange(T, device=x.device)
    if T * k < E:
        which = ids.reshape(-1)
        mix = torch.where(token[:, None] == token.repeat_interleave(k)[None], p.reshape(1, -1), 0.0)
    else:
        which = torch.arange(E, device=x.device)
        mix = torch.zeros((T, E), device=x.device).scatter_(1, ids, p)
    which = torch.cat([which, torch.arange(E, E + case["shared"], device=x.device)])
    mix = torch.cat([mix, torch.ones((T, case["shared"]), device=x.device)], 1)
    wg, wu, wd = (_values((s[m][0][which], s[m][1][which])) for m in ("wg", "wu", "wd"))
    g = (x @ wg.flatten(0, 1).t()).unflatten(1, (len(which), -1))
    u = (x @ wu.flatten(0, 1).t()).unflatten(1, (len(which), -1))
    h = _silu(g) * u * mix[:, :, None]
    out = h.flatten(1) @ wd.permute(0, 2, 1).flatten(0, 1)
    return out.to(s["x"].dtype), ids.to(torch.int32)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("residual", "train"):
        return _plain_residual(s)
    if op == "quantize":
        return _plain_quantize(s["x"], _DTYPES[case["y"]])
    if op == "moe":
        return _plain_moe(s)
    x = s["x"].float()
    if op == "matmul":
        y = x @ _values(s["w"]).t()
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(_DTYPES[case["y"]])
    return (_silu(x @ _values(s["wg"]).t()) * (x @ _values(s["wu"]).t())).to(s["x"].dtype)


# ---------------------------------------------------------------------- the definition, in 64 bits

def _exact_values(w):
    codes, scales = w
    c = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64,
                    device=codes.device)
    for half, part in enumerate((codes % 16, codes // 16)):
        m = (part % 8).double()
        # exponent 0 has no leading one
        v = torch.where(m < 2, m / 2, (1 + (m % 2) / 2) * 2 ** (torch.floor(m / 2) - 1))
        c[..., half::2] = torch.where(part >= 8, -v, v)
    return c * (2.0 ** (scales.double() - 127)).repeat_interleave(_GROUP, -1)


def _exact_residual(case, s):
    leaves = [k for k in ("x", "y", "w_post", "gate", "w_next") if s[k] is not None]
    v = {k: s[k].double().requires_grad_(case["op"] == "train") for k in leaves}

    def norm(a, w):
        return a / (a.pow(2).sum(1, keepdim=True) / a.shape[1] + _EPS).sqrt() * w

    z = norm(v["y"], v["w_post"]) if case["post"] else v["y"]
    if "gate" in v:
        rows, d = v["gate"].shape
        z = (z.view(rows, -1, d) * v["gate"].view(rows, 1, d)).view(-1, d)
    r = v["x"] + z / 2
    n = norm(r, v["w_next"]) if case["next"] else None
    if case["op"] == "residual":
        return (r, n) if case["next"] else r
    out = [r] + ([n] if case["next"] else [])
    at = [s["dr"].double()] + ([s["dn"].double()] if case["next"] else [])
    grads = dict(zip(leaves, torch.autograd.grad(out, [v[k] for k in leaves], at)))
    return (r.detach(), None if n is None else n.detach()) + tuple(
        grads.get(k) for k in ("x", "y", "w_post", "gate", "w_next"))


def _exact_quantize(case, s):
    x = s["x"].double().view(case["rows"], -1, _GROUP)
    top = x.abs().max(2).values
    m, e = torch.frexp(top)  # top = m * 2^e with m in [1/2, 1)
    e = torch.where(m <= 0.875, e - 3, e - 2)
    e = torch.where(top == 0, torch.zeros_like(e), e.clamp_min(-126))
    unit = (2.0 ** e.double()).unsqueeze(2)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64,
                        device=x.device)
    a = x.abs() / unit
    i = torch.searchsorted(grid, a, right=True) - 1  # the grid value at or below
    lo, hi = grid[i], grid[(i + 1).clamp_max(7)]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 1))
    q = torch.where(up, hi, lo) * unit
    return torch.where(x < 0, -q, q).view(case["rows"], -1), (e + 127).to(torch.uint8)


def _exact_moe(case, s):
    x, k = s["x"].double(), case["k"]
    logits = torch.mm(x, s["w_router"].double().T)
    out = torch.zeros_like(x)
    ids = torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k]
    p = torch.softmax(torch.gather(logits, 1, ids), 1)
    for e in range(case["E"] + case["shared"]):
        if e < case["E"]:
            weight = torch.where(ids == e, p, torch.zeros_like(p)).sum(1, keepdim=True)
        else:
            weight = torch.ones_like(p[:, :1])
        wg, wu, wd = (_exact_values((s[m][0][e], s[m][1][e])) for m in ("wg", "wu", "wd"))
        g = torch.mm(x, wg.T)
        out += weight * torch.mm(g * torch.sigmoid(g) * torch.mm(x, wu.T), wd.T)
    return out, ids.to(torch.int32)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("residual", "train"):
        return _exact_residual(case, s)
    if op == "quantize":
        return _exact_quantize(case, s)
    if op == "moe":
        return _exact_moe(case, s)
    x = s["x"].double()
    if op == "matmul":
        y = torch.mm(x, _exact_values(s["w"]).T)
        return y if s["bias"] is None else y + s["bias"].double()
    g = torch.mm(x, _exact_values(s["wg"]).T)
    return g * torch.sigmoid(g) * torch.mm(x, _exact_values(s["wu"]).T)


# ---------------------------------------------------------------------- what a pass cannot do without

def _mx4_bytes(values):
    return values // 2 + values // _GROUP


def work(case):
    op = case["op"]
    if op in ("residual", "train"):
        T, d = case["T"], case["d"]
        size, wsize = T * d * _BYTES[case["x"]], _BYTES[case["w"]]
        vectors = wsize * d * (case["post"] + case["next"] + _gate_rows(case))
        n = 1 if case["next"] else 0
        if op == "residual":  # x, y in; r, n out
            return dict(bytes=(3 + n) * size + vectors, flops=12 * T * d)
        # and dr, dn in; dx, dy and the vectors' gradients out
        return dict(bytes=(6 + 2 * n) * size + 2 * vectors, flops=40 * T * d)
    if op == "quantize":
        values = case["rows"] * case["cols"]
        # to codes and back
        return dict(bytes=values * (_BYTES[case["x"]] + _BYTES[case["y"]]) + 2 * _mx4_bytes(values),
                    flops=8 * values)
    T, d = case["T"], case["d"]
    if op == "matmul":
        n = case["n"]
        return dict(bytes=2 * T * d + _mx4_bytes(n * d) + (4 * n if case["bias"] else 0)
                    + T * n * _BYTES[case["y"]], flops=2 * T * d * n)
    f = case["f"]
    if op == "gated":
        return dict(bytes=2 * T * d + 2 * _mx4_bytes(f * d) + 2 * T * f, flops=4 * T * d * f)
    # experts that a batch of T picks, on the average of even picks
    E, k = case["E"], case["k"]
    active = E * (1.0 - (1.0 - k / E) ** T) + case["shared"]
    return dict(bytes=int(active * 3 * _mx4_bytes(d * f)) + 4 * E * d + 4 * T * d,
                flops=6 * T * (k + case["shared"]) * d * f + 2 * T * E * d)
