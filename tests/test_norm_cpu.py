"""Norms around a block: the 64-bit formulas against differences, and what the
entry points refuse (every call fails host validation, so nothing is enqueued
and no GPU is needed, or has no tokens)."""
import ctypes as C

import pytest
import torch

import norm_ref

fp8 = pytest.importorskip("fp8_moe_layer_amd", reason="libfp8moe.so not built")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_WORKSPACE = range(6)
MB = 1 << 20
P = [(i + 1) * 256 * MB for i in range(20)]  # distinct regions, never dereferenced
F32, BF16, F16 = 0, 1, 2


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [0, 1, 3, 6])
@pytest.mark.parametrize("nxt", [False, True])
def test_gradient_formulas_against_differences(post, gate, nxt):
    """A step along a random direction, six ways: the central difference's error
    is of order h^2 = 1e-10, its rounding 1e-16 / h."""
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    T, d = 6, 16
    v = dict(x=n(T, d), y=n(T, d), w_post=n(d) if post else None, gate=n(gate, d) if gate else None,
             w_next=n(d) if nxt else None)
    dr, dn = n(T, d), n(T, d) if nxt else None
    k = dict(scale=0.7, eps=1e-3, offset=0.5)

    def loss(v):
        (r, m, _, _), _ = norm_ref.forward(v["x"], v["y"], v["w_post"], v["gate"], v["w_next"], **k)
        return float((r * dr).sum() + ((m * dn).sum() if nxt else 0))

    grads, _ = norm_ref.backward(dr, dn, v["x"], v["y"], v["w_post"], v["gate"], v["w_next"], **k)
    for name, grad in zip(("x", "y", "w_post", "gate", "w_next"), grads):
        if v[name] is None:
            assert grad is None
            continue
        way, h = torch.randn(v[name].shape, generator=g, dtype=torch.float64), 1e-5
        up, down = (loss({**v, name: v[name] + s * h * way}) for s in (1, -1))
        assert abs((up - down) / (2 * h) - float((grad * way).sum())) < 1e-7, name


def dims(T=4, d=64, type=F32, w_type=F32, gate_rows=0, scale=1.0, offset=0.0, eps=1e-6):
    return fp8._NormDims(T, d, type, w_type, gate_rows, scale, offset, eps)


def forward(dm={}, x=P[0], ldx=64, y=P[1], ldy=64, w_post=None, gate=None, ldg=0, w_next=P[2], r=P[3],
            n=P[4], rstd_y=None, rstd_r=None):
    m = None if dm is None else C.byref(dims(**dm))
    return fp8._norm_residual(m, x, ldx, y, ldy, w_post, gate, ldg, w_next, r, n, rstd_y, rstd_r, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dm=None), ERR_NULL), (dict(x=None), ERR_NULL), (dict(y=None), ERR_NULL),
    (dict(r=None), ERR_NULL), (dict(n=None), ERR_NULL), (dict(w_next=None), ERR_NULL),
    (dict(y=None, r=None, w_post=P[5]), ERR_NULL), (dict(y=None, r=None, w_next=None, n=None), ERR_NULL),
    (dict(rstd_y=P[6]), ERR_NULL), (dict(w_next=None, n=None, rstd_r=P[6]), ERR_NULL),
    (dict(gate=P[5], ldg=64), ERR_NULL), (dict(dm=dict(gate_rows=1)), ERR_NULL),
    (dict(dm=dict(T=-1)), ERR_SHAPE), (dict(dm=dict(T=(1 << 21) + 1)), ERR_SHAPE),
    (dict(dm=dict(d=24)), ERR_SHAPE), (dict(dm=dict(d=0)), ERR_SHAPE),
    (dict(dm=dict(d=16400), ldx=16400, ldy=16400), ERR_SHAPE),
    (dict(dm=dict(gate_rows=3), gate=P[5], ldg=64), ERR_SHAPE),
    (dict(dm=dict(gate_rows=8), gate=P[5], ldg=64), ERR_SHAPE),
    (dict(dm=dict(gate_rows=-1)), ERR_SHAPE), (dict(dm=dict(eps=0.0)), ERR_SHAPE),
    (dict(dm=dict(eps=-1.0)), ERR_SHAPE), (dict(dm=dict(eps=float("nan"))), ERR_SHAPE),
    (dict(dm=dict(eps=float("inf"))), ERR_SHAPE), (dict(dm=dict(eps=1e-39)), ERR_SHAPE),
    (dict(ldx=60), ERR_SHAPE), (dict(ldx=66), ERR_SHAPE), (dict(ldy=48), ERR_SHAPE),
    (dict(dm=dict(gate_rows=2), gate=P[5], ldg=48), ERR_SHAPE), (dict(ldx=(1 << 20) + 4), ERR_SHAPE),
    (dict(dm=dict(type=3)), ERR_UNSUPPORTED), (dict(dm=dict(type=BF16, w_type=F16)), ERR_UNSUPPORTED),
    (dict(dm=dict(type=F32, w_type=BF16)), ERR_UNSUPPORTED),
    *[({k: p + 8}, ERR_ALIGN) for k, p in (("x", P[0]), ("y", P[1]), ("w_next", P[2]), ("r", P[3]), ("n", P[4]))],
    (dict(rstd_r=P[6] + 2), ERR_ALIGN),
    (dict(r=P[0]), ERR_SHAPE), (dict(n=P[3] + 1008), ERR_SHAPE), (dict(n=P[1] + 16), ERR_SHAPE),
    (dict(rstd_r=P[4]), ERR_SHAPE), (dict(r=P[2]), ERR_SHAPE),
])
def test_forward_refuses(kw, code):
    assert forward(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_norm_residual")


def backward(dm={}, dr=P[0], lddr=64, dn=P[1], lddn=64, x=P[2], ldx=64, y=P[3], ldy=64, rstd_y=None,
             rstd_r=P[4], w_post=None, gate=None, ldg=0, w_next=P[5], dx=P[6], dy=P[7], dw_post=None,
             dgate=None, dw_next=P[8], ws=P[9], wsb=MB):
    m = None if dm is None else C.byref(dims(**dm))
    return fp8._norm_bwd(m, dr, lddr, dn, lddn, x, ldx, y, ldy, rstd_y, rstd_r, w_post, gate, ldg, w_next,
                         dx, dy, dw_post, dgate, dw_next, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dm=None), ERR_NULL),
    *[({k: None}, ERR_NULL) for k in ("dn", "x", "y", "rstd_r", "w_next", "dw_next", "dx", "dy")],
    (dict(dr=None, w_next=None, dw_next=None), ERR_NULL),
    (dict(w_post=P[10]), ERR_NULL), (dict(w_post=P[10], dw_post=P[11]), ERR_NULL),
    (dict(y=None, dy=None, w_post=P[10], dw_post=P[11], rstd_y=P[12]), ERR_NULL),
    (dict(dm=dict(gate_rows=1), gate=P[10], ldg=64), ERR_NULL), (dict(dgate=P[10]), ERR_NULL),
    (dict(dm=dict(T=-1)), ERR_SHAPE), (dict(dm=dict(d=40), ), ERR_SHAPE), (dict(lddr=60), ERR_SHAPE),
    (dict(lddn=66), ERR_SHAPE), (dict(ldx=63), ERR_SHAPE), (dict(ldy=0), ERR_SHAPE),
    (dict(dm=dict(type=F16, w_type=BF16)), ERR_UNSUPPORTED),
    (dict(ws=None), ERR_WORKSPACE), (dict(wsb=64), ERR_WORKSPACE), (dict(ws=P[9] + 128), ERR_ALIGN),
    *[({k: p + 4}, ERR_ALIGN) for k, p in (("dr", P[0]), ("dn", P[1]), ("dx", P[6]), ("dw_next", P[8]))],
    (dict(dx=P[0]), ERR_SHAPE), (dict(dy=P[1]), ERR_SHAPE), (dict(dw_next=P[5]), ERR_SHAPE),
    (dict(dw_next=P[9] + 16), ERR_SHAPE), (dict(ws=P[2]), ERR_SHAPE),
])
def test_backward_refuses(kw, code):
    assert backward(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_norm_residual_backward")


def test_no_tokens_is_valid():
    assert forward(dm=dict(T=0), x=None, y=None, r=None, n=None) == OK
    assert fp8._norm_bwd_ws(C.byref(dims(T=0))) == 0


def test_workspace_sizes():
    ws = fp8.norm_backward_workspace_bytes
    assert 0 < ws(1, 64) < ws(4096, 4096)
    assert ws(4096, 4096) <= 32 * MB and ws(1 << 21, 16384) <= 128 * MB
    assert ws(1 << 21, 16384, 1 << 21) <= 128 * MB  # a gate row per token
    assert ws(4, 20) == 0 and b"d=20" in fp8._last_error()


def test_binding_refuses_host_tensors_autograd_and_mixed_types():
    x, w = torch.randn(4, 64), torch.ones(64)
    for call in (lambda: fp8.rms_norm(x, w), lambda: fp8.norm_residual(x, x, w_next=w),
                 lambda: fp8.norm_residual_backward(x, None, x, x, None, None)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
    with pytest.raises(RuntimeError, match="autograd"):
        fp8.rms_norm(x.requires_grad_(), w)
    with pytest.raises(ValueError, match="dn and w_next"):
        fp8.norm_residual_backward(x.detach(), x.detach(), x.detach(), x.detach(), None, None)
    with pytest.raises(ValueError, match="dr or dn"):
        fp8.norm_residual_backward(None, None, x.detach(), x.detach(), None, None)
    with pytest.raises(ValueError, match="2 dimensions"):
        fp8.rms_norm(x.detach()[0], w)
