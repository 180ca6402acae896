"""The norms around a block and their gradients in 64 bits, and how far a
kernel that computes in fp32 can be off.

Bounds, with u = 2^-24: a sum over a row of d <= 16384 values has at most 64
additions in a thread, 6 in a wave and 15 across waves, each off by u of what it
adds up, so 90u with the products' own roundings; an rstd is off by half of its
sum's error, the reciprocal square root's 2u and a rounding, under 50u; C = 100
u covers an rstd with the products around it.  The rest is carried through the
formulas term by term.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
C = 100 * U


def gate_of(gate, T):
    return 1.0 if gate is None else gate.double().repeat_interleave(T // gate.shape[0], 0)


def forward(x, y, w_post, gate, w_next, scale, eps, offset):
    """(r, n, rstd_y, rstd_r) and the errors of r and n; y None: no sum."""
    x = x.double()
    T = x.shape[0]
    rstd_y = rstd_r = n = err_n = None
    if y is None:
        r, err_r = x, torch.zeros_like(x)
    else:
        y, g = y.double(), gate_of(gate, T)
        z, err_z = y, torch.zeros_like(y)
        if w_post is not None:
            rstd_y = 1 / torch.sqrt((y * y).mean(1) + eps)
            z = y * rstd_y[:, None] * (offset + w_post.double())
            err_z = C * z.abs()
        part = scale * g * z
        r = x + part
        err_r = (scale * g * err_z).abs() if gate is not None else abs(scale) * err_z
        err_r = err_r + 4 * U * (x.abs() + part.abs())
    if w_next is not None:
        rstd_r = 1 / torch.sqrt((r * r).mean(1) + eps)
        w = (offset + w_next.double()) * rstd_r[:, None]
        n = r * w
        # the row's error moves its rstd by at most |err| / |r| in the 2-norm
        rel = err_r.norm(dim=1) / r.norm(dim=1).clamp_min(1e-300)
        err_n = err_r * w.abs() + n.abs() * (C + rel[:, None])
    return (r, n, rstd_y, rstd_r), (err_r, err_n)


def backward(dr, dn, x, y, w_post, gate, w_next, scale, eps, offset):
    """(dx, dy, dw_post, dgate, dw_next) and their errors; y None: no sum."""
    (r, _, sy, sr), (err_r, _) = forward(x, y, w_post, gate, w_next, scale, eps, offset)
    T, d = x.shape
    total = torch.zeros_like(r) if dr is None else dr.double()
    err_t = torch.zeros_like(r)
    dw_next = err_next = None
    if w_next is not None:
        sr, dn = sr[:, None], dn.double()
        rh, a = r * sr, dn * (offset + w_next.double())
        rel = err_r.norm(dim=1, keepdim=True) / r.norm(dim=1, keepdim=True).clamp_min(1e-300)
        err_rh = sr * err_r + (C + rel) * rh.abs()
        m = (a * rh).mean(1, keepdim=True)
        err_m = (a.abs() * err_rh).mean(1, keepdim=True) + 100 * U * (a * rh).abs().mean(1, keepdim=True)
        err_t = sr * (3 * U * a.abs() + m.abs() * err_rh + rh.abs() * err_m) \
            + (C + rel) * sr * (a.abs() + (rh * m).abs()) + 2 * U * total.abs()
        total = total + sr * (a - rh * m)
        dw_next = (dn * rh).sum(0)
        err_next = (dn.abs() * err_rh).sum(0) + (T + 20) * U * (dn * rh).abs().sum(0)
    if y is None:
        return (total, None, None, None, dw_next), (err_t, None, None, None, err_next)
    y, g = y.double(), gate_of(gate, T)
    absg = g.abs() if gate is not None else 1.0
    z, err_z = y, torch.zeros_like(y)
    if w_post is not None:
        wp = offset + w_post.double()
        yh = y * sy[:, None]
        z, err_z = yh * wp, C * (yh * wp).abs()
    dgate = err_gate = dw_post = err_post = None
    if gate is not None:
        G = gate.shape[0]
        rep = T // G
        dgate = (scale * total * z).view(G, rep, d).sum(1)
        err_gate = (abs(scale) * (err_t * z.abs() + total.abs() * err_z)
                    + (rep + 20) * U * (scale * total * z).abs()).view(G, rep, d).sum(1)
    c = scale * total * g
    err_c = abs(scale) * absg * err_t + 3 * U * c.abs()
    dy, err_dy = c, err_c
    if w_post is not None:
        dw_post = (c * yh).sum(0)
        err_post = (err_c * yh.abs() + (C + (T + 20) * U) * (c * yh).abs()).sum(0)
        b = c * wp
        err_b = wp.abs() * err_c + 3 * U * b.abs()
        m = (b * yh).mean(1, keepdim=True)
        err_m = (err_b * yh.abs()).mean(1, keepdim=True) + (C + 100 * U) * (b * yh).abs().mean(1, keepdim=True)
        s = sy[:, None]
        dy = s * (b - yh * m)
        err_dy = s * (err_b + yh.abs() * err_m) + C * s * (b.abs() + (yh * m).abs())
    return (total, dy, dw_post, dgate, dw_next), (err_t, err_dy, err_post, err_gate, err_next)
