"""4-bit weights in 64 bits: the quantisation, the values of codes and scales, and
the products, with how far a kernel that sums in fp32 can be off (u = 2^-24: a
matrix instruction adds 32 exact products, K/32 of them to an accumulator, each
addition off by at most 2u of what it adds up; the partial sums of up to 16 waves
or parts of K and the channel's factor are 20 more)."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x [rows, cols] (any float tensor) -> codes, scales (numpy uint8)."""
    v = x.detach().float().cpu().numpy().astype(np.float64)
    rows, cols = v.shape
    v = v.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(v).all(2)
    v = np.where(bad[..., None], 0.0, v)
    top = np.abs(v).max(2)
    e = np.full(top.shape, -126)
    for k in range(-126, 128):  # the smallest e with top <= 7 * 2^e
        e = np.where(top > 7.0 * 2.0 ** k, k + 1, e)
    e = np.where(top == 0, 0, e)
    a = np.abs(v) / (2.0 ** e.astype(np.float64))[..., None]
    lo = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 7)
    hi = np.minimum(lo + 1, 7)
    dl, dh = a - GRID[lo], GRID[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (lo % 2 == 1)), hi, lo)
    code = np.where(a >= 6, 7, code) | (np.signbit(v) * 8)
    code = np.where(bad[..., None], 0, code).reshape(rows, cols).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def values(codes, scales):
    """What codes and scales (tensors) stand for, fp64 on their device."""
    grid = torch.tensor(np.concatenate([GRID, -GRID]), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.nan, s)
    return grid[c] * s.repeat_interleave(32, -1)


def product(x, w):
    """(x w^T, its error) for fp64 w; with fp16 rows, weights below 2^-35 of their
    channel's largest scale are off by up to 2^-37 of it (the largest weight is at
    least half that scale)."""
    y = x.double() @ w.t()
    tol = (x.shape[1] / 32 + 52) * 2 * U * (x.double().abs() @ w.abs().t())
    if x.dtype == torch.float16:
        tol = tol + x.double().abs().sum(1, keepdim=True) * (w.abs().amax(1) * 2 * 2.0 ** -37)
    return y, tol


def gated(x, wg, wu):
    """SiLU moves by at most 1.1 of its argument's error; its exponential and
    reciprocal are within 8u together."""
    (g, eg), (u, eu) = product(x, wg), product(x, wu)
    s = g * torch.sigmoid(g)
    es = 1.1 * (eg + 2 * U * g.abs()) + 8 * U * s.abs()
    return s * u, es * (u.abs() + eu) + s.abs() * (eu + 2 * U * u.abs()) + 3 * U * (s * u).abs()


def routing(logits, k_max, k_per_token=None):
    """ids (-1 in empty slots) and weights in fp64 from fp32 logits: descending, ties
    to the lower index."""
    T, E = logits.shape
    order = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k_max]
    top = torch.gather(logits.double(), 1, order)
    kt = torch.full((T,), k_max, device=logits.device) if k_per_token is None else k_per_token
    there = torch.arange(k_max, device=logits.device)[None] < kt[:, None]
    p = torch.softmax(torch.where(there, top, -torch.inf), 1)
    return torch.where(there, order, -1), p


def layer(x, ids, p, experts, shared):
    """(out, its error) of the layer for given picks.  experts, shared: lists of
    (gate, up, down) values in fp64.  A routing weight is off by an exponential, a
    sum of up to 32 and a division, under 64u for logits within 30 of each other; h
    is held with 16 bits (2^-17, half a step); the sum over experts and channels runs
    through 2 x K/32 instructions."""
    T, d = x.shape
    out = torch.zeros((T, d), dtype=torch.float64, device=x.device)
    size, err = torch.zeros_like(out), torch.zeros_like(out)
    K = 0
    for e, (wg, wu, wd) in list(enumerate(experts)) + [(-2, w) for w in shared]:
        weight = torch.ones((T, 1), dtype=torch.float64, device=x.device) if e == -2 else \
            torch.where(ids == e, p, 0.0).sum(1, keepdim=True)
        if not bool((weight != 0).any()):
            continue
        h, eh = gated(x, wg, wu)
        h, eh = h * weight, eh * weight + (64 * U + 2.0 ** -17) * (h * weight).abs()
        out += h @ wd.t()
        size += h.abs() @ wd.abs().t()
        err += eh @ wd.abs().t()
        K += wd.shape[1]
    return out, err + 2 * (K / 32 + 52) * 2 * U * size
