"""Dense feed-forward operators at the ends of their types' ranges, on the GPU,
against 64 bits: gradients of small and of large dh, values near fp32's
largest, and rows that are not finite.  The bounds are those of
test_gpu_dense.py, where not said otherwise."""
import pytest
import torch

from gpu_common import dev, lib
from test_gpu_dense import (F16S, FLOATS, HALF, TINY, U, codes, gen, normal, quantize_ref, scales, within)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ gradients, small and large

def factor_floor(dg, du):
    """Half the smallest step of dg and du as they are held in fp16: they are
    multiplied by a power of two that brings the largest M of them (of those up
    to 2^24) to 2^15 .. 65504, where M is not in 2^-2 .. 65504 already.  So the
    step is 2^-24, or at most 2^-24 * M / 2^14 (M * factor >= 2^14 in any case)."""
    a = torch.cat([dg.abs().flatten(), du.abs().flatten()])
    m = float(a[a <= 2.0 ** 24].max())
    return max(2.0 ** -39 * m, TINY[torch.float16] if 0.24 < m < 65600 else 0.0)


def gradients_of(dh, x, wg, wu, gate, up):
    """Of the definition in 64 bits, each with its bound."""
    dtype = dh.dtype
    d64 = [t.double() for t in (dh, x, wg, wu, gate, up)]
    dh, x, wg, wu, g, u = d64
    s = torch.sigmoid(g)
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    floor = factor_floor(dg, du) if dtype == torch.float16 else TINY[dtype]
    eg = (dh * u).abs() * s * (1 + g.abs()) * 24 * U + HALF[dtype] * dg.abs() * (1 + 2 ** -8) + floor
    eu = du.abs() * 12 * U + HALF[dtype] * du.abs() * (1 + 2 ** -8) + floor
    sums = lambda k: (k / 32 + 32) * 2 * U
    ag, au, ax = (dg.abs() + eg).t().contiguous(), (du.abs() + eu).t().contiguous(), x.abs()
    f, T = wg.shape[0], x.shape[0]
    tx = eg @ wg.abs() + eu @ wu.abs() + sums(2 * f) * (ag.t() @ wg.abs() + au.t() @ wu.abs())
    tg = eg.t().contiguous() @ ax + sums(T) * (ag @ ax)
    tu = eu.t().contiguous() @ ax + sums(T) * (au @ ax)
    return ((dg @ wg + du @ wu, dg.t().contiguous() @ x, du.t().contiguous() @ x), (tx, tg, tu))


# one launch for both, both cut, both in tiles, one token, one of them cut
RANGE_SIZES = [(70, 256, 320), (40, 2048, 64), (7, 640, 1088), (1, 128, 64), (600, 64, 192), (8192, 128, 64)]


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("std", [2.0 ** -22, 2.0 ** -20, 2.0 ** -14, 2.0 ** -7, 2.0 ** 10, 2.0 ** 14])
@pytest.mark.parametrize("T,d,f", RANGE_SIZES)
def test_gradients_of_any_magnitude(T, d, f, std, dtype):
    """dh from fp16's smallest values to its largest, u of 30 where dh is
    large, so that dg and du pass 65504 though no gradient does."""
    g = gen(T + f)
    big = std > 1
    dh = normal(g, (T, f), std, dtype)
    dh = torch.where(dh.isfinite(), dh, torch.zeros_like(dh))  # 2^14: four standard deviations
    # so that dx and dW are ordinary numbers of the type
    scale = 2.0 ** -13 if big else 16.0
    x = normal(g, (T, d), scale, dtype)
    wg, wu = normal(g, (f, d), scale, dtype), normal(g, (f, d), scale, dtype)
    gate, up = normal(g, (T, f), 2.0), normal(g, (T, f), 30.0 if big else 1.0)
    got = lib().gated_ffn_backward(dh, x, wg, wu, gate, up)
    refs, tols = gradients_of(dh, x, wg, wu, gate, up)
    for o, ref, tol, name in zip(got, refs, tols, ("dx", "dw_gate", "dw_up")):
        within(o, ref, tol, f"T={T} d={d} f={f} {dtype} std {std} {name}")
    again = lib().gated_ffn_backward(dh, x, wg, wu, gate, up)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_gradients_that_are_not_finite_stay_where_they_are():
    """A token whose gradient is infinite or absurdly large does not choose
    the factor of the others, which are small."""
    g = gen(3)
    T, d, f = 70, 256, 320
    dtype = torch.float16
    dh = normal(g, (T, f), 2.0 ** -18, dtype)
    x, wg, wu = normal(g, (T, d), 1.0, dtype), normal(g, (f, d), 1.0, dtype), normal(g, (f, d), 1.0, dtype)
    gate, up = normal(g, (T, f), 2.0), normal(g, (T, f))
    want = lib().gated_ffn_backward(dh, x, wg, wu, gate, up)[0]
    keep = torch.arange(T, device=dev()) != 33
    for value in (torch.inf, torch.nan):
        bad = dh.clone()
        bad[33, 5] = value
        assert torch.equal(lib().gated_ffn_backward(bad, x, wg, wu, gate, up)[0][keep], want[keep])
    far = up.clone()
    far[33, 7], bad = 1e35, dh.clone()
    bad[33, 7] = 1.0
    got = lib().gated_ffn_backward(bad, x, wg, wu, gate, far)[0]
    # du of that channel is 1 * SiLU(gate), which is an ordinary value: factor 1
    refs, tols = gradients_of(bad, x, wg, wu, gate, far)
    within(got[keep], refs[0][keep], tols[0][keep] + 2 * f * TINY[dtype] * float(wg.abs().max()))


@pytest.mark.parametrize("T,d,f", [(70, 256, 320), (40, 2048, 64)])
def test_captured_with_gradients_of_changing_magnitude(T, d, f):
    g = gen(4)
    dtype = torch.float16
    x, dh = normal(g, (T, d), 1, dtype), normal(g, (T, f), 1, dtype)
    wg, wu = normal(g, (f, d), d ** -0.5, dtype), normal(g, (f, d), d ** -0.5, dtype)
    gate, up = normal(g, (T, f), 2.0), normal(g, (T, f))
    step = lambda: lib().gated_ffn_backward(dh, x, wg, wu, gate, up)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for std in (1.0, 2.0 ** -18, 2.0 ** 9, 0.5, 2.0 ** -20, 0.0):
        dh.copy_(normal(g, (T, f), std, dtype))
        up.copy_(normal(g, (T, f), 100.0 if std > 1 else 1.0))
        eager = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)), std


# ------------------------------------------------------------------ far values

FAR = [2.3e38, 2.4e38, 2.9e38, 3.3e38, 1e30, 200.0, 0.0]


@pytest.mark.parametrize("T", [14, 40, 300])
def test_silu_up_to_the_largest_numbers(T):
    """h is g * u for a large g and 0 for a large negative one, never NaN: bf16
    and int8 operands reach every fp32 value."""
    far = torch.tensor([s * v for v in FAR for s in (1, -1)], device=dev()).repeat(-(-T // 14))[:T]
    d = f = 64
    x = torch.zeros((T, d), device=dev())
    x[:, 0] = far / 2.0 ** 64
    wg, wu = torch.zeros((f, d), device=dev()), torch.zeros((f, d), device=dev())
    wg[:, 0], wu[:, 0] = 2.0 ** 64, 2.0 ** -64 / 2.0 ** 10
    b16 = lambda t: t.to(torch.bfloat16)
    h, gate, up = lib().gated_ffn(b16(x), b16(wg), b16(wu), save=True)
    g, u = gate.double(), up.double()
    assert bool(gate.isfinite().all()) and float(gate.max()) > 3e38
    ref = g * torch.sigmoid(g) * u
    within(h, ref, 400 * U * ref.abs())

    xq = torch.zeros((T, d), dtype=torch.int8, device=dev())
    xq[:, 0] = 1
    wq = xq[:1].expand(f, d).contiguous()
    sg, su = torch.full((f,), 2.0 ** 64, device=dev()), torch.full((f,), 2.0 ** -74, device=dev())
    for kind in FLOATS:
        h = lib().gated_ffn_i8(xq, far / 2.0 ** 64, wq, sg, wq, su, out_dtype=kind)
        g = far.double()[:, None].expand(T, f)
        ref = g * torch.sigmoid(g) * (g * 2.0 ** -138)
        if kind == torch.float16:
            ref = torch.where(ref > 65520, torch.full_like(ref, torch.inf), ref)
            assert torch.equal(h[ref.isinf()].double(), ref[ref.isinf()])
            h, ref = h[~ref.isinf()], ref[~ref.isinf()]
        within(h, ref, 400 * U * ref.abs())


def test_gradients_up_to_the_largest_numbers():
    """dg and du where g, u or dh is near the largest fp32 or bf16 number and
    the gradient itself is not: each is an ordinary number or 0, never NaN."""
    T, d, f = 4, 64, 64
    dtype = torch.bfloat16
    g = torch.zeros((T, f), device=dev())
    u, dh = torch.full((T, f), 2.0 ** -100, device=dev()), torch.full((T, f), 2.0 ** -60, device=dev())
    for i, v in enumerate(FAR):
        g[:, 2 * i], g[:, 2 * i + 1] = v, -v
    u[:, 20], g[:, 20] = 3e38, -200.0           # dh * u is finite, s = 0
    u[:, 21], g[:, 21], dh[:, 21] = 3e38, -200.0, 2.0 ** 100   # dh * u would be infinite
    dh[:, 22], g[:, 22] = 2.0 ** 120, -1e30     # dh * g would be infinite
    dh[:, 23], g[:, 23], u[:, 23] = 2.0 ** 120, -120.0, 2.0 ** 60
    x = torch.full((T, d), 1.0, device=dev()).to(dtype)
    w = torch.full((f, d), 2.0 ** -60, device=dev()).to(dtype)
    got = lib().gated_ffn_backward(dh.to(dtype), x, w, w, g, u)
    s = torch.sigmoid(g.double())
    dhd = dh.to(dtype).double()
    dg, du = dhd * u.double() * s * (1 + g.double() * (1 - s)), dhd * g.double() * s
    assert all(bool(t.isfinite().all()) for t in got)
    refs, tols = gradients_of(dh.to(dtype), x, w, w, g, u)
    # channels of s = e^-200 and e^-120: their sigmoid is 0 in fp32
    small = (g <= -100)
    lost_g, lost_u = torch.where(small, dg.abs(), 0 * dg), torch.where(small, du.abs(), 0 * du)
    wd, xd = w.double(), x.double()
    extra = (lost_g @ wd + lost_u @ wd, lost_g.t().contiguous() @ xd, lost_u.t().contiguous() @ xd)
    for o, ref, tol, e, name in zip(got, refs, tols, extra, ("dx", "dw_gate", "dw_up")):
        within(o, ref, tol + e, name)


# ------------------------------------------------------------------ rows that are not finite

@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("cols", [64, 192, 512, 1024, 4096, 8192, 16384, 32784])
def test_a_row_with_nan_has_a_nan_scale(cols, dtype):
    """And so everything made from it is NaN; a row with an infinity has an
    infinite scale; the other rows are what they are alone."""
    rows = 41
    x = normal(gen(cols), (rows, cols), 1.0, dtype)
    rq, rs = quantize_ref(x)
    bad = x.clone()
    nan, inf = [0, 7, 18, 40], [3, 22]
    for i, r in enumerate(nan):
        bad[r, [0, cols - 1, cols // 2, 33][i]] = torch.nan if i % 2 else -torch.nan
    bad[18] = torch.nan
    bad[40, 1] = torch.inf
    bad[3, cols - 1], bad[22, 5] = torch.inf, -torch.inf
    q, s = lib().quantize_rows_i8(bad)
    keep = [i for i in range(rows) if i not in nan + inf]
    assert bool(s[nan].isnan().all()) and bool((s[inf] == torch.inf).all())
    assert not bool(q[inf].any())
    assert torch.equal(s[keep].cpu(), torch.from_numpy(rs)[keep])
    assert torch.equal(q[keep].cpu(), torch.from_numpy(rq)[keep])
    if cols <= 4096:
        g = gen(1)
        y = lib().matmul_i8(q, s, codes(g, (65, cols)), scales(g, 65))
        w = codes(g, (64, cols))
        outs = [y] if cols % 64 else [y, lib().gated_ffn_i8(q, s, w, scales(g, 64), w, scales(g, 64))]
        for o in outs:
            assert bool(o[nan + inf].isnan().all()) and bool(o[keep].isfinite().all())


@pytest.mark.parametrize("T", [3, 12, 20, 70, 600])
def test_a_poisoned_token_changes_no_other(T):
    """Of the int8 gated block (its scale is NaN) and of the backward pass (its
    dh, and its g and u, are infinite or NaN): no other token's h or dx."""
    g = gen(T)
    d, f, at = 256, 320, T // 2
    keep = torch.arange(T, device=dev()) != at
    xq, sx, wg, wu = codes(g, (T, d)), scales(g, T), codes(g, (f, d)), codes(g, (f, d))
    sg, su = scales(g, f) * 0.1, scales(g, f) * 0.1
    want = lib().gated_ffn_i8(xq, sx, wg, sg, wu, su)
    bad = sx.clone()
    bad[at] = torch.nan
    got = lib().gated_ffn_i8(xq, bad, wg, sg, wu, su)
    assert torch.equal(got[keep], want[keep]) and bool(got[at].isnan().all())
    for dtype in F16S:
        x, dh = normal(g, (T, d), 1, dtype), normal(g, (T, f), 1, dtype)
        wg, wu = normal(g, (f, d), 1 / 16, dtype), normal(g, (f, d), 1 / 16, dtype)
        gate, up = normal(g, (T, f), 2.0), normal(g, (T, f))
        want = lib().gated_ffn_backward(dh, x, wg, wu, gate, up)[0]
        bdh, bg, bu = dh.clone(), gate.clone(), up.clone()
        bdh[at, ::3], bdh[at, 1::3], bg[at, ::7], bu[at, ::5] = torch.inf, torch.nan, -torch.inf, torch.nan
        got = lib().gated_ffn_backward(bdh, x, wg, wu, bg, bu)[0]
        assert torch.equal(got[keep], want[keep]), dtype
        assert bool(got[at].isnan().all())
