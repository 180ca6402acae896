"""The norms' backward pass on the GPU: infinities and NaN stay in their places."""
import pytest
import torch

from gpu_common import dev, lib
from test_gpu_dense import FLOATS, gen, normal

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DIMS = [48, 1024, 2064, 4096, 8192, 16384]  # every team width, and the longest rows


def spoil(v, t):
    """Infinities and a NaN in a few places of two rows (fp16: what an overflow leaves)."""
    v[1, 3], v[1, 17], v[4, 0] = torch.inf, -torch.inf, torch.inf
    v[4, 33] = torch.nan
    return v.to(t)


def same(a, b, tol):
    """Equal where b is no finite number (an infinity's sign counts), near elsewhere."""
    a, fin = a.double(), b.isfinite()
    return bool(((a == b) | (a.isnan() & b.isnan()))[~fin].all()) and \
        bool(((a - b).abs() <= tol)[fin].all())


@pytest.mark.parametrize("t", FLOATS)
@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("gate", [0, 1, 2, 6])
def test_without_norms_gradients_are_products(d, t, gate):
    """r = x + scale gate y: dx is dr, dy = scale dr gate exactly (powers of two), dgate
    the sum of scale dr y, whatever x and y hold."""
    T, g = 6, gen(d)
    x, y = (spoil(normal(g, (T, d)), t) for _ in range(2))
    dr = normal(g, (T, d), 1, t)
    w = torch.exp2(torch.randint(-2, 3, (gate, d), generator=g, device=dev()).float()) if gate else None
    dx, dy, dw_post, dgate, dw_next = lib().norm_residual_backward(dr, None, x, y, None, None, None, w, None, scale=-0.5)
    assert torch.equal(dx, dr) and dw_post is None and dw_next is None
    rows = 1.0 if w is None else w.repeat_interleave(T // gate, 0)
    assert torch.equal(dy, (dr.float() * -0.5 * rows).to(t))
    if gate:
        part = (-0.5 * dr.double() * y.double()).view(gate, T // gate, d)
        assert same(dgate, part.sum(1), (T + 3) * U * part.abs().sum(1).nan_to_num())


@pytest.mark.parametrize("t", FLOATS)
@pytest.mark.parametrize("d", DIMS)
def test_a_norm_of_y_alone(d, t):
    """z = norm(y) with rows of y that are no numbers: dx is dr everywhere, dy is no
    number in those rows alone, dw_post in their columns alone."""
    T, g = 6, gen(d + 1)
    x, y = normal(g, (T, d), 1, t), spoil(normal(g, (T, d)), t)
    w = 1 + 0.2 * normal(g, (d,))
    w = w if t == torch.float32 else w.to(t)
    _, _, sy, _ = lib().norm_residual(x, y, w, save=True)
    dr = normal(g, (T, d), 1, t)
    dx, dy, dw, _, _ = lib().norm_residual_backward(dr, None, x, y, sy, None, w)
    assert torch.equal(dx, dr)
    bad = torch.zeros(T, dtype=torch.bool, device=dev())
    bad[1], bad[4] = True, True
    assert bool(dy[~bad].isfinite().all()) and bool(dy[bad].isnan().all())
    finite = torch.ones(d, dtype=torch.bool, device=dev())
    finite[[3, 17]] = False
    # row 4 holds a NaN: its rstd is none, nor is any of its products
    assert bool(dw.isnan().all())
    dr[4] = 0
    y[4] = 1
    sy[4] = 1
    dw = lib().norm_residual_backward(dr, None, x, y, sy, None, w)[2]
    assert bool(dw[finite].isfinite().all()) and bool(dw[~finite].isnan().all())


@pytest.mark.parametrize("d", DIMS)
def test_a_next_norm_alone(d):
    """The sum without a norm of y, with the next one: a spoilt row of x is no number in
    its own row of dx and dy; dw_next in the columns that it spoils."""
    T, g, t = 6, gen(d + 2), torch.float16
    x, y = normal(g, (T, d), 1, t), normal(g, (T, d), 1, t)
    w = (1 + 0.2 * normal(g, (d,))).to(t)
    clean_r, clean_n, _, sr = lib().norm_residual(x, y, None, None, w, save=True)
    dr, dn = normal(g, (T, d), 1, t), normal(g, (T, d), 1, t)
    clean = lib().norm_residual_backward(dr, dn, x, y, None, sr, None, None, w)
    x[2, 5] = torch.inf
    r, n, _, sr = lib().norm_residual(x, y, None, None, w, save=True)
    got = lib().norm_residual_backward(dr, dn, x, y, None, sr, None, None, w)
    keep = torch.arange(T, device=dev()) != 2
    for a, b in zip((r, n) + got[:2], (clean_r, clean_n) + clean[:2]):
        assert torch.equal(a[keep], b[keep])
    assert bool(got[0][2].isnan().all()) and bool(got[1][2].isnan().all())
    ok = torch.arange(d, device=dev()) != 5
    assert bool(got[4][ok].isfinite().all()) and bool(got[4][5].isnan())


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 0.0, -3.0])
def test_scale_does_not_count_without_a_sum(scale):
    """The C entry points with y NULL: dims.scale belongs to the sum, and a caller may
    leave it unset."""
    import ctypes as C
    f, g, T, d = lib(), gen(7), 5, 96
    x, dn, w = normal(g, (T, d)), normal(g, (T, d)), 1 + 0.2 * normal(g, (d,))
    n, rstd = f.rms_norm(x, w, save=True)
    dx, dw = f.rms_norm_backward(dn, x, w, rstd)
    dims = f._NormDims(T, d, 0, 0, 0, scale, 0.0, 1e-6)
    n2, dx2, dw2 = (torch.empty_like(t) for t in (n, dx, dw))
    ws = torch.empty(f.norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=dev())
    stream = torch.cuda.current_stream().cuda_stream
    at = lambda t: t.data_ptr()
    f._check(f._norm_residual(C.byref(dims), at(x), d, None, 0, None, None, 0, at(w), None, at(n2), None, None, stream))
    f._check(f._norm_bwd(C.byref(dims), None, 0, at(dn), d, at(x), d, None, 0, None, at(rstd), None, None, 0, at(w),
                         at(dx2), None, None, None, at(dw2), at(ws), ws.numel(), stream))
    torch.cuda.synchronize()
    assert torch.equal(n, n2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
