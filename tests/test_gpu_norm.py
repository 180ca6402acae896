"""Norms around a block on the GPU, forward and backward, against the formulas
in 64 bits element by element (bounds: norm_ref.py)."""
import pytest
import torch

import norm_ref
from gpu_common import dev, lib
from test_gpu_dense import FLOATS, gen, guarded, normal, strided, within

pytestmark = pytest.mark.gpu

EPS = 1e-6
PAIRS = [(t, w) for t in FLOATS for w in dict.fromkeys((torch.float32, t))]
# T, d: a wave, parts of one, every team width, the longest rows, odd counts
SIZES = [(1, 16), (3, 48), (5, 512), (2, 1040), (7, 2048), (9, 4096), (3, 4112), (2, 8192), (2, 8208),
         (3, 16384), (1, 16368), (131, 256), (67, 1024)]


def inputs(T, d, t, w, post, gate, nxt, seed=0, pad=0):
    g = gen(seed + T * 31 + d)
    step = 16 // t.itemsize
    x = strided((normal(g, (T, d)) * torch.exp(normal(g, (T, 1)))).to(t), pad * step)
    y = strided((normal(g, (T, d)) * torch.exp(normal(g, (T, 1)))).to(t), 2 * pad * step)
    vec = lambda *s: (1 + 0.3 * normal(g, s)).to(w)
    return dict(x=x, y=y, w_post=vec(d) if post else None,
                gate=strided(vec(gate, d), pad * (16 // w.itemsize)) if gate else None,
                w_next=vec(d) if nxt else None), g


def check(got, ref, err, names, what):
    for name, a, b, e in zip(names, got, ref, err):
        assert (a is None) == (b is None), (what, name)
        if a is not None:
            within(a, b, e, f"{what} {name}")


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("T,d", SIZES)
def test_sizes_and_types(T, d, t, w):
    s, g = inputs(T, d, t, w, True, 1, True, pad=1)
    r, rok = guarded((T, d), t)
    n, nok = guarded((T, d), t)
    r, n, sy, sr = lib().norm_residual(*s.values(), scale=0.5, eps=EPS, r=r, n=n, save=True)
    rok(), nok()
    ref, err = norm_ref.forward(*s.values(), 0.5, EPS, 0.0)
    check((r, n), ref[:2], err, ("r", "n"), f"{T}x{d}")
    assert bool(((sy.double() - ref[2]).abs() <= norm_ref.C * ref[2]).all())
    dr, dn = normal(g, (T, d), 1, t), normal(g, (T, d), 1, t)
    dx, xok = guarded((T, d), t)
    dy, yok = guarded((T, d), t)
    got = lib().norm_residual_backward(dr, dn, s["x"], s["y"], sy, sr, s["w_post"], s["gate"], s["w_next"],
                                       scale=0.5, dx=dx, dy=dy)
    xok(), yok()
    ref, err = norm_ref.backward(dr, dn, *s.values(), 0.5, EPS, 0.0)
    check(got, ref, err, ("dx", "dy", "dw_post", "dgate", "dw_next"), f"{T}x{d}")


# (post, gate rows as a share of T = 24, next): every combination of what there is
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [0, 1, 3, 24])
@pytest.mark.parametrize("nxt", [False, True])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_every_combination(post, gate, nxt, offset):
    T, d, t = 24, 272, torch.bfloat16
    s, g = inputs(T, d, t, torch.float32, post, gate, nxt, seed=3)
    r, n, sy, sr = lib().norm_residual(*s.values(), scale=-1.5, eps=EPS, offset=offset, save=True)
    ref, err = norm_ref.forward(*s.values(), -1.5, EPS, offset)
    check((r, n), ref[:2], err, ("r", "n"), "forward")
    plain = lib().norm_residual(*s.values(), scale=-1.5, eps=EPS, offset=offset)
    for a, b in zip((plain if nxt else (plain,)), (r, n)):
        assert torch.equal(a, b)
    dn = normal(g, (T, d), 1, t) if nxt else None
    for dr in (normal(g, (T, d), 1, t), None):
        if dr is None and dn is None:
            continue
        got = lib().norm_residual_backward(dr, dn, s["x"], s["y"], sy, sr, s["w_post"], s["gate"],
                                           s["w_next"], scale=-1.5, offset=offset)
        ref, err = norm_ref.backward(dr, dn, *s.values(), -1.5, EPS, offset)
        check(got, ref, err, ("dx", "dy", "dw_post", "dgate", "dw_next"), f"dr {dr is not None}")


# gate rows against the backward pass's chunks: a row in parts, a row each, several rows to a chunk
@pytest.mark.parametrize("T,G", [(1, 1), (2000, 1), (2000, 2), (2000, 250), (513, 171), (1000, 500),
                                 (514, 257), (2080, 1040), (1500, 1500), (4100, 4100), (600, 300)])
def test_gate_rows(T, G):
    d, t = 64, torch.float16
    s, g = inputs(T, d, t, t, True, G, True, seed=G)
    r, n, sy, sr = lib().norm_residual(*s.values(), scale=0.25, eps=EPS, save=True)
    ref, err = norm_ref.forward(*s.values(), 0.25, EPS, 0.0)
    check((r, n), ref[:2], err, ("r", "n"), "forward")
    dr, dn = normal(g, (T, d), 0.1, t), normal(g, (T, d), 0.1, t)
    args = (dr, dn, s["x"], s["y"], sy, sr, s["w_post"], s["gate"], s["w_next"])
    got = lib().norm_residual_backward(*args, scale=0.25)
    ref, err = norm_ref.backward(dr, dn, *s.values(), 0.25, EPS, 0.0)
    check(got, ref, err, ("dx", "dy", "dw_post", "dgate", "dw_next"), "backward")
    again = lib().norm_residual_backward(*args, scale=0.25)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # equal calls, equal bits


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("T,d", [(1, 16), (33, 4096), (700, 528), (2, 16384)])
def test_rms_norm(T, d, t, w):
    s, g = inputs(T, d, t, w, False, 0, True, seed=5, pad=1)
    x, wn = s["x"], s["w_next"]
    n, rstd = lib().rms_norm(x, wn, EPS, offset=0.5, save=True)
    ref, err = norm_ref.forward(x, None, None, None, wn, 1.0, EPS, 0.5)
    within(n, ref[1], err[1], "n")
    dn, dr = normal(g, (T, d), 1, t), normal(g, (T, d), 1, t)
    for extra in (None, dr):
        got = lib().rms_norm_backward(dn, x, wn, rstd, offset=0.5, dr=extra)
        ref, err = norm_ref.backward(extra, dn, x, None, None, None, wn, 1.0, EPS, 0.5)
        within(got[0], ref[0], err[0], "dx")
        within(got[1], ref[4], err[4], "dw")


def test_gradient_against_differences_of_the_forward_pass():
    """The kernel's gradients along random directions against central differences
    of the formulas in 64 bits: h^2 and rounding leave 1e-6 of them, the kernel's
    own arithmetic what norm_ref bounds."""
    T, d = 12, 512
    s, g = inputs(T, d, torch.float32, torch.float32, True, 3, True, seed=9)
    dr, dn = normal(g, (T, d)), normal(g, (T, d))
    _, _, sy, sr = lib().norm_residual(*s.values(), scale=0.5, eps=EPS, save=True)
    got = lib().norm_residual_backward(dr, dn, s["x"], s["y"], sy, sr, s["w_post"], s["gate"], s["w_next"],
                                       scale=0.5)
    _, err = norm_ref.backward(dr, dn, *s.values(), 0.5, EPS, 0.0)

    def loss(v):
        (r, n, _, _), _ = norm_ref.forward(*v.values(), 0.5, EPS, 0.0)
        return float((r * dr.double()).sum() + (n * dn.double()).sum())

    wide = {k: v.double() for k, v in s.items()}
    for name, grad, e in zip(s, got, err):
        way, h = normal(g, grad.shape).double(), 1e-5
        up, down = (loss({**wide, name: wide[name] + sign * h * way}) for sign in (1, -1))
        slope, mine = (up - down) / (2 * h), float((grad.double() * way).sum())
        limit = float(((e + norm_ref.U * grad.abs()) * way.abs()).sum()) + 1e-6 * float((grad * way).abs().sum())
        assert abs(slope - mine) <= limit, name


def test_no_tokens():
    d, t = 64, torch.bfloat16
    x, w = torch.empty((0, d), dtype=t, device=dev()), torch.ones(d, dtype=t, device=dev())
    gate = torch.ones((1, d), dtype=t, device=dev())
    r, n = lib().norm_residual(x, x, w, gate, w)
    assert r.shape == n.shape == (0, d)
    e = torch.empty(0, device=dev())
    dx, dy, *vecs = lib().norm_residual_backward(x, x, x, x, e, e, w, gate, w)
    assert dx.shape == dy.shape == (0, d)
    assert [tuple(v.shape) for v in vecs] == [(d,), (1, d), (d,)] and all(bool((v == 0).all()) for v in vecs)
    none = lib().norm_residual_backward(x, x, x, x, e, e, w, torch.ones((0, d), dtype=t, device=dev()), w)
    assert none[3].shape == (0, d)


def test_edge_values():
    """Rows of zeros (the norm of nothing is nothing), of the smallest and of large
    values, and a NaN that stays in its row and the vectors' gradients."""
    t, d = torch.float32, 64
    x = torch.zeros((5, d), device=dev())
    x[1] = 1e-30
    x[2] = 1e18
    x[3, 5] = 3.0
    x[4] = torch.nan
    w = torch.full((d,), 2.0, device=dev())
    n, rstd = lib().rms_norm(x, w, EPS, save=True)
    ref, err = norm_ref.forward(x[:4], None, None, None, w, 1.0, EPS, 0.0)
    within(n[:4], ref[1], err[1], "n")
    assert bool(n[4].isnan().all())
    dx, dw = lib().rms_norm_backward(torch.ones_like(x), x, w, rstd)
    assert bool(dx[:4].isfinite().all()) and bool(dx[4].isnan().all())


def test_other_stream_and_graph():
    """Captured and replayed with new inputs, eager work between the replays; and
    on a side stream."""
    T, d, t = 300, 1024, torch.bfloat16
    s, g = inputs(T, d, t, t, True, 1, True, seed=11)
    dr, dn = normal(g, (T, d), 1, t), normal(g, (T, d), 1, t)

    def step(stream=None):
        r, n, sy, sr = lib().norm_residual(*s.values(), scale=0.5, save=True, stream=stream)
        return (r, n) + lib().norm_residual_backward(dr, dn, s["x"], s["y"], sy, sr, s["w_post"], s["gate"],
                                                     s["w_next"], scale=0.5, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        s["x"].copy_(normal(gen(50 + k), (T, d), 1, t))
        dn.copy_(normal(gen(60 + k), (T, d), 1, t))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out)), k


def test_refusals_on_the_device():
    x = torch.ones((4, 64), device=dev(), dtype=torch.bfloat16)
    w = torch.ones(64, device=dev(), dtype=torch.bfloat16)
    f = lib()
    with pytest.raises(TypeError, match="weights and gate"):
        f.rms_norm(x, w.half())
    with pytest.raises(TypeError, match="w_next"):
        f.norm_residual(x, x, w.float(), None, w)
    with pytest.raises(ValueError, match="gate: 3 rows"):
        f.norm_residual(x, x, None, torch.ones((3, 64), device=dev(), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="shape"):
        f.norm_residual(x, x[:3])
    with pytest.raises(ValueError, match="rows must be contiguous"):
        f.rms_norm(torch.ones((64, 64), device=dev(), dtype=torch.bfloat16).t(), w)
    with pytest.raises(ValueError, match="shape"):
        f.rms_norm(x, w[:32])
    with pytest.raises(f.MoEError, match="row stride"):
        f.rms_norm(torch.ones((4, 68), device=dev(), dtype=torch.bfloat16)[:, :64], w)
    with pytest.raises(f.MoEError, match="overlaps"):
        f.norm_residual(x, x, r=x)
    with pytest.raises(ValueError, match="n needs w_next"):
        f.norm_residual(x, x, n=torch.empty_like(x))
