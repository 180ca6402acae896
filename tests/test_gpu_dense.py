"""Dense feed-forward operators on the GPU against plain implementations in
64 bits, element by element.

Tolerances are worst-case bounds of the arithmetic, with u = 2^-24 (half an
ulp of fp32, relative):
- a sum of K 16-bit products in fp32: the products are exact; at most 32 are
  added inside one matrix instruction, and K/32 instructions add to the
  accumulator, each addition off by at most 2u of what it adds up, so
  (K/32 + 32) * 2u * sum|x w| in all;
- an int8 sum is exact; its conversion and two scalings are one rounding each;
- SiLU: a relative error e of g moves it by |1 + g (1 - sigmoid(g))| e <=
  (1 + |g|) e; exp and reciprocal are within 8u together (the exponential's
  compensated form a few ulp, the reciprocal 1);
- the output's rounding: half a step of its type.
"""
import ctypes as C

import numpy as np
import pytest
import torch

from gpu_common import dev, lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half the smallest step of a type's subnormal numbers
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
FLOATS = (torch.float32, torch.bfloat16, torch.float16)
F16S = (torch.bfloat16, torch.float16)


def gen(seed):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return g


def normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device=dev()).normal_(0, std, generator=g).to(dtype)


def codes(g, shape):
    return torch.randint(-128, 128, shape, device=dev(), generator=g, dtype=torch.int32).to(torch.int8)


def scales(g, n):
    return torch.rand((n,), device=dev(), generator=g) * 0.02 + 1e-4


def strided(t, pad):
    """The same rows, `pad` elements further apart, with rubbish in between."""
    if not pad:
        return t
    wide = torch.empty((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide.fill_(torch.nan if t.dtype.is_floating_point else 77)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def within(got, ref, tol, what=""):
    assert got.shape == ref.shape, what
    err = (got.double() - ref).abs()
    lim = tol + HALF[got.dtype] * (ref.abs() + tol) + TINY[got.dtype]
    bad = ~(err <= lim)  # a NaN is bad
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / lim).max()):.3g} x, "
        f"first at {bad.nonzero()[0].tolist()}")


def guarded(shape, dtype):
    """An output between two guard blocks: (view, check())."""
    n = int(np.prod(shape))
    g = 1024
    flat = torch.full((n + 2 * g,), 3.0, device=dev()).to(dtype)

    def check():
        assert bool((flat[:g] == 3).all()) and bool((flat[g + n:] == 3).all()), "written outside"
    return flat[g:g + n].view(shape), check


# ------------------------------------------------------------------ quantisation

def quantize_ref(x):
    x = x.float().cpu().numpy()
    a = np.abs(x).max(1)
    m = np.maximum(a, np.float32(2.0 ** -100))
    r = (np.float32(127) / m).astype(np.float32)
    s = np.where(a == 0, np.float32(1), m / np.float32(127)).astype(np.float32)
    q = np.rint(x.astype(np.float64) * r.astype(np.float64)[:, None])
    return q.astype(np.int8), s


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols,pad", [
    (1, 16, 0), (3, 48, 16), (5, 1008, 0), (17, 1024, 32), (2, 1040, 0), (9, 4096, 0), (4, 14336, 8),
    (3, 16384, 0), (2, 16400, 0), (1, 65536, 0), (1000, 64, 0), (257, 2048, 0), (67, 256, 0), (35, 272, 16),
    (18, 512, 0), (21, 528, 0), (1031, 192, 0)])
def test_quantize_rows_i8(rows, cols, pad, dtype):
    g = gen(rows * 7 + cols)
    x = (normal(g, (rows, cols)) * torch.exp(3 * normal(g, (rows, 1)))).clamp(-6e4, 6e4)
    x = strided(x.to(dtype), pad * (2 if dtype != torch.float32 else 1))
    q, check = guarded((rows, cols), torch.int8)
    q, s = lib().quantize_rows_i8(x, q=q)
    rq, rs = quantize_ref(x)
    check()
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


def test_quantize_edges():
    """Zero rows, ties, rows of tiny and of huge values, one value alone."""
    x = torch.zeros((7, 64), device=dev())
    x[1, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])      # r = 1: ties go to the even code
    x[2, :2] = torch.tensor([1e-38, -5e-39])              # below the floor: codes of 2^-100/127 steps
    x[3, :2] = torch.tensor([2.0 ** -99, -2.0 ** -100])
    x[4, :2] = torch.tensor([3.0e38, -3.0e38])
    x[5, 63] = -1e-30
    x[6] = 1.0
    q, s = lib().quantize_rows_i8(x)
    rq, rs = quantize_ref(x)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    assert q[1, :4].tolist() == [127, 0, 2, -2] and float(s[0]) == 1.0 and not bool(q[0].any())


# ------------------------------------------------------------------ int8 product

def matmul_ref(xq, sx, wq, sw, bias):
    acc = xq.double() @ wq.double().t()
    prod = acc * sx.double()[:, None] * sw.double()
    ref = prod if bias is None else prod + bias.double()
    tol = 4 * U * prod.abs() + (0 if bias is None else U * (prod.abs() + bias.double().abs()))
    return ref, tol


MATMUL = [(1, 16, 1), (1, 64, 16), (2, 48, 3), (15, 112, 31), (16, 128, 64), (17, 144, 65),
          (33, 256, 100), (48, 1408, 257), (64, 192, 200), (65, 2048, 128), (100, 14336, 130),
          (127, 320, 511), (129, 640, 1025), (255, 1408, 96), (256, 4096, 512), (257, 208, 769),
          (333, 1408, 2051), (1000, 96, 1000), (1, 14336, 4096), (7, 4096, 2048), (2100, 1024, 1536),
          (4100, 512, 2304), (9, 65536, 33), (4, 80, 70000), (16, 272, 9000), (24, 528, 8200),
          (8, 4096, 4111), (32, 1040, 16400), (8200, 128, 4100), (2000, 768, 300), (1000, 800, 4000), (2000, 800, 4000), (3256, 16, 1163),
          (130, 1424, 4111), (40, 16384, 33), (33, 8192, 321), (64, 14336, 4096), (130, 4112, 7),
          (300, 6160, 515), (20, 6400, 4200), (29, 6160, 8209), (19, 1040, 515), (32, 2064, 4096)]


@pytest.mark.parametrize("T,K,N", MATMUL)
def test_matmul_i8(T, K, N):
    g = gen(T + K + N)
    kind = FLOATS[(T + N) % 3]
    xq = strided(codes(g, (T, K)), 16 * (N % 3))
    wq, sx, sw = codes(g, (N, K)), scales(g, T), scales(g, N)
    bias = normal(g, (N,)) if T % 2 else None
    y, check = guarded((T, N), kind)
    y.fill_(5)
    lib().matmul_i8(xq, sx, wq, sw, bias=bias, out=y)
    ref, tol = matmul_ref(xq, sx, wq, sw, bias)
    check()
    within(y, ref, tol, f"T={T} K={K} N={N} {kind}")


@pytest.mark.parametrize("kind", FLOATS)
@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_matmul_i8_types_and_extreme_codes(T, kind):
    """Every code at -128 over a long row: the largest sum there is."""
    K, N = 4096, 80
    xq = torch.full((T, K), -128, dtype=torch.int8, device=dev())
    wq = torch.full((N, K), -128, dtype=torch.int8, device=dev())
    wq[1::2] = 127
    g = gen(3)
    sx, sw = scales(g, T) * 0.01, scales(g, N)
    y = lib().matmul_i8(xq, sx, wq, sw, out_dtype=kind)
    ref, tol = matmul_ref(xq, sx, wq, sw, None)
    within(y, ref, tol, f"{kind}")


@pytest.mark.parametrize("T", [1, 70])
def test_matmul_i8_longest_row(T):
    K, N = 65536, 17
    xq = torch.full((T, K), -128, dtype=torch.int8, device=dev())
    wq = torch.full((N, K), -128, dtype=torch.int8, device=dev())
    one = lambda n: torch.ones((n,), device=dev())
    y = lib().matmul_i8(xq, one(T), wq, one(N))
    assert bool((y == float(2 ** 30)).all())


@pytest.mark.parametrize("T,K,N", [(64, 16384, 64), (33, 8192, 321), (128, 14336, 515)])
def test_a_cut_product_equals_the_uncut_one(T, K, N):
    """int8 sums are exact, so cutting K (with a workspace, here one full of
    rubbish) changes no bit; and the workspace is written nowhere else."""
    m, g = lib(), gen(T)
    xq, wq, sx, sw = codes(g, (T, K)), codes(g, (N, K)), scales(g, T), scales(g, N)
    n = m._matmul_i8_ws(T, K, N)
    assert n > 0
    ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=dev())
    y, z = torch.empty((T, N), device=dev()), torch.empty((T, N), device=dev())
    args = (xq.data_ptr(), K, sx.data_ptr(), wq.data_ptr(), sw.data_ptr(), None, T, K, N, 0)
    st = torch.cuda.current_stream().cuda_stream
    assert m._matmul_i8(*args, y.data_ptr(), ws.data_ptr(), n, st) == 0
    assert m._matmul_i8(*args, z.data_ptr(), None, 0, st) == 0
    assert torch.equal(y, z) and torch.equal(y, m.matmul_i8(xq, sx, wq, sw))
    assert bool((ws[n:] == 0xFF).all())


# ------------------------------------------------------------------ gated block, int8

def silu_ref(g, u, eg, eu):
    """(h, bound) from g, u in 64 bits with absolute errors eg, eu."""
    s = torch.sigmoid(g)
    h = g * s * u
    slope = s * (1 + g.abs() * (1 - s))  # |SiLU'| <= this
    tol = (slope + eg) * eg * u.abs() + (g * s).abs() * eu + (slope + eg) * eg * eu
    return h, tol + 12 * U * h.abs()


@pytest.mark.parametrize("T,d,f", [(1, 64, 64), (3, 256, 192), (16, 128, 512), (17, 192, 64),
                                   (32, 320, 128), (63, 2048, 768), (65, 64, 1408), (130, 448, 320),
                                   (256, 256, 512), (300, 1408, 192), (700, 512, 1088),
                                   (1, 4096, 14336), (2050, 256, 2048), (5, 16384, 64),
                                   (130, 64, 16384), (8, 2048, 4160), (16, 4096, 4160),
                                   (31, 448, 8256), (1030, 192, 4096), (260, 832, 3456), (40, 16384, 64),
                                   (33, 8192, 320), (200, 6208, 192)])
def test_gated_i8(T, d, f):
    g = gen(T + d + f)
    kind = FLOATS[(T + f // 64) % 3]
    xq = strided(codes(g, (T, d)), 16 * (T % 3))
    wg, wu, sx = codes(g, (f, d)), codes(g, (f, d)), scales(g, T)
    sg, su = scales(g, f) * 0.1, scales(g, f) * 0.1
    h, check = guarded((T, f), kind)
    h.fill_(5)
    lib().gated_ffn_i8(xq, sx, wg, sg, wu, su, out=h)
    gr, _ = matmul_ref(xq, sx, wg, sg, None)
    ur, _ = matmul_ref(xq, sx, wu, su, None)
    ref, tol = silu_ref(gr, ur, 4 * U * gr.abs(), 4 * U * ur.abs())
    check()
    within(h, ref, tol, f"T={T} d={d} f={f} {kind}")


# ------------------------------------------------------------------ gated block, 16 bits

def sum_tol(a, b, k):
    """Bound of an fp32 sum of k exact products of a's rows with b's rows."""
    return (k / 32 + 32) * 2 * U * (a.double().abs() @ b.double().abs().t())


def gated_ref(x, wg, wu):
    g, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    d = x.shape[1]
    return g, u, sum_tol(x, wg, d), sum_tol(x, wu, d)


GATED = [(1, 64, 64), (2, 256, 192), (15, 128, 512), (16, 2048, 768), (17, 192, 64), (33, 64, 128),
         (64, 320, 256), (65, 1408, 192), (128, 256, 512), (129, 448, 320), (257, 192, 1408),
         (300, 2048, 64), (777, 512, 832), (2050, 256, 2048), (8, 512, 4160), (12, 192, 8256),
         (2500, 128, 192), (40, 1024, 2304), (1500, 1024, 320), (1100, 640, 2304), (5000, 64, 64), (260, 832, 3456), (40, 4096, 128), (90, 16384, 64),
         (200, 3136, 192), (23, 4096, 2112), (31, 640, 1088), (27, 3136, 8256)]

# and, for the gradients, sizes at which each tile is taken, by dx and dW alone and together
GRADIENTS = GATED + [(1044, 3136, 64), (1247, 640, 1088), (45, 2240, 896), (37, 1600, 1920),
                     (34, 3136, 1408), (1987, 832, 576), (4096, 1216, 64), (3215, 2368, 64),
                     (268, 2880, 64), (35, 3264, 320), (586, 2752, 64), (412, 3712, 320),
                     (626, 3712, 256), (1008, 3968, 576), (1081, 4096, 512), (7, 640, 11264),
                     (8192, 256, 192), (1, 1024, 4096), (3001, 128, 64), (70, 192, 8192)]


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("T,d,f", GATED)
def test_gated(T, d, f, dtype):
    g = gen(T + d + f)
    x = strided(normal(g, (T, d), 1.0, dtype), 8 * (T % 3))
    wg, wu = normal(g, (f, d), 2 * d ** -0.5, dtype), normal(g, (f, d), d ** -0.5, dtype)
    h, check = guarded((T, f), dtype)
    h.fill_(5)
    got, gate, up = lib().gated_ffn(x, wg, wu, out=h, save=True)
    assert got is h
    gr, ur, eg, eu = gated_ref(x, wg, wu)
    ref, tol = silu_ref(gr, ur, eg, eu)
    check()
    what = f"T={T} d={d} f={f} {dtype}"
    within(gate, gr, eg, what + " gate")
    within(up, ur, eu, what + " up")
    within(h, ref, tol, what)
    # without the kept products: the same h, bit for bit
    assert torch.equal(lib().gated_ffn(x, wg, wu), h)


def test_gated_far_values():
    """SiLU far out on both sides: h -> g * u, h -> 0, and never NaN."""
    d = f = 64
    x = torch.zeros((4, d), device=dev())
    x[0, 0], x[1, 0], x[2, 0] = 300.0, -300.0, -30.0
    w = torch.zeros((f, d), device=dev())
    w[:, 0] = 1.0
    for dtype in F16S:
        h = lib().gated_ffn(x.to(dtype), w.to(dtype), (w * 0.5).to(dtype))
        g = x.to(dtype)[:, :1].double()
        ref = (g * torch.sigmoid(g) * g * 0.5).expand(4, f)
        within(h, ref, 400 * U * ref.abs())


@pytest.mark.parametrize("T", [1, 20, 70, 300])
@pytest.mark.parametrize("dtype,small,w", [(torch.float16, 2.0 ** -20, 1.0),
                                           (torch.bfloat16, 2.0 ** -130, 2.0 ** 60)])
def test_subnormal_operands_count(dtype, small, w, T):
    """Powers of two, so the sums are exact: flushed operands would give 0."""
    x = torch.full((T, 64), small, device=dev()).to(dtype)
    wt = torch.full((64, 64), w, device=dev()).to(dtype)
    _, gate, up = lib().gated_ffn(x, wt, wt, save=True)
    assert bool((gate == 64 * small * w).all()) and torch.equal(gate, up)


def backward_ref(dh, x, wg, wu, gate, up, dtype):
    """Gradients from the kept products in 64 bits, each with its bound."""
    dh, x, wg, wu, g, u = (t.double() for t in (dh, x, wg, wu, gate, up))
    s = torch.sigmoid(g)
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    # fp32 evaluation: s within 8u, 1 - s within (8u + u) of 1, then a few products
    eg = (dh * u).abs() * s * (1 + g.abs()) * 24 * U + HALF[dtype] * dg.abs() * (1 + 2 ** -8) + TINY[dtype]
    eu = du.abs() * 12 * U + HALF[dtype] * du.abs() * (1 + 2 ** -8) + TINY[dtype]
    f, T = wg.shape[0], x.shape[0]
    sums = lambda k: (k / 32 + 32) * 2 * U
    ag, au, ax = dg.abs() + eg, du.abs() + eu, x.abs()
    dx = dg @ wg + du @ wu
    tx = eg @ wg.abs() + eu @ wu.abs() + sums(2 * f) * (ag @ wg.abs() + au @ wu.abs())
    tg = eg.t().contiguous() @ ax + sums(T) * (ag.t().contiguous() @ ax)
    tu = eu.t().contiguous() @ ax + sums(T) * (au.t().contiguous() @ ax)
    return (dx, dg.t().contiguous() @ x, du.t().contiguous() @ x), (tx, tg, tu)


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("T,d,f", GRADIENTS)
def test_gated_backward(T, d, f, dtype):
    g = gen(T + d + f + 1)
    x = strided(normal(g, (T, d), 1.0, dtype), 8 * (T % 3))
    dh = strided(normal(g, (T, f), 0.3, dtype), 8 * (T % 2))
    wg, wu = normal(g, (f, d), 2 * d ** -0.5, dtype), normal(g, (f, d), d ** -0.5, dtype)
    gate, up = normal(g, (T, f), 2.0), normal(g, (T, f), 1.0)
    outs = [guarded(s, dtype) for s in ((T, d), (f, d), (f, d))]
    n = lib().gated_ffn_backward_workspace_bytes(T, d, f)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev())  # a workspace full of NaN
    got = lib().gated_ffn_backward(dh, x, wg, wu, gate, up, *[o for o, _ in outs], workspace=ws)
    refs, tols = backward_ref(dh, x, wg, wu, gate, up, dtype)
    for o, (view, check), ref, tol, name in zip(got, outs, refs, tols, ("dx", "dw_gate", "dw_up")):
        check()
        assert o is view
        within(o, ref, tol, f"T={T} d={d} f={f} {dtype} {name}")
    again = lib().gated_ffn_backward(dh, x, wg, wu, gate, up)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_no_tokens():
    """T = 0: nothing but the weights' gradients is written, and those are zero."""
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev())
    w = z(128, 64)
    h, gate, up = lib().gated_ffn(z(0, 64), w, w, save=True)
    assert h.shape == (0, 128)
    dwg, dwu = z(128, 64) + 7, z(128, 64) + 7
    dx, _, _ = lib().gated_ffn_backward(z(0, 128), z(0, 64), w, w, gate, up, dw_gate=dwg, dw_up=dwu)
    assert dx.shape == (0, 64) and not bool(dwg.any()) and not bool(dwu.any())
    q, s = lib().quantize_rows_i8(z(0, 64))
    assert lib().matmul_i8(q, s, torch.zeros((5, 64), dtype=torch.int8, device=dev()),
                           torch.ones(5, device=dev())).shape == (0, 5)


def test_offsets_beyond_32_bits():
    """More than 2^32 bytes (and 2^31 values) in every array of T rows: the
    last tokens' rows, and a few channels of the weights' gradients."""
    T, d, f, last = 150_016, 64, 14_400, 300
    dtype = torch.bfloat16
    assert T * f > 2 ** 31
    g = gen(9)
    x = normal(g, (T, d), 1.0, dtype)
    wg, wu = normal(g, (f, d), 0.125, dtype), normal(g, (f, d), 0.125, dtype)
    h, gate, up = lib().gated_ffn(x, wg, wu, save=True)
    gr, ur, eg, eu = gated_ref(x[-last:], wg, wu)
    within(gate[-last:], gr, eg, "gate")
    ref, tol = silu_ref(gr, ur, eg, eu)
    within(h[-last:], ref, tol, "h")
    # h stands in for its own gradient
    dx, dwg, dwu = lib().gated_ffn_backward(h, x, wg, wu, gate, up)
    (rx, _, _), (tx, _, _) = backward_ref(h[-last:], x[-last:], wg, wu, gate[-last:], up[-last:], dtype)
    within(dx[-last:], rx, tx, "dx")
    c = slice(f - 8, f)
    (_, rg, ru), (_, tg, tu) = backward_ref(h[:, c].contiguous(), x, wg[c], wu[c], gate[:, c].contiguous(),
                                            up[:, c].contiguous(), dtype)
    within(dwg[c], rg, tg, "dw_gate")
    within(dwu[c], ru, tu, "dw_up")
    del gate, up, dx, dwg, dwu
    q, s = lib().quantize_rows_i8(h)
    rq, rs = quantize_ref(h[-last:])
    np.testing.assert_array_equal(q[-last:].cpu().numpy(), rq)
    w8, s8 = lib().quantize_rows_i8(wg)
    xq, sx = lib().quantize_rows_i8(x)
    y = lib().matmul_i8(xq, sx, w8, s8, out_dtype=dtype)
    ref, tol = matmul_ref(xq[-last:], sx[-last:], w8, s8, None)
    within(y[-last:], ref, tol, "y")
    down = codes(g, (3, f))
    sd = scales(g, 3)
    z = lib().matmul_i8(q, s, down, sd)
    ref, tol = matmul_ref(q[-last:], s[-last:], down, sd, None)
    within(z[-last:], ref, tol, "z")


@pytest.mark.parametrize("T", [3, 20, 70, 600])
def test_rows_do_not_touch_each_other(T):
    """A token of infinities and NaN changes no other token's outputs."""
    g = gen(T)
    d, f = 256, 320
    x = normal(g, (T, d), 1.0, torch.float16)
    wg, wu = normal(g, (f, d), 1 / 16, torch.float16), normal(g, (f, d), 1 / 16, torch.float16)
    want = lib().gated_ffn(x, wg, wu)
    bad = x.clone()
    bad[T // 2, ::3], bad[T // 2, 1::3] = torch.inf, torch.nan
    got = lib().gated_ffn(bad, wg, wu)
    keep = torch.arange(T, device=dev()) != T // 2
    assert torch.equal(got[keep], want[keep])
    xq, sx = lib().quantize_rows_i8(x)
    w8, s8 = lib().quantize_rows_i8(wg)
    y = lib().matmul_i8(xq, sx, w8, s8)
    sx2 = sx.clone()
    sx2[T // 2] = torch.nan
    assert torch.equal(lib().matmul_i8(xq, sx2, w8, s8)[keep], y[keep])


# ------------------------------------------------------------------ together

class _Block(torch.autograd.Function):
    """The gated block as a training program wraps it."""

    @staticmethod
    def forward(ctx, x, wg, wu):
        h, gate, up = lib().gated_ffn(x, wg, wu, save=True)
        ctx.save_for_backward(x, wg, wu, gate, up)
        return h

    @staticmethod
    def backward(ctx, dh):
        return lib().gated_ffn_backward(dh.contiguous(), *ctx.saved_tensors)


@pytest.mark.parametrize("T,d,f", [(37, 256, 512), (300, 128, 192)])
def test_a_training_step_against_differences(T, d, f):
    """Forward and backward through autograd, a down projection behind them:
    the gradients against central differences, in 64 bits, of the loss along a
    random direction.  The bound is the sum over all elements of |direction|
    times the gradient's own bound (the kept products are off by their sums'
    bound, which moves dg and du by at most their slopes times that)."""
    g = gen(5)
    dtype = torch.bfloat16
    x = normal(g, (T, d), 1.0, dtype).requires_grad_()
    wg = normal(g, (f, d), d ** -0.5, dtype).requires_grad_()
    wu = normal(g, (f, d), d ** -0.5, dtype).requires_grad_()
    dh = normal(g, (T, f), 0.25, dtype)
    h = _Block.apply(x, wg, wu)
    grads = torch.autograd.grad(h, (x, wg, wu), dh)
    x, wg, wu = x.detach(), wg.detach(), wu.detach()
    p = [t.double() for t in (x, wg, wu)]
    _, gate, up = lib().gated_ffn(x, wg, wu, save=True)
    _, tols = backward_ref(dh, x, wg, wu, gate, up, dtype)
    gr, ur, rg, ru = gated_ref(x, wg, wu)
    # |SiLU''| <= 1/2 and |SiLU'| <= 1.1 everywhere
    D = dh.double().abs()
    dgo, duo = D * (1.1 * ru + 0.5 * (ur.abs() + ru) * rg), D * 1.1 * rg
    extra = (dgo @ p[1].abs() + duo @ p[2].abs(), dgo.t().contiguous() @ p[0].abs(),
             duo.t().contiguous() @ p[0].abs())

    def loss(x, wg, wu):
        g_, u_ = x @ wg.t(), x @ wu.t()
        return (g_ * torch.sigmoid(g_) * u_ * dh.double()).sum()

    for i in range(3):
        v = torch.empty_like(p[i]).normal_(generator=gen(10 + i))
        e = 1e-4
        q, r = list(p), list(p)
        q[i], r[i] = p[i] + e * v, p[i] - e * v
        want = float((loss(*q) - loss(*r)) / (2 * e))
        got = float((grads[i].double() * v).sum())
        bound = float(((tols[i] + extra[i] + HALF[dtype] * grads[i].double().abs()) * v.abs()).sum())
        assert abs(got - want) <= bound + 1e-5 * abs(want), (i, got, want, bound)


def serve(x, wq):
    """The block as a server runs it, on quantised weights."""
    q, s = lib().quantize_rows_i8(x)
    h = lib().gated_ffn_i8(q, s, *wq["gate"], *wq["up"], out_dtype=torch.bfloat16)
    hq, sh = lib().quantize_rows_i8(h)
    return lib().matmul_i8(hq, sh, *wq["down"], out_dtype=torch.bfloat16), (q, s, h, hq, sh)


@pytest.mark.parametrize("T", [1, 16, 75, 513])
def test_trained_weights_served_in_int8(T):
    """Weights of a 16-bit block quantised per channel; the served block stage
    by stage, and its h against the 16-bit block's within the bound of the two
    quantisations (half a step of each operand)."""
    g = gen(T)
    d, f, n = 512, 768, 512
    x = normal(g, (T, d), 1.0, torch.bfloat16)
    w = {k: normal(g, s, s[1] ** -0.5, torch.bfloat16)
         for k, s in (("gate", (f, d)), ("up", (f, d)), ("down", (n, f)))}
    wq = {k: lib().quantize_rows_i8(v) for k, v in w.items()}
    y, (q, s, h, hq, sh) = serve(x, wq)
    ref, tol = matmul_ref(hq, sh, *wq["down"], None)
    within(y, ref, tol)
    rq, rs = quantize_ref(h)
    np.testing.assert_array_equal(hq.cpu().numpy(), rq)
    gr, ur, eg, eu = gated_ref(x, w["gate"], w["up"])
    step = lambda sc: sc.double()[:, None] * (0.5 + 2.0 ** -15)
    for key, e in (("gate", eg), ("up", eu)):
        e += (step(s) * torch.ones(1, d, device=dev(), dtype=torch.float64)) @ (
            w[key].double().abs() + step(wq[key][1])).t() + x.double().abs() @ (
            step(wq[key][1]) * torch.ones(1, d, device=dev(), dtype=torch.float64)).t()
    # |SiLU'| <= 1.1
    silu = (gr * torch.sigmoid(gr)).abs()
    tol = 1.1 * eg * (ur.abs() + eu) + silu * eu
    within(h, lib().gated_ffn(x, w["gate"], w["up"]).double(), tol * 1.01 + HALF[torch.bfloat16] * (
        gr * torch.sigmoid(gr) * ur).abs())


@pytest.mark.parametrize("T,d,f", [(70, 256, 320), (5, 256, 320), (40, 2048, 64)])
def test_captured_and_replayed_with_work_in_between(T, d, f):
    """The whole chain, training and serving, in one graph; every replay
    against the eager result on its own inputs, with eager calls of the same
    operators between the replays."""
    g = gen(1)
    dtype = torch.float16
    x, dh = normal(g, (T, d), 1, dtype), normal(g, (T, f), 1, dtype)
    wg, wu = normal(g, (f, d), d ** -0.5, dtype), normal(g, (f, d), d ** -0.5, dtype)
    wq = {"gate": lib().quantize_rows_i8(wg), "up": lib().quantize_rows_i8(wu),
          "down": lib().quantize_rows_i8(normal(g, (d, f), f ** -0.5))}

    def both():
        h, gate, up = lib().gated_ffn(x, wg, wu, save=True)
        return [h, *lib().gated_ffn_backward(dh, x, wg, wu, gate, up), serve(x, wq)[0]]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for i in range(4):
        x.copy_(normal(gen(20 + i), (T, d), 1, dtype))
        eager = [t.clone() for t in both()]
        for t in captured:
            t.zero_()
        graph.replay()
        if i % 2:
            torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)), i


def test_a_stream_of_its_own():
    """Calls given a stream run there, in order, and allocate for it."""
    g = gen(2)
    x = normal(g, (200, 256), 1, torch.bfloat16)
    w = normal(g, (256, 256), 1 / 16, torch.bfloat16)
    want = lib().gated_ffn(x, w, w)
    wh, gate, up = lib().gated_ffn(x, w, w, save=True)
    wantb = lib().gated_ffn_backward(wh, x, w, w, gate, up)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        h, ga, u = lib().gated_ffn(x, w, w, save=True, stream=s)
        grads = lib().gated_ffn_backward(h, x, w, w, ga, u, stream=s)
        q, sc = lib().quantize_rows_i8(h, stream=s)
        y = lib().matmul_i8(q, sc, q, sc, stream=s)
        s.synchronize()
        assert torch.equal(h, want)
        assert all(torch.equal(a, b) for a, b in zip(grads, wantb))
        ref, tol = matmul_ref(q, sc, q, sc, None)
        within(y, ref, tol)


def test_two_streams_at_once():
    """The same operators on two streams, each with its own inputs, at the same
    time: nothing is shared but the weights."""
    g = gen(8)
    wg, wu = normal(g, (320, 2048), 1 / 45, torch.bfloat16), normal(g, (320, 2048), 1 / 45, torch.bfloat16)
    xs = [normal(g, (n, 2048), 1, torch.bfloat16) for n in (300, 40)]

    def step(x, stream=None):
        h, ga, up = lib().gated_ffn(x, wg, wu, save=True, stream=stream)
        return [h, *lib().gated_ffn_backward(h, x, wg, wu, ga, up, stream=stream)]

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[step(x, s) for _ in range(8)] for x, s in zip(xs, ss)]
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, r))


def test_the_debug_build():
    """The device-checked build gives the same bits, and names a row that is
    not finite."""
    if not lib().DEBUG_LIB_PATH.exists():
        pytest.skip("libfp8moe_debug.so not built")
    dbg = C.CDLL(str(lib().DEBUG_LIB_PATH))
    for name in ("_quantize_rows_i8", "_gated_ffn", "_gated_bwd"):
        fn = getattr(lib(), name)
        getattr(dbg, fn.__name__).argtypes = fn.argtypes
    dbg.moe_last_error.restype = C.c_char_p
    g = gen(4)
    T, d, f = 50, 128, 192
    x = normal(g, (T, d), 1, torch.float16)
    wg, wu = normal(g, (f, d), 0.1, torch.float16), normal(g, (f, d), 0.1, torch.float16)
    h, ga, up = lib().gated_ffn(x, wg, wu, save=True)
    h2, ga2, up2 = torch.empty_like(h), torch.empty_like(ga), torch.empty_like(up)
    p = lambda t: t.data_ptr()
    torch.cuda.synchronize()
    assert dbg.moe_gated_ffn(p(x), d, p(wg), p(wu), 2, T, d, f, p(h2), p(ga2), p(up2), None, 0, None) == 0
    assert torch.equal(h, h2) and torch.equal(ga, ga2) and torch.equal(up, up2)
    want = lib().gated_ffn_backward(h, x, wg, wu, ga, up)
    got = [torch.empty_like(t) for t in want]
    n = lib().gated_ffn_backward_workspace_bytes(T, d, f)
    ws = torch.empty(n, dtype=torch.uint8, device=dev())
    torch.cuda.synchronize()
    assert dbg.moe_gated_ffn_backward(p(h), f, p(x), d, p(wg), p(wu), p(ga), p(up), 2, T, d, f,
                                      *map(p, got), p(ws), n, None) == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    q, s = torch.empty((T, d), dtype=torch.int8, device=dev()), torch.empty(T, device=dev())
    bad = x.clone()
    bad[3, 5] = torch.nan
    torch.cuda.synchronize()
    assert dbg.moe_quantize_rows_i8(p(x), 2, d, T, d, p(q), p(s), None) == 0
    assert dbg.moe_quantize_rows_i8(p(bad), 2, d, T, d, p(q), p(s), None) == 7
    assert b"non-finite" in dbg.moe_last_error()


def test_the_binding_refuses():
    b16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev())
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8, device=dev())
    f32 = lambda *s: torch.zeros(s, dtype=torch.float32, device=dev())
    m = lib()
    with pytest.raises(ValueError, match="rows must be contiguous"):
        m.quantize_rows_i8(f32(64, 64).t())
    with pytest.raises(m.MoEError, match="row stride 0"):
        m.quantize_rows_i8(f32(1, 64).expand(4, 64))
    with pytest.raises(TypeError):
        m.quantize_rows_i8(f32(4, 64).double())
    with pytest.raises(m.MoEError, match="multiple of 16"):
        m.quantize_rows_i8(f32(4, 40))
    with pytest.raises(ValueError, match="wq must be contiguous"):
        m.matmul_i8(i8(4, 64), f32(4), i8(64, 64).t(), f32(64))
    with pytest.raises(ValueError, match="sx: expected shape"):
        m.matmul_i8(i8(4, 64), f32(5), i8(8, 64), f32(8))
    with pytest.raises(TypeError, match="xq"):
        m.matmul_i8(f32(4, 64), f32(4), i8(8, 64), f32(8))
    with pytest.raises(TypeError):
        m.matmul_i8(i8(4, 64), f32(4), i8(8, 64), f32(8), out_dtype=torch.float64)
    with pytest.raises(TypeError):
        m.gated_ffn(f32(4, 64), f32(64, 64), f32(64, 64))
    with pytest.raises(TypeError, match="w_up"):
        m.gated_ffn(b16(4, 64), b16(64, 64), b16(64, 64).half())
    with pytest.raises(ValueError, match="w_up"):
        m.gated_ffn(b16(4, 64), b16(64, 64), b16(128, 64))
    with pytest.raises(m.MoEError, match="overlaps"):
        w = b16(64, 64)
        m.gated_ffn(w, w, b16(64, 64), out=w)
    with pytest.raises(m.MoEError, match="workspace"):
        m.gated_ffn_backward(b16(4, 64), b16(4, 64), b16(64, 64), b16(64, 64), f32(4, 64), f32(4, 64),
                             workspace=torch.empty(16, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError, match="x is on|w_gate is on"):
        m.gated_ffn(b16(4, 64), b16(64, 64).cpu(), b16(64, 64))
