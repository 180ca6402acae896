"""4-bit weights on the GPU: quantisation bit for bit, products element by element
against 64 bits (bounds: mx4_ref.py)."""
import numpy as np
import pytest
import torch

import mx4_ref
from gpu_common import dev, lib
from test_gpu_dense import F16S, FLOATS, gen, guarded, normal, strided, within

pytestmark = pytest.mark.gpu


def matrix(g, rows, cols, spread=1.0):
    """Codes and scales as a checkpoint has them, scales uneven over the groups."""
    codes = torch.randint(0, 256, (rows, cols // 2), generator=g, device=dev(), dtype=torch.int32).to(torch.uint8)
    e = 120 + spread * 2 * torch.randn((rows, cols // 32), generator=g, device=dev())
    return codes, e.round().clamp(1, 200).to(torch.uint8)


# ------------------------------------------------------------------ quantisation

@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 64, 16), (5, 96, 0), (257, 416, 8), (9, 4096, 0),
                                           (2, 16384, 8), (1, 65536, 0), (1031, 32, 0), (64, 1376, 0)])
def test_quantize_and_back(rows, cols, pad, dtype):
    g = gen(rows + cols)
    x = normal(g, (rows, cols)) * torch.exp(4 * normal(g, (rows, 1)))
    x[0, :32] = 0
    x = strided(x.clamp(-6e4, 6e4).to(dtype), pad * (2 if dtype != torch.float32 else 1))
    codes, cok = guarded((rows, cols // 2), torch.uint8)
    scales, sok = guarded((rows, cols // 32), torch.uint8)
    lib().quantize_rows_mx4(x, codes=codes, scales=scales)
    cok(), sok()
    rc, rs = mx4_ref.quantize(x)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    for out in FLOATS:
        y, yok = guarded((rows, cols), out)
        lib().dequantize_rows_mx4(codes, scales, out=y)
        yok()
        assert torch.equal(y.double(), mx4_ref.values(codes, scales).to(out).double())


def test_quantize_edges():
    """Ties, the borders between two scales, the smallest and largest values, zeros
    of both signs, infinities and NaN in one group of a row."""
    x = torch.zeros((12, 64), device=dev())
    x[0, :16] = torch.tensor([7.0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0])
    x[1, :2] = torch.tensor([7.0000005, 1.0])
    x[2, :2] = torch.tensor([3.5, -3.5000002])
    x[3, :3] = torch.tensor([1e-45, -1e-40, 3e-39])
    x[4, :2] = torch.tensor([3.4e38, -1e38])
    x[5, :2] = torch.tensor([2.0 ** -124, -(2.0 ** -126)])
    x[6, 3] = torch.inf
    x[7, 40] = torch.nan
    x[8, 1], x[8, 2] = torch.nan, -torch.inf
    x[9] = -0.0
    x[10, 0], x[10, 33] = 1e-30, -1e30
    x[11, :2] = torch.tensor([6.9999995, 6.5])
    codes, scales = lib().quantize_rows_mx4(x)
    rc, rs = mx4_ref.quantize(x)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    y = lib().dequantize_rows_mx4(codes, scales)
    assert bool(y[6, :32].isnan().all()) and bool((y[6, 32:] == 0).all()) and bool(y[8, :32].isnan().all())


def test_dequantize_every_code_and_scale():
    """Every code with every scale byte, the smallest (2^-127) and 255 among them."""
    codes = torch.arange(256, device=dev()).to(torch.uint8).repeat(256, 1)
    scales = torch.arange(256, device=dev()).to(torch.uint8)[:, None].repeat(1, 16)
    for out in FLOATS:
        y = lib().dequantize_rows_mx4(codes, scales, out)
        ref = mx4_ref.values(codes, scales)
        ref = ref.float().to(out)  # fp32 holds them all (those past it are infinite)
        assert torch.equal(y.nan_to_num(nan=7e3, posinf=8e3, neginf=-8e3),
                           ref.nan_to_num(nan=7e3, posinf=8e3, neginf=-8e3)), out


# ------------------------------------------------------------------ products

# T, K, N: K that ends in a tile's every quarter, one group, whole tiles and pieces; odd
# counts of channels; every form's tokens and their borders
PRODUCTS = [(1, 32, 1), (1, 64, 33), (2, 96, 16), (3, 128, 31), (1, 160, 32), (7, 512, 64), (16, 544, 40),
            (17, 1056, 100), (31, 2048, 257), (32, 4096, 48), (5, 14336, 32), (33, 32, 5), (40, 224, 70),
            (64, 256, 129), (65, 1024, 300), (127, 96, 64), (128, 4128, 128), (129, 544, 260), (333, 1408, 2051),
            (1000, 64, 17), (257, 2048, 512)]


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("T,K,N", PRODUCTS)
def test_matmul(T, K, N, dtype):
    g = gen(T * 7 + K + N)
    codes, scales = matrix(g, N, K)
    w = mx4_ref.values(codes, scales)
    packed = lib().pack_mx4(codes, scales)
    x = strided(normal(g, (T, K), 1, dtype), 8 if T % 2 else 0)
    bias = normal(g, (N,)) if N % 2 else None
    ref, tol = mx4_ref.product(x, w)
    if bias is not None:
        ref = ref + bias.double()
    for out in (dtype, torch.float32):
        y, ok = guarded((T, N), out)
        lib().matmul_mx4(x, packed, bias=bias, out=y)
        ok()
        within(y, ref, tol + 2 * mx4_ref.U * ref.abs(), f"{T}x{K}x{N}")
        assert torch.equal(y, lib().matmul_mx4(x, packed, bias=bias, out_dtype=out))


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("T,d,f", [(1, 32, 32), (1, 2048, 768), (2, 96, 64), (13, 2048, 1408), (16, 160, 96),
                                   (17, 544, 32), (32, 1024, 256), (33, 64, 96), (64, 4096, 160), (100, 256, 512),
                                   (128, 96, 32), (200, 1056, 352), (513, 512, 768)])
def test_gated(T, d, f, dtype):
    g = gen(T + d + f)
    (cg, sg), (cu, su) = matrix(g, f, d), matrix(g, f, d)
    x = strided(normal(g, (T, d), 1, dtype), 16 if T % 2 else 0)
    h, ok = guarded((T, f), dtype)
    lib().gated_ffn_mx4(x, lib().pack_mx4(cg, sg), lib().pack_mx4(cu, su), out=h)
    ok()
    ref, tol = mx4_ref.gated(x, mx4_ref.values(cg, sg), mx4_ref.values(cu, su))
    within(h, ref, tol, f"{T}x{d}x{f}")


# every kernel, cut along K and not, with every count of waves along the channels (mx4_form)
FORMS = [
    ("stream 16", False, 1, [(3, 544, 33), (1, 288, 96)]), ("stream 16", False, 2, [(2, 96, 8190), (2, 96, 8192)]),
    ("stream 16", False, 4, [(9, 160, 14335), (9, 160, 14336)]), ("stream 16", True, 4, [(13, 6176, 65), (13, 6176, 96)]),
    ("stream 32", False, 1, [(31, 544, 70), (17, 800, 64)]), ("stream 32", False, 2, [(19, 160, 14336), (19, 160, 8192)]),
    ("stream 32", False, 4, [None, (32, 96, 14336)]), ("stream 32", True, 4, [(17, 4128, 100), None]),
    ("stream 32", True, 8, [None, (27, 4128, 96)]),
    ("tile 32x128", False, 0, [(45, 160, 67), (45, 160, 96)]), ("tile 32x128", True, 0, [(65, 2080, 35), (33, 2080, 32)]),
    ("tile 64x128", False, 0, [(500, 160, 2051), (500, 160, 1056)]),
    ("tile 64x128", True, 0, [(1500, 8192, 95), (1500, 3200, 32)]),
    ("tile 64x256", False, 0, [(500, 96, 2051), (500, 96, 1056)]),
    ("tile 64x256", True, 0, [(500, 6176, 2051), (500, 6176, 1056)]),
    ("tile 128x256", False, 0, [(1000, 96, 4097), (2047, 96, 1056)]),
    ("tile 128x256", True, 0, [(500, 6176, 4097), (500, 6176, 2080)]),
]


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name,cut,along,sizes", FORMS)
def test_every_form(name, cut, along, sizes, gated, dtype):
    if sizes[gated] is None:
        pytest.skip("the rule does not give this form")
    T, K, N = sizes[gated]
    form = lib().mx4_form("gated_ffn_mx4" if gated else "matmul_mx4", T, K, N)
    assert (form[0], form[1] > 1, form[2]) == (name, cut, along), form
    g = gen(T + K + N)
    x = strided(normal(g, (T, K), 1, dtype), 8)
    (cg, sg), (cu, su) = matrix(g, N, K, 0.5), matrix(g, N, K, 0.5)
    w = lib().pack_mx4(cg, sg)
    if gated:
        h, ok = guarded((T, N), dtype)
        lib().gated_ffn_mx4(x, w, lib().pack_mx4(cu, su), out=h)
        ok()
        within(h, *mx4_ref.gated(x, mx4_ref.values(cg, sg), mx4_ref.values(cu, su)), str(form))
        return
    bias = normal(g, (N,))
    ref, tol = mx4_ref.product(x, mx4_ref.values(cg, sg))
    ref += bias.double()
    for out in (dtype, torch.float32):
        y, ok = guarded((T, N), out)
        lib().matmul_mx4(x, w, bias=bias, out=y)
        ok()
        within(y, ref, tol + 2 * mx4_ref.U * ref.abs(), str(form))


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("T", [1, 20, 70])
def test_uneven_scales(T, dtype):
    """Scales over 60 binades in one row, rows of zeros, groups of zeros with a scale
    larger than the others', and rows of very small and large weights."""
    K, N = 512, 48
    g = gen(T)
    codes, scales = matrix(g, N, K, spread=8.0)
    scales[0], scales[1] = 20, 100
    codes[2] = 0
    codes[3, :16], scales[3, 0] = 0x88, 250  # zeros
    scales[4, 1:] = 60
    scales[4, 0] = 122
    scales[5] = 1
    w = mx4_ref.values(codes, scales)
    ref, tol = mx4_ref.product(normal(gen(T + 1), (T, K), 1, dtype), w)
    y = lib().matmul_mx4(normal(gen(T + 1), (T, K), 1, dtype), lib().pack_mx4(codes, scales), out_dtype=torch.float32)
    within(y, ref, tol, "uneven")


@pytest.mark.parametrize("T", [2, 24, 80])
def test_scales_that_are_none_and_poisoned_tokens_stay_where_they_are(T):
    K, N = 256, 64
    g = gen(T)
    codes, scales = matrix(g, N, K)
    scales[7, 3], scales[33, 0] = 255, 252
    x = normal(g, (T, K), 1, torch.bfloat16)
    clean = lib().matmul_mx4(x, lib().pack_mx4(codes, scales))
    none = torch.zeros(N, dtype=torch.bool, device=dev())
    none[7] = none[33] = True
    assert bool(clean[:, none].isnan().all()) and bool(clean[:, ~none].isfinite().all())
    x[1] = torch.nan
    y = lib().matmul_mx4(x, lib().pack_mx4(codes, scales))
    assert bool(y[1].isnan().all())
    keep = torch.arange(T, device=dev()) != 1
    assert torch.equal(y[keep][:, ~none], clean[keep][:, ~none])


def test_no_tokens_and_no_rows():
    codes, scales = matrix(gen(1), 32, 64)
    w = lib().pack_mx4(codes, scales)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=dev())
    assert lib().matmul_mx4(x, w).shape == (0, 32) and lib().gated_ffn_mx4(x, w, w).shape == (0, 32)
    c, s = lib().quantize_rows_mx4(x)
    assert c.shape == (0, 32) and s.shape == (0, 2) and lib().dequantize_rows_mx4(c, s).shape == (0, 64)


def test_block_as_it_is_served():
    """Weights quantised and packed; norm, gated block, down projection, residual sum:
    each step against its own formula on what the step before gave."""
    import norm_ref
    T, d, f, t = 5, 256, 544, torch.bfloat16
    g = gen(4)
    parts = [lib().quantize_rows_mx4(normal(g, s, s[1] ** -0.5, t)) for s in ((f, d), (f, d), (d, f))]
    wg, wu, wd = (lib().pack_mx4(*p) for p in parts)
    vg, vu, vd = (mx4_ref.values(*p) for p in parts)
    x, wn = normal(g, (T, d), 1, t), (1 + 0.2 * normal(g, (d,))).to(t)
    n = lib().rms_norm(x, wn)
    h = lib().gated_ffn_mx4(n, wg, wu)
    y = lib().matmul_mx4(h, wd)
    r, m = lib().norm_residual(x, y, wn, None, wn, scale=0.5)
    within(h, *mx4_ref.gated(n, vg, vu), "h")
    within(y, *mx4_ref.product(h, vd), "y")
    ref, err = norm_ref.forward(x, y, wn, None, wn, 0.5, 1e-6, 0.0)
    within(r, ref[0], err[0], "r")
    within(m, ref[1], err[1], "m")


def test_streams_and_graphs():
    """Captured and replayed on new inputs with eager work between, and two streams
    at once."""
    g = gen(8)
    (cg, sg), (cu, su) = matrix(g, 768, 1024), matrix(g, 768, 1024)
    wg, wu = lib().pack_mx4(cg, sg), lib().pack_mx4(cu, su)
    for T in (1, 20, 150):
        x = normal(g, (T, 1024), 1, torch.float16)
        want = lib().gated_ffn_mx4(x, wg, wu)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = lib().gated_ffn_mx4(x, wg, wu)
        for k in range(3):
            x.copy_(normal(gen(k), (T, 1024), 1, torch.float16))
            graph.replay()
            eager = lib().gated_ffn_mx4(x, wg, wu)
            torch.cuda.synchronize()
            assert torch.equal(eager, out)
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        for s in (a, b):
            s.wait_stream(torch.cuda.current_stream())
        got = [lib().gated_ffn_mx4(x, wg, wu, stream=s) for s in (a, b, a, b)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, eager) for o in got) and want.shape == out.shape


def test_refusals_on_the_device():
    f = lib()
    codes, scales = matrix(gen(1), 32, 64)
    w = f.pack_mx4(codes, scales)
    x = torch.ones((4, 64), device=dev(), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="expected one of"):
        f.matmul_mx4(x.float(), w)
    with pytest.raises(ValueError, match="inputs"):
        f.matmul_mx4(x[:, :32], w)
    with pytest.raises(f.MoEError, match="y_type"):
        f.matmul_mx4(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="w_up: expected"):
        f.gated_ffn_mx4(x, w, f.Mx4Matrix(w.data, 64, 64))
    with pytest.raises(ValueError, match="shape"):
        f.gated_ffn_mx4(x, w, f.Mx4Matrix(w.data[:-16], 32, 64))
    with pytest.raises(ValueError, match="scales: expected shape"):
        f.pack_mx4(codes, scales[:, :1])
    with pytest.raises(ValueError, match="multiple of 32"):
        f.pack_mx4(codes[:, :20].contiguous(), scales)
    with pytest.raises(f.MoEError, match="multiple of 32"):
        f.quantize_rows_mx4(torch.ones((2, 48), device=dev()))
