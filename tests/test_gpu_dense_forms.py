"""Every form of the int8 products with every output type: the sizes below take
the form they are listed under (tests/test_dense_forms_cpu.py asserts it), so
that none is left to the sizes of another test."""
import pytest
import torch

from gpu_common import dev, lib
from test_gpu_dense import (FLOATS, U, codes, gen, guarded, matmul_ref, normal, scales, silu_ref, strided,
                            within)

pytestmark = pytest.mark.gpu

MATMUL_FORMS = {
    "stream 8": (5, 4112, 1025), "stream 16": (13, 1040, 2051), "stream 32": (27, 2064, 1003),
    "stream 32 wide": (21, 6416, 4201), "cut": (35, 4144, 201), "tile 64x64": (33, 336, 205),
    "tile 64x128": (65, 336, 8289), "tile 128x128": (4149, 336, 411), "tile 128x256": (649, 336, 5421),
    "tile 256x256": (3599, 336, 2053),
}
GATED_I8_FORMS = {
    "stream 8": (7, 192, 320), "stream 16": (11, 1088, 192), "stream 32": (23, 448, 2048),
    "stream 32 wide": (19, 6208, 2112), "cut": (33, 4032, 192), "tile 64x64": (61, 320, 192),
    "tile 64x128": (65, 192, 4160), "tile 128x128": (69, 192, 8384), "tile 128x256": (131, 192, 8512),
    "tile 256x256": (397, 192, 8256),
}
# the widest stream at more of the channels that take it
MORE_WIDE = [(24, 448, 2112), (17, 64, 2176), (32, 4096, 4096), (17, 8192, 4160)]


@pytest.mark.parametrize("kind", FLOATS, ids=str)
@pytest.mark.parametrize("form", MATMUL_FORMS)
def test_matmul_i8_form(form, kind):
    T, K, N = MATMUL_FORMS[form]
    g = gen(T + K)
    xq, wq, sx, sw = strided(codes(g, (T, K)), 16), codes(g, (N, K)), scales(g, T), scales(g, N)
    for bias in (None, normal(g, (N,))):
        y, check = guarded((T, N), kind)
        lib().matmul_i8(xq, sx, wq, sw, bias=bias, out=y)
        check()
        within(y, *matmul_ref(xq, sx, wq, sw, bias), f"{form} {kind}")


@pytest.mark.parametrize("kind", FLOATS, ids=str)
@pytest.mark.parametrize("T,d,f", [*GATED_I8_FORMS.values(), *MORE_WIDE])
def test_gated_i8_form(T, d, f, kind):
    g = gen(T + d + f)
    xq, sx = strided(codes(g, (T, d)), 32), scales(g, T)
    wg, wu, sg, su = codes(g, (f, d)), codes(g, (f, d)), scales(g, f) * 0.1, scales(g, f) * 0.1
    h, check = guarded((T, f), kind)
    lib().gated_ffn_i8(xq, sx, wg, sg, wu, su, out=h)
    check()
    gr, ur = matmul_ref(xq, sx, wg, sg, None)[0], matmul_ref(xq, sx, wu, su, None)[0]
    within(h, *silu_ref(gr, ur, 4 * U * gr.abs(), 4 * U * ur.abs()), f"T={T} d={d} f={f} {kind}")
