"""The form of the 4-bit products that test_gpu_mx4's list of forms lacks: 17 to 32 tokens,
four waves along the channels, K in one part."""
import pytest
import torch

import mx4_ref
from gpu_common import lib
from test_gpu_dense import F16S, gen, guarded, normal, strided, within
from test_gpu_mx4 import matrix

pytestmark = pytest.mark.gpu

MORE_FORMS = [("stream 32", False, 4, [(20, 96, 28675), (32, 2048, 30016), (17, 160, 28672)])]
SIZES = [(form[:3], size) for form in MORE_FORMS for size in form[3]]


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("form,size", SIZES)
def test_product(form, size, dtype):
    T, K, N = size
    got = lib().mx4_form("matmul_mx4", T, K, N)
    assert (got[0], got[1] > 1, got[2]) == form
    g = gen(T + K + N)
    x, bias = strided(normal(g, (T, K), 1, dtype), 8), normal(g, (N,))
    codes, scales = matrix(g, N, K, 0.5)
    w = lib().pack_mx4(codes, scales)
    ref, tol = mx4_ref.product(x, mx4_ref.values(codes, scales))
    ref += bias.double()
    for out in (dtype, torch.float32):
        y, ok = guarded((T, N), out)
        lib().matmul_mx4(x, w, bias=bias, out=y)
        ok()
        within(y, ref, tol + 2 * mx4_ref.U * ref.abs(), str(got))
