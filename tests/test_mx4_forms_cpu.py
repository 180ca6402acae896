"""Which kernels the 4-bit products take (moe_mx4_form), and that the GPU tests' sizes
reach all of them."""
import math
import random

import pytest

fp8 = pytest.importorskip("fp8_moe_layer_amd", reason="libfp8moe.so not built")

from test_gpu_mx4 import FORMS
from test_gpu_mx4_forms import SIZES

OPS = ("matmul_mx4", "gated_ffn_mx4")


def kind(op, T, K, N):
    name, parts, along = fp8.mx4_form(op, T, K, N)
    return name, parts > 1, along


def listed(op):
    forms = {(tuple(form), sizes[op == OPS[1]]) for *form, sizes in FORMS}
    return {(f, s) for f, s in forms if s} | ({(f, s) for f, s in SIZES} if op == OPS[0] else set())


@pytest.mark.parametrize("op", OPS)
def test_each_listed_size_takes_its_form(op):
    for form, size in listed(op):
        assert kind(op, *size) == form, size


@pytest.mark.parametrize("op", OPS)
def test_the_lists_hold_every_form_that_sizes_give(op):
    """Over the whole range of sizes, by their logarithm; no listed form is one that no
    size gives."""
    r, seen = random.Random(1), set()
    size = lambda low, high, step=1: max(low, int(math.exp(r.uniform(math.log(low), math.log(high)))) // step * step)
    for i in range(40000):
        T = r.randint(1, 40) if i % 2 else size(1, 1 << 16)
        K, N = (size(32, 65536, 32), size(1, 1 << 17)) if op == OPS[0] else (size(32, 16384, 32), size(32, 16384, 32))
        seen.add(kind(op, T, K, N))
    assert seen == {form for form, _ in listed(op)}
