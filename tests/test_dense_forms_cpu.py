"""Which kernels the dense operators take (moe_dense_form), and that the GPU
tests' sizes reach all of them, in every type."""
import csv
import ctypes as C
import math
import pathlib

import pytest

fp8 = pytest.importorskip("fp8_moe_layer_amd", reason="libfp8moe.so not built")

import test_gpu_dense as gpu
from test_gpu_dense_forms import GATED_I8_FORMS, MATMUL_FORMS, MORE_WIDE

OK, ERR_NULL, ERR_SHAPE, _, ERR_UNSUPPORTED = range(5)
NAMES = set(fp8._FORMS.values()) - {"none"}
PRODUCT = {n for n in NAMES if not n.startswith("pair")}
SINGLE = {n for n in PRODUCT if not n.startswith("stream")}  # of the gradients' products
PAIR = {n for n in NAMES if n.startswith("pair")}


@pytest.mark.parametrize("op,sizes", [("matmul_i8", MATMUL_FORMS), ("gated_ffn_i8", GATED_I8_FORMS)])
def test_each_listed_size_takes_its_form(op, sizes):
    assert set(sizes) == PRODUCT
    for form, size in sizes.items():
        assert fp8.dense_form(op, *size) == form
    assert all(fp8.dense_form("gated_ffn_i8", *s) == "stream 32 wide" for s in MORE_WIDE)


def test_the_16_bit_lists_reach_every_form():
    """Both lists run in both types."""
    assert {fp8.dense_form("gated_ffn", *s) for s in gpu.GATED} == PRODUCT
    both = [fp8.dense_form("gated_ffn_backward", *s) for s in gpu.GRADIENTS]
    assert {a for a, _ in both if a in PAIR} == PAIR
    assert {a for a, _ in both} - PAIR == SINGLE  # dx
    assert {b for _, b in both} - PAIR == SINGLE  # dW
    assert all((a in PAIR) == (b in PAIR) for a, b in both)


def test_forms_without_a_workspace_or_tokens():
    forms = (C.c_int32 * 2)()
    T, K, N = MATMUL_FORMS["cut"]
    assert fp8._dense_form(0, T, K, N, 0, forms) == OK and fp8._FORMS[forms[0]] == "tile 64x64"
    assert forms[1] == 0
    assert fp8.dense_form("gated_ffn", 0, 64, 64) == "none"
    dx, dw = fp8.dense_form("gated_ffn_backward", 0, 64, 64)
    assert dx == "none" and dw != "none"


def test_a_workspace_is_asked_for_where_the_product_is_cut():
    for op, size, lists in (("matmul_i8", fp8._matmul_i8_ws, gpu.MATMUL), ("gated_ffn", fp8._gated_ffn_ws, gpu.GATED)):
        for s in lists:
            assert (size(*s) > 0) == (fp8.dense_form(op, *s) == "cut"), (op, s)


@pytest.mark.parametrize("args,code", [
    ((4, 4, 64, 64), ERR_UNSUPPORTED), ((-1, 4, 64, 64), ERR_UNSUPPORTED), ((0, -1, 64, 64), ERR_SHAPE),
    ((0, 4, 24, 64), ERR_SHAPE), ((0, 4, 64, 0), ERR_SHAPE), ((1, 4, 96, 64), ERR_SHAPE),
    ((3, 4, 64, 16448), ERR_SHAPE), ((2, (1 << 21) + 1, 64, 64), ERR_SHAPE)])
def test_dense_form_refuses(args, code):
    forms = (C.c_int32 * 2)(7, 7)
    assert fp8._dense_form(*args, 1, forms) == code
    assert list(forms) == [7, 7] and fp8._last_error().startswith(b"moe_dense_form")
    assert fp8._dense_form(0, 4, 64, 64, 1, None) == ERR_NULL


def test_the_stream_is_chosen_where_it_was_faster():
    """Both sides of the choice at 17 to 32 tokens, as measured: the form taken
    costs 2 % over the better one at most, on average."""
    path = pathlib.Path(__file__).parent.parent / "profiles" / "dense_few_tokens.csv"
    cost, taken = [], set()
    for row in csv.DictReader(path.open()):
        op, kbytes, groups = row["operator"], int(row["row_bytes"]), int(row["groups_of_16_rows"])
        inner = kbytes // 2 if op == "gated_ffn" else kbytes
        outputs = groups * 16 if op == "matmul_i8" else groups * 8
        form = fp8.dense_form(op, int(row["tokens"]), inner, outputs)
        t = {True: float(row["stream_us"]), False: float(row["tiles_us"])}
        cost.append(t[form.startswith("stream")] / min(t.values()))
        taken.add(form.startswith("stream"))
    assert len(cost) > 700 and taken == {True, False}
    assert math.exp(sum(map(math.log, cost)) / len(cost)) < 1.02
