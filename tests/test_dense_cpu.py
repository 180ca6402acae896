"""Dense feed-forward entry points, what they refuse: every call below fails
host validation (so nothing is enqueued and no GPU is needed) or has no tokens
to work on."""
import ctypes as C
import os
import re

import pytest
import torch

fp8 = pytest.importorskip("fp8_moe_layer_amd", reason="libfp8moe.so not built")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_WORKSPACE = range(6)
MB = 1 << 20
# distinct 16 MiB regions that are never dereferenced
P = [(i + 1) * 256 * MB for i in range(16)]
F32, BF16, F16 = 0, 1, 2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_dense_symbol_is_exported_by_both_libraries():
    src = open(os.path.join(ROOT, "include", "fp8moe.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = {n for n in re.findall(r"\b(moe_\w+)\s*\(", src) if "_i8" in n or "gated" in n}
    assert len(names) == 9
    for path in (fp8.LIB_PATH, fp8.DEBUG_LIB_PATH):
        if path.exists():
            lib = C.CDLL(str(path))
            assert all(hasattr(lib, n) for n in names)


def quantize(x=P[0], kind=F32, ldx=64, rows=4, cols=64, q=P[1], scale=P[2]):
    return fp8._quantize_rows_i8(x, kind, ldx, rows, cols, q, scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ERR_NULL), (dict(q=None), ERR_NULL), (dict(scale=None), ERR_NULL),
    (dict(rows=-1), ERR_SHAPE), (dict(cols=0), ERR_SHAPE), (dict(cols=40), ERR_SHAPE),
    (dict(cols=65552, ldx=65552), ERR_SHAPE), (dict(ldx=63), ERR_SHAPE), (dict(ldx=66), ERR_SHAPE),
    (dict(kind=BF16, ldx=68), ERR_SHAPE), (dict(ldx=(1 << 20) + 4), ERR_SHAPE),
    (dict(rows=(1 << 21) + 1), ERR_SHAPE),
    (dict(kind=3), ERR_UNSUPPORTED), (dict(kind=-1), ERR_UNSUPPORTED),
    (dict(x=P[0] + 8), ERR_ALIGN), (dict(q=P[1] + 4), ERR_ALIGN), (dict(scale=P[2] + 2), ERR_ALIGN),
    (dict(q=P[0] + 1008), ERR_SHAPE), (dict(scale=P[1] + 252), ERR_SHAPE),
])
def test_quantize_refuses(kw, code):
    assert quantize(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_quantize_rows_i8")


def matmul(xq=P[0], ldx=64, sx=P[1], wq=P[2], sw=P[3], bias=None, T=4, K=64, N=7, kind=F32, y=P[4],
           ws=None, wsb=0):
    return fp8._matmul_i8(xq, ldx, sx, wq, sw, bias, T, K, N, kind, y, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("xq", "sx", "wq", "sw", "y")],
    (dict(T=-1), ERR_SHAPE), (dict(T=(1 << 21) + 1), ERR_SHAPE), (dict(K=0, ldx=64), ERR_SHAPE),
    (dict(K=24), ERR_SHAPE), (dict(K=65552, ldx=65552), ERR_SHAPE), (dict(N=0), ERR_SHAPE),
    (dict(N=(1 << 21) + 1), ERR_SHAPE), (dict(ldx=48), ERR_SHAPE), (dict(ldx=72), ERR_SHAPE),
    (dict(ldx=(1 << 22) + 16), ERR_SHAPE), (dict(kind=3), ERR_UNSUPPORTED),
    (dict(xq=P[0] + 4), ERR_ALIGN), (dict(wq=P[2] + 8), ERR_ALIGN), (dict(y=P[4] + 4), ERR_ALIGN),
    (dict(sw=P[3] + 1), ERR_ALIGN), (dict(bias=P[5] + 2), ERR_ALIGN),
    (dict(y=P[0] + 240), ERR_SHAPE), (dict(y=P[2] + 432), ERR_SHAPE), (dict(bias=P[4] + 108), ERR_SHAPE),
])
def test_matmul_refuses(kw, code):
    assert matmul(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_matmul_i8")


def gated_i8(xq=P[0], ldx=128, sx=P[1], wg=P[2], sg=P[3], wu=P[4], su=P[5], T=4, d=128, f=64,
             kind=BF16, h=P[6], ws=None, wsb=0):
    return fp8._gated_ffn_i8(xq, ldx, sx, wg, sg, wu, su, T, d, f, kind, h, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("xq", "sx", "wg", "sg", "wu", "su", "h")],
    (dict(T=-1), ERR_SHAPE), (dict(d=96, ldx=96), ERR_SHAPE), (dict(d=16448, ldx=16448), ERR_SHAPE),
    (dict(f=32), ERR_SHAPE), (dict(f=16448), ERR_SHAPE), (dict(ldx=112), ERR_SHAPE),
    (dict(kind=7), ERR_UNSUPPORTED), (dict(wu=P[4] + 8), ERR_ALIGN), (dict(su=P[5] + 2), ERR_ALIGN),
    (dict(h=P[0] + 496), ERR_SHAPE),
])
def test_gated_i8_refuses(kw, code):
    assert gated_i8(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_gated_ffn_i8")


def gated(x=P[0], ldx=128, wg=P[1], wu=P[2], kind=BF16, T=4, d=128, f=64, h=P[3], gate=P[4], up=P[5],
          ws=None, wsb=0):
    return fp8._gated_ffn(x, ldx, wg, wu, kind, T, d, f, h, gate, up, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("x", "wg", "wu", "h", "gate", "up")],
    (dict(T=-1), ERR_SHAPE), (dict(T=(1 << 21) + 1), ERR_SHAPE), (dict(d=96), ERR_SHAPE),
    (dict(f=0), ERR_SHAPE), (dict(ldx=120), ERR_SHAPE), (dict(ldx=132), ERR_SHAPE),
    (dict(kind=F32), ERR_UNSUPPORTED), (dict(x=P[0] + 8), ERR_ALIGN), (dict(up=P[5] + 8), ERR_ALIGN),
    (dict(h=P[4] + 256), ERR_SHAPE), (dict(gate=P[1]), ERR_SHAPE), (dict(gate=P[5]), ERR_SHAPE),
])
def test_gated_refuses(kw, code):
    assert gated(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_gated_ffn:")


def backward(dh=P[0], lddh=64, x=P[1], ldx=128, wg=P[2], wu=P[3], gate=P[4], up=P[5], kind=F16, T=4,
             d=128, f=64, dx=P[6], dwg=P[7], dwu=P[8], ws=P[9], wsb=16 * MB):
    return fp8._gated_bwd(dh, lddh, x, ldx, wg, wu, gate, up, kind, T, d, f, dx, dwg, dwu, ws, wsb,
                          None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("dh", "x", "wg", "wu", "gate", "up", "dx", "dwg", "dwu")],
    (dict(ws=None), ERR_WORKSPACE), (dict(wsb=0), ERR_WORKSPACE),
    (dict(wsb=fp8.gated_ffn_backward_workspace_bytes(4, 128, 64) - 1), ERR_WORKSPACE),
    (dict(ws=P[9] + 16), ERR_ALIGN), (dict(dh=P[0] + 8), ERR_ALIGN),
    (dict(T=-1), ERR_SHAPE), (dict(d=100), ERR_SHAPE), (dict(f=100), ERR_SHAPE),
    (dict(lddh=60), ERR_SHAPE), (dict(ldx=130), ERR_SHAPE), (dict(kind=F32), ERR_UNSUPPORTED),
    (dict(dx=P[1]), ERR_SHAPE), (dict(dwg=P[8]), ERR_SHAPE), (dict(ws=P[7]), ERR_SHAPE),
    (dict(dx=P[0] + 256), ERR_SHAPE),
])
def test_backward_refuses(kw, code):
    assert backward(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_gated_ffn_backward")


def test_optional_workspaces():
    """Products with few outputs and a long sum can be cut; what they then ask
    for is checked, and so is where it lies."""
    assert fp8._matmul_i8_ws(64, 16384, 64) > 0 and fp8._gated_ffn_ws(64, 4096, 64) > 0
    assert fp8._gated_ffn_i8_ws(64, 8192, 64) > 0
    for few in (fp8._matmul_i8_ws(16, 16384, 64), fp8._matmul_i8_ws(8192, 4096, 4096),
                fp8._matmul_i8_ws(64, 64, 64), fp8._matmul_i8_ws(0, 4096, 64)):
        assert few == 0
    for bad in (fp8._matmul_i8_ws(64, 100, 64), fp8._matmul_i8_ws(-1, 4096, 64),
                fp8._gated_ffn_ws(64, 100, 64), fp8._gated_ffn_i8_ws(64, 128, 100)):
        assert bad == 0 and fp8._last_error()
    big = dict(T=64, K=16384, ldx=16384, N=64)
    n = fp8._matmul_i8_ws(64, 16384, 64)
    assert matmul(**big, ws=P[9], wsb=n - 1) == ERR_WORKSPACE
    assert matmul(**big, ws=P[9] + 16, wsb=n) == ERR_ALIGN
    assert matmul(**big, ws=P[4], wsb=n) == ERR_SHAPE       # over y
    assert matmul(**big, ws=P[2], wsb=n) == ERR_SHAPE       # over the weights
    n = fp8._gated_ffn_i8_ws(64, 8192, 64)
    assert gated_i8(T=64, d=8192, ldx=8192, ws=P[9], wsb=n - 1) == ERR_WORKSPACE
    assert gated_i8(T=64, d=8192, ldx=8192, ws=P[6], wsb=n) == ERR_SHAPE
    n = fp8._gated_ffn_ws(64, 4096, 64)
    assert gated(T=64, d=4096, ldx=4096, ws=P[9], wsb=n - 1) == ERR_WORKSPACE
    assert gated(T=64, d=4096, ldx=4096, ws=P[5], wsb=n) == ERR_SHAPE


def test_backward_workspace_size():
    small = fp8.gated_ffn_backward_workspace_bytes(1, 256, 512)
    big = fp8.gated_ffn_backward_workspace_bytes(4096, 256, 512)
    assert 0 < small < big
    for bad in ((-1, 256, 512), (4, 100, 512), (4, 256, 96), ((1 << 21) + 1, 256, 512)):
        assert fp8.gated_ffn_backward_workspace_bytes(*bad) == 0
        assert fp8._last_error()


def test_no_tokens_is_valid_and_enqueues_nothing():
    assert quantize(x=None, q=None, scale=None, rows=0) == OK
    assert matmul(xq=None, sx=None, y=None, T=0) == OK
    assert gated_i8(xq=None, sx=None, h=None, T=0) == OK
    assert gated(x=None, h=None, gate=None, up=None, T=0) == OK


def test_the_binding_refuses_host_tensors_and_recorded_ones():
    x = torch.zeros(4, 64)
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        fp8.quantize_rows_i8(x)
    with pytest.raises(ValueError, match="2 dimensions"):
        fp8.quantize_rows_i8(x[0])
    with pytest.raises(ValueError, match="device tensors"):
        fp8.gated_ffn(x.bfloat16(), w, w)
    with pytest.raises(RuntimeError, match="not recorded by autograd"):
        fp8.gated_ffn(x.bfloat16(), w.requires_grad_(), w)
