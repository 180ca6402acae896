"""4-bit weights: the reference quantiser against its definition, and what the
entry points refuse (every call fails host validation, so nothing is enqueued
and no GPU is needed, or has no tokens)."""
import ctypes as C

import numpy as np
import pytest
import torch

import mx4_ref

fp8 = pytest.importorskip("fp8_moe_layer_amd", reason="libfp8moe.so not built")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_WORKSPACE = range(6)
MB = 1 << 20
P = [(i + 1) * 256 * MB for i in range(8)]  # distinct regions, never dereferenced
F32, BF16, F16 = 0, 1, 2


def test_reference_quantiser_picks_the_nearest_code():
    """Every value within one unit of its scale of what its codes stand for, and no
    code nearer; the scale the smallest that holds the group."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn((7, 256), generator=g) * torch.exp(3 * torch.randn((7, 1), generator=g))
    codes, scales = (torch.from_numpy(a) for a in mx4_ref.quantize(x))
    v, s = mx4_ref.values(codes, scales), torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    grid = torch.tensor(np.concatenate([mx4_ref.GRID, -mx4_ref.GRID]))
    best = ((x.double() / s)[..., None] - grid).abs().amin(-1) * s
    assert bool(((x.double() - v).abs() <= best * (1 + 1e-12)).all()) and bool(((x.double() - v).abs() <= s).all())
    top = x.double().abs().view(7, 8, 32).amax(2)
    unit = torch.exp2(scales.double() - 127)
    assert bool((top <= 7 * unit).all()) and bool((top > 3.5 * unit).all())


def quantize(x=P[0], kind=F32, ldx=64, rows=4, cols=64, codes=P[1], scales=P[2]):
    return fp8._quantize_rows_mx4(x, kind, ldx, rows, cols, codes, scales, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("x", "codes", "scales")],
    (dict(rows=-1), ERR_SHAPE), (dict(rows=(1 << 21) + 1), ERR_SHAPE), (dict(cols=0), ERR_SHAPE),
    (dict(cols=48), ERR_SHAPE), (dict(cols=65568, ldx=65568), ERR_SHAPE), (dict(ldx=60), ERR_SHAPE),
    (dict(ldx=66), ERR_SHAPE), (dict(kind=3), ERR_UNSUPPORTED), (dict(kind=-1), ERR_UNSUPPORTED),
    (dict(x=P[0] + 8), ERR_ALIGN), (dict(codes=P[1] + 4), ERR_ALIGN),
    (dict(codes=P[0] + 1008), ERR_SHAPE), (dict(scales=P[1] + 127), ERR_SHAPE),
])
def test_quantize_refuses(kw, code):
    assert quantize(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_quantize_rows_mx4")


def dequantize(codes=P[0], scales=P[1], rows=4, cols=64, kind=F32, y=P[2]):
    return fp8._dequantize_rows_mx4(codes, scales, rows, cols, kind, y, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("codes", "scales", "y")],
    (dict(rows=-1), ERR_SHAPE), (dict(cols=16), ERR_SHAPE), (dict(kind=4), ERR_UNSUPPORTED),
    (dict(codes=P[0] + 4), ERR_ALIGN), (dict(y=P[2] + 8), ERR_ALIGN), (dict(y=P[0] + 112), ERR_SHAPE),
    (dict(scales=P[2] + 1023), ERR_SHAPE),
])
def test_dequantize_refuses(kw, code):
    assert dequantize(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_dequantize_rows_mx4")


def pack(codes=P[0], scales=P[1], rows=40, cols=64, packed=P[2]):
    return fp8._pack_mx4(codes, scales, rows, cols, packed, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("codes", "scales", "packed")],
    (dict(rows=0), ERR_SHAPE), (dict(rows=-5), ERR_SHAPE), (dict(cols=33), ERR_SHAPE),
    (dict(codes=P[0] + 8), ERR_ALIGN), (dict(packed=P[2] + 4), ERR_ALIGN),
    (dict(packed=P[0] + 1264), ERR_SHAPE), (dict(scales=P[2] + 16), ERR_SHAPE),
])
def test_pack_refuses(kw, code):
    assert pack(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_pack_mx4")


def test_packed_size():
    # 32 channels of 128 inputs: two blocks of a tile with its scales, 16 factors
    assert fp8.packed_mx4_bytes(1, 32) == fp8.packed_mx4_bytes(32, 128) == 2 * (1024 + 64 + 64)
    assert fp8.packed_mx4_bytes(33, 544) == 4 * (5 * 1024 + 5 * 64 + 64)
    assert fp8.packed_mx4_bytes(0, 32) == fp8.packed_mx4_bytes(4, 40) == 0 and fp8._last_error()
    assert fp8.packed_mx4_bytes(1 << 40, 32) == fp8.packed_mx4_bytes(4, 1 << 40) == 0


def matmul(x=P[0], ldx=64, w=P[1], bias=None, x_type=BF16, T=4, K=64, N=40, y_type=F32, y=P[2], ws=None, wsb=0):
    return fp8._matmul_mx4(x, ldx, w, bias, x_type, T, K, N, y_type, y, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("x", "w", "y")],
    (dict(T=-1), ERR_SHAPE), (dict(T=(1 << 21) + 1), ERR_SHAPE), (dict(K=80, ldx=80), ERR_SHAPE),
    (dict(K=0), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(N=(1 << 21) + 1), ERR_SHAPE),
    (dict(ldx=56), ERR_SHAPE), (dict(ldx=68), ERR_SHAPE), (dict(ldx=(1 << 21) + 8), ERR_SHAPE),
    (dict(x_type=F32), ERR_UNSUPPORTED), (dict(y_type=F16), ERR_UNSUPPORTED), (dict(x_type=7), ERR_UNSUPPORTED),
    (dict(x=P[0] + 8), ERR_ALIGN), (dict(w=P[1] + 8), ERR_ALIGN), (dict(y=P[2] + 4), ERR_ALIGN),
    (dict(bias=P[3] + 2), ERR_ALIGN), (dict(y=P[0] + 496), ERR_SHAPE), (dict(y=P[1] + 4464), ERR_SHAPE),
    (dict(bias=P[2] + 636), ERR_SHAPE),
])
def test_matmul_refuses(kw, code):
    assert matmul(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_matmul_mx4")


def gated(x=P[0], ldx=64, wg=P[1], wu=P[2], kind=F16, T=4, d=64, f=96, h=P[3], ws=None, wsb=0):
    return fp8._ffn_mx4(x, ldx, wg, wu, kind, T, d, f, h, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, ERR_NULL) for n in ("x", "wg", "wu", "h")],
    (dict(T=-2), ERR_SHAPE), (dict(d=48), ERR_SHAPE), (dict(d=16416, ldx=16416), ERR_SHAPE),
    (dict(f=40), ERR_SHAPE), (dict(f=16416), ERR_SHAPE), (dict(f=0), ERR_SHAPE), (dict(ldx=32), ERR_SHAPE),
    (dict(kind=F32), ERR_UNSUPPORTED), (dict(wu=P[2] + 8), ERR_ALIGN), (dict(h=P[0]), ERR_SHAPE),
    (dict(h=P[2] + 64), ERR_SHAPE),
])
def test_gated_refuses(kw, code):
    assert gated(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_ffn_mx4")


def test_forms_and_workspaces():
    form = fp8.mx4_form
    assert form("matmul_mx4", 1, 14336, 4096) == ("stream 16", 1, 1)
    assert form("gated_ffn_mx4", 32, 2048, 768)[0] == "stream 32" and form("gated_ffn_mx4", 33, 2048, 768)[0][:4] == "tile"
    assert form("gated_ffn_mx4", 8192, 4096, 14336) == ("tile 128x256", 1, 0)
    assert form("matmul_mx4", 0, 64, 64) == ("none", 0, 0)
    for T in (1, 5, 16, 17, 32, 33, 64, 300, 5000):
        for K, N in ((32, 1), (1408, 2051), (14336, 4096), (65536, 96)):
            parts = form("matmul_mx4", T, K, N)[1]
            size = fp8._matmul_mx4_ws(T, K, N)
            # a part's fp32 sums, tokens in sixteens and channels in 32s, or nothing
            assert (size == 0) == (parts == 1)
            assert size == 0 or size == parts * -(-T // 16) * 16 * -(-N // 32) * 32 * 4
    for bad in (("matmul_mx4", 1, 40, 64), ("gated_ffn_mx4", 1, 64, 40), ("matmul_mx4", -1, 64, 64)):
        with pytest.raises(fp8.MoEError, match="moe_mx4_form"):
            form(*bad)


def test_no_tokens_is_valid():
    assert quantize(rows=0, x=None, codes=None, scales=None) == OK
    assert dequantize(rows=0, codes=None, scales=None, y=None) == OK
    assert matmul(T=0, x=None, y=None) == OK and gated(T=0, x=None, h=None) == OK


def test_binding_refuses_host_tensors_and_autograd():
    x, u8 = torch.randn(4, 64), torch.zeros((4, 32), dtype=torch.uint8)
    w = fp8.Mx4Matrix(torch.zeros(fp8.packed_mx4_bytes(32, 64), dtype=torch.uint8), 32, 64)
    for call in (lambda: fp8.quantize_rows_mx4(x), lambda: fp8.dequantize_rows_mx4(u8, u8[:, :2]),
                 lambda: fp8.pack_mx4(u8, u8[:, :2]), lambda: fp8.matmul_mx4(x.bfloat16(), w),
                 lambda: fp8.gated_ffn_mx4(x.bfloat16(), w, w)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
    p = x.bfloat16().requires_grad_()
    for call in (lambda: fp8.matmul_mx4(p, w), lambda: fp8.gated_ffn_mx4(p, w, w),
                 lambda: fp8.quantize_rows_mx4(p)):
        with pytest.raises(RuntimeError, match="autograd"):
            call()


# ------------------------------------------------------------------ the layer

def layer(dm={}, kind=BF16, x=P[0], ldx=64, router=P[1], bias=None, kpt=None, w={}, override=None, out=P[2],
          ids=None, tw=None, ws=P[3], wsb=MB):
    m = None if dm is None else C.byref(fp8.dims(**{**dict(T=4, d=64, f=32, E=8, k_max=2), **dm}))
    parts = {**dict(w_gate=P[4], w_up=P[5], w_down=P[6]), **w} if w is not None else None
    return fp8._mx4_forward(m, kind, x, ldx, router, bias, kpt,
                            None if parts is None else C.byref(fp8._Mx4Weights(**parts)), override, out, ids, tw,
                            ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dm=None), ERR_NULL), (dict(w=None), ERR_NULL),
    *[({n: None}, ERR_NULL) for n in ("x", "router", "out")],
    *[(dict(w={n: None}), ERR_NULL) for n in ("w_gate", "w_up", "w_down")],
    (dict(dm=dict(n_shared=1)), ERR_NULL),
    (dict(dm=dict(T=33)), ERR_SHAPE), (dict(dm=dict(T=-1)), ERR_SHAPE), (dict(dm=dict(d=48), ldx=48), ERR_SHAPE),
    (dict(dm=dict(f=16)), ERR_SHAPE), (dict(dm=dict(d=16416), ldx=16416), ERR_SHAPE), (dict(dm=dict(E=0)), ERR_SHAPE),
    (dict(dm=dict(E=513)), ERR_SHAPE), (dict(dm=dict(k_max=0)), ERR_SHAPE), (dict(dm=dict(k_max=9)), ERR_SHAPE),
    (dict(dm=dict(E=64, k_max=33)), ERR_SHAPE), (dict(dm=dict(n_shared=33)), ERR_SHAPE), (dict(ldx=56), ERR_SHAPE),
    (dict(dm=dict(no_requant=True)), ERR_UNSUPPORTED), (dict(kind=F32), ERR_UNSUPPORTED),
    (dict(ws=None), ERR_WORKSPACE), (dict(wsb=512), ERR_WORKSPACE), (dict(ws=P[3] + 64), ERR_ALIGN),
    (dict(x=P[0] + 8), ERR_ALIGN), (dict(out=P[2] + 4), ERR_ALIGN), (dict(w=dict(w_up=P[5] + 8)), ERR_ALIGN),
    (dict(ids=P[7] + 2), ERR_ALIGN), (dict(kpt=P[7] + 1), ERR_ALIGN),
    (dict(out=P[0]), ERR_SHAPE), (dict(ws=P[5]), ERR_SHAPE), (dict(ids=P[3] + 16), ERR_SHAPE),
    (dict(ids=P[7], tw=P[7] + 28), ERR_SHAPE), (dict(out=P[1] + 2032), ERR_SHAPE), (dict(tw=P[6]), ERR_SHAPE),
])
def test_layer_refuses(kw, code):
    assert layer(**kw) == code, fp8._last_error()
    assert fp8._last_error().startswith(b"moe_mx4_forward")


def test_layer_workspace_and_no_tokens():
    size = lambda **kw: fp8._mx4_workspace_bytes(C.byref(fp8.dims(**{**dict(T=4, d=64, f=32, E=8, k_max=2), **kw})))
    # scores, a list of experts, and h's two halves by (token, pick) rows
    assert 4 * 8 * 4 + 2 * 8 * 32 * 2 < size() < size(T=32) < size(T=32, f=16384, n_shared=2) < 64 * MB
    assert size(T=33) == 0 and b"T=33" in fp8._last_error()
    assert layer(dm=dict(T=0), x=None, out=None, ws=None) == OK
