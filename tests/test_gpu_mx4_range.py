"""Norms and 4-bit operators where offsets pass 32 bits, and with long rows and strides:
the last rows of outputs of several GiB against 64 bits."""
import numpy as np
import pytest
import torch

import mx4_ref
import norm_ref
from gpu_common import dev, lib
from test_gpu_dense import gen, normal, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_norm_rows_past_4_gib():
    T, d = (1 << 17) + 3, 16384  # 2^31 values and more: 4.3 GB an array
    g = gen(1)
    x = torch.empty((T, d), dtype=BF, device=dev()).normal_(generator=g)
    y = torch.empty((T, d), dtype=BF, device=dev()).normal_(generator=g)
    w = (1 + 0.2 * normal(g, (d,))).to(BF)
    r, n, sy, sr = lib().norm_residual(x, y, w, None, w, scale=0.5, save=True)
    dx, dy, dw, _, dn = lib().norm_residual_backward(r, n, x, y, sy, sr, w, None, w, scale=0.5)
    rows = torch.tensor([0, T // 2, T - 2, T - 1], device=dev())
    part = [t[rows].contiguous() for t in (x, y, r, n, dx, dy)]
    ref, err = norm_ref.forward(part[0], part[1], w, None, w, 0.5, 1e-6, 0.0)
    within(part[2], ref[0], err[0], "r")
    within(part[3], ref[1], err[1], "n")
    ref, err = norm_ref.backward(part[2], part[3], part[0], part[1], w, None, w, 0.5, 1e-6, 0.0)
    within(part[4], ref[0], err[0], "dx")
    within(part[5], ref[1], err[1], "dy")
    assert bool(dw.isfinite().all()) and bool(dn.isfinite().all())


def test_quantised_rows_past_4_gib():
    rows, cols = 70001, 65536  # 4.6e9 values
    x = torch.empty((rows, cols), dtype=BF, device=dev()).normal_(generator=gen(2))
    codes, scales = lib().quantize_rows_mx4(x)
    y = lib().dequantize_rows_mx4(codes, scales, BF)
    for i in (0, rows // 2, rows - 1):
        rc, rs = mx4_ref.quantize(x[i:i + 1])
        np.testing.assert_array_equal(codes[i:i + 1].cpu().numpy(), rc)
        np.testing.assert_array_equal(scales[i:i + 1].cpu().numpy(), rs)
        assert torch.equal(y[i:i + 1].double(), mx4_ref.values(codes[i:i + 1], scales[i:i + 1]))


@pytest.mark.parametrize("T", [1, 20, 40])
def test_weights_past_4_gib(T):
    N, K = (1 << 20) + 70, 8192  # 4.6 GB packed
    g = gen(3)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev(), dtype=torch.uint8)
    scales = torch.randint(115, 122, (N, K // 32), generator=g, device=dev(), dtype=torch.uint8)
    w = lib().pack_mx4(codes, scales)
    assert w.data.numel() > 1 << 32
    x = normal(g, (T, K), 1, BF)
    y = lib().matmul_mx4(x, w, out_dtype=torch.float32)
    for at in (slice(0, 40), slice(N // 2, N // 2 + 40), slice(N - 70, N)):
        ref, tol = mx4_ref.product(x, mx4_ref.values(codes[at], scales[at]))
        within(y[:, at], ref, tol, str(at))


def test_outputs_past_4_gib():
    T, K, N = 40010, 64, 65540  # 2.6e9 outputs
    g = gen(4)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev(), dtype=torch.uint8)
    scales = torch.randint(115, 122, (N, K // 32), generator=g, device=dev(), dtype=torch.uint8)
    x = normal(g, (T, K), 1, torch.float16)
    y = lib().matmul_mx4(x, lib().pack_mx4(codes, scales))
    rows = torch.tensor([0, 1, T // 2, T - 130, T - 1], device=dev())
    ref, tol = mx4_ref.product(x[rows], mx4_ref.values(codes, scales))
    within(y[rows], ref, tol, "y")


@pytest.mark.parametrize("T", [3, 32, 130])
def test_longest_rows_and_strides(T):
    """K of 65536, rows 4 MiB apart (the longest stride), the last one ending its memory."""
    K, N, ld = 65536, 64, 1 << 21
    g = gen(5)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev(), dtype=torch.uint8)
    scales = torch.randint(115, 122, (N, K // 32), generator=g, device=dev(), dtype=torch.uint8)
    flat = torch.full(((T - 1) * ld + K,), torch.nan, dtype=BF, device=dev())
    x = flat.as_strided((T, K), (ld, 1))
    x.copy_(normal(g, (T, K), 1, BF))
    ref, tol = mx4_ref.product(x, mx4_ref.values(codes, scales))
    within(lib().matmul_mx4(x, lib().pack_mx4(codes, scales), out_dtype=torch.float32), ref, tol, "y")
    with pytest.raises(lib().MoEError, match="row stride"):
        lib().matmul_mx4(torch.empty((2, ld + 8), dtype=BF, device=dev())[:, :K], lib().pack_mx4(codes, scales))


@pytest.mark.parametrize("T", [2, 30])
def test_experts_past_4_gib(T):
    """The last experts of matrices of more than 4 GiB give what they give alone."""
    d, f, E = 4096, 8192, 256
    g = gen(6)
    two = lib().Mx4Experts.empty(2, d, f, 1)
    many = lib().Mx4Experts.empty(E, d, f, 1)
    assert many.w_gate.numel() > 1 << 32 and many.w_down.numel() > 1 << 32
    for i, e in enumerate((E - 2, E - 1)):
        for which, shape in (("gate", (f, d)), ("up", (f, d)), ("down", (d, f))):
            codes, scales = lib().quantize_rows_mx4(normal(g, shape, shape[1] ** -0.5))
            two.set_expert(which, i, codes, scales)
            many.set_expert(which, e, codes, scales)
            if i == 0:
                for w in (two, many):
                    w.set_expert(which, 0, codes, scales, shared=True)
    x = normal(g, (T, d), 1, BF)
    logits = torch.zeros((T, E), device=dev())
    logits[:, -2:] = normal(g, (T, 2)) + 50
    ids = torch.empty((T, 2), dtype=torch.int32, device=dev())
    y = lib().Mx4MoELayer(many, None, 2).forward(x, logits_override=logits, topk_ids=ids)
    assert bool((ids >= E - 2).all()) and bool(y.isfinite().all())
    want = lib().Mx4MoELayer(two, None, 2).forward(x, logits_override=logits[:, -2:].contiguous())
    # both round once to bf16 (half a step each); the sums are the same products in another order
    within(y, want.double(), 2.0 ** -8 * want.double().abs() + 2.0 ** -14 * want.double().abs().max(), "y")
