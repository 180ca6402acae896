"""The dense operators' Python binding, what it refuses before it looks for a
GPU: tensors that autograd would have to record, sizes that its 32-bit integers
cannot hold."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

fp8 = pytest.importorskip("fp8_moe_layer_amd", reason="libfp8moe.so not built")


def _args(dtype=torch.bfloat16):
    x, w = torch.ones(4, 64, dtype=dtype), torch.ones(64, 64, dtype=dtype)
    g = torch.ones(4, 64)
    q, wq, s, sw = torch.ones(4, 64, dtype=torch.int8), torch.ones(64, 64, dtype=torch.int8), torch.ones(4), torch.ones(64)
    return {
        "quantize_rows_i8": (dict(x=x), ("x",)),
        "matmul_i8": (dict(xq=q, sx=s, wq=wq, sw=sw, bias=sw.clone()), ("sx", "sw", "bias")),
        "gated_ffn_i8": (dict(xq=q, sx=s, w_gate=wq, s_gate=sw, w_up=wq, s_up=sw.clone()),
                         ("sx", "s_gate", "s_up")),
        "gated_ffn": (dict(x=x, w_gate=w, w_up=w.clone()), ("x", "w_gate", "w_up")),
        "gated_ffn_backward": (dict(dh=x, x=x.clone(), w_gate=w, w_up=w.clone(), gate=g, up=g.clone()),
                               ("dh", "x", "w_gate", "w_up", "gate", "up")),
    }


CASES = [(fn, name) for fn, (_, names) in _args().items() for name in names]


@pytest.mark.parametrize("fn,name", CASES)
def test_what_autograd_would_record_is_refused(fn, name):
    kw = dict(_args()[fn][0])
    kw[name] = kw[name].clone().requires_grad_()
    with pytest.raises(RuntimeError, match=f"{fn} is not recorded by autograd"):
        getattr(fp8, fn)(**kw)
    for allowed in (lambda: torch.no_grad(), lambda: torch.inference_mode()):
        with allowed(), pytest.raises(ValueError, match="device tensors"):  # the next check
            getattr(fp8, fn)(**kw)
    kw[name] = kw[name].detach()
    with pytest.raises(ValueError, match="device tensors"):
        getattr(fp8, fn)(**kw)


@pytest.mark.parametrize("fn,name", CASES)
def test_forward_mode_tangents_are_refused(fn, name):
    kw = dict(_args()[fn][0])
    with fwad.dual_level():
        plain = dict(kw)
        kw[name] = fwad.make_dual(kw[name], torch.ones_like(kw[name]))
        for mode in (torch.enable_grad, torch.no_grad):
            with mode(), pytest.raises(RuntimeError, match=f"{fn} has no forward-mode derivative"):
                getattr(fp8, fn)(**kw)
        with pytest.raises(ValueError, match="device tensors"):
            getattr(fp8, fn)(**plain)


HUGE = 2 ** 32 + 4  # 4 in 32 bits


@pytest.mark.parametrize("fn,name", [
    ("quantize_rows_i8", "x"), ("matmul_i8", "xq"), ("matmul_i8", "wq"), ("gated_ffn_i8", "xq"),
    ("gated_ffn_i8", "w_gate"), ("gated_ffn", "x"), ("gated_ffn", "w_gate"), ("gated_ffn_backward", "x"),
    ("gated_ffn_backward", "w_gate")])
def test_sizes_past_32_bits_are_refused(fn, name):
    for shape in ((HUGE, 64), (4, HUGE)):
        kw = dict(_args()[fn][0])
        kw[name] = kw[name][:1, :1].expand(shape)
        with pytest.raises(ValueError, match=f"{name}: shape .* is past the operators' limits"):
            getattr(fp8, fn)(**kw)


def test_workspace_of_sizes_past_32_bits():
    assert fp8.gated_ffn_backward_workspace_bytes(4, 64, 64) > 0
    for bad in ((HUGE, 64, 64), (4, 2 ** 32 + 64, 64), (4, 64, 2 ** 32 + 64), (4 - 2 ** 32, 64, 64)):
        assert fp8.gated_ffn_backward_workspace_bytes(*bad) == 0
        assert fp8._last_error()


@pytest.mark.parametrize("T,outputs", [(1, 64), (33, 64), (5000, 50000)])
def test_the_library_alone_says_whether_a_call_gets_a_workspace(T, outputs):
    call = object.__new__(fp8._Call)
    call.alloc, call.dev = None, torch.device("cpu")
    ws, at, n = call.workspace(lambda *sizes: 512 if sizes == (T, 128, outputs) else 0, T, 128, outputs)
    assert n == 512 and ws.numel() == 512 and at == ws.data_ptr()
    assert call.workspace(lambda *sizes: 0, T, 128, outputs) == (None, None, 0)
