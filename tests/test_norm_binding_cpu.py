"""The norms' Python binding: what its calls give the library."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

from host_call import host_calls

fp8 = pytest.importorskip("fp8_moe_layer_amd", reason="libfp8moe.so not built")

X, V, RSTD = torch.ones(4, 64), torch.ones(64), torch.ones(4)
# the call, its scalars
CALLS = {
    "rms_norm": (lambda **kw: fp8.rms_norm(X, V, **kw), ("eps", "offset")),
    "norm_residual": (lambda **kw: fp8.norm_residual(X, X, V, None, V, **kw), ("scale", "eps", "offset")),
    "rms_norm_backward": (lambda **kw: fp8.rms_norm_backward(X, X, V, RSTD, **kw), ("offset",)),
    "norm_residual_backward": (lambda **kw: fp8.norm_residual_backward(X, X, X, X, RSTD, RSTD, V, None, V, **kw),
                               ("scale", "offset")),
}
CASES = [(fn, name) for fn, (_, names) in CALLS.items() for name in names]


@pytest.mark.parametrize("make", [torch.tensor, lambda v: torch.nn.Parameter(torch.tensor(v), requires_grad=False)])
@pytest.mark.parametrize("fn,name", CASES)
def test_a_scalar_tensor_counts_with_its_value_at_the_call(fn, name, make, monkeypatch):
    calls = host_calls(monkeypatch, fp8)
    s, seen = make(0.5), []
    for v in (0.5, 2.0, 0.25, 2.0):
        with torch.no_grad():
            s.fill_(v)
        CALLS[fn][0](**{name: s})
        seen.append(getattr(calls[-1][1][0]._obj, name))
    assert seen == [0.5, 2.0, 0.25, 2.0]


@pytest.mark.parametrize("fn,name", CASES)
def test_scalars_of_other_kinds(fn, name, monkeypatch):
    import numpy as np
    calls = host_calls(monkeypatch, fp8)
    for v in (2, True, 0.5, np.float32(0.5), np.float64(0.5), np.array(0.5), torch.tensor(3), torch.tensor([0.5])):
        CALLS[fn][0](**{name: v})
        assert getattr(calls[-1][1][0]._obj, name) == float(v)
    for bad in ("0.5", None, 1j, torch.ones(2)):
        with pytest.raises((TypeError, ValueError)):
            CALLS[fn][0](**{name: bad})


@pytest.mark.parametrize("fn,name", CASES)
def test_a_scalar_that_autograd_would_record_is_refused(fn, name, monkeypatch):
    calls = host_calls(monkeypatch, fp8)
    s = torch.nn.Parameter(torch.tensor(0.5))
    with pytest.raises(RuntimeError, match=f"{fn} is not recorded by autograd"):
        CALLS[fn][0](**{name: s})
    with fwad.dual_level():
        with pytest.raises(RuntimeError, match=f"{fn} has no forward-mode derivative"):
            CALLS[fn][0](**{name: fwad.make_dual(s.detach(), torch.tensor(1.0))})
    assert not calls
    with torch.no_grad():
        CALLS[fn][0](**{name: s})
    assert len(calls) == 1


def test_workspace_of_sizes_past_32_bits():
    size = fp8.norm_backward_workspace_bytes
    assert size(4, 64) > 0 and size(4, 64, 2) > 0
    for bad in ((2 ** 32 + 4, 64), (4, 2 ** 32 + 64), (4, 64, 2 ** 32 + 2), (4 - 2 ** 32, 64), (4, 64, 2 - 2 ** 32)):
        assert size(*bad) == 0
        assert fp8._last_error().startswith(b"moe_norm_residual_backward_workspace_bytes")


def test_a_refused_size_is_named_each_time():
    for d in (20, 24, 20, 24):
        assert fp8.norm_backward_workspace_bytes(4, d) == 0 and f"d={d}".encode() in fp8._last_error()
