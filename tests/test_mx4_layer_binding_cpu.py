"""The 4-bit MoE layer's Python binding: what its steps give the library."""
import ctypes as C

import pytest
import torch

from host_call import host_calls

fp8 = pytest.importorskip("fp8_moe_layer_amd", reason="libfp8moe.so not built")

NAMES = ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")


def experts(E=4, d=64, f=32, S=1):
    return fp8.Mx4Experts.empty(E, d, f, S, device="cpu")


def make(**kw):
    w = experts(**kw)
    return fp8.Mx4MoELayer(w, torch.zeros(w.E, w.d), 2, torch.zeros(w.E))


def seen(calls):
    """(dims, router, bias, matrices' addresses) of the last call."""
    dims, _, _, _, router, bias, _, w = calls[-1][1][:8]
    return dims._obj, router, bias, [getattr(w._obj, n) for n in NAMES]


def addresses(layer):
    w = [getattr(layer.w, n) for n in NAMES]
    return (layer.w_router.data_ptr(), layer.router_bias.data_ptr(), [None if t is None else t.data_ptr() for t in w])


def test_a_step_reads_the_tensors_that_the_layer_has(monkeypatch):
    """A replaced router, bias, matrix, set of experts, or storage of one: the next step
    reads the new one (the old one may be gone)."""
    calls = host_calls(monkeypatch, fp8)
    layer, x = make(), torch.zeros(3, 64, dtype=torch.bfloat16)
    keep = []  # the old tensors live, so that no new one takes their address

    def step():
        layer.forward(x)
        assert seen(calls)[1:] == addresses(layer)

    step()
    for name in ("w_router", "router_bias"):
        keep.append(getattr(layer, name))
        setattr(layer, name, keep[-1].clone())
        step()
    for name in NAMES:
        keep.append(getattr(layer.w, name))
        setattr(layer.w, name, keep[-1].clone())
        step()
    keep.append(layer.w_router.data)
    layer.w_router.data = layer.w_router.data.clone()
    step()
    keep.append(layer.w)
    layer.w = experts()
    step()
    layer.router_bias = None
    layer.forward(x)
    assert seen(calls)[2] is None


def test_a_step_goes_by_the_sizes_that_the_layer_has(monkeypatch):
    calls = host_calls(monkeypatch, fp8)
    layer, x = make(), torch.zeros(3, 64, dtype=torch.bfloat16)
    layer.forward(x)
    assert (seen(calls)[0].k_max, seen(calls)[0].n_shared) == (2, 1)
    layer.k_max = 3
    layer.forward(x, topk_ids=torch.zeros((3, 3), dtype=torch.int32))
    assert seen(calls)[0].k_max == 3
    layer.w = experts(f=96, S=0)
    layer.forward(x)
    dm = seen(calls)[0]
    assert (dm.f, dm.n_shared) == (96, 0) and seen(calls)[3][3:] == [None] * 3
    # and the workspace is one for these sizes
    fn, args = calls[-1]
    assert args[-1] >= fp8._mx4_workspace_bytes(C.byref(dm))
    layer.k_max = 5
    with pytest.raises(fp8.MoEError, match="k_max"):
        layer.forward(x)


def test_a_replaced_tensor_that_does_not_fit_is_refused(monkeypatch):
    host_calls(monkeypatch, fp8)
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    for change, error, text in [
            (lambda l: setattr(l, "w_router", torch.zeros(3, 64)), ValueError, "w_router"),
            (lambda l: setattr(l, "router_bias", torch.zeros(4).double()), TypeError, "router_bias"),
            (lambda l: setattr(l.w, "w_up", l.w.w_up[:3]), ValueError, "w_up"),
            (lambda l: setattr(l.w, "w_down", l.w.w_down.to(torch.int8)), TypeError, "w_down"),
            (lambda l: setattr(l, "w", experts(E=8)), ValueError, "w_router")]:
        layer = make()
        layer.forward(x)
        change(layer)
        with pytest.raises(error, match=text):
            layer.forward(x)


def test_threads_do_not_meet_in_a_workspace(monkeypatch):
    """A step's launches write and read its workspace one after the other; a second
    thread's step on the same stream must not come between them."""
    import threading
    import time
    inside, met, steps = {}, [], []

    def run(fn, args):
        ws = args[-2]
        met.append(inside.get(ws, 0))
        inside[ws] = inside.get(ws, 0) + 1
        time.sleep(0.01)  # as ctypes does, the others are let on
        inside[ws] -= 1
        steps.append(args[-1])

    host_calls(monkeypatch, fp8, run)
    layer = make()
    # steps of several sizes: a larger workspace takes the place of a smaller one
    work = lambda T: [layer.forward(torch.zeros(T, 64, dtype=torch.bfloat16)) for _ in range(4)]
    threads = [threading.Thread(target=work, args=(T,)) for T in (1, 3, 20, 32)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(steps) == 16 and met == [0] * 16


def test_a_refused_step_leaves_the_layer_usable(monkeypatch):
    def run(fn, args):
        if not calls[1:]:
            raise fp8.MoEError(2)

    calls = host_calls(monkeypatch, fp8, run)
    layer, x = make(), torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(fp8.MoEError):
        layer.forward(x)
    layer.forward(x)
    assert len(calls) == 2


def test_sizes_past_32_bits_are_refused(monkeypatch):
    host_calls(monkeypatch, fp8)
    layer = make()
    layer.k_max = 2 ** 32 + 2  # 2 in 32 bits
    with pytest.raises(fp8.MoEError, match="k_max"):
        layer.forward(torch.zeros(3, 64, dtype=torch.bfloat16))
    for op in ("matmul_mx4", "gated_ffn_mx4"):
        assert fp8.mx4_form(op, 1, 64, 64)[0] == "stream 16"
        for bad in ((2 ** 32 + 1, 64, 64), (1, 2 ** 32 + 64, 64), (1, 64, 2 ** 32 + 64), (1 - 2 ** 32, 64, 64)):
            with pytest.raises(fp8.MoEError, match="moe_mx4_form"):
                fp8.mx4_form(op, *bad)


def test_workspaces_of_two_devices_are_two(monkeypatch):
    """A layer whose tensors moved to another device: the default streams have one handle."""
    host_calls(monkeypatch, fp8)
    layer, kept = make(), []
    for index in (0, 1, 0, 1):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: index)
        c = fp8._Call(layer.w_router, None)
        c.index = index
        kept.append(layer._workspace(c, 512).data_ptr())
    assert kept[0] == kept[2] != kept[1] == kept[3]
