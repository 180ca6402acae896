"""The 4-bit mixture-of-experts layer as an object that a server keeps: its tensors
replaced between steps, and threads that share it."""
import pytest
import torch

from gpu_common import dev, lib
from test_gpu_dense import normal
from test_gpu_mx4_moe import Layer

pytestmark = pytest.mark.gpu


def matrices(w):
    return [n for n in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down") if getattr(w, n) is not None]


@pytest.mark.parametrize("T", [3, 20])
def test_replaced_tensors(T):
    """After each replacement a step gives the bits of a layer made from the same tensors."""
    f, a, b = lib(), Layer(256, 128, 8, 2, 1, bias=True, seed=1), Layer(256, 128, 8, 2, 1, bias=True, seed=2)
    x = normal(a.g, (T, 256), 1, torch.bfloat16)
    first = a.op.forward(x)

    def step():
        y = a.op.forward(x)
        torch.cuda.synchronize()
        assert torch.equal(y, f.Mx4MoELayer(a.op.w, a.op.w_router, a.op.k_max, a.op.router_bias).forward(x))
        return y

    last = step()
    assert torch.equal(last, first)
    for name in ("w_router", "router_bias"):
        setattr(a.op, name, getattr(b.op, name))
        y = step()
        assert not torch.equal(y, last), name
        last = y
    for name in matrices(b.op.w):
        setattr(a.op.w, name, getattr(b.op.w, name))
        y = step()
        assert not torch.equal(y, last), name
        last = y
    assert torch.equal(last, b.op.forward(x))
    a.op.k_max = 3
    assert not torch.equal(step(), last)
    a.op.w = Layer(256, 512, 8, 2, 0, seed=3).op.w  # other sizes, a larger workspace
    step()
    a.op.w_router = torch.zeros((7, 256), device=dev())
    with pytest.raises(ValueError, match="w_router"):
        a.op.forward(x)


@pytest.mark.parametrize("streams", [1, 2])
def test_threads_share_a_layer(streams):
    """Four threads' steps of several sizes at once, on one stream or on two: the bits
    that a thread alone gets."""
    import threading
    layer = Layer(512, 1056, 16, 4, 1, bias=True)
    sizes = (1, 7, 13, 32)
    xs = {T: [normal(layer.g, (T, 512), 1, torch.bfloat16) for _ in range(5)] for T in sizes}
    fresh = lib().Mx4MoELayer(layer.op.w, layer.op.w_router, layer.op.k_max, layer.op.router_bias)
    want = {T: [layer.op.forward(x) for x in xs[T]] for T in sizes}
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(streams)] if streams > 1 else [None]
    got, failed, start = {}, [], threading.Barrier(len(sizes))

    def work(i, T):
        try:
            start.wait(timeout=30)
            got[T] = [fresh.forward(xs[T][k % 5], stream=side[i % streams]) for k in range(60)]
        except Exception as e:  # noqa: BLE001 -- told by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i, T)) for i, T in enumerate(sizes)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    torch.cuda.synchronize()
    assert not failed, failed
    for T in sizes:
        assert all(torch.equal(y, want[T][k % 5]) for k, y in enumerate(got[T])), T


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [4, 20])
@pytest.mark.parametrize("d,f", [(64, 96), (2048, 1056)])
def test_an_infinite_activation_stays_an_infinity(d, f, T, dtype):
    """All weights of one sign to an output: a token whose gate and up are infinite gets
    infinities of those signs, as the formula has them, and the others their own values."""
    m, E = lib(), 4
    w = m.Mx4Experts.empty(E, d, f, 1)
    one = torch.ones((f, d), device=dev()) / d
    sign = torch.where(torch.arange(d, device=dev()) % 3 == 0, -1.0, 1.0)
    for e in range(E + 1):
        for which, v in (("gate", one), ("up", one), ("down", sign[:, None] * torch.ones((d, f), device=dev()) / f)):
            w.set_expert(which, e % E, *m.quantize_rows_mx4(v), shared=e == E)
    layer = m.Mx4MoELayer(w, None, 2)
    logits = torch.zeros((T, E), device=dev())
    x = torch.ones((T, d), device=dev(), dtype=dtype)
    clean = layer.forward(x, logits_override=logits)
    assert bool(clean.isfinite().all())
    x[1, 5] = torch.inf
    if dtype == torch.bfloat16:
        x[3] = 3e38  # g and u are finite, their product is not
    got = layer.forward(x, logits_override=logits)
    bad = [1, 3] if dtype == torch.bfloat16 else [1]
    keep = torch.ones(T, dtype=torch.bool, device=dev())
    keep[bad] = False
    assert torch.equal(got[keep], clean[keep])
    for t in bad:
        assert torch.equal(got[t].float(), sign * torch.inf), t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 4, 20, 32])
def test_a_scale_that_is_none_stays_with_its_expert(T, dtype):
    """A scale byte of 255 in one expert's down projection: that channel of its tokens."""
    layer = Layer(64, 96, 4, 2, 1)
    codes, scales = lib().quantize_rows_mx4(normal(layer.g, (64, 96), 0.1))
    layer.op.w.set_expert("down", 0, codes, scales)
    x = normal(layer.g, (T, 64), 1, dtype)
    logits = torch.zeros((T, 4), device=dev())
    logits[:, 0] = -9
    logits[T // 2, 0] = 9  # one token alone is on expert 0
    clean = layer.op.forward(x, logits_override=logits)
    scales[7, 1] = 255
    layer.op.w.set_expert("down", 0, codes, scales)
    got = layer.op.forward(x, logits_override=logits)
    want = clean.clone()
    want[T // 2, 7] = torch.nan
    assert bool(clean.isfinite().all()) and torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())
