"""The 4-bit mixture-of-experts layer of a few tokens on the GPU: picks exactly,
outputs element by element against 64 bits (bounds: mx4_ref.py)."""
import pytest
import torch

import mx4_ref
from gpu_common import dev, lib
from test_gpu_dense import F16S, gen, guarded, normal, strided, within

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, d, f, E, k, S=0, bias=False, seed=0):
        g = self.g = gen(seed + d + f + E)
        self.d, self.f, self.E, self.k = d, f, E, k
        self.router = normal(g, (E, d), d ** -0.5)
        self.bias = normal(g, (E,)) if bias else None
        w = lib().Mx4Experts.empty(E, d, f, S)
        self.values = []
        for e in range(E + S):
            three = []
            for which, shape in (("gate", (f, d)), ("up", (f, d)), ("down", (d, f))):
                codes, scales = lib().quantize_rows_mx4(normal(g, shape, shape[1] ** -0.5))
                w.set_expert(which, e if e < E else e - E, codes, scales, shared=e >= E)
                three.append(mx4_ref.values(codes, scales))
            self.values.append(tuple(three))
        self.op = lib().Mx4MoELayer(w, self.router, k, self.bias)

    def logits(self, x):
        s = x.double() @ self.router.double().t()
        return (s if self.bias is None else s + self.bias.double()).float()

    def check(self, x, kpt=None, override=None, what=""):
        T = x.shape[0]
        ids = torch.full((T, self.k), -7, dtype=torch.int32, device=dev())
        w = torch.full((T, self.k), -7.0, device=dev())
        out, ok = guarded((T, self.d), x.dtype)
        self.op.forward(x, k_per_token=kpt, logits_override=override, out=out, topk_ids=ids, topk_w=w)
        ok()
        rid, p = mx4_ref.routing(self.logits(x) if override is None else override, self.k, kpt)
        assert torch.equal(ids.long(), rid), what
        assert float((w.double() - p).abs().max()) <= 64 * mx4_ref.U
        ref, tol = mx4_ref.layer(x, rid, p, self.values[:self.E], self.values[self.E:])
        within(out, ref, tol, what)
        assert torch.equal(out, self.op.forward(x, k_per_token=kpt, logits_override=override))
        return out


@pytest.mark.parametrize("dtype", F16S)
@pytest.mark.parametrize("d,f,E,k,S", [(32, 32, 1, 1, 0), (64, 96, 4, 2, 0), (256, 512, 8, 2, 1),
                                       (544, 160, 70, 5, 2), (2048, 768, 128, 8, 0), (160, 1056, 130, 6, 0),
                                       (96, 64, 512, 32, 3), (1056, 2080, 3, 3, 0)])
def test_tokens_and_shapes(d, f, E, k, S, dtype):
    layer = Layer(d, f, E, k, S, bias=E % 2 == 0)
    for T in (1, 2, 3, 15, 16, 17, 31, 32):
        layer.check(strided(normal(layer.g, (T, d), 1, dtype), 8 if T % 2 else 0), what=f"T {T}")


@pytest.mark.parametrize("T,d,f,E,k", [
    (8, 6144, 32, 3, 2), (8, 6176, 32, 3, 2), (8, 8192, 256, 64, 8), (8, 8224, 256, 64, 8),
    (8, 8224, 512, 64, 8), (16, 3200, 32, 5, 4), (32, 2048, 512, 40, 8), (32, 2080, 512, 40, 8),
    (32, 2080, 512, 64, 8), (9, 4096, 1056, 16, 16)])
def test_activations_at_the_ends_of_what_lds_holds(T, d, f, E, k):
    """The most that fits beside the plan, with items for a wave each and for several
    waves together, and a little more than that."""
    layer = Layer(d, f, E, k)
    layer.check(normal(layer.g, (T, d), 1, torch.float16), what=f"T {T} d {d}")


def test_per_token_budgets_ties_and_given_logits():
    layer = Layer(128, 64, 16, 6, 1)
    for T in (5, 32):
        x = normal(layer.g, (T, 128), 1, torch.bfloat16)
        kpt = torch.randint(1, 7, (T,), device=dev(), generator=layer.g, dtype=torch.int32)
        layer.check(x, kpt=kpt)
        layer.check(x, override=torch.zeros((T, 16), device=dev()))  # all tie
        lumps = torch.randint(-2, 3, (T, 16), device=dev(), generator=layer.g).float()
        layer.check(x, kpt=kpt, override=lumps)
        one = torch.zeros((T, 16), device=dev())
        one[:, 9], one[:, 3] = 20, 10  # every token on the same experts
        layer.check(x, override=one)


def test_logits_are_summed_in_64_bits():
    """Two experts whose scores differ by less than an fp32 sum's rounding."""
    d, E = 4096, 8
    layer = Layer(d, 32, E, 2)
    x = (normal(layer.g, (4, d)) * 100).bfloat16()
    layer.router[:] = layer.router[0]
    layer.router[:, 0] += torch.arange(E, device=dev()) * 2.0 ** -22
    layer.check(x)


@pytest.mark.parametrize("T", [4, 20])
def test_a_poisoned_token_stays_alone(T):
    layer = Layer(256, 128, 8, 2, 1)
    x = normal(layer.g, (T, 256), 1, torch.bfloat16)
    clean = layer.op.forward(x)
    x[2] = torch.nan
    ids = torch.empty((T, 2), dtype=torch.int32, device=dev())
    got = layer.op.forward(x, topk_ids=ids)
    keep = torch.arange(T, device=dev()) != 2
    assert torch.equal(got[keep], clean[keep]) and bool(got[2].isnan().all())
    assert bool(((ids >= 0) & (ids < 8)).all())


def test_no_tokens_other_sizes_and_a_workspace_that_was_filled():
    """Steps of changing size on one layer; what a workspace held before does not matter."""
    layer = Layer(96, 96, 8, 2, 1)
    assert layer.op.forward(torch.empty((0, 96), dtype=torch.bfloat16, device=dev())).shape == (0, 96)
    for T in (3, 32, 1, 9, 32):
        x = normal(layer.g, (T, 96), 1, torch.bfloat16)
        a = layer.check(x, what=f"T {T}")
        for ws in layer.op._ws.values():
            ws.fill_(0xFF)
        assert torch.equal(a, layer.op.forward(x))


def test_streams_and_graphs():
    """Two streams at once, each with a workspace of its own; graphs captured and
    replayed with eager steps of the same layer between."""
    layer = Layer(512, 256, 16, 4, 1)
    xs = [normal(layer.g, (T, 512), 1, torch.float16) for T in (1, 12, 32)]
    want = [layer.op.forward(x) for x in xs]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    got = [[layer.op.forward(x, stream=s) for s in (a, b)] for _ in range(3) for x in xs]
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        assert all(torch.equal(o, want[i % 3]) for o in pair)
    graphs = []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer.op.forward(x)
        graphs.append((graph, out))
    for k in range(4):
        for x in xs:
            x.copy_(normal(gen(k), tuple(x.shape), 1, torch.float16))
        for graph, _ in graphs:
            graph.replay()
        eager = [layer.op.forward(x) for x in xs]
        torch.cuda.synchronize()
        assert all(torch.equal(o, e) for (_, o), e in zip(graphs, eager)), k


def test_a_decode_step_as_it_is_served():
    """Norm, layer, norms and residual sum of a step on the same stream, eager and as a
    replayed graph: each step against its own formula on what the step before gave."""
    import norm_ref
    layer = Layer(512, 256, 16, 4, 1)
    g, t = layer.g, torch.bfloat16
    w = [(1 + 0.2 * normal(g, (512,))).to(t) for _ in range(3)]
    for T in (1, 7, 32):
        x = normal(g, (T, 512), 1, t)

        def step():
            n = lib().rms_norm(x, w[0])
            y = layer.op.forward(n)
            return (n, y) + lib().norm_residual(x, y, w[1], None, w[2], scale=0.5)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for k in range(3):
            x.copy_(normal(gen(k + T), (T, 512), 1, t))
            graph.replay()
            eager = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, eager)), k
        n, y, r, m = eager
        ref, err = norm_ref.forward(x, None, None, None, w[0], 1.0, 1e-6, 0.0)
        within(n, ref[1], err[1], "n")
        ids, p = mx4_ref.routing(layer.logits(n), layer.k)
        within(y, *mx4_ref.layer(n, ids, p, layer.values[:16], layer.values[16:]), "y")
        ref, err = norm_ref.forward(x, y, w[1], None, w[2], 0.5, 1e-6, 0.0)
        within(r, ref[0], err[0], "r")
        within(m, ref[1], err[1], "m")


def debug_calls(monkeypatch):
    """The package's new calls go to the device-checked build."""
    import ctypes as C
    m = lib()
    if not m.DEBUG_LIB_PATH.exists():
        pytest.fail("libfp8moe_debug.so is not built (fp8_moe_layer_amd/build.py --debug)")
    dbg = C.CDLL(str(m.DEBUG_LIB_PATH))
    for name, symbol in (("_mx4_forward", "moe_mx4_forward"), ("_matmul_mx4", "moe_matmul_mx4"),
                         ("_ffn_mx4", "moe_ffn_mx4"), ("_norm_residual", "moe_norm_residual"),
                         ("_norm_bwd", "moe_norm_residual_backward")):
        fn, old = getattr(dbg, symbol), getattr(m, name)
        fn.restype, fn.argtypes = old.restype, old.argtypes
        monkeypatch.setattr(m, name, fn)


@pytest.mark.parametrize("T", [2, 20])
def test_debug_build(T, monkeypatch):
    """The same bits as the release library on valid inputs; a budget outside its range
    and a logit that is no number are named, and stay within bounds (the kernels clamp
    the one and give the other's token some experts)."""
    layer = Layer(256, 128, 8, 4, 1)
    x = normal(layer.g, (T, 256), 1, torch.bfloat16)
    w = torch.ones(256, device=dev(), dtype=torch.bfloat16)

    def outputs():
        y = layer.op.forward(x)
        r, n, sy, sr = lib().norm_residual(x, y, w, None, w, save=True)
        return (y, r, n) + lib().norm_residual_backward(r, n, x, y, sy, sr, w, None, w)

    want = [o for o in outputs() if o is not None]
    debug_calls(monkeypatch)
    got = [o for o in outputs() if o is not None]
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    kpt = torch.full((T,), 4, dtype=torch.int32, device=dev())
    kpt[1] = 9
    with pytest.raises(lib().MoEError) as e:
        layer.op.forward(x, k_per_token=kpt)
    assert e.value.status == 7
    logits = torch.zeros((T, 8), device=dev())
    logits[0, 3] = torch.nan
    with pytest.raises(lib().MoEError) as e:
        layer.op.forward(x, logits_override=logits)
    assert e.value.status == 7


def test_refusals_on_the_device():
    f = lib()
    layer = Layer(64, 32, 4, 2)
    x = torch.ones((2, 64), dtype=torch.bfloat16, device=dev())
    with pytest.raises(f.MoEError, match="T=33"):
        layer.op.forward(x[:1].repeat(33, 1))
    with pytest.raises(TypeError, match="expected one of"):
        layer.op.forward(x.float())
    with pytest.raises(ValueError, match="shape"):
        layer.op.forward(x[:, :32])
    with pytest.raises(ValueError, match="topk_ids"):
        layer.op.forward(x, topk_ids=torch.empty((2, 3), dtype=torch.int32, device=dev()))
    with pytest.raises(f.MoEError, match="k_max"):
        f.Mx4MoELayer(layer.op.w, layer.router, 5).forward(x)
    with pytest.raises(f.MoEError, match="logits_override is required"):
        f.Mx4MoELayer(layer.op.w, None, 2).forward(x)
    with pytest.raises(ValueError, match="w_router"):
        f.Mx4MoELayer(layer.op.w, layer.router[:2], 2)
    with pytest.raises(ValueError, match="codes: expected shape"):
        layer.op.w.set_expert("gate", 0, *f.quantize_rows_mx4(torch.ones((64, 32), device=dev())))


def test_inputs_that_autograd_records_are_refused():
    """Every call of the set, for each tensor whose gradient would be lost; under
    no_grad they pass, and forward-mode tangents are refused too."""
    f = lib()
    new = lambda *shape, dtype=torch.bfloat16: torch.ones(shape, dtype=dtype, device=dev())
    layer = Layer(64, 32, 4, 2, bias=True)
    w = f.pack_mx4(*f.quantize_rows_mx4(new(32, 64)))
    x, y, v, rstd = new(2, 64), new(2, 64), new(64), new(2, dtype=torch.float32)
    calls = [
        (f.quantize_rows_mx4, [x]), (lambda a, b: f.matmul_mx4(a, w, b), [x, new(32, dtype=torch.float32)]),
        (lambda a: f.gated_ffn_mx4(a, w, w), [x]), (f.rms_norm, [x, v]),
        (f.norm_residual, [x, y, v, new(1, 64), v]),
        (lambda a, b, c, d: f.rms_norm_backward(a, b, c, rstd, dr=d), [x, y, v, x]),
        (lambda a, b, c, d, e, g, h: f.norm_residual_backward(a, b, c, d, rstd, rstd, e, g, h),
         [x, x, y, y, v, new(1, 64), v]),
        (layer.op.forward, [x]),
        (lambda a, b: f.Mx4MoELayer(layer.op.w, a, 2, b).forward(x), [layer.router, layer.bias]),
    ]
    for call, tensors in calls:
        call(*tensors)
        for i in range(len(tensors)):
            one = [t.clone().requires_grad_(j == i) for j, t in enumerate(tensors)]
            with pytest.raises(RuntimeError, match="not recorded by autograd"):
                call(*one)
            with torch.no_grad():
                call(*one)
            with torch.autograd.forward_ad.dual_level():
                dual = [torch.autograd.forward_ad.make_dual(t, t) if j == i else t
                        for j, t in enumerate(tensors)]
                with pytest.raises(RuntimeError):
                    call(*dual)
