"""The vectors' gradients of the norms' backward pass over many rows, exactly: on small
integers every product and every sum is an integer below 2^24, which fp32 holds in any
order, so that a row left out or counted twice shows in whole numbers."""
import pytest
import torch

from gpu_common import dev, lib
from test_gpu_dense import U, gen, within

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def integers(g, shape, low, high, t=F32):
    return torch.randint(low, high + 1, shape, generator=g, device=dev(), dtype=torch.int8).to(t)


def pairs(g, shape, low, high, t=F32, sign=1):
    """Columns 2i and 2i + 1 equal, or (sign -1) opposite."""
    v = integers(g, (*shape[:-1], shape[-1] // 2), low, high, t)
    return torch.stack([v, sign * v], -1).flatten(-2)


# T, d, gate rows: a gate row in hundreds of parts, the last one short; a few; one each; and
# several to a chunk, of one token or of many, behind the last chunk's end or not
@pytest.mark.parametrize("T,d,G,t", [
    (131075, 16384, 1, BF), (131075, 64, 0, BF), (131075, 512, 131075, BF), (131075, 1024, 1225, F16),
    (131075, 256, 5243, BF), (131075, 2048, 25, F16), (70001, 4096, 1, F32), (40003, 16384, 0, F32),
    (40000, 8192, 250, BF), (40000, 8192, 4000, F16), (8193, 1024, 1, BF), (1009, 512, 1009, F32),
    (513, 16384, 513, BF), (9000, 16384, 300, F16)])
def test_sums_over_many_rows(T, d, G, t):
    """With rstd of 1 the norms' rows are what they scale, and dn in opposite pairs
    against equal pairs of r leaves no mean: D = dr + dn w_next."""
    g = gen(T + d + G)
    x, y = pairs(g, (T, d), -2, 2, t), pairs(g, (T, d), -2, 2, t)
    dn, dr = pairs(g, (T, d), -2, 2, t, -1), integers(g, (T, d), -2, 2, t)
    w_post, w_next = pairs(g, (d,), 1, 2), pairs(g, (d,), 1, 2)
    gate = pairs(g, (G, d), -2, 2) if G else None
    one = torch.ones(T, device=dev())
    dx, dy, dw_post, dgate, dw_next = lib().norm_residual_backward(dr, dn, x, y, one, one, w_post, gate, w_next)
    sums = torch.zeros((2, d), dtype=torch.float64, device=dev())
    gsum = torch.zeros((max(G, 1), d), dtype=torch.float64, device=dev())
    wp, wn = w_post.double(), w_next.double()
    step = max(1, (1 << 25) // d)
    for a in range(0, T, step):
        rows = slice(a, min(a + step, T))
        of = torch.arange(rows.start, rows.stop, device=dev()) // (T // max(G, 1))
        xs, ys, ds, ns = (v[rows].double() for v in (x, y, dr, dn))
        gs = gate[of].double() if G else 1.0
        z = ys * wp
        D, r = ds + ns * wn, xs + gs * z
        assert torch.equal(dx[rows].double(), D)
        b = D * gs * wp
        m = (b * ys).mean(1, keepdim=True)
        # the mean and the difference are roundings of what they join; then the output's
        within(dy[rows], b - ys * m, 4 * U * (b.abs() + (ys * m).abs()), f"dy {a}")
        sums[0] += (D * gs * ys).sum(0)
        sums[1] += (ns * r).sum(0)
        gsum.index_add_(0, of, D * z)
    assert float(sums.abs().max()) < 2 ** 24 and float(gsum.abs().max()) < 2 ** 24
    assert torch.equal(dw_post.double(), sums[0]) and torch.equal(dw_next.double(), sums[1])
    if G:
        assert torch.equal(dgate.double(), gsum)
