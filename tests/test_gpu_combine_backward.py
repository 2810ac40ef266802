"""Gradient of the combine on the GPU: dy bit-exact (one rounding of an fp32
product), the gates' gradient within the bound of its fp32 sums."""
import numpy as np
import pytest

from experts_harness import guarded, layout_of_ids, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import torch
    import __graft_entry__ as ge
    ge.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import combine_moe_layout_04_gb300 as m
    return m


def _run(moe, prob, lay, dout, y, w):
    import torch
    dy, t0 = guarded(tuple(y.shape), torch.bfloat16, 0xC3)
    dw, t1 = guarded(tuple(w.shape), torch.float32, 0xC3)
    moe.moe_combine_backward(prob, lay, dout, y, w, dy, dw)
    torch.cuda.synchronize()
    assert bool((t0 == 0xC3).all()) and bool((t1 == 0xC3).all())
    return dy, dw


def _problem(moe, T, k, E, h, seed=0):
    ids = np.argsort(np.random.default_rng(seed).random((T, E)), axis=1)[:, :k]
    return layout_of_ids(moe, ids, E, hidden=h)


@pytest.mark.parametrize("T,k,E,h", [(1, 1, 1, 8), (1, 8, 256, 7168), (3, 2, 4, 16), (131, 8, 16, 1000), (257, 9, 12, 2056),
                                     (64, 32, 40, 264), (500, 4, 8, 4104), (2, 17, 33, 32768)])
def test_matches_definition(moe, T, k, E, h):
    import torch
    prob, lay = _problem(moe, T, k, E, h)
    dout, y = randn((T, h), 1), randn((T * k, h), 2)
    w = torch.rand((T, k), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    dy, dw = _run(moe, prob, lay, dout, y, w)
    pos = lay.pos.long()
    want = torch.empty_like(dy)
    want[pos.reshape(-1)] = (w[..., None] * dout.float()[:, None, :]).to(torch.bfloat16).flatten(0, 1)
    assert torch.equal(dy, want)
    a, b = dout.double()[:, None, :], y.double()[pos]
    ref, mag = (a * b).sum(-1), (a * b).abs().sum(-1)
    # fp32 fma chains of h / 256 steps of 8, then 13 additions of partial sums: a rounding of the running magnitude each
    assert bool(((dw.double() - ref).abs() <= mag * (h / 256 + 8 + 16) * 2.0 ** -24).all())


@pytest.mark.parametrize("T,k,h", [(700, 3, 8), (700, 2, 256), (700, 2, 264), (640, 2, 512), (650, 9, 520), (615, 3, 1032),
                                   (620, 2, 7168), (160, 3, 1032), (160, 2, 4096), (151, 2, 2056), (100, 1, 520),
                                   (700, 1, 520), (700, 4, 264), (640, 5, 256), (151, 4, 7168), (160, 5, 2056), (20, 5, 1032)])
def test_every_block_size(moe, T, k, h):
    """Many, some and few tokens at row widths on both sides of each block size."""
    import torch
    prob, lay = _problem(moe, T, k, 12, h)
    dout, y = randn((T, h), 1), randn((T * k, h), 2)
    w = torch.rand((T, k), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    dy, dw = _run(moe, prob, lay, dout, y, w)
    pos = lay.pos.long()
    want = torch.empty_like(dy)
    want[pos.reshape(-1)] = (w[..., None] * dout.float()[:, None, :]).to(torch.bfloat16).flatten(0, 1)
    assert torch.equal(dy, want)
    a, b = dout.double()[:, None, :], y.double()[pos]
    # groups of 8 products, at most h / 256 groups a thread, 5 additions over lanes and at most 16 over warps
    assert bool(((dw.double() - (a * b).sum(-1)).abs() <= (a * b).abs().sum(-1) * (8 + h / 256 + 1 + 21) * 2.0 ** -24).all())


def test_gates_of_zero_and_values_that_are_not_finite(moe):
    import torch
    prob, lay = _problem(moe, 10, 3, 6, 64)
    dout, y = randn((10, 64), 1), randn((30, 64), 2)
    w = torch.rand((10, 3), device="cuda")
    w[4] = 0.0
    dout[2, 5] = float("inf")
    dy, dw = _run(moe, prob, lay, dout, y, w)
    pos = lay.pos.long()
    assert bool((dy[pos[4]] == 0).all())
    assert not bool(torch.isfinite(dw[2]).any())
    keep = [t for t in range(10) if t != 2]
    assert bool(torch.isfinite(dw[keep]).all())


def test_bad_positions_are_skipped(moe):
    """Positions out of range: nothing is written for them and their gate gradient is 0."""
    import torch
    prob, lay = _problem(moe, 6, 2, 4, 64)
    lay.pos[1, 0], lay.pos[3, 1] = -5, 12
    dout, y, w = randn((6, 64), 1), randn((12, 64), 2), torch.ones((6, 2), device="cuda")
    dy, dw = _run(moe, prob, lay, dout, y, w)
    assert float(dw[1, 0]) == 0 and float(dw[3, 1]) == 0
    rows = lay.pos[lay.pos.ge(0) & lay.pos.lt(12)].long()
    left = [r for r in range(12) if r not in rows.tolist()]
    assert len(left) == 2 and bool((dy[left].view(torch.uint8) == 0xC3).all())


def test_gradient_against_differences(moe):
    """The slope of sum(combine(y, w) * dout) along changes of y and w; the sum is bilinear, so the
    difference of 64-bit values is exact up to its rounding."""
    import torch
    T, k, h = 40, 4, 136
    prob, lay = _problem(moe, T, k, 9, h)
    dout, y = randn((T, h), 1), randn((T * k, h), 2)
    w = torch.rand((T, k), device="cuda")
    dy, dw = _run(moe, prob, lay, dout, y, w)
    pos = lay.pos.long()
    way_y, way_w = randn(y.shape, 7).double(), randn(w.shape, 8).double()

    def value(y, w):
        return ((w[..., None] * y[pos]).sum(1) * dout.double()).sum()
    step = 2.0 ** -10
    base = [y.double(), w.double()]
    slope_y = (value(base[0] + step * way_y, base[1]) - value(base[0] - step * way_y, base[1])) / (2 * step)
    slope_w = (value(base[0], base[1] + step * way_w) - value(base[0], base[1] - step * way_w)) / (2 * step)
    got_y, got_w = dy.double() * way_y, dw.double() * way_w
    assert abs(float(slope_y - got_y.sum())) <= 2.0 ** -8 * float(got_y.abs().sum())
    assert abs(float(slope_w - got_w.sum())) <= 1e-5 * float((dout.double()[:, None, :] * y.double()[pos] * way_w[..., None]).abs().sum())
