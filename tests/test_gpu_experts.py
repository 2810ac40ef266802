"""The experts' grouped products on the GPU against 64-bit products: forward
(plain and gated), gradients of rows (plain and through the activation) and of
weights, over ragged groups, odd widths and placements."""
import numpy as np
import pytest

from experts_harness import (close, gated, gated_slack, guarded, layout_of_counts, layout_of_ids, products, randn,
                             spans, sum_slack)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import torch
    import __graft_entry__ as ge
    ge.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import combine_moe_layout_04_gb300 as m
    yield m
    assert m.moe_move_faults() == 0


# rows per expert: none, one, around the tile sizes, many, empty experts at both ends
COUNTS = {
    "one row": [0, 0, 1, 0],
    "tile edges": [1, 127, 128, 129, 0, 255, 256, 257],
    "skewed": [0, 3, 700, 0, 16, 17, 64, 1, 0],
    "a little over a tile": [257, 272, 300, 0, 320, 321, 255, 290],
    "a tile and a half": [384, 360, 385, 350, 400, 0, 391],
    "some dozens": [40, 64, 65, 33, 50, 0, 17],
    "about a hundred": [90, 104, 128, 129, 72, 0, 100],
    "few each": [2, 1, 0, 3, 1, 1, 2, 0, 0, 1, 4, 1, 0, 1, 2, 1],
}
# (in_cols, out_cols): multiples of 8 that fill no tile, one tile, several
WIDTHS = [(8, 8), (64, 128), (72, 136), (200, 264), (1024, 512), (520, 1016)]


def _forward(moe, prob, lay, K, N, act, seed=0, rows=None, weights=None, want_pre=True):
    import torch
    R, E = prob.num_tokens * prob.topk, prob.num_experts
    W = 2 * N if act else N
    rows = randn((R, K), seed) if rows is None else rows
    weights = randn((E, W, K), seed + 1, K ** -0.5) if weights is None else weights
    x = moe.Experts(K, N, weights, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)
    out, tail = guarded((R, N), torch.bfloat16, 0xC3)
    pre, pre_tail = guarded((R, W), torch.bfloat16, 0xC3) if act and want_pre else (None, None)
    moe.moe_expert_forward(prob, lay, x, rows, out, pre=pre)
    torch.cuda.synchronize()
    assert bool((tail == 0xC3).all()) and (pre is None or bool((pre_tail == 0xC3).all()))
    return rows, weights, out, pre


def _check_forward(lay, rows, weights, out, pre, act):
    ref, mag = products(lay, rows, weights)
    slack = sum_slack(mag, rows.shape[1])
    if not act:
        return close(out, ref, slack)
    if pre is not None:
        close(pre, ref, slack)
    close(out, gated(ref), gated_slack(ref, slack))


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
def test_forward(moe, counts, K, N, act):
    prob, lay = layout_of_counts(moe, counts)
    _check_forward(lay, *_forward(moe, prob, lay, K, N, act), act)


def test_gate_far_out(moe):
    """Gates from -100 to 100 (one weight, so that a row is its own gate): silu keeps its relative accuracy where
    exp(-g) nears and passes the largest float, and its gradient too."""
    import torch
    g = torch.linspace(-100, 100, 4096, device="cuda").to(torch.bfloat16)
    counts = [4096]
    prob, lay = layout_of_counts(moe, counts)
    rows = torch.zeros((4096, 8), dtype=torch.bfloat16, device="cuda")
    rows[:, 0], rows[:, 1] = g, 3.0
    w = torch.zeros((1, 16, 8), dtype=torch.bfloat16, device="cuda")
    w[0, :8, 0], w[0, 8:, 1] = 1.0, 1.0
    out = torch.empty((4096, 8), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_forward(prob, lay, moe.Experts(8, 8, w, act=moe.MOE_ACT_SWIGLU), rows, out)
    x = g.double()
    # exp(-g) past the largest float is infinity: 0 there (the true value is below 2^-121)
    close(out[:, 0], 3 * x * torch.sigmoid(x), 2.0 ** -20 * 3 * (x * torch.sigmoid(x)).abs() + 2.0 ** -119 * (x < -88))
    pre = torch.stack((g, torch.full_like(g, 3.0)), 1).repeat_interleave(8, 1).contiguous()
    dout = torch.ones((4096, 8), dtype=torch.bfloat16, device="cuda")
    eye = torch.eye(8, dtype=torch.bfloat16, device="cuda")[None].contiguous()
    drows = torch.empty((4096, 16), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_backward_rows(prob, lay, moe.Experts(8, 8, eye), dout, drows, pre=pre)
    s = torch.sigmoid(x)
    low = 2.0 ** -119 * (x < -88)
    close(drows[:, 0], 3 * s * (1 + x * (1 - s)), 2.0 ** -20 * 3 * s * (1 + x.abs()) + low)
    close(drows[:, 8], x * s, 2.0 ** -20 * (x * s).abs() + low)


def test_forward_without_pre(moe):
    prob, lay = layout_of_counts(moe, COUNTS["tile edges"])
    a = _forward(moe, prob, lay, 136, 200, True)
    b = _forward(moe, prob, lay, 136, 200, True, want_pre=False)
    assert (a[2].view(b[2].dtype) == b[2]).all()


@pytest.mark.parametrize("act", [False, True])
def test_forward_many_rows(moe, act):
    """Groups of several row tiles and contractions of many steps."""
    prob, lay = layout_of_counts(moe, [900, 0, 1300, 411])
    _check_forward(lay, *_forward(moe, prob, lay, 2048, 776, act), act)


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1], [5, 64, 0, 65], [17] * 8, [1] * 20])
@pytest.mark.parametrize("K", [768, 2056, 7168])
def test_few_tiles_and_long_sums(moe, counts, K):
    """Contractions that are cut into parts because there are few tiles, every way round."""
    prob, lay = layout_of_counts(moe, counts)
    for act, N in ((True, 72), (False, 520)):
        _check_forward(lay, *_forward(moe, prob, lay, K, N, act), act)
    weights, dout, rows, pre, drows, dw = _backward(moe, prob, lay, 136, K, False, True)
    _check_rows(lay, weights, dout, pre, drows)
    _check_weights(lay, rows, dout, dw)
    again = _backward(moe, prob, lay, 136, K, False, True)
    assert (drows.view(torch_uint16()) == again[4].view(torch_uint16())).all()


def torch_uint16():
    import torch
    return torch.int16


def test_forward_top_k_and_placement(moe):
    """Top-8 of 64 experts on 8 ranks out of order: offsets do not ascend with the expert."""
    rng = np.random.default_rng(3)
    ids = np.argsort(rng.random((173, 64)), axis=1)[:, :8]
    e2r = rng.permutation(np.repeat(np.arange(8), 8))
    prob, lay = layout_of_ids(moe, ids, 64, e2r.tolist(), 8)
    off = [s[1] for s in spans(lay)]
    assert off != sorted(off)
    _check_forward(lay, *_forward(moe, prob, lay, 328, 264, True), True)
    _check_forward(lay, *_forward(moe, prob, lay, 328, 264, False), False)


def test_forward_1024_experts(moe):
    counts = np.random.default_rng(8).integers(0, 4, 1024)
    counts[[0, 500, 1023]] = 0, 130, 1
    prob, lay = layout_of_counts(moe, counts.tolist())
    _check_forward(lay, *_forward(moe, prob, lay, 64, 72, True), True)


def _backward(moe, prob, lay, K, N, act, through, seed=0, rows=None, dout=None, weights=None):
    import torch
    R, E = prob.num_tokens * prob.topk, prob.num_experts
    W = 2 * N if act else N
    weights = randn((E, W, K), seed + 1, W ** -0.5) if weights is None else weights
    dout = randn((R, W), seed + 2) if dout is None else dout
    rows = randn((R, K), seed + 3) if rows is None else rows
    pre = randn((R, 2 * K), seed + 4, 2.0) if through else None
    x = moe.Experts(K, N, weights, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)
    drows, t0 = guarded((R, 2 * K if through else K), torch.bfloat16, 0xC3)
    dw, t1 = guarded((E, W, K), torch.bfloat16, 0xC3)
    moe.moe_expert_backward_rows(prob, lay, x, dout, drows, pre=pre)
    moe.moe_expert_backward_weights(prob, lay, x, rows, dout, dw)
    torch.cuda.synchronize()
    assert bool((t0 == 0xC3).all()) and bool((t1 == 0xC3).all())
    return weights, dout, rows, pre, drows, dw


def _check_rows(lay, weights, dout, pre, drows):
    import torch
    dh, mag = products(lay, dout, weights.transpose(1, 2))
    slack = sum_slack(mag, dout.shape[1])
    if pre is None:
        return close(drows, dh, slack)
    g, u = pre.double().chunk(2, dim=1)
    s = torch.sigmoid(g)
    # fp32 evaluation: at most 16 roundings of the factors' magnitudes
    fu, fg = u * s * (1 + g * (1 - s)), g * s
    mu = u.abs() * s * (1 + g.abs())
    close(drows, torch.cat((dh * fu, dh * fg), 1),
          torch.cat((slack * (fu.abs() + 2.0 ** -20 * mu) + 2.0 ** -20 * dh.abs() * mu,
                     slack * (1 + 2.0 ** -20) * fg.abs() + 2.0 ** -20 * (dh * fg).abs()), 1))


def _check_weights(lay, rows, dout, dw):
    for e, r0, n in spans(lay):
        d, x = dout[r0:r0 + n].double(), rows[r0:r0 + n].double()
        if n == 0:
            assert bool((dw[e].view(dtype=dw.dtype) == 0).all())
        else:
            close(dw[e], d.T @ x, sum_slack(d.abs().T @ x.abs(), n))


@pytest.mark.parametrize("through", [False, True])
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
def test_backward(moe, counts, K, N, through):
    prob, lay = layout_of_counts(moe, counts)
    weights, dout, rows, pre, drows, dw = _backward(moe, prob, lay, K, N, False, through)
    _check_rows(lay, weights, dout, pre, drows)
    _check_weights(lay, rows, dout, dw)


def test_backward_of_gated_weights(moe):
    """The gate and up product's own backward: dout is the gradient of pre, [R, 2 * out_cols]."""
    prob, lay = layout_of_counts(moe, COUNTS["tile edges"])
    weights, dout, rows, pre, drows, dw = _backward(moe, prob, lay, 264, 136, True, False)
    _check_rows(lay, weights, dout, pre, drows)
    _check_weights(lay, rows, dout, dw)


def test_backward_many_rows_and_placement(moe):
    rng = np.random.default_rng(4)
    ids = np.argsort(rng.random((700, 12)), axis=1)[:, :3]
    prob, lay = layout_of_ids(moe, ids, 12, rng.permutation(np.repeat(np.arange(4), 3)).tolist(), 4)
    weights, dout, rows, pre, drows, dw = _backward(moe, prob, lay, 1096, 776, False, True)
    _check_rows(lay, weights, dout, pre, drows)
    _check_weights(lay, rows, dout, dw)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_neighbours_do_not_leak(moe, bad):
    """Rows and weights of one expert that are not finite leave every other expert's results as they are:
    tiles reach over the ends of groups and of weights, and must not mix them in."""
    import torch
    counts, K, N = [130, 5, 0, 77, 128], 136, 200
    prob, lay = layout_of_counts(moe, counts)
    R = sum(counts)
    hurt = 1
    own = torch.zeros(R, dtype=torch.bool, device="cuda")
    _, r0, n = spans(lay)[hurt]
    own[r0:r0 + n] = True
    rows, dout = randn((R, K), 1), randn((R, N), 2)
    wf, wb = randn((5, 2 * N, K), 3, K ** -0.5), randn((5, N, K), 4, N ** -0.5)

    def run(rows, dout, wf, wb):
        f = _forward(moe, prob, lay, K, N, True, rows=rows, weights=wf)
        b = _backward(moe, prob, lay, K, N, False, False, rows=rows, dout=dout, weights=wb)
        return f[2], f[3], b[4], b[5]
    clean = run(rows, dout, wf, wb)
    rows2, dout2, wf2, wb2 = rows.clone(), dout.clone(), wf.clone(), wb.clone()
    rows2[own], dout2[own], wf2[hurt], wb2[hurt] = bad, bad, bad, bad
    hurt_out = run(rows2, dout2, wf2, wb2)
    for a, b in zip(clean[:3], hurt_out[:3]):
        assert torch.equal(a[~own], b[~own])
        assert not bool(torch.isfinite(b[own]).any())
    others = [e for e in range(5) if e != hurt]
    assert torch.equal(clean[3][others], hurt_out[3][others])


def test_no_tokens(moe):
    """No tokens: nothing is read, and the weights' gradient is zero."""
    import torch
    prob = moe.Problem(0, 1024, 2, 4, 1, 1)
    lay = moe.Layout(prob)
    lay.expert_count.zero_()
    lay.expert_offset.zero_()
    none = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = randn((4, 64, 64), 1)
    dw = torch.full_like(w, 3.0)
    moe.moe_expert_forward(prob, lay, moe.Experts(64, 64, w), none, none)
    moe.moe_expert_backward_rows(prob, lay, moe.Experts(64, 64, w), none, none)
    moe.moe_expert_backward_weights(prob, lay, moe.Experts(64, 64), none, none, dw)
    assert bool((dw == 0).all())


def test_repeatable_and_on_another_stream(moe):
    """Two runs, one of them on another stream beside other work, give the same bits."""
    import torch
    prob, lay = layout_of_counts(moe, COUNTS["skewed"])
    a = _backward(moe, prob, lay, 200, 264, False, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _backward(moe, prob, lay, 200, 264, False, True)
    torch.cuda.synchronize()
    assert torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])


def test_two_streams_at_once(moe):
    """Two problems on two streams, their kernels side by side on the GPU: the bits of each alone."""
    import torch
    jobs = []
    for i, counts in enumerate((COUNTS["skewed"], COUNTS["few each"])):
        prob, lay = layout_of_counts(moe, counts)
        R, E, K, N = prob.num_tokens, prob.num_experts, 1024, 520
        rows, w = randn((R, K), i), randn((E, 2 * N, K), 10 + i, K ** -0.5)
        out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
        x = moe.Experts(K, N, w, act=moe.MOE_ACT_SWIGLU)
        moe.moe_expert_forward(prob, lay, x, rows, out)
        jobs.append((prob, lay, x, rows, out, out.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for j in jobs:
        j[4].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for prob, lay, x, rows, out, _, stream in jobs:
            moe.moe_expert_forward(prob, lay, x, rows, out, stream=stream)
    torch.cuda.synchronize()
    for j in jobs:
        assert torch.equal(j[4], j[5])


def test_least_alignment(moe):
    """Arrays that start on 16 bytes and no more."""
    import torch

    def off(t):
        raw = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        assert raw.data_ptr() % 256 == 0
        v = raw[8:].view(t.shape)
        v.copy_(t)
        return v
    prob, lay = layout_of_counts(moe, COUNTS["tile edges"])
    R, K, N = prob.num_tokens, 72, 136
    rows, w, dout, pre = randn((R, K), 1), randn((8, N, K), 2, K ** -0.5), randn((R, N), 3), randn((R, 2 * K), 4)
    for fix in (lambda t: t, off):
        out, dw, drows = (fix(torch.zeros(s, dtype=torch.bfloat16, device="cuda")) for s in ((R, N), (8, N, K), (R, 2 * K)))
        x = moe.Experts(K, N, fix(w))
        moe.moe_expert_forward(prob, lay, x, fix(rows), out)
        moe.moe_expert_backward_rows(prob, lay, x, fix(dout), drows, pre=fix(pre))
        moe.moe_expert_backward_weights(prob, lay, x, fix(rows), fix(dout), dw)
        torch.cuda.synchronize()
        if fix is off:
            assert all(torch.equal(a, b) for a, b in zip(first, (out, dw, drows)))
        else:
            first = (out, dw, drows)


def test_captured_in_a_graph(moe):
    import torch
    prob, lay = layout_of_counts(moe, COUNTS["tile edges"])
    R, K, N = prob.num_tokens, 200, 264
    rows, w = randn((R, K), 1), randn((8, 2 * N, K), 2, K ** -0.5)
    x = moe.Experts(K, N, w, act=moe.MOE_ACT_SWIGLU)
    out, want = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda"), None
    moe.moe_expert_forward(prob, lay, x, rows, out)
    want = out.clone()
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_expert_forward(prob, lay, x, rows, out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_gradient_against_differences(moe):
    """The directional slope of sum(out * dout) along a change of rows and of weights, by differences of 64-bit
    forwards, is what the gradients give (bf16 gradients: 2^-8 relative a term, in magnitude)."""
    import torch
    prob, lay = layout_of_counts(moe, [9, 0, 33, 130])
    K, N = 64, 72
    weights, dout, rows, pre, drows, dw = _backward(moe, prob, lay, K, N, False, True, seed=11)
    way = randn(pre.shape, 21).double()
    way_w = randn(weights.shape, 22).double()
    h = 2.0 ** -12

    def value(pre, weights):
        return (products(lay, gated(pre), weights)[0] * dout.double()).sum()
    slope = (value(pre.double() + h * way, weights.double()) - value(pre.double() - h * way, weights.double())) / (2 * h)
    got, size = (drows.double() * way).sum(), (drows.double() * way).abs().sum()
    assert abs(float(slope - got)) <= 2.0 ** -8 * float(size)
    hidden = gated(pre).to(torch.bfloat16)
    dw = torch.empty_like(weights)
    moe.moe_expert_backward_weights(prob, lay, moe.Experts(K, N), hidden, dout, dw)

    def value_w(w):
        return (products(lay, hidden, w)[0] * dout.double()).sum()
    slope = (value_w(weights.double() + h * way_w) - value_w(weights.double() - h * way_w)) / (2 * h)
    got, size = (dw.double() * way_w).sum(), (dw.double() * way_w).abs().sum()
    assert abs(float(slope - got)) <= 2.0 ** -8 * float(size)
