"""The router on the GPU against its definition in 64 bits: ids exact (ties,
masked experts, NaN, empty rows), gates and logit gradients within the bound of
their fp32 arithmetic."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import torch
    import __graft_entry__ as ge
    ge.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import combine_moe_layout_04_gb300 as m
    return m


def _softmax(x):
    top = x.max(axis=1, keepdims=True)
    z = np.exp(x - np.where(np.isneginf(top), 0.0, top))
    s = z.sum(axis=1, keepdims=True)
    return np.divide(z, s, out=np.zeros_like(z), where=s != 0)


def _reference(logits32, bias32, k, score, renorm, scale, dgates):
    """ids, gates, dlogits (and the magnitude its terms have) in 64 bits; keys are fp32 by definition."""
    key = logits32 if bias32 is None else (logits32 + bias32).astype(np.float32)
    ranked = np.where(np.isnan(key), -np.inf, key).astype(np.float64)
    T, E = key.shape
    # NaN after -infinity after every number, equal keys by index
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -ranked, np.isnan(key)), axis=1)
    ids = order[:, :k]
    with np.errstate(all="ignore"):
        x = logits32.astype(np.float64)
        on = np.zeros((T, E), bool)
        np.put_along_axis(on, ids, True, 1)
        if score == "softmax":
            w = _softmax(np.where(on, x, -np.inf) if renorm else x)
            slope = np.ones_like(w)
        else:
            s = 1 / (1 + np.exp(-x))
            total = np.where(on, s, 0).sum(1, keepdims=True) if renorm else np.ones((T, 1))
            w = np.divide(np.where(on, s, 0), total, out=np.zeros_like(s), where=total != 0)
            slope = 1 - s
        gates = scale * np.take_along_axis(w, ids, 1)
        a = np.zeros((T, E))
        np.put_along_axis(a, ids, scale * dgates.astype(np.float64), 1)
        wa = np.where(on, w * a, 0)
        if score == "softmax" or renorm:
            mean, size = wa.sum(1, keepdims=True), np.abs(wa).sum(1, keepdims=True)
            live = w if score == "softmax" and not renorm else np.where(on, w, 0)
            d = live * (a - mean) * slope
            size = live * (np.abs(a) + size)
        else:
            d = wa * slope
            size = np.abs(wa)
    live = live_or(on, score, renorm)
    return ids, gates, np.where(live, d, 0), np.where(live, size, 0)


def live_or(on, score, renorm):
    return np.ones_like(on) if score == "softmax" and not renorm else on


def _run(moe, logits, k, score, renorm, scale, bias, dgates):
    import torch
    T, E = logits.shape
    prob = moe.Problem(T, 1024, k, E, 1, 1)
    r = moe.Routing(moe.MOE_SCORE_SOFTMAX if score == "softmax" else moe.MOE_SCORE_SIGMOID, renorm, scale)
    ids = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    gates = torch.full((T, k), -7.0, device="cuda")
    dl = torch.full_like(logits, -5.0)
    moe.moe_route(prob, r, logits, ids, gates, bias=bias)
    moe.moe_route_backward(prob, r, logits, ids, dgates, dl)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), gates.cpu().numpy(), dl.float().cpu().numpy()


def _check(moe, logits, k, score, renorm, scale=1.0, bias=None, seed=0):
    import torch
    T, E = logits.shape
    dg = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, k)).astype(np.float32)).cuda()
    ids, gates, dl = _run(moe, logits, k, score, renorm, scale, bias, dg)
    x = logits.float().cpu().numpy()
    rids, rgates, rdl, size = _reference(x, None if bias is None else bias.cpu().numpy(), k, score, renorm, scale,
                                         dg.cpu().numpy())
    assert np.array_equal(ids, rids)
    # fp32: the difference v - max is off by 2^-24 |v - max|, which expf turns into that relative error; expf,
    # the sums (at most 32 + 5 additions) and the divisions add less than 64 roundings; beyond 128 below the
    # maximum (or beyond +-128, for a sigmoid) the fp32 exponential is exactly 0 and nothing is off
    finite = min(128.0, float(np.abs(np.where(np.isfinite(x), x, 0)).max(initial=0.0)))
    rel = 2.0 ** -24 * (64 + 4 * 2 * finite)
    ok = ~np.isnan(rgates)
    assert np.array_equal(np.isnan(gates), np.isnan(rgates))
    assert np.all(np.abs(gates - rgates)[ok] <= rel * np.abs(rgates[ok]) + 1e-37)
    bound = 4 * rel * abs(scale) * size + 1e-37
    if logits.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(rdl)
    ok = ~np.isnan(rdl)
    assert np.array_equal(np.isnan(dl), np.isnan(rdl))
    assert np.all(np.abs(dl - rdl)[ok] <= bound[ok])


FORMS = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


@pytest.mark.parametrize("score,renorm", FORMS)
@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 256, 8, "f32"), (1, 1, 1, "f32"), (3, 2, 2, "bf16"), (130, 31, 3, "f32"), (67, 32, 32, "bf16"),
    (33, 33, 6, "f32"), (500, 61, 4, "bf16"), (1025, 128, 8, "f32"), (77, 160, 8, "bf16"), (259, 384, 8, "f32"),
    (19, 1000, 32, "f32"), (5, 1024, 16, "bf16")])
def test_route_matches_definition(moe, T, E, k, dtype, score, renorm):
    import torch
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = (3 * torch.randn((T, E), generator=g)).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    _check(moe, logits, k, score, renorm)
    bias = (0.5 * torch.randn(E, generator=g)).cuda()
    _check(moe, logits, k, score, renorm, scale=2.5, bias=bias)


@pytest.mark.parametrize("score,renorm", FORMS)
def test_route_ties_masks_and_empty_rows(moe, score, renorm):
    import torch
    E, k = 70, 5
    rows = np.zeros((8, E), np.float32)
    rows[0] = 1.25                                  # all equal: the lowest indexes
    rows[1, ::2] = -0.0                             # -0 and +0 tie
    rows[2] = -np.inf                               # an empty row
    rows[3] = -np.inf
    rows[3, [9, 40, 65]] = [1.0, 2.0, 1.0]          # fewer than k left
    rows[4] = np.finfo(np.float32).min              # a mask by the type's lowest value
    rows[4, [3, 69]] = [0.5, 0.5]
    rows[5] = np.arange(E) % 7
    rows[6] = 80.0 * np.sin(np.arange(E))           # wide: exp underflows
    rows[7, 10:] = -np.inf
    _check(moe, torch.from_numpy(rows).cuda(), k, score, renorm)


@pytest.mark.parametrize("E,k", [(129, 32), (256, 32), (257, 8), (384, 32), (511, 16), (512, 32), (700, 32), (1024, 32)])
def test_route_ties_of_many_experts(moe, E, k):
    """Keys of few values, so that a lane's keys and those of other lanes tie all the time; choices from one lane's keys."""
    import torch
    rng = np.random.default_rng(E)
    rows = rng.integers(0, 4, (40, E)).astype(np.float32)
    rows[0] = 0.5
    rows[1] = -np.inf
    rows[2, :] = -np.inf
    rows[2, E - k:] = 1.0
    rows[3], rows[3, 5::32] = -2.0, np.arange(len(rows[3, 5::32]))        # lane 5 holds the largest, rising
    rows[4], rows[4, 31::32] = -2.0, -np.arange(len(rows[4, 31::32])) + 9.0
    rows[5], rows[5, ::32] = -2.0, 3.0
    for score, renorm in (("softmax", True), ("sigmoid", False)):
        _check(moe, torch.from_numpy(rows).cuda(), k, score, renorm)
        _check(moe, torch.from_numpy(rows).cuda().to(torch.bfloat16), k, score, renorm)


def test_route_nan_is_chosen_last(moe):
    import torch
    E, k = 40, 6
    rows = np.tile(np.linspace(-1, 1, E, dtype=np.float32), (3, 1))
    rows[0, [0, 20, 39]] = np.nan                   # never chosen: plenty of numbers
    rows[1, :36] = np.nan                           # four numbers, then the lowest NaN indexes
    rows[2] = np.nan
    rows[1, 0] = -np.inf
    for score, renorm in (("softmax", True), ("sigmoid", False)):
        _check(moe, torch.from_numpy(rows).cuda(), k, score, renorm)


def test_route_feeds_the_layout(moe):
    """The ids are what moe_layout takes: distinct and in range, no status bit."""
    import torch
    T, E, k = 777, 96, 6
    logits = torch.randn((T, E), device="cuda")
    logits[5] = float("-inf")
    logits[6] = float("nan")
    prob = moe.Problem(T, 1024, k, E, 4, 2)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    gates = torch.empty((T, k), device="cuda")
    moe.moe_route(prob, moe.Routing(), logits, ids, gates)
    lay, ws = moe.Layout(prob), moe.alloc_workspace(prob)
    moe.moe_layout(prob, ids, ws, lay)
    assert moe.moe_status(ws) == (moe.MOE_OK, 0)


def test_route_backward_ignores_bad_ids(moe):
    import torch
    logits = torch.randn((2, 16), device="cuda")
    prob = moe.Problem(2, 1024, 2, 16, 1, 1)
    ids = torch.tensor([[3, 99], [-4, 7]], dtype=torch.int32, device="cuda")
    dg, dl = torch.ones((2, 2), device="cuda"), torch.full((2, 16), 9.0, device="cuda")
    moe.moe_route_backward(prob, moe.Routing(moe.MOE_SCORE_SIGMOID, False), logits, ids, dg, dl)
    want = torch.zeros((2, 16), dtype=torch.float64)
    for t, e in ((0, 3), (1, 7)):
        s = torch.sigmoid(logits[t, e].double().cpu())
        want[t, e] = s * (1 - s)
    assert torch.allclose(dl.double().cpu(), want, rtol=1e-5, atol=0)


@pytest.mark.parametrize("score,renorm", FORMS)
def test_route_gradient_over_its_logits(moe, score, renorm):
    """dlogits may be logits itself: the same bits as in a buffer of its own."""
    import torch
    T, E, k = 301, 160, 6
    logits = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    dg = torch.randn((T, k), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    for x in (logits, logits.to(torch.bfloat16)):
        ids, _, dl = _run(moe, x, k, score, renorm, 1.5, None, dg)
        prob = moe.Problem(T, 1024, k, E, 1, 1)
        r = moe.Routing(moe.MOE_SCORE_SOFTMAX if score == "softmax" else moe.MOE_SCORE_SIGMOID, renorm, 1.5)
        moe.moe_route_backward(prob, r, x, torch.from_numpy(ids).cuda(), dg, x)
        torch.cuda.synchronize()
        assert np.array_equal(x.float().cpu().numpy(), dl)


@pytest.mark.parametrize("score,renorm", FORMS)
def test_route_gradient_against_differences(moe, score, renorm):
    """dlogits is the slope of sum(gates * dgates) along a direction (central differences of the forward
    call's own gates; step 2^-6: the second-order term is below 2^-12 of the third derivative, at most 1)."""
    import torch
    T, E, k = 64, 48, 5
    g = torch.Generator().manual_seed(5)
    logits = torch.randn((T, E), generator=g)
    logits += 4 * (torch.rand((T, E), generator=g) < 0.2)    # wide gaps: the choice does not change
    way = 2.0 ** -6 * torch.randn((T, E), generator=g).clamp(-2, 2)
    dg = torch.randn((T, k), generator=g).cuda()
    prob, r = moe.Problem(T, 1024, k, E, 1, 1), moe.Routing(
        moe.MOE_SCORE_SOFTMAX if score == "softmax" else moe.MOE_SCORE_SIGMOID, renorm)

    def gates_of(x):
        ids, gates = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
        moe.moe_route(prob, r, x.cuda(), ids, gates)
        return ids, gates.double()
    ids, _ = gates_of(logits)
    up, down = gates_of(logits + way), gates_of(logits - way)
    same = (up[0] == ids).all(1) & (down[0] == ids).all(1)
    slope = ((up[1] - down[1]) * dg.double()).sum(1) / 2
    dl = torch.empty((T, E), device="cuda")
    moe.moe_route_backward(prob, r, logits.cuda(), ids, dg, dl)
    want = (dl.double() * way.cuda().double()).sum(1)
    assert int(same.sum()) >= T // 2
    # third-order remainder: |way|^3 / 6 times the third derivative, over at most E terms
    bound = (way.abs().double() ** 3).sum(1).cuda() * dg.abs().sum(1).double() * 4 + 1e-6
    assert torch.all(((slope - want).abs() <= bound) | ~same)


# ---- sigmoid gates far out ----------------------------------------------------------
#
# The reference works with logarithms, so that nothing of it underflows or cancels: log s = -log(1 + exp(-v)),
# 1 - s = exp(-log(1 + exp(v))).


def _sigmoid_reference(x, ids, renorm, a):
    v = np.take_along_axis(x.astype(np.float64), ids, 1)
    log_s, rest = -np.logaddexp(0, -v), np.exp(-np.logaddexp(0, v))
    w = np.exp(log_s - (log_s.max(axis=1, keepdims=True) if renorm else 0))
    w = w / w.sum(axis=1, keepdims=True) if renorm else w
    d, size = np.zeros_like(x, dtype=np.float64), np.zeros_like(x, dtype=np.float64)
    mean, spread = ((w * a).sum(1, keepdims=True), np.abs(w * a).sum(1, keepdims=True)) if renorm else (0, 0)
    np.put_along_axis(d, ids, w * rest * (a - mean), 1)
    np.put_along_axis(size, ids, w * rest * (np.abs(a) + spread), 1)
    return w, d, size


def _check_sigmoid(moe, rows, k, renorm, what):
    """Chosen by the largest logits; the bounds of _check, the gradient's with the slope in it."""
    import torch
    x = np.ascontiguousarray(rows, np.float32)
    T, E = x.shape
    dg = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    ids, gates, dl = _run(moe, torch.from_numpy(x).cuda(), k, "sigmoid", renorm, 1.0, None, torch.from_numpy(dg).cuda())
    assert np.array_equal(ids, np.argsort(-x, axis=1, kind="stable")[:, :k])
    w, d, size = _sigmoid_reference(x, ids, renorm, dg.astype(np.float64))
    rel = 2.0 ** -24 * (64 + 8 * min(128.0, float(np.abs(x).max())))
    got, want, bound = (gates, w, rel * w + 1e-37) if what == "gates" else (dl, d, 4 * rel * size + 1e-37)
    off = np.abs(got - want)
    assert np.all(off <= bound), (float((off / np.maximum(bound, 1e-300)).max()), got[off > bound][:4], want[off > bound][:4])


def _rows_up(E):
    """Confident experts: logits of 8 to 30, alone or with low ones."""
    rng = np.random.default_rng(8)
    rows = rng.uniform(8, 30, (40, E))
    rows[20:] = np.where(rng.random((20, E)) < 0.1, rows[20:], rng.uniform(-30, 0, (20, E)))
    rows[0, :4] = 12.0, 15.0, 17.0, 29.0
    return rows


@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_gradient_of_confident_experts(moe, renorm):
    """s (1 - s) where s is one but for its last bits: the slope keeps its relative accuracy."""
    _check_sigmoid(moe, _rows_up(64), 6, renorm, "gradient")


def _rows_down(E):
    """Every logit so low that exp(-v) nears or passes the largest float: the chosen ones still share 1."""
    rng = np.random.default_rng(9)
    rows = rng.uniform(-120, -80, (40, E))
    rows[0] = -95.0
    rows[1] = -95.0 + 1e-3 * np.arange(E)
    rows[2] = np.finfo(np.float32).min              # a whole row under a mask of the type's lowest value
    rows[3] = -1e30
    rows[4] = np.linspace(-90, -88, E)
    rows[5] = np.linspace(-500, -100, E)
    rows[6:12, ::3] = rng.uniform(-5, 30, rows[6:12, ::3].shape)
    rows[12, :2] = 20.0, -87.0
    return rows


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("what", ["gates", "gradient"])
def test_sigmoid_gates_of_low_logits(moe, renorm, what):
    _check_sigmoid(moe, _rows_down(70), 5, renorm, what)
    _check_sigmoid(moe, _rows_up(64), 6, renorm, what)


def test_sigmoid_of_infinities(moe):
    """+infinity has a sigmoid of 1 (a share of it when renormalised), -infinity one of 0, and rows of -infinity have
    gates 0; a NaN that is chosen makes the renormalised gates of its row NaN and no other."""
    import torch
    E, k, inf = 40, 3, np.inf
    rows = np.full((5, E), -inf, np.float32)
    rows[0, :2] = inf, 0.0
    rows[1, :3] = inf, inf, -200.0
    rows[3, 7] = -300.0
    rows[4, :2], rows[4, 2:] = (-100.0, -101.0), np.nan
    dg = torch.ones((5, k), device="cuda")
    one = _run(moe, torch.from_numpy(rows).cuda(), k, "sigmoid", False, 1.0, None, dg)[1]
    assert np.allclose(one[:4], [[1, 0.5, 0], [1, 1, 0], [0, 0, 0], [0, 0, 0]], rtol=1e-6, atol=0)
    share = _run(moe, torch.from_numpy(rows).cuda(), k, "sigmoid", True, 1.0, None, dg)[1]
    assert np.allclose(share[:4], [[2 / 3, 1 / 3, 0], [0.5, 0.5, 0], [0, 0, 0], [1, 0, 0]], rtol=1e-6, atol=0)
    assert np.isnan(share[4]).all()
