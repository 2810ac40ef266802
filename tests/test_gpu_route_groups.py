"""The router's choice limited to groups, on the GPU, against its definition in 64 bits: ids exact wherever 64 bits
tell the keys and the groups' values apart by more than fp32 can move them (ties, masks, NaN and empty rows are made of
equal bits, so they are exact too), gates within the bound of their fp32 arithmetic, and the gradient of the gates."""
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


# A score is off by the difference to the maximum (2^-24 of up to 32 for the logits below), expf, a sum and a division:
# less than 2^-24 (32 + 8) of itself; the bias's addition and a group's sum of two add 2^-23 each, of a score and a bias.
# So two keys or values that differ by more than this, of the row's largest score and the largest bias, are told apart.
GAP = 2.0 ** -24 * 64


def _scores(x, score):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-x))
        top = x.max(axis=1, keepdims=True)
        z = np.where(np.isneginf(x), 0.0, np.exp(x - np.where(np.isneginf(top), 0.0, top)))
        s = z.sum(axis=1, keepdims=True)
        return np.divide(z, s, out=np.zeros_like(z), where=s != 0)


def _order(v):
    """Indexes in falling order, equal values by index."""
    return np.lexsort((np.broadcast_to(np.arange(v.shape[1]), v.shape), -v), axis=1)


def _reference(x, bias, G, kept, top, k, score):
    """ids [T, k] and how near a row's decisions are: the least difference between neighbours in order, of the groups'
    values and of the keys (equal logits apart) of the groups that stay, over the largest score and bias."""
    T, E = x.shape
    s = _scores(x.astype(np.float64), score)
    s32 = s.astype(np.float32)                       # keys are fp32 by definition, which makes equals of near ones
    if score == "sigmoid":
        with np.errstate(all="ignore"):
            s32 = np.float32(1) / (np.float32(1) + np.exp(-x.astype(np.float64)).astype(np.float32))
    key = (s32 if bias is None else s32 + bias).astype(np.float64)
    key = np.where((s32 == 0) | np.isnan(key), -np.inf, key)
    best = -np.sort(-key.reshape(T, G, E // G), axis=2)
    value = best[..., 0].copy()
    if top == 2 and E > G:
        value = value + np.where(np.isneginf(best[..., 1]), 0, best[..., 1])
    rank = _order(value)
    on = np.zeros((T, G), bool)
    np.put_along_axis(on, rank[:, :kept], True, 1)
    on = np.repeat(on, E // G, axis=1)

    def near(v, n, ties):
        v = -np.sort(-v, axis=1)[:, : n + 1]
        with np.errstate(all="ignore"):
            d = v[:, :-1] - v[:, 1:]
        return np.where((ties & (d == 0)) | ~np.isfinite(d), np.inf, d).min(axis=1, initial=np.inf)
    key64 = np.where(np.isneginf(key), key, s if bias is None else s + bias.astype(np.float64))
    size = np.nan_to_num(s).max(axis=1) + (0 if bias is None else float(np.abs(np.nan_to_num(bias)).max()))
    gap = np.minimum(near(value, kept, False), near(np.where(on, key64, -np.inf), k, True)) / np.maximum(size, 1e-300)
    # an expert of a group that stays comes before any other, whatever its key
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -key, ~on), axis=1)
    return order[:, :k], gap


def _gates(x, ids, score, renorm, scale):
    x = x.astype(np.float64)
    chosen = np.take_along_axis(x, ids, 1)
    with np.errstate(all="ignore"):
        if score == "softmax":
            return scale * (_scores(chosen, score) if renorm else np.take_along_axis(_scores(x, score), ids, 1))
        s = 1 / (1 + np.exp(-chosen))
        total = s.sum(1, keepdims=True) if renorm else np.ones((len(x), 1))
        return scale * np.divide(s, total, out=np.zeros_like(s), where=total != 0)


def _run(moe, logits, bias, G, kept, top, k, score, renorm=True, scale=1.0):
    import torch
    T, E = logits.shape
    prob = moe.Problem(T, 1024, k, E, 1, 1)
    r = moe.Routing(moe.MOE_SCORE_SOFTMAX if score == "softmax" else moe.MOE_SCORE_SIGMOID, renorm, scale)
    ids = torch.full((T + 1, k), -9, dtype=torch.int32, device="cuda")
    gates = torch.full((T + 1, k), -7.0, device="cuda")
    moe.moe_route_groups(prob, r, moe.Grouping(G, kept, top), logits, ids[:T], gates[:T], bias=bias)
    torch.cuda.synchronize()
    assert bool((ids[T] == -9).all()) and bool((gates[T] == -7).all())
    return prob, r, ids[:T], gates[:T]


def _check(moe, logits, bias, G, kept, top, k, score, renorm=True, scale=1.0, exact=False, decided=0.9):
    x = logits.float().cpu().numpy()
    b = None if bias is None else bias.cpu().numpy()
    want, gap = _reference(x, b, G, kept, top, k, score)
    far = np.ones(len(x), bool) if exact else gap > GAP
    assert far.mean() >= decided                     # (rows that decide on less than fp32 can tell say nothing)
    prob, r, ids, gates = _run(moe, logits, bias, G, kept, top, k, score, renorm, scale)
    got = ids.cpu().numpy()
    E = x.shape[1]
    assert ((got >= 0) & (got < E)).all() and all(len(set(row)) == k for row in got)
    assert all(len(set(row // (E // G))) <= kept for row in got)
    assert np.array_equal(got[far], want[far])
    g = gates.cpu().numpy()
    ref = _gates(x, got, score, renorm, scale)
    finite = min(128.0, float(np.abs(np.where(np.isfinite(x), x, 0)).max(initial=0.0)))
    rel = 2.0 ** -24 * (64 + 8 * finite)             # the difference to the maximum, then less than 64 roundings
    ok = ~np.isnan(ref)
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    assert np.all(np.abs(g - ref)[ok] <= rel * np.abs(ref[ok]) + 1e-37)
    return prob, r, ids, gates


CASES = [  # T, E, G, kept, k
    (1, 256, 8, 4, 8), (1, 1, 1, 1, 1), (5, 2, 2, 1, 1), (130, 60, 5, 2, 3), (67, 32, 32, 32, 32), (33, 64, 32, 3, 6),
    (500, 160, 8, 3, 6), (1025, 128, 4, 1, 8), (259, 384, 8, 4, 8), (77, 192, 6, 5, 4), (19, 1000, 20, 7, 32),
    (9, 1023, 31, 2, 17), (31, 192, 8, 2, 8), (45, 176, 8, 8, 9), (60, 384, 8, 2, 6), (12, 768, 16, 3, 8), (21, 1023, 11, 4, 9), (5, 1024, 1, 1, 16), (300, 512, 16, 4, 8), (40, 96, 3, 1, 32)]


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T,E,G,kept,k", CASES)
def test_groups_match_definition(moe, T, E, G, kept, k, top, score, renorm):
    import torch
    g = torch.Generator().manual_seed(T * 1000 + E + top)
    for dtype in (torch.float32, torch.bfloat16):
        # separate keys: a permutation of evenly spread scores in every row, far more apart than GAP
        rank = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).double()
        p = (rank + 0.5) / E
        logits = (torch.log(p / (1 - p)) if score == "sigmoid" else torch.log(p)).to(dtype).cuda()
        # sums of two evenly spread scores, (i + j + 1) / E, are often equal, and so tie but for the last bit; logits rounded
        # to bf16 are, too
        _check(moe, logits, None, G, kept, top, k, score, renorm, decided=0.9 if top == 1 and dtype == torch.float32 else 0)
        bias = (0.2 / (E if score == "softmax" else 1) * torch.randn(E, generator=g)).cuda()
        noise = (3 * torch.randn((T, E), generator=g)).to(dtype).cuda()
        want, gap = _reference(noise.float().cpu().numpy(), bias.cpu().numpy(), G, kept, top, k, score)
        rows = torch.from_numpy(np.nonzero(gap > GAP)[0]).cuda()
        if len(rows):
            _check(moe, noise[rows].contiguous(), bias, G, kept, top, k, score, renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,G,kept,k", [(70, 7, 2, 5), (72, 8, 3, 7), (64, 32, 4, 8), (256, 8, 1, 32), (60, 20, 2, 6)])
def test_ties_masks_and_empty_rows(moe, E, G, kept, k, top, score):
    import torch
    size = E // G
    rows = np.zeros((10, E), np.float32)
    rows[0] = 1.25                                   # all equal: the first groups, the lowest indexes
    rows[1, ::2] = -0.0                              # -0 and +0 tie
    rows[2] = -np.inf                                # an empty row
    rows[3] = -np.inf
    rows[3, [E - 1, E // 2]] = [1.0, 2.0]            # fewer experts than k left
    rows[4] = np.finfo(np.float32).min               # a mask by the type's lowest value
    rows[4, [3, E - 1]] = 0.5
    rows[5] = np.arange(E) % size                    # every group alike: equal values
    rows[6, : E - size] = -np.inf                    # only the last group is open
    rows[7] = -np.inf
    rows[7, ::size] = 1.0                            # one expert a group: no second key
    rows[8] = -200.0                                 # sigmoids of 0, softmax of equals
    rows[9, 0] = -np.inf
    logits = torch.from_numpy(rows).cuda()
    for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.5, device="cuda"), torch.full((E,), -2.0, device="cuda")):
        _check(moe, logits, bias, G, kept, top, k, score, exact=True)
    # a bias never opens a masked expert while open ones are left: +8 on every masked one
    shut = torch.from_numpy(np.where(np.arange(E) % size == 0, -np.inf, 0.25).astype(np.float32)).cuda().expand(3, E).contiguous()
    if size > 1 and k <= kept * (size - 1):
        bias = torch.where(torch.isinf(shut[0]), 8.0, 0.0)
        _, _, ids, gates = _check(moe, shut, bias, G, kept, top, k, score, exact=True)
        assert bool((ids % size != 0).all()) and bool((gates > 0).all())


def test_nan_and_infinities_stay_in_range(moe):
    import torch
    E, G = 64, 8
    rows = np.zeros((4, E), np.float32)
    rows[0, :40] = np.nan                            # whole groups of NaN
    rows[1] = np.nan
    rows[2, 5] = np.inf
    rows[3, ::8] = np.nan
    logits = torch.from_numpy(rows).cuda()
    for score in ("sigmoid", "softmax"):
        for bias in (None, torch.full((E,), float("nan"), device="cuda")):
            _, _, ids, gates = _run(moe, logits, bias, G, 3, 2, 8, score)
            got = ids.cpu().numpy()
            assert ((got >= 0) & (got < E)).all() and all(len(set(r)) == 8 for r in got)
            assert all(len(set(r // 8)) <= 3 for r in got)
    want, _ = _reference(rows, None, G, 3, 2, 8, "sigmoid")
    assert np.array_equal(_run(moe, logits, None, G, 3, 2, 8, "sigmoid")[2].cpu().numpy(), want)


def test_one_group_is_the_plain_choice(moe):
    """With one group and no bias the ids are moe_route's, where fp32 tells the scores apart."""
    import torch
    T, E, k = 257, 96, 8
    p = (torch.stack([torch.randperm(E) for _ in range(T)]).double() + 0.5) / E
    logits = torch.log(p / (1 - p)).float().cuda()
    for score in ("sigmoid", "softmax"):
        prob, r, ids, gates = _run(moe, logits, None, 1, 1, 2, k, score)
        plain, g = torch.empty_like(ids), torch.empty_like(gates)
        moe.moe_route(prob, r, logits, plain, g)
        assert torch.equal(ids, plain) and torch.equal(gates, g)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_of_the_gates(moe, score, renorm):
    """moe_route_backward takes these ids: against 64-bit autograd of the gates, and against differences of the gates
    that the call itself gives for moved logits (the choice stays)."""
    import torch
    T, E, G, kept, k = 33, 64, 8, 3, 6
    g = torch.Generator().manual_seed(4)
    logits = (2 * torch.randn((T, E), generator=g)).cuda()
    bias = (0.1 * torch.randn(E, generator=g)).cuda()
    prob, r, ids, gates = _run(moe, logits, bias, G, kept, 2, k, score, renorm, 1.5)
    dg = torch.randn((T, k), generator=g).cuda()
    dl = torch.empty_like(logits)
    moe.moe_route_backward(prob, r, logits, ids, dg, dl)

    def gates64(x):
        chosen = x.gather(1, ids.long())
        if score == "softmax":
            return 1.5 * (torch.softmax(chosen, 1) if renorm else torch.softmax(x, 1).gather(1, ids.long()))
        s = torch.sigmoid(chosen)
        return 1.5 * (s / s.sum(1, keepdim=True) if renorm else s)
    x = logits.double().requires_grad_(True)
    want, = torch.autograd.grad((gates64(x) * dg.double()).sum(), x)
    # gates of at most 1.5, gradients of sums of k such terms: 64 roundings of terms below 1.5 k max|dg|
    slack = 2.0 ** -24 * 128 * 1.5 * k * float(dg.abs().max())
    assert float((dl.double() - want).abs().max()) <= slack
    step = 2.0 ** -7
    v = torch.randn((T, E), generator=g).cuda()
    moved = []
    for sign in (1, -1):
        _, _, ids2, gates2 = _run(moe, logits + sign * step * v, bias, G, kept, 2, k, score, renorm, 1.5)
        moved.append((ids2, gates2.double()))
    same = (moved[0][0] == ids).all(1) & (moved[1][0] == ids).all(1)
    assert int(same.sum()) >= 10
    slope = ((moved[0][1] - moved[1][1]) / (2 * step) * dg.double()).sum(1)
    along = (dl.double() * v.double()).sum(1)
    # third derivatives of a gate along v: at most 6 |v|^3 1.5 a gate, times step^2 / 6; and fp32 gates over 2 step
    size = v.double().abs().amax(1) * 2
    bound = (step ** 2 * 1.5 * size ** 3 + 2.0 ** -24 * 128 * 1.5 / step) * dg.double().abs().sum(1)
    assert bool(((slope - along).abs() <= bound)[same].all())


def test_streams_graphs_and_two_calls_at_once(moe):
    import torch
    T, E = 2000, 256
    logits = [torch.randn((T, E), device="cuda") for _ in range(2)]
    bias = 0.1 * torch.randn(E, device="cuda")
    want = [_run(moe, x, bias, 8, 4, 2, 8, "sigmoid")[2:] for x in logits]
    prob, r, gr = moe.Problem(T, 1024, 8, E, 1, 1), moe.Routing(moe.MOE_SCORE_SIGMOID), moe.Grouping(8, 4)
    out = [(torch.empty((T, 8), dtype=torch.int32, device="cuda"), torch.empty((T, 8), device="cuda")) for _ in logits]
    streams = [torch.cuda.Stream() for _ in logits]
    torch.cuda.synchronize()
    for x, (i, g), s in zip(logits, out, streams):
        moe.moe_route_groups(prob, r, gr, x, i, g, bias=bias, stream=s)
    torch.cuda.synchronize()
    for (i, g), w in zip(out, want):
        assert torch.equal(i, w[0]) and torch.equal(g, w[1])
    graph, x = torch.cuda.CUDAGraph(), logits[0].clone()
    with torch.cuda.graph(graph):
        moe.moe_route_groups(prob, r, gr, x, *out[0], bias=bias)
    x.copy_(logits[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], want[1][0]) and torch.equal(out[0][1], want[1][1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_least_alignment_gives_the_same(moe, dtype):
    """Logits and bias that start on their type's own size alone: the same bits as aligned ones."""
    import torch
    T, E = 65, 160
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(9)
    logits, bias = torch.randn((T, E), generator=g).to(kind).cuda(), (0.1 * torch.randn(E, generator=g)).cuda()
    raw, raw_bias = torch.empty(T * E + 8, dtype=kind, device="cuda"), torch.empty(E + 4, device="cuda")
    want = _run(moe, logits, bias, 8, 3, 2, 6, "sigmoid")[2:]
    for shift in (1, 2, 3):
        x, b = raw[shift:shift + T * E].view(T, E), raw_bias[shift:shift + E]
        x.copy_(logits)
        b.copy_(bias)
        for lo, bi in ((x, bias), (logits, b), (x, b)):
            got = _run(moe, lo, bi, 8, 3, 2, 6, "sigmoid")[2:]
            assert all(torch.equal(p, q) for p, q in zip(got, want))
