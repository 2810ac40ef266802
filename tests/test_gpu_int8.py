"""The experts in 8-bit integers on the GPU: codes and scales bit for bit against their definition, products against
64-bit products of the values, over ragged groups, odd widths, every code and cut contractions."""
import numpy as np
import pytest

from experts_harness import close, gated, gated_slack, guarded, layout_of_counts, layout_of_ids, randn, spans

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


def quantise(x):
    """Integers and scales of rows x (bf16 [n, cols]) by the definition: fp32 divisions and products, on the CPU."""
    import torch
    v = x.float().cpu().numpy()
    m = np.abs(v).max(axis=1, keepdims=True)
    bad = ~np.isfinite(m)
    with np.errstate(all="ignore"):
        lift = np.where(m < 2.0 ** -100, np.float32(2.0 ** 100), np.float32(1))
        c = np.rint((v * lift) * (np.float32(127) / (m * lift)))
        c = np.where(bad | (m == 0), 0, c)
        s = np.where(bad, np.float32("nan"), np.where(m == 0, np.float32(1), m / np.float32(127)))
    return torch.from_numpy(c.astype(np.int8)).cuda(), torch.from_numpy(s[:, 0].astype(np.float32)).cuda()


def _rows_call(moe, x):
    import torch
    n, cols = x.shape
    codes, t0 = guarded((n, cols), torch.int8, 0xC3)
    scales, t1 = guarded((n,), torch.float32, 0xC3)
    moe.moe_quant8_rows(moe.Problem(n, 1024, 1, 1, 1, 1), x, codes, scales)
    torch.cuda.synchronize()
    assert bool((t0 == 0xC3).all()) and bool((t1 == 0xC3).all())
    return codes, scales


def _same(got, want):
    import torch
    codes, scales = got
    assert torch.equal(codes, want[0])
    assert torch.equal(torch.nan_to_num(scales, nan=-1.0), torch.nan_to_num(want[1], nan=-1.0))


@pytest.mark.parametrize("n,cols", [(1, 16), (3, 7168), (300, 48), (1000, 528), (77, 2048), (33, 4112), (5, 16400), (2, 1 << 20),
                                    (4000, 1024), (130, 8192), (9, 32), (17, 12304)])
def test_rows(moe, n, cols):
    x = randn((n, cols), n + cols)
    _same(_rows_call(moe, x), quantise(x))


def test_rows_at_the_ends_of_the_types(moe):
    """Zeros, the smallest and largest numbers, half steps, infinities and NaN, a largest value at either end."""
    import torch
    cols = 272
    x = randn((24, cols), 1)
    x[0], x[1], x[2] = 0, 2.0 ** -133, torch.finfo(torch.bfloat16).max
    x[3] *= 2.0 ** -126
    x[4] = (torch.arange(cols, device="cuda") - 127.5).clamp(-127, 127).to(torch.bfloat16)   # ties
    x[5], x[5, 0] = 0, 1
    x[6], x[6, -1] = 0, -3
    x[7, 100], x[8, 0], x[9, -1] = float("inf"), float("nan"), -float("inf")
    x[10] = 2.0 ** -100
    x[11] = 2.0 ** -101
    x[12] = -0.0
    x[13] = 1e38 * x[13].clamp(-3, 3)
    x[14] *= 2.0 ** -130
    got = _rows_call(moe, x)
    _same(got, quantise(x))
    assert int(got[0].abs().max()) <= 127
    assert bool(torch.isnan(got[1][7:10]).all()) and not bool(got[0][7:10].any())


def test_rows_stay_apart_and_least_alignment(moe):
    """Rows that start 16 bytes past a line, more rows than a grid dimension of the GPU's second axis holds."""
    import torch
    raw = randn((70001 * 16 + 8,), 2)
    x = raw[8:].view(70001, 16)
    _same(_rows_call(moe, x), quantise(x))


@pytest.mark.parametrize("act", [False, True])
def test_weights(moe, act):
    import torch
    E, K, N = 5, 272, 40
    w = randn((E, 2 * N if act else N, K), 3)
    x = moe.Experts(K, N, w, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)
    codes, t0 = guarded(w.shape, torch.int8, 0xC3)
    scales, t1 = guarded(w.shape[:2], torch.float32, 0xC3)
    moe.moe_quant8_weights(moe.Problem(8, 1024, 1, E, 1, 1), x, codes, scales)
    want = quantise(w.view(-1, K))
    _same((codes.view(-1, K), scales.view(-1)), want)
    assert bool((t0 == 0xC3).all()) and bool((t1 == 0xC3).all())


def integers(shape, seed, low=-127, high=127):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(low, high + 1, shape, generator=g, device="cuda", dtype=torch.int8)


def scales_of(shape, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp(torch.randn(shape, generator=g, device="cuda")) * 1e-3


def _forward(moe, prob, lay, codes, scales, weights, wscales, act, want_pre=True):
    import torch
    R, K = codes.shape
    N = weights.shape[1] // (2 if act else 1)
    x = moe.Experts(K, N, weights, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE, scales=wscales)
    out, t0 = guarded((R, N), torch.bfloat16, 0xC3)
    pre, t1 = guarded((R, 2 * N), torch.bfloat16, 0xC3) if act and want_pre else (None, None)
    moe.moe_expert_forward8(prob, lay, x, codes, scales, out, pre=pre)
    torch.cuda.synchronize()
    assert bool((t0 == 0xC3).all()) and (pre is None or bool((t1 == 0xC3).all()))
    return out, pre


def _check(lay, codes, scales, weights, wscales, act, out, pre):
    """The sums of integers are exact in fp32 below 2^24, else off by 2^-23 of the running magnitude a term; two products
    with the scales, one rounding each."""
    import torch
    R, K = codes.shape
    ref = torch.zeros((R, weights.shape[1]), dtype=torch.float64, device="cuda")
    slack = torch.zeros_like(ref)
    for e, r0, n in spans(lay):
        a, b = codes[r0:r0 + n].double(), weights[e].double()
        size = a.abs() @ b.abs().T
        s = scales[r0:r0 + n, None].double() * wscales[e].double()
        ref[r0:r0 + n] = (a @ b.T) * s
        slack[r0:r0 + n] = torch.where(size < 2 ** 24, 0, size * (K + 16) * 2.0 ** -23) * s
    slack += 2.0 ** -22 * ref.abs()
    if not act:
        return close(out, ref, slack)
    if pre is not None:
        close(pre, ref, slack)
    close(out, gated(ref), gated_slack(ref, slack))


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
WIDTHS = [(16, 8), (64, 128), (80, 136), (208, 264), (1024, 512), (528, 1016), (128, 8), (4112, 72)]


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
def test_forward(moe, counts, K, N, act):
    prob, lay = layout_of_counts(moe, counts)
    E, W = len(counts), 2 * N if act else N
    codes, weights = integers((sum(counts), K), 4), integers((E, W, K), 5)
    scales, wscales = scales_of(sum(counts), 6), scales_of((E, W), 7)
    _check(lay, codes, scales, weights, wscales, act, *_forward(moe, prob, lay, codes, scales, weights, wscales, act))


def test_every_code_is_exact(moe):
    """Weights that pick a column, times every integer: the product of any two integers, -128 among them."""
    import torch
    counts, K, N = [256, 0, 256], 256, 256
    prob, lay = layout_of_counts(moe, counts)
    every = torch.arange(-128, 128, device="cuda").to(torch.int8)
    codes = every[:, None].expand(256, K).repeat(2, 1).contiguous()
    weights = torch.zeros((3, N, K), dtype=torch.int8, device="cuda")
    at = torch.arange(N, device="cuda")
    for e in range(3):
        weights[e, at, (at * 37 + e) % K] = every
    one = torch.ones(512, device="cuda")
    out, _ = _forward(moe, prob, lay, codes, one, weights, torch.ones((3, N), device="cuda"), False)
    want = codes[:, :1].double() * every.double()
    assert torch.equal(out, want.to(torch.bfloat16))


def test_neighbours_do_not_leak(moe):
    """Scales of other experts' rows, and of other experts' features, may be anything."""
    import torch
    counts, K, N = [5, 129, 0, 31], 144, 72
    prob, lay = layout_of_counts(moe, counts)
    codes, weights = integers((sum(counts), K), 8), integers((4, 2 * N, K), 9)
    scales, wscales = scales_of(sum(counts), 10), scales_of((4, 2 * N), 11)
    clean = _forward(moe, prob, lay, codes, scales, weights, wscales, True)
    s, w = scales.clone(), wscales.clone()
    s[5:134], w[1] = float("nan"), float("inf")
    codes[5:134] = -128
    out, pre = _forward(moe, prob, lay, codes, s, weights, w, True)
    keep = torch.ones(sum(counts), dtype=torch.bool, device="cuda")
    keep[5:134] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(pre[keep], clean[1][keep])
    assert bool(torch.isnan(out[5:134]).all())


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("counts,K,N", [([1], 7168, 1024), ([3, 0, 1, 2], 4096, 264), ([300], 7168, 256), ([20, 0, 40], 3712, 520)])
def test_few_tiles_and_long_contractions(moe, counts, K, N, act):
    prob, lay = layout_of_counts(moe, counts)
    E, W = len(counts), 2 * N if act else N
    codes, weights = integers((sum(counts), K), 12), integers((E, W, K), 13)
    scales, wscales = scales_of(sum(counts), 14), scales_of((E, W), 15)
    _check(lay, codes, scales, weights, wscales, act, *_forward(moe, prob, lay, codes, scales, weights, wscales, act, want_pre=False))


def test_many_experts_and_a_layer_in_integers(moe):
    """1024 experts top-4; and rows quantised, multiplied, quantised and multiplied again, against 64 bits."""
    import torch
    T, k, E, K, N = 100, 4, 1024, 128, 64
    ids = np.stack([np.random.default_rng(t).permutation(E)[:k] for t in range(T)])
    prob, lay = layout_of_ids(moe, ids, E)
    up, down = randn((E, 2 * N, K), 16, K ** -0.5), randn((E, K, N), 17, N ** -0.5)
    made = []
    for w, act in ((up, moe.MOE_ACT_SWIGLU), (down, moe.MOE_ACT_NONE)):
        c, s = torch.empty(w.shape, dtype=torch.int8, device="cuda"), torch.empty(w.shape[:2], device="cuda")
        n = w.shape[1] // (2 if act else 1)
        moe.moe_quant8_weights(prob, moe.Experts(w.shape[2], n, w, act=act), c, s)
        made.append(moe.Experts(w.shape[2], n, c, act=act, scales=s))
    x = randn((T * k, K), 18)
    c0, s0 = torch.empty((T * k, K), dtype=torch.int8, device="cuda"), torch.empty(T * k, device="cuda")
    hidden, y = (torch.empty((T * k, n), dtype=torch.bfloat16, device="cuda") for n in (N, K))
    c1, s1 = torch.empty((T * k, N), dtype=torch.int8, device="cuda"), torch.empty(T * k, device="cuda")
    moe.moe_quant8_rows(prob, x, c0, s0)
    moe.moe_expert_forward8(prob, lay, made[0], c0, s0, hidden)
    moe.moe_quant8_rows(prob, hidden, c1, s1)
    moe.moe_expert_forward8(prob, lay, made[1], c1, s1, y)
    _same((c0, s0), quantise(x))
    _check(lay, c0, s0, made[0].weights, made[0].scales, True, hidden, None)
    _same((c1, s1), quantise(hidden))
    _check(lay, c1, s1, made[1].weights, made[1].scales, False, y, None)


def test_streams_graphs_and_repeats(moe):
    import torch
    counts, K, N = [30, 60, 0, 200, 1], 2048, 136
    prob, lay = layout_of_counts(moe, counts)
    E, R = len(counts), sum(counts)
    weights, wscales = integers((E, N, K), 19), scales_of((E, N), 20)
    inputs = [randn((R, K), 21 + i) for i in range(2)]
    made = [_rows_call(moe, x) for x in inputs]
    want = [_forward(moe, prob, lay, c, s, weights, wscales, False)[0] for c, s in made]
    x = moe.Experts(K, N, weights, scales=wscales)
    got = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for (c, s), o in zip(made, got):
        moe.moe_expert_forward8(prob, lay, x, c, s, o, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    rows, (c, s), o = inputs[0].clone(), (torch.empty_like(made[0][0]), torch.empty_like(made[0][1])), got[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_quant8_rows(prob, rows, c, s)
        moe.moe_expert_forward8(prob, lay, x, c, s, o)
    rows.copy_(inputs[1])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[1])
