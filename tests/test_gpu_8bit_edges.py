"""The 8-bit calls at the ends of what they document: the widest rows and results, experts placed on ranks out of order,
layouts that do not fit, a gated product on the way back, a step in a hundred thousand tokens of choice."""
import pytest

from experts_harness import close, gated, gated_slack, guarded, layout_of_counts, randn, spans, sum_slack
from test_gpu_int8 import _check as check_int8, _forward as forward_int8, integers, quantise, scales_of
from test_gpu_kept import _back, _check_back, _check_forward, _forward, _random_kept, values8

pytestmark = pytest.mark.gpu
WIDEST = 1 << 20


@pytest.fixture(scope="module")
def moe():
    import torch
    import __graft_entry__ as ge
    ge.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import combine_moe_layout_04_gb300 as m
    yield m
    assert m.moe_move_faults() == 0
    torch.cuda.empty_cache()


def test_integers_of_the_widest_rows(moe):
    """A contraction of 2^20, all of one sign in one row: sums far beyond 2^24, in fp32 as documented."""
    import torch
    counts, K, N = [2, 0, 1], WIDEST, 8
    prob, lay = layout_of_counts(moe, counts)
    codes, weights = integers((3, K), 1), integers((3, N, K), 2)
    codes[0], weights[0, 3] = 127, -128
    scales, wscales = scales_of(3, 3), scales_of((3, N), 4)
    check_int8(lay, codes, scales, weights, wscales, False, *forward_int8(moe, prob, lay, codes, scales, weights, wscales, False))


@pytest.mark.parametrize("act", [False, True])
def test_integers_to_the_widest_results(moe, act):
    import torch
    counts, K, N = [3, 1], 16, WIDEST
    prob, lay = layout_of_counts(moe, counts)
    W = 2 * N if act else N
    codes, weights = integers((4, K), 5), integers((2, W, K), 6)
    scales, wscales = scales_of(4, 7), scales_of((2, W), 8)
    check_int8(lay, codes, scales, weights, wscales, act, *forward_int8(moe, prob, lay, codes, scales, weights, wscales, act))


def test_kept_of_the_widest_results(moe):
    counts, K, N = [2, 0, 1], 16, WIDEST
    prob, lay = layout_of_counts(moe, counts)
    rows, weights = randn((3, K), 9), randn((3, 2 * N, K), 10, 0.25)
    out, kept, scales = _forward(moe, prob, lay, rows, weights)
    _check_forward(lay, rows, weights, out, kept, scales)
    dout, down = randn((3, 8), 11), randn((3, 8, N), 12, 0.25)
    _check_back(lay, dout, down, kept, scales, *_back(moe, prob, lay, dout, down, kept, scales))


def test_experts_placed_out_of_order(moe):
    """Receive rows lie by rank, then by expert: offsets do not rise with the expert."""
    counts, e2r = [40, 3, 0, 129, 77, 1, 300, 64], [2, 0, 3, 1, 0, 2, 1, 3]
    K, N, R = 144, 72, sum(counts)
    prob, lay = layout_of_counts(moe, counts, expert_to_rank=e2r, num_ranks=4)
    firsts = [r0 for _, r0, n in spans(lay) if n]
    assert firsts != sorted(firsts)
    codes, weights = integers((R, K), 13), integers((8, 2 * N, K), 14)
    scales, wscales = scales_of(R, 15), scales_of((8, 2 * N), 16)
    check_int8(lay, codes, scales, weights, wscales, True, *forward_int8(moe, prob, lay, codes, scales, weights, wscales, True))
    rows, w = randn((R, K), 17), randn((8, 2 * N, K), 18, K ** -0.5)
    out, kept, ks = _forward(moe, prob, lay, rows, w)
    _check_forward(lay, rows, w, out, kept, ks)
    dout, down = randn((R, K), 19), randn((8, K, N), 20, N ** -0.5)
    _check_back(lay, dout, down, kept, ks, *_back(moe, prob, lay, dout, down, kept, ks))


def test_way_back_of_a_gated_product(moe):
    """experts of a gated product: dout has both its halves' columns."""
    import torch
    counts, K, N = [33, 0, 140], 104, 72
    R = sum(counts)
    prob, lay = layout_of_counts(moe, counts)
    dout, weights = randn((R, 2 * N), 21), randn((3, 2 * N, K), 22, K ** -0.5)
    kept, scales = _random_kept(R, K, 23)
    drows, act = torch.empty((R, 2 * K), dtype=torch.bfloat16, device="cuda"), torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_backward_kept(prob, lay, moe.Experts(K, N, weights, act=moe.MOE_ACT_SWIGLU), dout, kept, scales, drows, act=act)
    _check_back(lay, dout, weights, kept, scales, drows, act)


def test_layouts_that_do_not_fit_stay_inside(moe):
    """Counts and offsets from nowhere: rows outside [0, T*k) are neither read nor written; rows no expert owns stay."""
    import torch
    R, E, K, N = 50, 4, 64, 40
    prob = moe.Problem(R, 1024, 1, E, 1, 1)
    lay = moe.Layout.__new__(moe.Layout)
    codes, scales = integers((R, K), 24), scales_of(R, 25)
    weights, wscales = integers((E, 2 * N, K), 26), scales_of((E, 2 * N), 27)
    rows, w16, down = randn((R, K), 28), randn((E, 2 * N, K), 29, 0.125), randn((E, K, N), 30, 0.125)
    for counts, offsets in (([10, -5, 2 ** 31 - 1, 7], [0, 3, 45, -9, 0]), ([0, 0, 0, 0], [0, 0, 0, 0, 0]),
                            ([60, 60, 60, 60], [-1, 2 ** 31 - 1, 49, 20, 0])):
        lay.expert_count = torch.tensor(counts, dtype=torch.int32, device="cuda")
        lay.expert_offset = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        owned = torch.zeros(R, dtype=torch.bool)
        for c, o in zip(counts, offsets):
            first = min(max(o, 0), R)
            owned[first:first + min(max(c, 0), R - first)] = True
        out, _ = forward_int8(moe, prob, lay, codes, scales, weights, wscales, True)
        free = ~owned.cuda()
        assert bool((out[free].view(torch.uint8) == 0xC3).all())
        out, kept, ks = _forward(moe, prob, lay, rows, w16)
        for t in (out.view(torch.uint8), kept, ks):
            assert bool((t[free] == 0xC3).all())
        kept.masked_fill_(kept == 0xC3, 0)
        drows, act = _back(moe, prob, lay, rows, down, kept, ks)
        assert bool((drows[free].view(torch.uint8) == 0xC3).all()) and bool((act[free].view(torch.uint8) == 0xC3).all())


def test_choice_of_many_tokens(moe):
    """More tokens than a grid's second axis could hold, against the same call in pieces."""
    import torch
    T, E, k = 300_001, 64, 4
    g = torch.Generator(device="cuda").manual_seed(31)
    logits = torch.randn((T, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")

    def call(x):
        n = x.shape[0]
        ids, gates = torch.empty((n, k), dtype=torch.int32, device="cuda"), torch.empty((n, k), device="cuda")
        moe.moe_route_groups(moe.Problem(n, 1024, k, E, 1, 1), moe.Routing(moe.MOE_SCORE_SIGMOID), moe.Grouping(8, 2), x, ids, gates,
                             bias=bias)
        return ids, gates
    ids, gates = call(logits)
    for at in (0, 100_000, 262_143, T - 1000):
        i, w = call(logits[at:at + 1000].contiguous())
        assert torch.equal(ids[at:at + 1000], i) and torch.equal(gates[at:at + 1000], w)
