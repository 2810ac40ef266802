"""The 8-bit calls where an element's offset passes 32 bits: kept pre-activations, integer rows and integer weights of more
than 2^31 bytes, checked at both ends and around the crossing."""
import pytest

from experts_harness import close, gated, gated_slack, sum_slack
from test_gpu_int8 import integers, quantise
from test_gpu_kept import values8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import torch
    import __graft_entry__ as ge
    ge.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    import combine_moe_layout_04_gb300 as m
    yield m
    assert m.moe_move_faults() == 0
    torch.cuda.empty_cache()


def _layout(moe, counts):
    """A problem and the two layout arrays that the experts' calls read."""
    import torch
    R = sum(counts)
    prob = moe.Problem(R, 1024, 1, len(counts), 1, 1)
    lay = moe.Layout.__new__(moe.Layout)
    lay.expert_count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    lay.expert_offset = torch.cat((torch.zeros(1), torch.tensor(counts).cumsum(0))).int().cuda()
    return prob, lay, R


def _places(R, crossing):
    import torch
    at = [0, 1, crossing - 1, crossing, crossing + 1, R - 2, R - 1]
    return torch.tensor(sorted(set(min(max(a, 0), R - 1) for a in at)), device="cuda")


def test_kept(moe):
    import torch
    N, K, counts = 512, 64, [1_100_000, 1, 1_050_000, 7]
    prob, lay, R = _layout(moe, counts)
    assert R * 2 * N > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((R, K), generator=gen, device="cuda", dtype=torch.bfloat16)
    weights = torch.randn((4, 2 * N, K), generator=gen, device="cuda", dtype=torch.bfloat16) / 8
    x = moe.Experts(K, N, weights, act=moe.MOE_ACT_SWIGLU)
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    kept = torch.empty((R, 2 * N), dtype=torch.uint8, device="cuda")
    scales = torch.empty((R, 2, N // 32), dtype=torch.uint8, device="cuda")
    moe.moe_expert_forward_kept(prob, lay, x, rows, out, kept, scales)
    at = _places(R, 2 ** 31 // (2 * N))
    expert = torch.searchsorted(lay.expert_offset[1:].long(), at, right=True)
    pre = torch.einsum("rk,rnk->rn", rows[at].double(), weights[expert].double())
    mag = torch.einsum("rk,rnk->rn", rows[at].double().abs(), weights[expert].double().abs())
    slack = sum_slack(mag, K)
    close(out[at], gated(pre), gated_slack(pre, slack))
    v, X = values8(kept[at], scales[at], N)
    assert bool(((v - pre).abs() <= torch.maximum(2.0 ** -4 * (pre.abs() + slack), 2.0 ** -10 * X) + slack).all())

    down = torch.randn((4, K, N), generator=gen, device="cuda", dtype=torch.bfloat16) / 16
    drows, act = torch.empty((R, 2 * N), dtype=torch.bfloat16, device="cuda"), out
    moe.moe_expert_backward_kept(prob, lay, moe.Experts(N, K, down), rows, kept, scales, drows, act=act)
    g, u = v.chunk(2, dim=1)
    s = torch.sigmoid(g)
    dh = torch.einsum("rn,rnk->rk", rows[at].double(), down[expert].double())
    mag = torch.einsum("rn,rnk->rk", rows[at].double().abs(), down[expert].double().abs())
    near = sum_slack(mag, K) + 2.0 ** -20 * dh.abs()
    close(act[at], g * s * u, 2.0 ** -20 * (g * u).abs())
    close(drows[at, :N], dh * u * s * (1 + g * (1 - s)), near * u.abs() * (1 + g.abs()))
    close(drows[at, N:], dh * g * s, near * g.abs())


def test_integer_rows(moe):
    import torch
    K, N, counts = 4096, 16, [300_000, 5, 230_000]
    prob, lay, R = _layout(moe, counts)
    assert R * K > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn((R, K), generator=gen, device="cuda", dtype=torch.bfloat16)
    codes, scales = torch.empty((R, K), dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    moe.moe_quant8_rows(prob, rows, codes, scales)
    weights, wscales = integers((3, N, K), 3), torch.rand((3, N), generator=gen, device="cuda")
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_forward8(prob, lay, moe.Experts(K, N, weights, scales=wscales), codes, scales, out)
    at = _places(R, 2 ** 31 // K)
    want = quantise(rows[at])
    assert torch.equal(codes[at], want[0]) and torch.equal(scales[at], want[1])
    expert = torch.searchsorted(lay.expert_offset[1:].long(), at, right=True)
    by = scales[at, None].double() * wscales[expert].double()
    sums = torch.einsum("rk,rnk->rn", codes[at].double(), weights[expert].double())
    mag = torch.einsum("rk,rnk->rn", codes[at].double().abs(), weights[expert].double().abs())
    close(out[at], sums * by, by * (mag * (K + 16) * 2.0 ** -23 + 2.0 ** -22 * sums.abs()))


def test_integer_weights(moe):
    import torch
    K, N, E = 8192, 4096, 70
    counts = [0] * E
    counts[0], counts[63], counts[64], counts[69] = 3, 2, 1, 5
    prob, lay, R = _layout(moe, counts)
    assert E * N * K > 2 ** 31
    weights, codes = integers((E, N, K), 4), integers((R, K), 5)
    scales, wscales = torch.rand(R, device="cuda"), torch.rand((E, N), device="cuda")
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_forward8(prob, lay, moe.Experts(K, N, weights, scales=wscales), codes, scales, out)
    first = 0
    for e in (0, 63, 64, 69):
        r = slice(first, first + counts[e])
        first += counts[e]
        by = scales[r, None].double() * wscales[e].double()
        sums = codes[r].double() @ weights[e].double().T
        mag = codes[r].double().abs() @ weights[e].double().abs().T
        close(out[r], sums * by, by * (mag * (K + 16) * 2.0 ** -23 + 2.0 ** -22 * sums.abs()))
    del weights
    w16 = torch.randn((20, 2 * N, K), device="cuda", dtype=torch.bfloat16)   # more than 2^31 bytes, and elements over all rows
    x = moe.Experts(K, N, w16, act=moe.MOE_ACT_SWIGLU)
    c, s = torch.empty(w16.shape, dtype=torch.int8, device="cuda"), torch.empty(w16.shape[:2], device="cuda")
    moe.moe_quant8_weights(moe.Problem(1, 1024, 1, 20, 1, 1), x, c, s)
    for e, n in ((0, 0), (15, 2 * N - 1), (16, 0), (19, 2 * N - 1)):
        want = quantise(w16[e, n:n + 1])
        assert torch.equal(c[e, n:n + 1], want[0]) and torch.equal(s[e, n:n + 1], want[1])
