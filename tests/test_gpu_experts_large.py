"""Arrays whose element offsets pass 32 bits: results at both ends and in
between against 64-bit products of sampled rows."""
import pytest

from experts_harness import (close, layout_of_counts, quantise4, randn, row_scales, spans, sum_slack, unpack4, values4)

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
    torch.cuda.empty_cache()


def _sample(n, lay):
    """Rows at the ends of the array and of the groups, and their experts."""
    at = {0, 1, n - 1, n // 2}
    owner = {}
    for e, r0, c in spans(lay):
        at |= {r0, r0 + c - 1, r0 + c // 2}
    for e, r0, c in spans(lay):
        owner.update({r: e for r in at if r0 <= r < r0 + c})
    return sorted(owner), owner


def test_products_with_results_past_32_bits(moe):
    import torch
    counts, K, N = [100000, 7, 162040, 105], 64, 8200
    R = sum(counts)
    assert R * N > 1 << 31
    prob, lay = layout_of_counts(moe, counts)
    rows, w = randn((R, K), 1), randn((4, N, K), 2, K ** -0.5)
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_forward(prob, lay, moe.Experts(K, N, w), rows, out)
    at, owner = _sample(R, lay)
    for r in at:
        a, b = rows[r].double(), w[owner[r]].double()
        close(out[r], b @ a, sum_slack(b.abs() @ a.abs(), K))
    # the same array as the gradient that comes in, and as the rows' gradient that goes out
    wide = moe.Experts(N, K, randn((4, K, N), 3, N ** -0.5))
    d = rows
    moe.moe_expert_backward_rows(prob, lay, wide, d, out)
    for r in at:
        a, b = d[r].double(), wide.weights[owner[r]].double()
        close(out[r], a @ b, sum_slack(a.abs() @ b.abs(), K))


def test_weight_gradient_past_32_bits(moe):
    import torch
    counts, K, W = [3] * 30 + [0, 200] + [17] * 32, 8200, 4104
    E, R = len(counts), sum(counts)
    assert E * W * K > 1 << 31
    prob, lay = layout_of_counts(moe, counts)
    rows, dout = randn((R, K), 1), randn((R, W), 2)
    dw = torch.full((E, W, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_backward_weights(prob, lay, moe.Experts(K, W), rows, dout, dw)
    for e, r0, n in spans(lay):
        if e not in (0, 30, 31, 63):
            continue
        for m in (0, 4095, W - 1):
            d, x = dout[r0:r0 + n, m].double(), rows[r0:r0 + n].double()
            close(dw[e, m], d @ x, sum_slack(d.abs() @ x.abs(), n))


def test_4_bit_rows_past_32_bits(moe):
    import torch
    counts, K, N = [140001, 0, 160000], 7168, 64
    R = sum(counts)
    assert R * K > 1 << 31
    prob, lay = layout_of_counts(moe, counts)
    rows = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    for r in range(0, R, 32768):
        rows[r:r + 32768] = randn((min(32768, R - r), K), r)
    codes = torch.empty((R, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty(moe.moe_quant4_row_scale_bytes(prob, K), dtype=torch.uint8, device="cuda")
    moe.moe_quant4_rows(prob, lay, rows, codes, scales)
    at, owner = _sample(R, lay)
    want, byte = quantise4(rows[at])
    assert torch.equal(unpack4(codes[at]), want)
    got = row_scales(lay, scales, K)[at]
    assert torch.equal(got[:, : K // 32], byte)
    w = moe.Experts(K, N, randn((3, N, K), 5, K ** -0.5))
    wc = torch.empty((3, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.empty(moe.moe_quant4_weight_scale_bytes(prob, w), dtype=torch.uint8, device="cuda")
    moe.moe_quant4_weights(prob, w, wc, ws)
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_forward4(prob, lay, moe.Experts(K, N, wc, scales=ws), codes, scales, out)
    value = values4(want, byte)
    for i, r in enumerate(at):
        b = values4(*quantise4(w.weights[owner[r]]))
        close(out[r], b @ value[i], sum_slack(b.abs() @ value[i].abs(), K))


def test_combine_gradient_past_32_bits(moe):
    import torch
    T, k, h = 40000, 8, 7168
    assert T * k * h > 1 << 31
    prob = moe.Problem(T, h, k, 16, 1, 1)
    ids = torch.rand((T, 16), device="cuda").topk(k, dim=1).indices.int().contiguous()
    lay, ws = moe.Layout(prob), moe.alloc_workspace(prob)
    moe.moe_layout(prob, ids, ws, lay)
    dout = randn((T, h), 1)
    y = torch.empty((T * k, h), dtype=torch.bfloat16, device="cuda")
    for r in range(0, T * k, 32768):
        y[r:r + 32768] = randn((min(32768, T * k - r), h), r)
    w = torch.rand((T, k), device="cuda")
    dy, dw = torch.full_like(y, float("nan")), torch.empty_like(w)
    moe.moe_combine_backward(prob, lay, dout, y, w, dy, dw)
    for t in (0, 1, T // 2, T - 1):
        pos = lay.pos[t].long()
        assert torch.equal(dy[pos], (w[t][:, None] * dout[t].float()).to(torch.bfloat16))
        a, b = dout[t].double(), y[pos].double()
        assert bool(((dw[t].double() - b @ a).abs() <= (b.abs() @ a.abs()) * (h / 256 + 24) * 2.0 ** -24).all())
    assert bool(torch.isfinite(dy[:: 997].float()).all())


def test_rows_past_the_plain_sums_of_counts(moe):
    """So many rows that the counts of tiles are added up with checks: rows at both ends of every expert."""
    import torch
    counts, K, N = [1, (1 << 26) - 70, 0, 131, 5], 32, 8
    R, E = sum(counts), len(counts)
    assert R >= 1 << 26
    prob = moe.Problem(R, 1024, 1, E, 1, 1)
    lay = moe.Layout.__new__(moe.Layout)            # the two arrays that the experts' calls read
    lay.expert_count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    lay.expert_offset = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    lay.expert_offset[1:] = lay.expert_count.cumsum(0)
    lay.recv_src = torch.empty(0, device="cuda")
    rows = torch.empty((R, K), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w = moe.Experts(K, N, randn((E, N, K), 2, K ** -0.5))
    out = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_forward(prob, lay, w, rows, out)
    at, owner = _sample(R, lay)
    for r in at:
        a, b = rows[r].double(), w.weights[owner[r]].double()
        close(out[r], b @ a, sum_slack(b.abs() @ a.abs(), K))
    assert bool(torch.isfinite(out).all())
    codes = torch.empty((R, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty(moe.moe_quant4_row_scale_bytes(prob, K), dtype=torch.uint8, device="cuda")
    moe.moe_quant4_rows(prob, lay, rows, codes, scales)
    wc = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.empty(moe.moe_quant4_weight_scale_bytes(prob, w), dtype=torch.uint8, device="cuda")
    moe.moe_quant4_weights(prob, w, wc, ws)
    out.fill_(float("nan"))
    moe.moe_expert_forward4(prob, lay, moe.Experts(K, N, wc, scales=ws), codes, scales, out)
    want, byte = quantise4(rows[at])
    assert torch.equal(unpack4(codes[at]), want)
    value = values4(want, byte)
    for i, r in enumerate(at):
        b = values4(*quantise4(w.weights[owner[r]]))
        close(out[r], b @ value[i], sum_slack(b.abs() @ value[i].abs(), K))
    assert bool(torch.isfinite(out).all())


def test_weight_gradient_of_experts_that_take_seconds(moe):
    """Experts whose sums over their rows take longer than a second (0.23 us for 64 rows): nothing that waits for them
    gives up, nor what waits for a later expert on the same SMs (77 experts, a tile each, on at most 76 pairs of SMs)."""
    import torch
    counts, K = [300_000_000, 300_000_003] + [0] * 73 + [7, 5], 8
    R, E = sum(counts), len(counts)
    prob = moe.Problem(R, 1024, 1, E, 1, 1)
    lay = moe.Layout.__new__(moe.Layout)
    lay.expert_count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    lay.expert_offset = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    lay.expert_offset[1:] = lay.expert_count.cumsum(0)
    rows, dout = (torch.zeros((R, K), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = torch.tensor([0, 63, 64, 1 << 20, (1 << 28) + 1, counts[0] - 70, counts[0] - 1], device="cuda")
    rows[at], dout[at], rows[counts[0] + at], dout[counts[0] + at] = 2.0, 1.0, 3.0, 1.0
    rows[R - 12:], dout[R - 12:] = 1.0, 5.0
    dw = torch.full((E, K, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_backward_weights(prob, lay, moe.Experts(K, K), rows, dout, dw)
    assert moe.moe_move_faults() == 0
    for e, want in ((0, 2 * len(at)), (1, 3 * len(at)), (2, 0), (E - 2, 35), (E - 1, 25)):
        assert bool((dw[e] == want).all()), e
