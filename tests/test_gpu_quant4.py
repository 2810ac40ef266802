"""Microscaled 4 bits on the GPU: codes and scales bit-exact against a 64-bit
search over the grid, and the grouped product against 64-bit products of the
values that codes and scales stand for."""
import numpy as np
import pytest

from experts_harness import (close, gated, gated_slack, guarded, layout_of_counts, products, quantise4, randn,
                             row_scales, spans, sum_slack, unpack4, values4, weight_scales)
from test_gpu_experts import COUNTS

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


def _quant_rows(moe, prob, lay, rows):
    import torch
    R, K = rows.shape
    codes, t0 = guarded((R, K // 2), torch.uint8, 0xC3)
    scales, t1 = guarded((moe.moe_quant4_row_scale_bytes(prob, K),), torch.uint8, 0xC3)
    moe.moe_quant4_rows(prob, lay, rows, codes, scales)
    torch.cuda.synchronize()
    assert bool((t0 == 0xC3).all()) and bool((t1 == 0xC3).all())
    return codes, scales


def _wild(n, K, seed):
    """Rows with zero blocks, one-value blocks, tiny and huge magnitudes, exact ties and both zeros."""
    import torch
    x = randn((n, K), seed).float().view(n, -1, 32)
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    x *= torch.pow(2.0, torch.randint(-90, 90, (n, K // 32, 1), generator=g, device="cuda").float())
    pick = torch.randint(0, 8, (n, K // 32), generator=g, device="cuda")
    x[pick == 0] = 0.0
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, device="cuda")
    x[pick == 1] = ties * torch.where(torch.arange(32, device="cuda") % 3 == 0, -1.0, 1.0)
    x[pick == 2] = -0.0
    tiny = torch.full((32,), 2.0 ** -133, device="cuda")
    tiny[::2] *= 3
    x[pick == 3] = tiny
    one = torch.zeros(32, device="cuda")
    one[5] = -3.0e38
    x[pick == 4] = one
    return x.view(n, K).to(torch.bfloat16)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 1024, 1056, 2208])
@pytest.mark.parametrize("counts", [COUNTS["one row"], COUNTS["tile edges"], COUNTS["skewed"]])
def test_row_codes_and_scales_exact(moe, counts, K):
    import torch
    prob, lay = layout_of_counts(moe, counts)
    rows = _wild(sum(counts), K, K)
    codes, scales = _quant_rows(moe, prob, lay, rows)
    want, byte = quantise4(rows)
    got = row_scales(lay, scales, K)
    assert torch.equal(got[:, : K // 32], byte)
    assert bool((got[:, K // 32:] == 0).all())
    assert torch.equal(unpack4(codes), want)


@pytest.mark.parametrize("counts", [[0] * 20 + [1000, 3] + [0] * 18, [300, 0, 129, 31]])
def test_blocks_of_rows_whole_and_shared(moe, counts):
    """Few rows an expert on average, and one with many: a block takes 128 rows; many on average: four blocks share them."""
    import torch
    K = 1056
    prob, lay = layout_of_counts(moe, counts)
    rows = _wild(sum(counts), K, K)
    codes, scales = _quant_rows(moe, prob, lay, rows)
    want, byte = quantise4(rows)
    assert torch.equal(row_scales(lay, scales, K)[:, : K // 32], byte) and torch.equal(unpack4(codes), want)


@pytest.mark.parametrize("K", [32, 544, 1056, 2208])
def test_rows_on_16_bytes_only(moe, K):
    """Rows that start 16 bytes past a 32-byte boundary: the same codes and scales."""
    import torch
    counts = [3, 0, 130, 7]
    prob, lay = layout_of_counts(moe, counts)
    n = sum(counts)
    rows = torch.empty(n * K + 8, dtype=torch.bfloat16, device="cuda")[8:].view(n, K)
    rows.copy_(_wild(n, K, K))
    assert rows.data_ptr() % 32 == 16
    codes, scales = _quant_rows(moe, prob, lay, rows)
    want, byte = quantise4(rows)
    assert torch.equal(row_scales(lay, scales, K)[:, : K // 32], byte) and torch.equal(unpack4(codes), want)


def test_not_finite_blocks(moe):
    import torch
    prob, lay = layout_of_counts(moe, [3, 2])
    rows = randn((5, 128), 1)
    rows[0, 3], rows[1, 40], rows[2, 127], rows[3, 64] = float("inf"), float("nan"), float("-inf"), float("nan")
    codes, scales = _quant_rows(moe, prob, lay, rows)
    want, byte = quantise4(rows)
    assert torch.equal(row_scales(lay, scales, 128), byte) and torch.equal(unpack4(codes), want)
    assert int((byte == 255).sum()) == 4


def _quant_weights(moe, prob, x, weights):
    import torch
    E, W, K = weights.shape
    codes, t0 = guarded((E, W, K // 2), torch.uint8, 0xC3)
    scales, t1 = guarded((moe.moe_quant4_weight_scale_bytes(prob, x),), torch.uint8, 0xC3)
    moe.moe_quant4_weights(prob, x, codes, scales)
    torch.cuda.synchronize()
    assert bool((t0 == 0xC3).all()) and bool((t1 == 0xC3).all())
    return codes, scales


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("K,N", [(32, 8), (96, 136), (1152, 72), (256, 264)])
def test_weight_codes_and_scales_exact(moe, K, N, act):
    import torch
    prob, _ = layout_of_counts(moe, [1, 2, 0])
    x = moe.Experts(K, N, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)
    W = x.weight_rows
    x.weights = _wild(3 * W, K, N).view(3, W, K)
    codes, scales = _quant_weights(moe, prob, x, x.weights)
    want, byte = quantise4(x.weights.view(3 * W, K))
    got = weight_scales(x, 3, scales)
    assert torch.equal(unpack4(codes).view(3 * W, K), want)
    assert torch.equal(got[..., : K // 32].reshape(3 * W, -1), byte)
    assert bool((got[..., K // 32:] == 0).all())


def _product(moe, prob, lay, K, N, act, rows, weights, want_pre=True):
    import torch
    R, E = rows.shape[0], weights.shape[0]
    x = moe.Experts(K, N, weights, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)
    wc, ws = _quant_weights(moe, prob, x, weights)
    rc, rs = _quant_rows(moe, prob, lay, rows)
    x4 = moe.Experts(K, N, wc, act=x.act, scales=ws)
    out, t0 = guarded((R, N), torch.bfloat16, 0xC3)
    pre, t1 = guarded((R, x.weight_rows), torch.bfloat16, 0xC3) if act and want_pre else (None, None)
    moe.moe_expert_forward4(prob, lay, x4, rc, rs, out, pre=pre)
    torch.cuda.synchronize()
    assert bool((t0 == 0xC3).all()) and (pre is None or bool((t1 == 0xC3).all()))
    values = values4(unpack4(rc), row_scales(lay, rs, K)[:, : K // 32])
    wv = values4(unpack4(wc).view(E * x.weight_rows, K), weight_scales(x, E, ws)[..., : K // 32].reshape(E * x.weight_rows, -1))
    return out, pre, values, wv.view(E, -1, K)


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("K,N", [(32, 8), (64, 128), (96, 136), (288, 264), (1024, 520), (2080, 264)])
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
def test_product(moe, counts, K, N, act):
    prob, lay = layout_of_counts(moe, counts)
    rows = randn((sum(counts), K), 5)
    weights = randn((len(counts), 2 * N if act else N, K), 6, K ** -0.5)
    out, pre, values, wv = _product(moe, prob, lay, K, N, act, rows, weights)
    ref, mag = products(lay, values, wv)
    slack = sum_slack(mag, K)
    if act:
        close(pre, ref, slack)
        close(out, gated(ref), gated_slack(ref, slack))
    else:
        close(out, ref, slack)


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 130], [17] * 8])
@pytest.mark.parametrize("K,N,act", [(8224, 72, True), (10272, 264, False), (4128, 136, True)])
def test_product_of_few_tiles(moe, counts, K, N, act):
    """Contractions that are cut into parts because there are few tiles."""
    prob, lay = layout_of_counts(moe, counts)
    rows = randn((sum(counts), K), 5)
    weights = randn((len(counts), 2 * N if act else N, K), 6, K ** -0.5)
    out, pre, values, wv = _product(moe, prob, lay, K, N, act, rows, weights)
    ref, mag = products(lay, values, wv)
    slack = sum_slack(mag, K)
    close(out, gated(ref) if act else ref, gated_slack(ref, slack) if act else slack)


def test_product_wide_scales(moe):
    """Scales far from one, a different one for every block: 2^-40 .. 2^40 on rows and weights."""
    import torch
    counts, K, N = [40, 0, 129, 3], 512, 136
    prob, lay = layout_of_counts(moe, counts)
    g = torch.Generator(device="cuda").manual_seed(9)

    def spread(shape):
        x = randn(shape, shape[-2]).float()
        s = torch.randint(-40, 41, shape[:-1] + (shape[-1] // 32,), generator=g, device="cuda").float()
        return (x * torch.pow(2.0, s).repeat_interleave(32, dim=-1)).to(torch.bfloat16)
    out, _, values, wv = _product(moe, prob, lay, K, N, False, spread((172, K)), spread((4, N, K)))
    ref, mag = products(lay, values, wv)
    close(out, ref, sum_slack(mag, K))


@pytest.mark.parametrize("counts,K,N", [([300, 0, 384, 290, 321, 129], 512, 136), ([257, 385, 310], 96, 264),
                                        ([1000, 1153, 0, 1152, 900], 288, 72)])
@pytest.mark.parametrize("act", [False, True])
def test_product_wide_tiles(moe, counts, K, N, act):
    """Tiles of two products, a different scale for every block: 2^-20 .. 2^20 on rows, up to 2^4 on weights."""
    import torch
    prob, lay = layout_of_counts(moe, counts)
    g = torch.Generator(device="cuda").manual_seed(9)

    def spread(shape, most):
        x = randn(shape, shape[-2], K ** -0.5)
        s = torch.randint(-most, most + 1, shape[:-1] + (K // 32,), generator=g, device="cuda").float()
        return (x.float() * torch.pow(2.0, s).repeat_interleave(32, dim=-1)).to(torch.bfloat16)
    out, pre, values, wv = _product(moe, prob, lay, K, N, act, spread((sum(counts), K), 20),
                                    spread((len(counts), 2 * N if act else N, K), 4))
    ref, mag = products(lay, values, wv)
    slack = sum_slack(mag, K)
    if act:
        close(pre, ref, slack)
    else:
        close(out, ref, slack)


def test_rows_that_are_not_finite_stay_alone(moe):
    """A row with an infinity gives NaN in its own results and changes no other row; so do weights."""
    import torch
    counts, K, N = [100, 30], 256, 136
    prob, lay = layout_of_counts(moe, counts)
    rows, weights = randn((130, K), 1), randn((2, 2 * N, K), 2, K ** -0.5)
    clean = _product(moe, prob, lay, K, N, True, rows, weights)[0]
    rows2, weights2 = rows.clone(), weights.clone()
    rows2[7, 100], weights2[1, 5, 31] = float("inf"), float("nan")
    hurt = _product(moe, prob, lay, K, N, True, rows2, weights2)[0]
    bad = torch.zeros((130, N), dtype=torch.bool, device="cuda")
    bad[7] = True
    _, r0, n = spans(lay)[1]
    bad[r0:r0 + n, 5] = True
    assert bool(torch.isnan(hurt[bad]).all())
    assert torch.equal(hurt[~bad], clean[~bad])
