"""Every way that the experts' products are cut: tiles of all widths, tiles shared by two and four pairs at each
width, and teams of pairs that take a second tile, against 64-bit products."""
import pytest

from experts_harness import close, gated, gated_slack, layout_of_counts, products, randn, sum_slack
from test_gpu_experts import _backward, _check_forward, _check_rows, _forward
from test_gpu_quant4 import _product

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


# means of 311 to 365 rows: tiles of 384 columns, one tile or two an expert, the second product of 16 to 256 columns
AROUND_384 = {
    "all kinds of rows": [384, 383, 384, 257, 273, 369, 385],
    "one too many": [384, 360, 385, 350, 300],
    "as few as there are": [311, 311, 312, 312],
    "skewed": [1, 769, 700, 17, 330],
}


@pytest.mark.parametrize("K,N", [(8, 8), (72, 136), (200, 264), (1024, 512)])
@pytest.mark.parametrize("counts", AROUND_384.values(), ids=AROUND_384.keys())
def test_tiles_of_384_columns(moe, counts, K, N):
    assert 310 < sum(counts) / len(counts) <= 365
    prob, lay = layout_of_counts(moe, counts)
    for act in (False, True):
        _check_forward(lay, *_forward(moe, prob, lay, K, N, act), act)
    for through in (False, True):
        weights, dout, rows, pre, drows, dw = _backward(moe, prob, lay, K, N, False, through)
        _check_rows(lay, weights, dout, pre, drows)


def test_tiles_of_384_columns_and_many_stages(moe):
    prob, lay = layout_of_counts(moe, [340, 384, 330, 355])
    _check_forward(lay, *_forward(moe, prob, lay, 4104, 1160, True), True)
    weights, dout, rows, pre, drows, dw = _backward(moe, prob, lay, 1160, 4104, False, True)
    _check_rows(lay, weights, dout, pre, drows)


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("counts", [[1000, 1024, 769, 1152, 900], [1152, 1153, 1151, 385]])
@pytest.mark.parametrize("K,N", [(96, 136), (1056, 264)])
def test_4_bit_tiles_of_three_an_expert(moe, counts, K, N, act):
    """Means of 769 to 1152 rows: 384 columns in 4 bits, three tiles an expert."""
    assert 768 < sum(counts) / len(counts) <= 1152
    prob, lay = layout_of_counts(moe, counts)
    rows = randn((sum(counts), K), 5)
    weights = randn((len(counts), 2 * N if act else N, K), 6, K ** -0.5)
    out, pre, values, wv = _product(moe, prob, lay, K, N, act, rows, weights)
    ref, mag = products(lay, values, wv)
    slack = sum_slack(mag, K)
    close(out, gated(ref) if act else ref, gated_slack(ref, slack) if act else slack)


# Few tiles and a long contraction: two or four pairs share a tile.  (counts, features, contraction); a gated tile has 128
# features, any other 256.  Tiles of 64, 128, 256, 320 and 384 columns, then more tiles than teams run at once (36 of two
# pairs, 15 of four), so that a team's barriers, blocks and ends of tensor memory go on from one tile to the next.
SHARED = {
    "128 columns, four pairs": ([80], 1024, 7168),
    "256 columns, four pairs": ([150], 1024, 7168),
    "320 columns, four pairs": ([300], 1024, 7176),
    "384 columns, four pairs": ([350], 1032, 7168),
    "256 columns, two pairs": ([200, 190], 1024, 7168),
    "320 columns, two pairs": ([300, 0, 301, 320], 520, 7168),
    "second tile, two pairs": ([4, 3, 4, 1, 0, 9, 4, 4], 1280, 7168),
    "second tile, four pairs": ([4, 1, 7, 4, 2], 1024, 16384),
    "second wide tile, four pairs": ([300, 257, 320], 1024, 16384),
}


def _twice(run):
    """The results of a run, and that another one gives the same bits."""
    import torch
    a, b = run(), run()
    for x, y in zip(a, b):
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    return a


@pytest.mark.parametrize("counts,N,K", SHARED.values(), ids=SHARED.keys())
def test_shared_tiles_forward(moe, counts, N, K):
    prob, lay = layout_of_counts(moe, counts)
    for act, n in ((True, N), (False, 2 * N)):
        _check_forward(lay, *_twice(lambda: _forward(moe, prob, lay, K, n, act)), act)


@pytest.mark.parametrize("counts,half,N", SHARED.values(), ids=SHARED.keys())
def test_shared_tiles_of_the_rows_gradient(moe, counts, half, N):
    import torch
    prob, lay = layout_of_counts(moe, counts)
    K = 2 * half
    weights, dout, pre = randn((len(counts), N, K), 1, N ** -0.5), randn((sum(counts), N), 2), randn((sum(counts), 2 * K), 3, 2.0)
    for p in (None, pre):
        def run():
            drows = torch.full((sum(counts), K if p is None else 2 * K), float("nan"), dtype=torch.bfloat16, device="cuda")
            moe.moe_expert_backward_rows(prob, lay, moe.Experts(K, N, weights), dout, drows, pre=p)
            return (drows,)
        _check_rows(lay, weights, dout, p, *_twice(run))


@pytest.mark.parametrize("counts,N,K", [([80], 1024, 8224), ([150], 1024, 8224), ([300], 1024, 8224), ([350, 340], 520, 8224),
                                        ([4, 3, 4, 1, 0, 9, 4, 4], 1280, 28672), ([4, 1, 7, 4, 2], 1024, 65536),
                                        ([300, 257, 384], 1024, 65536)])
def test_shared_tiles_in_4_bits(moe, counts, N, K):
    prob, lay = layout_of_counts(moe, counts)
    rows, weights = randn((sum(counts), K), 5), randn((len(counts), 2 * N, K), 6, K ** -0.5)
    first = _product(moe, prob, lay, K, N, True, rows, weights)
    out, pre, values, wv = first
    again = _twice(lambda: _product(moe, prob, lay, K, N, True, rows, weights)[:2])
    assert bool((again[0] == out).all()) and bool((again[1] == pre).all())
    ref, mag = products(lay, values, wv)
    slack = sum_slack(mag, K)
    close(pre, ref, slack)
    close(out, gated(ref), gated_slack(ref, slack))
