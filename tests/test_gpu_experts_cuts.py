"""Every way that the experts' products are cut: tiles of all widths, against 64-bit products."""
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
