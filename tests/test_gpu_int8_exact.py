"""Integer products whose sums are exact at any length of the contraction, so that results are compared bit for bit: a
lost or doubled stage, piece or part of a long contraction shows, however long it is."""
import pytest

from experts_harness import layout_of_counts, spans
from test_gpu_int8 import _forward, integers, moe  # noqa: F401

pytestmark = pytest.mark.gpu

# counts, K, N: contractions shared by four and two pairs and by none, short ones with three store groups (below 3200, tiles of
# 256), a last stage of 16, 48 and 112 columns, one row to several tiles
CASES = [([2, 0, 1], 1 << 20, 8), ([1], (1 << 20) - 16, 264), ([60, 0, 70], 65536 + 48, 72), ([1], 7168, 1024),
         ([3, 0, 1, 2], 8192, 264), ([300], 8192 + 112, 520), ([130, 0, 257, 60], 7168, 4096), ([140, 1, 512, 0, 200], 3712, 1032),
         ([300, 257, 0, 512], 2064, 2568), ([130, 400], 3184, 136), ([16, 0, 31, 1], 2048, 512)]


def _sums(lay, codes, weights):
    """The sums in 64 bits (far below 2^24, so exact in fp32 too)."""
    import torch
    out = torch.zeros((codes.shape[0], weights.shape[1]), dtype=torch.float64, device="cuda")
    for e, r0, n in spans(lay):
        for at in range(0, weights.shape[1], 256):   # (weights of 2^20 columns in 64 bits are 8 MB a row)
            out[r0:r0 + n, at:at + 256] = codes[r0:r0 + n].double() @ weights[e, at:at + 256].double().T
    return out


def _compare(moe, counts, codes, weights, act):
    import torch
    prob, lay = layout_of_counts(moe, counts)
    R, one = sum(counts), torch.ones
    out, pre = _forward(moe, prob, lay, codes, one(R, device="cuda"), weights, one(weights.shape[:2], device="cuda"), act)
    want = _sums(lay, codes, weights).to(torch.bfloat16)
    assert torch.equal(pre if act else out, want)
    return want


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_small_integers(moe, counts, K, N, act):
    """Every term counts: integers in -3 .. 3, sums of magnitudes at most 9 K <= 9 * 2^20 < 2^24."""
    W = 2 * N if act else N
    _compare(moe, counts, integers((sum(counts), K), K + N, -3, 3), integers((len(counts), W, K), K + N + 1, -3, 3), act)


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_places_of_a_contraction(moe, counts, K, N, act):
    """26 terms a sum, of 9 at most each, so that bf16 holds every sum (<= 234 < 256): at both ends, on either side of
    where pieces, stages and parts of the contraction meet, and in other places for every row."""
    import torch
    W, R = 2 * N if act else N, sum(counts)
    stages = -(-K // 128)
    meet = {0, 15, 16, 63, 64, 127, 128, K - 1, K - 16, K - 17}
    for part in (1, 2, 3):
        at = stages * part // 4 * 128
        meet |= {at - 1, at}
    places = torch.tensor(sorted(p for p in meet if 0 <= p < K), device="cuda")
    codes = torch.zeros((R, K), dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(K + N)
    others = torch.randint(0, K, (R, 26 - len(places)), generator=g, device="cuda")
    values = integers((R, 26), K, 1, 3) * (1 - 2 * integers((R, 26), K + 1, 0, 1))
    codes.scatter_(1, torch.cat((others, places.expand(R, -1)), dim=1), values)
    weights = integers((len(counts), W, K), N, 1, 3) * (1 - 2 * integers((len(counts), W, K), N + 1, 0, 1))
    assert int(_compare(moe, counts, codes, weights, act).abs().max()) <= 234
