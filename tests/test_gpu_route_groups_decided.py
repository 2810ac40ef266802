"""The grouped choice by the sum of two keys, and from bf16 logits, on rows most of which are decided by more than fp32
can move: their share is asked for."""
import pytest

from test_gpu_route_groups import _check, moe  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [  # T, E, G, kept, k
    (1, 256, 8, 4, 8), (509, 256, 8, 4, 8), (300, 160, 8, 3, 6), (200, 64, 8, 2, 4), (77, 384, 8, 4, 8), (60, 512, 16, 4, 8),
    (90, 60, 5, 2, 3), (33, 1000, 20, 7, 16), (25, 1024, 4, 1, 8)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T,E,G,kept,k", CASES)
def test_most_rows_are_decided(moe, T, E, G, kept, k, top, score):
    import torch
    g = torch.Generator().manual_seed(7 * T + E + top)
    for dtype in (torch.float32, torch.bfloat16):
        noise = (2 * torch.randn((T, E), generator=g)).to(dtype)
        bias = 0.2 / (E if score == "softmax" else 1) * torch.randn(E, generator=g)
        _check(moe, noise.cuda(), bias.cuda(), G, kept, top, k, score, decided=0.9)
