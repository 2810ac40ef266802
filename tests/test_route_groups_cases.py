"""That the grouped choice's cases on the GPU compare something: the share of their rows that decide by more than fp32
can move, made anew on the CPU (no GPU needed)."""
import numpy as np
import pytest

from test_gpu_route_groups import CASES, GAP, _reference


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T,E,G,kept,k", CASES)
def test_rows_decide(T, E, G, kept, k, top, score):
    import torch
    g = torch.Generator().manual_seed(T * 1000 + E + top)
    for dtype in (torch.float32, torch.bfloat16):
        rank = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).double()
        p = (rank + 0.5) / E
        logits = (torch.log(p / (1 - p)) if score == "sigmoid" else torch.log(p)).to(dtype)
        assert (_reference(logits.float().numpy(), None, G, kept, top, k, score)[1] > GAP).mean() >= 0.3
        bias = 0.2 / (E if score == "softmax" else 1) * torch.randn(E, generator=g)
        noise = (3 * torch.randn((T, E), generator=g)).to(dtype)
        assert (_reference(noise.float().numpy(), bias.numpy(), G, kept, top, k, score)[1] > GAP).mean() >= 0.5
