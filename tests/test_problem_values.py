"""A problem's struct says what its fields hold at the call, however they are held (no GPU needed)."""
import numpy as np
import pytest

from test_experts_refusals import moe  # noqa: F401


def _bytes(moe, p):
    return bytes(moe.Problem(*[int(v) for v in (p.num_tokens, p.hidden, p.topk, p.num_experts, p.num_ranks, p.ranks_per_host,
                                                p.num_src_ranks, p.dtype)]).c())


@pytest.mark.parametrize("kind", ["tensor", "array"])
def test_fields_changed_in_place_are_seen(moe, kind):
    """A count of tokens (or any other field) that a program keeps in a tensor or an array and changes there."""
    import torch
    made = torch.tensor if kind == "tensor" else np.array
    p = moe.Problem(*[made(v) for v in (256, 1024, 2, 16, 4, 2, 1, 0)])
    names = ("num_tokens", "hidden", "topk", "num_experts", "num_ranks", "ranks_per_host", "num_src_ranks", "dtype")
    assert bytes(p.c()) == _bytes(moe, p)
    for name in names:
        getattr(p, name)[...] = int(getattr(p, name)) + 1
        assert bytes(p.c()) == _bytes(moe, p)
        assert bytes(p.c()) == _bytes(moe, p)


def test_plain_fields_are_kept(moe):
    p = moe.Problem(256, 1024, 2, 16, 4, 2)
    assert p.c() is p.c()
    p.num_tokens = np.int64(100)                     # (never changes in place; not kept)
    assert bytes(p.c()) == _bytes(moe, p)
    p.num_tokens = 100
    assert p.c() is p.c() and bytes(p.c()) == _bytes(moe, p)
