"""The type of the logits that the library is told is that of the tensor that was checked, whatever else a torch's tensors
say of themselves (no GPU needed: the entry points are replaced by ones that look at their arguments)."""
import types

import pytest

from test_experts_refusals import GOOD, On, _p, first_gpu, moe  # noqa: F401


@pytest.mark.parametrize("which", ["moe_route", "moe_route_groups", "moe_route_backward"])
def test_type_follows_the_tensor(moe, first_gpu, monkeypatch, which):
    import torch
    told = []

    def entry(problem, routing, *rest):
        told.append(routing._obj.logits_dtype)
        return moe.MOE_OK
    monkeypatch.setattr(moe, "_lib", types.SimpleNamespace(**{which: entry}))
    p, r = _p(moe), moe.Routing()
    ids, gates = On(torch.int32, 256, 2), On(torch.float32, 256, 2)

    def call(logits):
        if which == "moe_route":
            moe.moe_route(p, r, logits, ids, gates, stream=0)
        elif which == "moe_route_groups":
            moe.moe_route_groups(p, r, moe.Grouping(4, 2), logits, ids, gates, stream=0)
        else:
            moe.moe_route_backward(p, r, logits, ids, gates, logits, stream=0)
        return told[-1]
    assert call(On(torch.float32, 256, 16)) == moe.MOE_LOGITS_F32
    assert call(On(torch.bfloat16, 256, 16)) == moe.MOE_LOGITS_BF16  # (a stand-in has no itemsize, as tensors of an older torch)
    assert call(GOOD) == moe.MOE_LOGITS_F32                          # nothing but an address
