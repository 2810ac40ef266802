"""What a grouped choice's structs say is what its routing and grouping hold at the call, however their fields are
held (no GPU needed: the library's entry point is replaced by one that looks at its arguments)."""
import types

import numpy as np
import pytest

from test_experts_refusals import _p, moe  # noqa: F401


@pytest.fixture
def said(moe, monkeypatch):
    """Makes the call and returns the bytes of the structs that the library was given."""
    seen = []

    def entry(problem, routing, grouping, *rest):
        seen.append((bytes(routing._obj), bytes(grouping._obj)))
        return moe.MOE_OK
    monkeypatch.setattr(moe, "_lib", types.SimpleNamespace(moe_route_groups=entry))
    moe._CHOICE.clear()

    def call(r, g):
        moe.moe_route_groups(_p(moe, num_tokens=0), r, g, None, None, None, stream=0)
        return seen[-1]
    return call


def _plain(moe, r, g):
    return (bytes(moe.Routing(int(r.score), bool(r.renormalise), float(r.scale)).c(None)),
            bytes(moe.Grouping(int(g.groups), int(g.kept), int(g.top)).c()))


def test_fields_changed_in_place_are_seen(moe, said):
    """A model's buffer as the scale, or any field, that is loaded or counted on between two calls."""
    import torch
    r = moe.Routing(torch.tensor(0), torch.tensor(True), torch.tensor(1.5))
    g = moe.Grouping(torch.tensor(4), torch.tensor(2), torch.tensor(2))
    assert said(r, g) == _plain(moe, r, g)
    for change in (lambda: r.scale.fill_(3.0), lambda: r.renormalise.fill_(False), lambda: r.score.fill_(1),
                   lambda: g.groups.fill_(8), lambda: g.kept.fill_(3), lambda: g.top.fill_(1)):
        change()
        assert said(r, g) == _plain(moe, r, g)


def test_arrays_of_no_dimension_are_taken(moe, said):
    """As moe_route takes them; the next value of the same array too."""
    r, g = moe.Routing(np.array(0), np.array(True), np.array(1.5)), moe.Grouping(np.array(4), np.array(2), np.array(2))
    assert said(r, g) == _plain(moe, r, g)
    r.scale[...], g.kept[...] = 0.25, 4
    assert said(r, g) == _plain(moe, r, g)


def test_zeros_keep_their_sign(moe, said):
    for scale in (0.0, -0.0, 0.0):
        r, g = moe.Routing(scale=scale), moe.Grouping(4, 2)
        assert said(r, g) == _plain(moe, r, g)


def test_plain_values_are_kept(moe, said):
    r, g = moe.Routing(scale=2), moe.Grouping(4, 2)
    for scale in (2, 2.5, 2.0):
        r.scale = scale
        assert said(r, g) == _plain(moe, r, g)
    assert len(moe._CHOICE) == 2


def test_values_of_no_number_are_refused_each_time(moe, said):
    good = moe.Grouping(4, 2)
    for r, g in ((moe.Routing(scale="2"), good), (moe.Routing(score=None), good), (moe.Routing(), moe.Grouping([4], 2)),
                 (moe.Routing(score=0.0), good), (moe.Routing(), moe.Grouping(4.0, 2))):
        said(moe.Routing(), good)
        for _ in range(2):
            with pytest.raises(TypeError):
                said(r, g)
