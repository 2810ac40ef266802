"""The binding's checks hold on a torch that lacks one of the types they name, and no failure inside a check counts as
an object with nothing but an address (no GPU needed)."""
import pytest

from test_experts_refusals import On, _lay, _p, first_gpu, moe  # noqa: F401


@pytest.fixture
def without_e8m0(moe, first_gpu, monkeypatch):
    """A torch without 8-bit powers of two."""
    import torch
    monkeypatch.delattr(torch, "float8_e8m0fnu", raising=False)
    monkeypatch.setattr(moe, "_KINDS", moe._Kinds())


def _kept_calls(moe):
    import torch
    bf, u8, p = torch.bfloat16, torch.uint8, _p(moe)
    lay = _lay(moe, expert_count=On(torch.int32, 16), expert_offset=On(torch.int32, 17))
    up = moe.Experts(64, 40, On(bf, 16, 80, 64), act=moe.MOE_ACT_SWIGLU)
    down = moe.Experts(40, 64, On(bf, 16, 64, 40))
    return (lambda scales: moe.moe_expert_forward_kept(p, lay, up, On(bf, 512, 64), On(bf, 512, 40), On(u8, 512, 80), scales, stream=0),
            lambda scales: moe.moe_expert_backward_kept(p, lay, down, On(bf, 512, 64), On(u8, 512, 80), scales, On(bf, 512, 80), stream=0))


@pytest.mark.parametrize("which", [0, 1])
def test_scales_are_checked_without_the_type(moe, without_e8m0, which):
    import torch
    u8, call = torch.uint8, _kept_calls(moe)[which]
    for bad in (torch.zeros((512, 2, 2), dtype=u8), On(u8, 512, 2, 2, gpu=1), On(torch.float32, 512, 2, 2),
                On(u8, 512, 2, 2, dense=False), On(u8, 511, 2, 2)):
        with pytest.raises(moe.MoeError) as ei:
            call(bad)
        assert ei.value.code == moe.MOE_ERR_INVALID


def test_a_failing_check_is_not_an_address(moe, first_gpu, monkeypatch):
    """Nor is a tensor an address because the question on which GPU it lies could not be asked."""
    import torch

    def lost():
        raise AttributeError("no such thing")
    monkeypatch.setattr(moe, "_get_device", lost)
    with pytest.raises(AttributeError):
        moe.moe_quant8_rows(_p(moe, num_tokens=0), On(torch.bfloat16, 0, 64), On(torch.int8, 0, 64), On(torch.float32, 0), stream=0)


def test_a_failing_check_is_not_an_array_of_the_layout(moe, first_gpu, monkeypatch):
    import torch

    def lost():
        raise AttributeError("no such thing")
    monkeypatch.setattr(moe, "_get_device", lost)
    for lay in (_lay(moe, expert_count=On(torch.int32, 16)), _lay(moe, expert_offset=On(torch.int32, 17))):
        with pytest.raises(AttributeError):
            moe.moe_expert_forward(_p(moe, num_tokens=0), lay, moe.Experts(64, 64), None, None, stream=0)
    with pytest.raises(AttributeError):
        moe.moe_combine_backward(_p(moe, num_tokens=0), _lay(moe, pos=On(torch.int32, 0)), None, None, None, None, None, stream=0)
