"""Arguments that the grouped router's, the 8-bit integers' and the kept activations' calls refuse on the host, before
anything is enqueued (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from test_experts_refusals import GOOD, ODD, At, On, _lay, _p, _refused, first_gpu, moe  # noqa: F401


def _mirror_check(tmp_path, mirrors):
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe_layout.h"', "int main(void) {"]
    for name, cls in mirrors.items():
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "s.c"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()]
    want = []
    for cls in mirrors.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_grouping_struct_matches_the_header(moe, tmp_path):
    _mirror_check(tmp_path, {"moe_grouping": moe._GroupingC})


def test_route_groups_refusals(moe):
    r, good = moe.Routing(), moe.Grouping(4, 2)

    def refused(code, p, g, *args, routing=r, **kw):
        _refused(moe, code, moe.moe_route_groups, p, routing, g, *args, **kw)
    for g in (moe.Grouping(0, 1), moe.Grouping(-4, 1), moe.Grouping(3, 1), moe.Grouping(32, 1), moe.Grouping(4, 0),
              moe.Grouping(4, 5), moe.Grouping(4, -1), moe.Grouping(4, 2, top=0), moe.Grouping(4, 2, top=3),
              moe.Grouping(16, 1)):                                  # (one expert is less than top-2)
        refused(moe.MOE_ERR_INVALID, _p(moe), g, GOOD, GOOD, GOOD)
    refused(moe.MOE_ERR_INVALID, _p(moe, num_experts=64, num_ranks=1, ranks_per_host=1), moe.Grouping(64, 9), GOOD, GOOD, GOOD)
    for bad in (moe.Routing(score=2), moe.Routing(scale=float("nan"))):
        refused(moe.MOE_ERR_INVALID, _p(moe), good, GOOD, GOOD, GOOD, routing=bad)
    for args in ((None, GOOD, GOOD), (GOOD, None, GOOD), (GOOD, GOOD, None)):
        refused(moe.MOE_ERR_INVALID, _p(moe), good, *args)
    off = At(0x20002)
    for args in ((off, GOOD, GOOD), (GOOD, off, GOOD), (GOOD, GOOD, off)):
        refused(moe.MOE_ERR_ALIGN, _p(moe), good, *args)
    refused(moe.MOE_ERR_ALIGN, _p(moe), good, GOOD, GOOD, GOOD, bias=off)
    gc = good.c()
    gc.reserved = 1
    lib, p, rc = moe.load_library(), _p(moe).c(), r.c(GOOD)
    for g in (ctypes.byref(gc), None):
        assert lib.moe_route_groups(ctypes.byref(p), ctypes.byref(rc), g, 0x20000, None, 0x20000, 0x20000,
                                    None) == moe.MOE_ERR_INVALID
    moe.moe_route_groups(_p(moe, num_tokens=0), r, good, None, None, None, stream=0)


def test_choice_structs_follow_their_values(moe):
    """The structs of a routing and a grouping are kept by value: changed fields give others, and the store stays small."""
    r, g = moe.Routing(scale=1.5), moe.Grouping(4, 2)
    moe._CHOICE.clear()
    p = _p(moe, num_tokens=0)
    moe.moe_route_groups(p, r, g, None, None, None, stream=0)
    (key, (rc, gc)), = moe._CHOICE.items()
    assert bytes(rc._obj) == bytes(r.c(None)) and bytes(gc._obj) == bytes(g.c())
    r.score, g.kept = moe.MOE_SCORE_SIGMOID, 3
    moe.moe_route_groups(p, r, g, None, None, None, stream=0)
    assert len(moe._CHOICE) == 2
    r.score, g.top = 7, 2                                              # refused each time, also from the store
    for _ in range(2):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_route_groups, _p(moe), r, g, GOOD, GOOD, GOOD)
    for i in range(200):
        moe.moe_route_groups(p, moe.Routing(scale=float(i)), moe.Grouping(4, 2), None, None, None, stream=0)
    assert len(moe._CHOICE) <= 64


def _tensors_refused(moe, tensors, call):
    """Every tensor in turn on the host, on another GPU, of another type, with gaps or of another shape."""
    import torch
    for i in range(len(tensors)):
        kind, *shape = tensors[i]
        other = torch.float64
        for bad in (torch.zeros(shape, dtype=kind), On(kind, *shape, gpu=1), On(other, *shape), On(kind, *shape, dense=False),
                    On(kind, shape[0] - 1, *shape[1:])):
            args = [On(*t) for t in tensors]
            args[i] = bad
            with pytest.raises(moe.MoeError) as ei:
                call(*args)
            assert ei.value.code == moe.MOE_ERR_INVALID, (i, bad)


def test_binding_refuses_tensors_of_the_grouped_router(moe, first_gpu):
    import torch
    f32, i32 = torch.float32, torch.int32
    _tensors_refused(moe, [(f32, 256, 16), (i32, 256, 2), (f32, 256, 2), (f32, 16)],
                     lambda a, b, c, d: moe.moe_route_groups(_p(moe), moe.Routing(), moe.Grouping(4, 2), a, b, c, bias=d, stream=0))


def test_kept_refusals(moe):
    p, lay = _p(moe), _lay(moe)
    x, down = moe.Experts(64, 64, GOOD, act=moe.MOE_ACT_SWIGLU), moe.Experts(64, 64, GOOD)
    forward = (moe.moe_expert_forward_kept, x, [GOOD] * 4)
    backward = (moe.moe_expert_backward_kept, down, [GOOD] * 4)
    for call, experts, good in (forward, backward):
        for i in range(4):
            _refused(moe, moe.MOE_ERR_INVALID, call, p, lay, experts, *good[:i], None, *good[i + 1:])
            odd = At(0x20002) if i == (3 if call is forward[0] else 2) else ODD     # scales: 4 bytes
            _refused(moe, moe.MOE_ERR_ALIGN, call, p, lay, experts, *good[:i], odd, *good[i + 1:])
        for bad in (dict(weights=None), dict(in_cols=12), dict(out_cols=4), dict(act=2), dict(in_cols=(1 << 20) + 8)):
            kw = {**dict(in_cols=64, out_cols=64, weights=GOOD, act=experts.act), **bad}
            _refused(moe, moe.MOE_ERR_INVALID, call, p, lay, moe.Experts(**kw), *good)
        _refused(moe, moe.MOE_ERR_ALIGN, call, p, lay, moe.Experts(64, 64, ODD, act=experts.act), *good)
        _refused(moe, moe.MOE_ERR_INVALID, call, p, _lay(moe, expert_count=At(None)), experts, *good)
        _refused(moe, moe.MOE_ERR_INVALID, call, _p(moe, topk=0), lay, experts, *good)
        call(_p(moe, num_tokens=0), lay, experts, None, None, None, None, stream=0)
    # kept pre-activations are a gated activation's
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward_kept, p, lay, down, *[GOOD] * 4)
    _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_expert_backward_kept, p, lay, down, *[GOOD] * 4, act=ODD)


def test_binding_refuses_tensors_of_kept_calls(moe, first_gpu):
    import torch
    bf, u8, p = torch.bfloat16, torch.uint8, _p(moe)
    lay = _lay(moe, expert_count=On(torch.int32, 16), expert_offset=On(torch.int32, 17))
    _tensors_refused(moe, [(bf, 16, 80, 64), (bf, 512, 64), (bf, 512, 40), (u8, 512, 80), (u8, 512, 2, 2)],
                     lambda w, *t: moe.moe_expert_forward_kept(p, lay, moe.Experts(64, 40, w, act=moe.MOE_ACT_SWIGLU), *t, stream=0))
    _tensors_refused(moe, [(bf, 16, 64, 40), (bf, 512, 64), (u8, 512, 80), (u8, 512, 2, 2), (bf, 512, 80), (bf, 512, 40)],
                     lambda w, *t: moe.moe_expert_backward_kept(p, lay, moe.Experts(40, 64, w), *t[:4], act=t[4], stream=0))
    for call in (lambda l: moe.moe_expert_forward_kept(p, l, moe.Experts(64, 40, On(bf, 16, 80, 64), act=moe.MOE_ACT_SWIGLU),
                                                       On(bf, 512, 64), On(bf, 512, 40), On(u8, 512, 80), On(u8, 512, 2, 2), stream=0),
                 lambda l: moe.moe_expert_backward_kept(p, l, moe.Experts(40, 64, On(bf, 16, 64, 40)), On(bf, 512, 64),
                                                        On(u8, 512, 80), On(u8, 512, 2, 2), On(bf, 512, 80), stream=0)):
        for bad in (dict(expert_count=On(torch.int32, 15)), dict(expert_offset=On(torch.int32, 16)),
                    dict(expert_offset=On(torch.int64, 17)), dict(expert_count=On(torch.int32, 16, gpu=1))):
            with pytest.raises(moe.MoeError) as ei:
                call(_lay(moe, **{**dict(expert_count=On(torch.int32, 16), expert_offset=On(torch.int32, 17)), **bad}))
            assert ei.value.code == moe.MOE_ERR_INVALID


def test_int8_refusals(moe):
    p, lay = _p(moe), _lay(moe)
    codes = At(0x30000, (512, 64))
    for args in ((None, codes, GOOD), (GOOD, At(None, (512, 64)), GOOD), (GOOD, codes, None)):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant8_rows, p, *args)
    for args in ((ODD, codes, GOOD), (GOOD, At(0x30008, (512, 64)), GOOD), (GOOD, codes, At(0x20002))):
        _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_quant8_rows, p, *args)
    for cols in (0, 8, 24, -16, (1 << 20) + 16):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant8_rows, p, GOOD, At(0x30000, (512, cols)), GOOD)
    for shape in ((), (512 * 64,), (512, 64, 1)):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant8_rows, p, GOOD, At(0x30000, shape), GOOD)
    most = _p(moe, num_tokens=(1 << 31) - 256, topk=1, num_ranks=1, ranks_per_host=1)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant8_rows, most, GOOD, codes, GOOD)
    moe.moe_quant8_rows(_p(moe, num_tokens=0), None, At(None, (0, 64)), None, stream=0)

    x = moe.Experts(64, 64, GOOD, scales=GOOD)
    for bad in (dict(in_cols=8), dict(in_cols=72), dict(in_cols=0), dict(in_cols=(1 << 20) + 16), dict(out_cols=4), dict(act=2)):
        kw = {**dict(in_cols=64, out_cols=64, weights=GOOD, scales=GOOD), **bad}
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward8, p, lay, moe.Experts(**kw), GOOD, GOOD, GOOD)
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant8_weights, p, moe.Experts(**kw), GOOD, GOOD)
    for i in range(3):
        good = [GOOD] * 3
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward8, p, lay, x, *good[:i], None, *good[i + 1:])
        odd = At(0x20002) if i == 1 else ODD
        _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_expert_forward8, p, lay, x, *good[:i], odd, *good[i + 1:])
    for kw, code in ((dict(weights=None, scales=GOOD), "INVALID"), (dict(weights=GOOD, scales=None), "INVALID"),
                     (dict(weights=ODD, scales=GOOD), "ALIGN"), (dict(weights=GOOD, scales=ODD), "ALIGN")):
        _refused(moe, getattr(moe, "MOE_ERR_" + code), moe.moe_expert_forward8, p, lay, moe.Experts(64, 64, **kw), GOOD, GOOD, GOOD)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward8, p, lay, x, GOOD, GOOD, GOOD, pre=GOOD)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward8, p, _lay(moe, expert_offset=At(None)), x, GOOD, GOOD, GOOD)
    gated = moe.Experts(64, 64, GOOD, act=moe.MOE_ACT_SWIGLU, scales=GOOD)
    _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_expert_forward8, p, lay, gated, GOOD, GOOD, GOOD, pre=ODD)
    moe.moe_expert_forward8(_p(moe, num_tokens=0), lay, moe.Experts(64, 64), None, None, None, stream=0)
    for args in ((None, GOOD), (GOOD, None)):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant8_weights, p, x, *args)
    for args in ((ODD, GOOD), (GOOD, ODD)):
        _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_quant8_weights, p, x, *args)


def test_binding_refuses_tensors_of_int8_calls(moe, first_gpu):
    import torch
    bf, i8, f32, p = torch.bfloat16, torch.int8, torch.float32, _p(moe)
    lay = _lay(moe, expert_count=On(torch.int32, 16), expert_offset=On(torch.int32, 17))
    _tensors_refused(moe, [(bf, 512, 64), (i8, 512, 64), (f32, 512)], lambda *t: moe.moe_quant8_rows(p, *t, stream=0))
    _tensors_refused(moe, [(bf, 16, 40, 64), (i8, 16, 40, 64), (f32, 16, 40)],
                     lambda w, *t: moe.moe_quant8_weights(p, moe.Experts(64, 40, w), *t, stream=0))
    _tensors_refused(moe, [(i8, 16, 80, 64), (f32, 16, 80), (i8, 512, 64), (f32, 512), (bf, 512, 40), (bf, 512, 80)],
                     lambda w, s, *t: moe.moe_expert_forward8(p, lay, moe.Experts(64, 40, w, act=moe.MOE_ACT_SWIGLU, scales=s),
                                                              *t[:3], pre=t[3], stream=0))
    for bad in (dict(expert_count=On(torch.int32, 15)), dict(expert_offset=On(torch.int32, 16))):
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_expert_forward8(p, _lay(moe, **{**dict(expert_count=On(torch.int32, 16), expert_offset=On(torch.int32, 17)), **bad}),
                                    moe.Experts(64, 40, On(i8, 16, 40, 64), scales=On(f32, 16, 40)), On(i8, 512, 64),
                                    On(f32, 512), On(bf, 512, 40), stream=0)
        assert ei.value.code == moe.MOE_ERR_INVALID
