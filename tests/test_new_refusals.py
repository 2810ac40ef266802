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
