"""Arguments that the router's and the experts' calls refuse on the host,
before anything is enqueued (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_04_gb300 import _build
    _build.build()
    import combine_moe_layout_04_gb300 as m
    m.load_library()
    return m


class At:
    """A pointer-shaped stand-in: the checks decide from the address alone."""

    def __init__(self, addr, shape=()):
        self.addr, self.shape = addr, shape

    def data_ptr(self):
        return self.addr


GOOD, ODD = At(0x20000), At(0x20008)


def _p(moe, **kw):
    base = dict(num_tokens=256, hidden=1024, topk=2, num_experts=16, num_ranks=4, ranks_per_host=2)
    base.update(kw)
    return moe.Problem(**base)


def _lay(moe, **kw):
    lay = moe.Layout.__new__(moe.Layout)
    for n in moe._LAYOUT_FIELDS:
        setattr(lay, n, kw.get(n, At(0x10000)))
    return lay


def _refused(moe, code, call, *args, **kw):
    with pytest.raises(moe.MoeError) as ei:
        call(*args, **kw, stream=0)
    assert ei.value.code == code


def test_structs_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    import combine_moe_layout_04_gb300 as m
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    mirrors = {"moe_routing": m._RoutingC, "moe_experts": m._ExpertsC}
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


def test_route_refusals(moe):
    r = moe.Routing()
    for bad in (moe.Routing(score=2), moe.Routing(score=-1), moe.Routing(scale=float("nan")),
                moe.Routing(scale=float("inf"))):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_route, _p(moe), bad, GOOD, GOOD, GOOD)
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_route_backward, _p(moe), bad, GOOD, GOOD, GOOD, GOOD)
    few = _p(moe, num_experts=4, topk=5)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_route, few, r, GOOD, GOOD, GOOD)
    for args in ((None, GOOD, GOOD), (GOOD, None, GOOD), (GOOD, GOOD, None)):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_route, _p(moe), r, *args)
    for args in ((None, GOOD, GOOD, GOOD), (GOOD, None, GOOD, GOOD), (GOOD, GOOD, None, GOOD), (GOOD, GOOD, GOOD, None)):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_route_backward, _p(moe), r, *args)
    off = At(0x20002)
    _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_route, _p(moe), r, off, GOOD, GOOD)
    _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_route, _p(moe), r, GOOD, off, GOOD)
    _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_route, _p(moe), r, GOOD, GOOD, GOOD, bias=off)
    rc = r.c(GOOD)
    rc.reserved[2] = 1
    lib = moe.load_library()
    assert lib.moe_route(ctypes.byref(_p(moe).c()), ctypes.byref(rc), 0x20000, None, 0x20000, 0x20000,
                         None) == moe.MOE_ERR_INVALID
    assert lib.moe_route(ctypes.byref(_p(moe).c()), None, 0x20000, None, 0x20000, 0x20000, None) == moe.MOE_ERR_INVALID
    assert lib.moe_route(None, ctypes.byref(r.c(GOOD)), 0x20000, None, 0x20000, 0x20000, None) == moe.MOE_ERR_INVALID


def _calls(moe, p, lay, x):
    """Every expert call with good arguments, as (call, positional arguments)."""
    return [(moe.moe_expert_forward, [p, lay, x, GOOD, GOOD]),
            (moe.moe_expert_backward_rows, [p, lay, x, GOOD, GOOD]),
            (moe.moe_expert_backward_weights, [p, lay, x, GOOD, GOOD, GOOD]),
            (moe.moe_expert_forward4, [p, lay, x, GOOD, GOOD, GOOD])]


@pytest.mark.parametrize("bad", [dict(in_cols=0), dict(in_cols=12), dict(in_cols=-8), dict(out_cols=4), dict(out_cols=20),
                                 dict(in_cols=(1 << 20) + 32), dict(out_cols=(1 << 20) + 8), dict(act=2), dict(act=-1)])
def test_expert_shapes_refused(moe, bad):
    x = moe.Experts(**{**dict(in_cols=64, out_cols=64, weights=GOOD, scales=GOOD), **bad})
    for call, args in _calls(moe, _p(moe), _lay(moe), x):
        _refused(moe, moe.MOE_ERR_INVALID, call, *args)
    with pytest.raises(moe.MoeError):
        moe.moe_quant4_weight_scale_bytes(_p(moe), x)


def test_expert_pointers_refused(moe):
    p, lay, x = _p(moe), _lay(moe), moe.Experts(64, 64, GOOD, scales=GOOD)
    for call, args in _calls(moe, p, lay, x):
        for i in range(3, len(args)):
            _refused(moe, moe.MOE_ERR_INVALID, call, *args[:i], None, *args[i + 1:])
            _refused(moe, moe.MOE_ERR_ALIGN, call, *args[:i], ODD, *args[i + 1:])
        if call is not moe.moe_expert_backward_weights:
            _refused(moe, moe.MOE_ERR_INVALID, call, p, lay, moe.Experts(64, 64, None, scales=GOOD), *args[3:])
            _refused(moe, moe.MOE_ERR_ALIGN, call, p, lay, moe.Experts(64, 64, ODD, scales=GOOD), *args[3:])
        _refused(moe, moe.MOE_ERR_INVALID, call, p, _lay(moe, expert_count=At(None)), x, *args[3:])
        _refused(moe, moe.MOE_ERR_INVALID, call, p, _lay(moe, expert_offset=At(None)), x, *args[3:])
        _refused(moe, moe.MOE_ERR_INVALID, call, _p(moe, topk=0), lay, x, *args[3:])
    # pre is what a gated activation leaves behind; 4-bit weights need scales and columns in blocks of 32
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward, p, lay, x, GOOD, GOOD, pre=GOOD)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward4, p, lay, moe.Experts(64, 64, GOOD), GOOD, GOOD, GOOD)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward4, p, lay, moe.Experts(72, 64, GOOD, scales=GOOD), GOOD, GOOD, GOOD)
    # more weight rows than an int holds
    many = moe.Experts(64, 1 << 20, GOOD, moe.MOE_ACT_SWIGLU)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward, _p(moe, num_experts=1024), lay, many, GOOD, GOOD)


def test_quant4_sizes_and_refusals(moe):
    p = _p(moe)
    assert moe.moe_quant4_row_scale_bytes(p, 32) == (512 // 128 + 16) * 512
    assert moe.moe_quant4_row_scale_bytes(p, 160) == (512 // 128 + 16) * 2 * 512
    assert moe.moe_quant4_weight_scale_bytes(p, moe.Experts(160, 136)) == 16 * 2 * 2 * 512
    assert moe.moe_quant4_weight_scale_bytes(p, moe.Experts(160, 136, act=moe.MOE_ACT_SWIGLU)) == 16 * 3 * 2 * 512
    for act in (moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU):
        for cols, n in ((32, 8), (160, 136), (256, 64), (1056, 1000)):
            x = moe.Experts(cols, n, act=act)
            assert moe._row_scale_bytes(p, cols) == moe.moe_quant4_row_scale_bytes(p, cols)
            assert moe._weight_scale_bytes(p, x) == moe.moe_quant4_weight_scale_bytes(p, x)
    for cols in (0, 16, -32, 100, (1 << 20) + 32):
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_quant4_row_scale_bytes(p, cols)
        assert ei.value.code == moe.MOE_ERR_INVALID
    lay, codes = _lay(moe), At(0x30000, (512, 32))
    for args in ((None, codes, GOOD), (GOOD, At(None, (512, 32)), GOOD), (GOOD, codes, None)):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant4_rows, p, lay, *args)
    for args in ((ODD, codes, GOOD), (GOOD, At(0x30004, (512, 32)), GOOD), (GOOD, codes, ODD)):
        _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_quant4_rows, p, lay, *args)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant4_rows, p, lay, GOOD, At(0x30000, (512, 20)), GOOD)
    x = moe.Experts(64, 64, GOOD)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant4_weights, p, moe.Experts(64, 64), GOOD, GOOD)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant4_weights, p, moe.Experts(72, 64, GOOD), GOOD, GOOD)
    _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_quant4_weights, p, x, ODD, GOOD)
    _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_quant4_weights, p, x, GOOD, ODD)


def test_combine_backward_refusals(moe):
    p, lay = _p(moe), _lay(moe)
    good = [GOOD] * 5
    for i in range(5):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_combine_backward, p, lay, *good[:i], None, *good[i + 1:])
    for i in (0, 1, 3):
        _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_combine_backward, p, lay, *good[:i], ODD, *good[i + 1:])
    for i in (2, 4):
        _refused(moe, moe.MOE_ERR_ALIGN, moe.moe_combine_backward, p, lay, *good[:i], At(0x20002), *good[i + 1:])
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_combine_backward, p, _lay(moe, pos=At(None)), *good)


def test_binding_refuses_other_shapes_types_and_strides(moe):
    """Tensors whose type, shape or strides are not the call's are refused by the binding."""
    import torch
    p, lay = _p(moe), _lay(moe)
    x = moe.Experts(64, 32, torch.empty((16, 32, 64), dtype=torch.bfloat16))
    rows, out = torch.empty((512, 64), dtype=torch.bfloat16), torch.empty((512, 32), dtype=torch.bfloat16)
    for bad_rows, bad_out in ((rows.float(), out), (rows[:, :32], out), (rows[:511], out), (rows, out.half()),
                              (torch.empty((64, 512), dtype=torch.bfloat16).T, out), (rows, out[:, :16])):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward, p, lay, x, bad_rows, bad_out)
    wrong = moe.Experts(64, 32, torch.empty((16, 64, 64), dtype=torch.bfloat16))
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_expert_forward, p, lay, wrong, rows, out)
    scales = torch.empty(100, dtype=torch.uint8)
    codes = torch.empty((512, 32), dtype=torch.uint8)
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant4_rows, p, lay, rows, codes, scales)
    logits = torch.empty((256, 16))
    _refused(moe, moe.MOE_ERR_INVALID, moe.moe_route_backward, p, moe.Routing(), logits,
             torch.empty((256, 2), dtype=torch.int32), torch.empty((256, 2)), logits.bfloat16())


def test_no_tokens_is_no_work(moe):
    p = _p(moe, num_tokens=0)
    moe.moe_route(p, moe.Routing(), None, None, None, stream=0)
    moe.moe_route_backward(p, moe.Routing(), None, None, None, None, stream=0)
    moe.moe_combine_backward(p, _lay(moe), None, None, None, None, None, stream=0)
    moe.moe_expert_forward(p, _lay(moe), moe.Experts(64, 64, None), None, None, stream=0)


def test_problem_struct_follows_its_fields(moe):
    """The C struct is made once for plain sizes; a changed field, a placement or a tuning makes another, and
    copies and pickles carry the fields alone."""
    import copy
    import pickle
    p = _p(moe)
    assert p.c() is p.c() and p.c().num_tokens == 256
    p.num_tokens = 64
    assert p.c().num_tokens == 64
    p.tuning = moe.Tuning(layout_kind=moe.MOE_LAYOUT_FUSED)
    assert p.c() is not p.c() and p.c().tuning.contents.layout_kind == moe.MOE_LAYOUT_FUSED
    p.tuning = None
    assert not p.c().tuning
    p.expert_to_rank = At(0x5000)
    assert p.c().expert_to_rank == 0x5000
    p.expert_to_rank = None
    p.c()
    for other in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert other == p and other.c().num_tokens == 64
        other.hidden = 2048
        assert p.c().hidden == 1024 and other.c().hidden == 2048


def test_problem_struct_is_never_of_other_sizes(moe, monkeypatch):
    """Fields set past the class, by another thread while the struct is made, and a struct that its holder edited:
    the next call takes the problem's own fields."""
    p = _p(moe)
    p.c()
    vars(p)["num_tokens"] = 32
    assert p.c().num_tokens == 32
    object.__setattr__(p, "num_tokens", 48)
    assert p.c().num_tokens == 48
    p.c().hidden = 8
    p.c().tuning = ctypes.pointer(moe.Tuning(dispatch_sms=3).c())
    assert p.c().hidden == 1024 and not p.c().tuning
    make, other = moe._ProblemC, []

    def meanwhile(*args):
        pc = make(*args)
        if not other:
            other.append(1)
            p.num_tokens = 64                       # what another thread may do here
        return pc
    p.num_tokens = 96
    monkeypatch.setattr(moe, "_ProblemC", meanwhile)
    p.c()
    assert p.c().num_tokens == 64
    p.num_tokens = 96
    assert p.c().num_tokens == 96
    with pytest.raises(AttributeError):             # not a field: computed from the others
        p.num_hosts = 5


class On:
    """A tensor-shaped stand-in on a GPU of this number: nothing behind its address is ever read."""

    def __init__(self, dtype, *shape, gpu=0, dense=True):
        self.dtype, self.shape, self.gpu, self.dense = dtype, tuple(shape), gpu, dense
        self.device, self.is_cuda = f"cuda:{gpu}", True

    def data_ptr(self):
        return 0x20000

    def get_device(self):
        return self.gpu

    def is_contiguous(self):
        return self.dense

    def stride(self):
        return (1,) * len(self.shape)

    def numel(self):
        n = 1
        for v in self.shape:
            n *= v
        return n


@pytest.fixture
def first_gpu(moe, monkeypatch):
    """The current GPU is number 0 of several, whatever this machine has."""
    moe._KINDS["float32"]  # (looked up with the types)
    monkeypatch.setattr(moe, "_get_device", lambda: 0, raising=False)
    monkeypatch.setattr(moe, "_one_gpu", False, raising=False)


def _every_call(moe, p):
    """(call, arguments of `make` for every tensor in its order, how to call it) of the router's, the experts' and the
    combine gradient's calls, with good types and shapes."""
    import torch
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    T, k, E, h, R = 256, 2, 16, 1024, 512
    lay, r = _lay(moe), moe.Routing()

    def with_weights(call, kind, *dims, **kw):
        return lambda w, *rest: call(p, lay, moe.Experts(64, 32, w, **kw), *rest, stream=0)
    x = On(u8, 1 << 20)
    return [
        ((f32, T, E), (i32, T, k), (f32, T, k), (f32, E), lambda a, b, c, d: moe.moe_route(p, r, a, b, c, bias=d, stream=0)),
        ((f32, T, E), (i32, T, k), (f32, T, k), (f32, T, E), lambda *t: moe.moe_route_backward(p, r, *t, stream=0)),
        ((bf, T, h), (bf, R, h), (f32, T, k), (bf, R, h), (f32, T, k),
         lambda *t: moe.moe_combine_backward(p, lay, *t, stream=0)),
        ((bf, E, 32, 64), (bf, R, 64), (bf, R, 32), with_weights(moe.moe_expert_forward, bf)),
        ((bf, E, 32, 64), (bf, R, 32), (bf, R, 64), with_weights(moe.moe_expert_backward_rows, bf)),
        ((bf, R, 64), (bf, R, 32), (bf, E, 32, 64),
         lambda *t: moe.moe_expert_backward_weights(p, lay, moe.Experts(64, 32), *t, stream=0)),
        ((bf, R, 64), (u8, R, 32), (u8, 1 << 20), lambda *t: moe.moe_quant4_rows(p, lay, *t, stream=0)),
        ((bf, E, 32, 64), (u8, E, 32, 32), (u8, 1 << 20),
         lambda w, *t: moe.moe_quant4_weights(p, moe.Experts(64, 32, w), *t, stream=0)),
        ((u8, E, 32, 32), (u8, R, 32), (u8, 1 << 20), (bf, R, 32), with_weights(moe.moe_expert_forward4, u8, scales=x)),
    ]


@pytest.mark.parametrize("which", range(9))
def test_binding_refuses_tensors_that_are_not_on_the_current_gpu(moe, first_gpu, which):
    import torch
    *tensors, call = _every_call(moe, _p(moe))[which]
    for i in range(len(tensors)):
        for bad in (torch.zeros(tensors[i][1:], dtype=tensors[i][0]), On(*tensors[i], gpu=1)):
            args = [On(*t) for t in tensors]
            args[i] = bad
            with pytest.raises(moe.MoeError) as ei:
                call(*args)
            assert ei.value.code == moe.MOE_ERR_INVALID and "current GPU" in str(ei.value), (i, str(ei.value))


def test_one_gpu_takes_no_host_tensor(moe, first_gpu, monkeypatch):
    import torch
    monkeypatch.setattr(moe, "_one_gpu", True)
    *tensors, call = _every_call(moe, _p(moe))[0]
    for i in range(len(tensors)):
        args = [On(*t) for t in tensors]
        args[i] = torch.zeros(tensors[i][1:], dtype=tensors[i][0])
        with pytest.raises(moe.MoeError) as ei:
            call(*args)
        assert ei.value.code == moe.MOE_ERR_INVALID and "current GPU" in str(ei.value)


def _layout_calls(moe, p):
    """The calls that read a layout's arrays, with good tensors: call(layout)."""
    import torch
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    w, rows, out = On(bf, 16, 32, 64), On(bf, 512, 64), On(bf, 512, 32)
    x, x4 = moe.Experts(64, 32, w), moe.Experts(64, 32, On(u8, 16, 32, 32), scales=On(u8, 1 << 20))
    codes, scales, gates, wide = On(u8, 512, 32), On(u8, 1 << 20), On(f32, 256, 2), On(bf, 512, 1024)
    groups = [lambda l: moe.moe_expert_forward(p, l, x, rows, out, stream=0),
              lambda l: moe.moe_expert_backward_rows(p, l, x, out, rows, stream=0),
              lambda l: moe.moe_expert_backward_weights(p, l, x, rows, out, w, stream=0),
              lambda l: moe.moe_quant4_rows(p, l, rows, codes, scales, stream=0),
              lambda l: moe.moe_expert_forward4(p, l, x4, codes, scales, out, stream=0)]
    return groups, lambda l: moe.moe_combine_backward(p, l, On(bf, 256, 1024), wide, gates, wide, gates, stream=0)


def test_binding_refuses_layouts_of_other_problems(moe, first_gpu):
    """A layout array that is too short, of another type, with gaps or not on this GPU is not read."""
    import torch
    p, i32 = _p(moe), torch.int32
    groups, combine = _layout_calls(moe, p)

    def refused(call, **arrays):
        good = dict(expert_count=On(i32, 16), expert_offset=On(i32, 17), pos=On(i32, 256, 2))
        with pytest.raises(moe.MoeError) as ei:
            call(_lay(moe, **{**good, **arrays}))
        assert ei.value.code == moe.MOE_ERR_INVALID, arrays
    for name, n in (("expert_count", 16), ("expert_offset", 17)):
        for bad in (On(i32, n - 1), On(torch.int64, n), On(i32, n, dense=False), On(i32, n, gpu=1),
                    torch.zeros(n, dtype=i32)):
            for call in groups:
                refused(call, **{name: bad})
    for bad in (On(i32, 255, 2), On(torch.int64, 256, 2), On(i32, 256, 2, dense=False), torch.zeros((256, 2), dtype=i32)):
        refused(combine, pos=bad)


def test_binding_refuses_codes_that_are_no_matrix(moe, first_gpu):
    import torch
    p, rows, scales = _p(moe), On(torch.bfloat16, 512, 64), On(torch.uint8, 1 << 20)
    for codes in (None, On(torch.uint8, 512 * 32), On(torch.uint8, 512, 32, 1)):
        _refused(moe, moe.MOE_ERR_INVALID, moe.moe_quant4_rows, p, _lay(moe), rows, codes, scales)
