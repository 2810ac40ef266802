"""The example's MoE layer with its choice limited to groups, its pre-activations kept in 8 bits and its experts in
8-bit integers: all calls together, as a program strings them, against 64 bits."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    import __graft_entry__ as ge
    ge.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _layer(example, T, h, inter, E, k, kept=True):
    import torch
    moe = example.moe
    torch.manual_seed(T)
    layer = example.MoeLayer(T, h, inter, E, k, routing=moe.Routing(moe.MOE_SCORE_SIGMOID, scale=2.0),
                             grouping=moe.Grouping(4, 2), bias=0.05 * torch.randn(E, device="cuda"), kept=kept)
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    return layer, x, torch.randn((T, E), device="cuda"), torch.randn((T, h), device="cuda").to(torch.bfloat16)


def _kept_values(layer, inter):
    import torch
    power = torch.exp2(layer.scales8.double() - 127).repeat_interleave(32, dim=2)[:, :, :inter]
    return layer.codes8.view(torch.float8_e4m3fn).double().view(-1, 2, inter) * power


@pytest.mark.parametrize("T,h,inter,E,k", [(300, 256, 192, 8, 2), (1, 64, 72, 8, 4), (77, 128, 104, 16, 3)])
def test_way_back_from_what_was_kept(example, T, h, inter, E, k):
    """The gradients are those of the layer whose gated pre-activations are the kept values (the forward result is made
    of the unrounded ones): 64-bit autograd, with the kept values put in the place of the products."""
    import torch
    layer, x, logits, dout = _layer(example, T, h, inter, E, k)
    out = layer.forward(x, logits).double().clone()
    got = [g.double() for g in layer.backward(logits, dout)]
    ids = layer.ids.long()
    assert all(len(set((row // (E // 4)).tolist())) <= 2 for row in ids.cpu())
    leaves = [t.double().requires_grad_(True) for t in (x, layer.up.weights, layer.down.weights, logits)]
    xd, up, down, lg = leaves
    s = torch.sigmoid(lg.gather(1, ids))
    gates = 2.0 * s / s.sum(1, keepdim=True)
    kept = _kept_values(layer, inter)[layer.layout.pos.long()]          # [T, k, 2, inter]
    plain, moved = torch.zeros((T, h), dtype=torch.float64, device="cuda"), torch.zeros((T, h), dtype=torch.float64, device="cuda")
    y_made = layer.y.double()[layer.layout.pos.long()]                  # the gates' gradient takes the forward's rows
    for j in range(k):
        pre = torch.einsum("th,tnh->tn", xd, up[ids[:, j]])
        g, u = pre.chunk(2, dim=1)
        plain = plain + (gates[:, j:j + 1] * torch.einsum("tn,thn->th", torch.nn.functional.silu(g) * u, down[ids[:, j]])).detach()
        held = pre + (kept[:, j].flatten(1) - pre).detach()             # kept values forward, products backward
        g, u = held.chunk(2, dim=1)
        y = torch.einsum("tn,thn->th", torch.nn.functional.silu(g) * u, down[ids[:, j]])
        moved = moved + gates[:, j:j + 1].detach() * y + gates[:, j:j + 1] * y_made[:, j]
    grads = torch.autograd.grad(moved, leaves, dout.double())
    # at most six bf16 roundings behind a result, 2^-9 relative each in the mean, in random directions: below 2^-7 in norm
    assert float((out - plain).norm() / plain.norm()) < 2.0 ** -7
    for a, b in zip(got, grads):
        assert float((a - b).norm() / b.norm()) < 2.0 ** -7


def test_layer_in_8_bit_integers(example):
    """Gaussian rows and weights: the step is 2 m / 254 for a largest value m of 3 to 4 deviations (5 to 8 for the gated
    rows), off by its 12th root, so 0.7 to 1.8 % an operand and less than 4 % over both products, and not below 0.5 %."""
    import torch
    layer, x, logits, _ = _layer(example, 257, 512, 256, 16, 4, kept=False)
    out = layer.forward(x, logits).float().clone()
    layer.quantise(8)
    off = float((layer.serve(x, logits).float() - out).norm() / out.norm())
    assert 0.005 < off < 0.04


def test_example_runs(example):
    example.main(["--tokens", "65", "--hidden", "256", "--inter", "128"])


CHILD = r"""
import importlib.util, sys
sys.path.insert(0, {root!r})
import torch
spec = importlib.util.spec_from_file_location("example", {root!r} + "/examples/moe_layer.py")
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)
moe = example.moe
torch.manual_seed(3)
layer = example.MoeLayer(40, 2048, 256, 8, 2, grouping=moe.Grouping(4, 2), routing=moe.Routing(moe.MOE_SCORE_SIGMOID), kept=True)
x = torch.randn((40, 2048), device="cuda").to(torch.bfloat16)
logits = torch.randn((40, 8), device="cuda")
dout = torch.randn((40, 2048), device="cuda").to(torch.bfloat16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    layer.forward(x, logits)
    outs = list(layer.backward(logits, dout))
    layer.quantise(8)
    eight = layer.serve(x, logits).clone()
for o in outs:
    o.zero_()
g.replay()
torch.cuda.synchronize()
replayed = [o.clone() for o in outs] + [eight.clone()]
layer.forward(x, logits)
for o, r in zip(layer.backward(logits, dout), replayed):
    assert torch.equal(o, r)
assert torch.equal(layer.serve(x, logits), replayed[-1])
assert moe.moe_move_faults() == 0
print("cold capture ok")
"""


def test_a_process_s_first_calls_inside_a_graph_capture(example):
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "cold capture ok" in r.stdout
