"""The example's MoE layer, all its calls together: forward and every gradient
against 64-bit autograd of the same layer, and the 4-bit forward against the
bf16 one."""
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


@pytest.mark.parametrize("T,h,inter,E,k", [(300, 256, 192, 8, 2), (1, 64, 64, 4, 4), (77, 128, 96, 5, 3)])
def test_layer_against_autograd(example, T, h, inter, E, k):
    import torch
    torch.manual_seed(T)
    layer = example.MoeLayer(T, h, inter, E, k)
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), device="cuda")
    dout = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    out = layer.forward(x, logits).double()
    got = [g.double() for g in layer.backward(logits, dout)]

    leaves = [t.double().requires_grad_(True) for t in (x, layer.up.weights, layer.down.weights, logits)]
    xd, up, down, lg = leaves
    ids = layer.ids.long()
    gates = torch.softmax(lg.gather(1, ids), dim=1)
    want = torch.zeros((T, h), dtype=torch.float64, device="cuda")
    for j in range(k):
        pre = torch.einsum("th,tnh->tn", xd, up[ids[:, j]])
        g, u = pre.chunk(2, dim=1)
        want = want + gates[:, j:j + 1] * torch.einsum("tn,thn->th", torch.nn.functional.silu(g) * u, down[ids[:, j]])
    grads = torch.autograd.grad(want, leaves, dout.double())
    # each bf16 intermediate rounds by 2^-9 relative in the mean; a result has at most six behind it, in random
    # directions and in norm: sqrt(6) 2^-9 is below 2^-7
    assert float((out - want.detach()).norm() / want.detach().norm()) < 2.0 ** -7
    for a, b in zip(got, grads):
        assert float((a - b).norm() / b.norm()) < 2.0 ** -7


def test_layer_in_4_bits(example):
    """Gaussian rows and weights in 4 bits: each product's relative error is about that of its two operands together
    (E2M1 with a power-of-two scale is 0.11 to 0.14 off in norm), two products one after the other."""
    off = example.main(["--tokens", "257", "--hidden", "512", "--inter", "256"])
    assert 0.05 < off < 0.45


CHILD = r"""
import importlib.util, sys
sys.path.insert(0, {root!r})
import torch
spec = importlib.util.spec_from_file_location("example", {root!r} + "/examples/moe_layer.py")
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)
torch.manual_seed(3)
layer = example.MoeLayer(40, 2048, 256, 8, 2)
x = torch.randn((40, 2048), device="cuda").to(torch.bfloat16)
logits = torch.randn((40, 8), device="cuda")
dout = torch.randn((40, 2048), device="cuda").to(torch.bfloat16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = [layer.forward(x, logits), *layer.backward(logits, dout)]
    layer.quantise()
    four = layer.serve(x, logits).clone()
for o in outs:
    o.zero_()
g.replay()
torch.cuda.synchronize()
replayed = [o.clone() for o in outs[1:]] + [four.clone()]
layer.forward(x, logits)
eager = list(layer.backward(logits, dout))
for o, r in zip(eager, replayed):
    assert torch.equal(o, r)
assert torch.equal(layer.serve(x, logits), replayed[-1])
print("cold capture ok")
"""


def test_a_process_s_first_calls_inside_a_graph_capture(example):
    """The launch-shape lookups of a first call are legal in a capture, and the replay gives the eager results."""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "cold capture ok" in r.stdout
