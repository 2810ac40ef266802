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
