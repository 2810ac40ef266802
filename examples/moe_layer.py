"""One MoE layer on one GPU, put together from the library's calls.

    python examples/moe_layer.py [--tokens 2048] [--hidden 1024] [--inter 512] [--experts 16] [--topk 2]

Training: route -> layout -> dispatch -> gated experts -> down experts -> combine, and the whole way back to
the gradients of the tokens, of both weight matrices and of the router's logits.  Serving: the same layer with
its experts in 4 bits.  Prints how far the 4-bit result is from the bf16 one and what a step takes.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_moe_layout_04_gb300 as moe  # noqa: E402


class MoeLayer:
    """Weights, buffers and handles of one layer for batches of T tokens."""

    def __init__(self, T, h, inter, E, k, device="cuda"):
        self.problem = moe.Problem(T, h, k, E, num_ranks=1, ranks_per_host=1)
        self.layout = moe.Layout(self.problem, device)
        self.workspace = moe.alloc_workspace(self.problem, device)
        self.routing = moe.Routing()
        R = T * k

        def bf16(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=device)
        up = (torch.randn((E, 2 * inter, h), device=device) / math.sqrt(h)).to(torch.bfloat16)
        down = (torch.randn((E, h, inter), device=device) / math.sqrt(inter)).to(torch.bfloat16)
        self.up = moe.Experts(h, inter, up, act=moe.MOE_ACT_SWIGLU)
        self.down = moe.Experts(inter, h, down)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=device)
        self.gates = torch.empty((T, k), device=device)
        self.ones = torch.ones((T, k), device=device)
        self.recv, self.y, self.out = bf16(R, h), bf16(R, h), bf16(T, h)
        self.hidden, self.pre = bf16(R, inter), bf16(R, 2 * inter)
        # gradients
        self.dy, self.dgates = bf16(R, h), torch.empty((T, k), device=device)
        self.dpre, self.drecv, self.dx = bf16(R, 2 * inter), bf16(R, h), bf16(T, h)
        self.dup, self.ddown = torch.empty_like(up), torch.empty_like(down)
        self.dlogits = torch.empty((T, E), device=device)

    def forward(self, x, logits):
        p, lay = self.problem, self.layout
        moe.moe_route(p, self.routing, logits, self.ids, self.gates)
        moe.moe_layout(p, self.ids, self.workspace, lay)
        moe.moe_dispatch(p, lay, x, None, self.recv, None)
        moe.moe_expert_forward(p, lay, self.up, self.recv, self.hidden, pre=self.pre)
        moe.moe_expert_forward(p, lay, self.down, self.hidden, self.y)
        moe.moe_combine(p, lay, self.y, self.gates, self.out)
        return self.out

    def backward(self, logits, dout):
        p, lay = self.problem, self.layout
        moe.moe_combine_backward(p, lay, dout, self.y, self.gates, self.dy, self.dgates)
        moe.moe_expert_backward_weights(p, lay, self.down, self.hidden, self.dy, self.ddown)
        moe.moe_expert_backward_rows(p, lay, self.down, self.dy, self.dpre, pre=self.pre)
        moe.moe_expert_backward_weights(p, lay, self.up, self.recv, self.dpre, self.dup)
        moe.moe_expert_backward_rows(p, lay, self.up, self.dpre, self.drecv)
        moe.moe_combine(p, lay, self.drecv, self.ones, self.dx)  # the gradient of the dispatch
        moe.moe_route_backward(p, self.routing, logits, self.ids, self.dgates, self.dlogits)
        return self.dx, self.dup, self.ddown, self.dlogits

    def quantise(self):
        """The experts in 4 bits, once; serve() then reads a quarter of the weights."""
        p = self.problem

        def in4(x):
            codes = torch.empty((*x.weights.shape[:2], x.in_cols // 2), dtype=torch.uint8, device=x.weights.device)
            scales = torch.empty(moe.moe_quant4_weight_scale_bytes(p, x), dtype=torch.uint8, device=codes.device)
            moe.moe_quant4_weights(p, x, codes, scales)
            return moe.Experts(x.in_cols, x.out_cols, codes, act=x.act, scales=scales)
        self.up4, self.down4 = in4(self.up), in4(self.down)
        self.codes = [torch.empty((self.recv.shape[0], x.in_cols // 2), dtype=torch.uint8, device=self.recv.device)
                      for x in (self.up, self.down)]
        self.scales = [torch.empty(moe.moe_quant4_row_scale_bytes(p, x.in_cols), dtype=torch.uint8,
                                   device=self.recv.device) for x in (self.up, self.down)]

    def serve(self, x, logits):
        p, lay = self.problem, self.layout
        moe.moe_route(p, self.routing, logits, self.ids, self.gates)
        moe.moe_layout(p, self.ids, self.workspace, lay)
        moe.moe_dispatch(p, lay, x, None, self.recv, None)
        moe.moe_quant4_rows(p, lay, self.recv, self.codes[0], self.scales[0])
        moe.moe_expert_forward4(p, lay, self.up4, self.codes[0], self.scales[0], self.hidden)
        moe.moe_quant4_rows(p, lay, self.hidden, self.codes[1], self.scales[1])
        moe.moe_expert_forward4(p, lay, self.down4, self.codes[1], self.scales[1], self.y)
        moe.moe_combine(p, lay, self.y, self.gates, self.out)
        return self.out


def step_us(step, reps=20):
    for _ in range(3):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    for _ in range(reps):
        step()
    end.record()
    torch.cuda.synchronize()
    return 1e3 * start.elapsed_time(end) / reps


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("hidden", 1024), ("inter", 512), ("experts", 16), ("topk", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    layer = MoeLayer(a.tokens, a.hidden, a.inter, a.experts, a.topk)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    router = torch.randn((a.hidden, a.experts), device="cuda") / math.sqrt(a.hidden)
    logits = x.float() @ router
    dout = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)

    out = layer.forward(x, logits).float()
    grads = layer.backward(logits, dout)
    assert all(bool(torch.isfinite(g.float()).all()) for g in grads)
    layer.quantise()
    off = (layer.serve(x, logits).float() - out).norm() / out.norm()
    assert moe.moe_status(layer.workspace) == (moe.MOE_OK, 0) and moe.moe_move_faults() == 0
    print(f"{a.tokens} tokens, hidden {a.hidden}, {a.experts} experts top-{a.topk} of width {a.inter}")
    print(f"4-bit experts: {100 * float(off):.1f}% off the bf16 result (2-norm)")
    print(f"forward {step_us(lambda: layer.forward(x, logits)):.0f} us, "
          f"forward and backward {step_us(lambda: (layer.forward(x, logits), layer.backward(logits, dout))):.0f} us, "
          f"4-bit forward {step_us(lambda: layer.serve(x, logits)):.0f} us")
    return float(off)


if __name__ == "__main__":
    main()
