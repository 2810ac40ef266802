"""One MoE layer on one GPU, put together from the library's calls.

    python examples/moe_layer.py [--tokens 2048] [--hidden 1024] [--inter 512] [--experts 16] [--topk 2]

Training: route -> layout -> dispatch -> gated experts -> down experts -> combine, and the whole way back to
the gradients of the tokens, of both weight matrices and of the router's logits; what the way back needs of the
gated experts' products is kept in bf16, or in 8 bits (kept).  The router may choose from a few groups of experts
alone (grouping).  Serving: the same layer with its experts in 4 bits or in 8-bit integers.  Prints how far those
results are from the bf16 one and what a step takes.
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

    def __init__(self, T, h, inter, E, k, device="cuda", routing=None, grouping=None, bias=None, kept=False):
        self.problem = moe.Problem(T, h, k, E, num_ranks=1, ranks_per_host=1)
        self.layout = moe.Layout(self.problem, device)
        self.workspace = moe.alloc_workspace(self.problem, device)
        self.routing, self.grouping, self.bias, self.kept = routing or moe.Routing(), grouping, bias, kept
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
        self.hidden, self.pre = bf16(R, inter), None if kept else bf16(R, 2 * inter)
        if kept:                       # half the memory, and hidden is made anew on the way back
            self.codes8 = torch.empty((R, 2 * inter), dtype=torch.uint8, device=device)
            self.scales8 = torch.empty((R, 2, -(-inter // 32)), dtype=torch.uint8, device=device)
        # gradients
        self.dy, self.dgates = bf16(R, h), torch.empty((T, k), device=device)
        self.dpre, self.drecv, self.dx = bf16(R, 2 * inter), bf16(R, h), bf16(T, h)
        self.dup, self.ddown = torch.empty_like(up), torch.empty_like(down)
        self.dlogits = torch.empty((T, E), device=device)

    def receive(self, x, logits):
        """Tokens to the receive rows of their experts."""
        p, lay = self.problem, self.layout
        if self.grouping is None:
            moe.moe_route(p, self.routing, logits, self.ids, self.gates, bias=self.bias)
        else:
            moe.moe_route_groups(p, self.routing, self.grouping, logits, self.ids, self.gates, bias=self.bias)
        moe.moe_layout(p, self.ids, self.workspace, lay)
        moe.moe_dispatch(p, lay, x, None, self.recv, None)

    def forward(self, x, logits):
        p, lay = self.problem, self.layout
        self.receive(x, logits)
        if self.kept:
            moe.moe_expert_forward_kept(p, lay, self.up, self.recv, self.hidden, self.codes8, self.scales8)
        else:
            moe.moe_expert_forward(p, lay, self.up, self.recv, self.hidden, pre=self.pre)
        moe.moe_expert_forward(p, lay, self.down, self.hidden, self.y)
        moe.moe_combine(p, lay, self.y, self.gates, self.out)
        return self.out

    def backward(self, logits, dout):
        p, lay = self.problem, self.layout
        moe.moe_combine_backward(p, lay, dout, self.y, self.gates, self.dy, self.dgates)
        if self.kept:
            moe.moe_expert_backward_kept(p, lay, self.down, self.dy, self.codes8, self.scales8, self.dpre, act=self.hidden)
        else:
            moe.moe_expert_backward_rows(p, lay, self.down, self.dy, self.dpre, pre=self.pre)
        moe.moe_expert_backward_weights(p, lay, self.down, self.hidden, self.dy, self.ddown)
        moe.moe_expert_backward_weights(p, lay, self.up, self.recv, self.dpre, self.dup)
        moe.moe_expert_backward_rows(p, lay, self.up, self.dpre, self.drecv)
        moe.moe_combine(p, lay, self.drecv, self.ones, self.dx)  # the gradient of the dispatch
        moe.moe_route_backward(p, self.routing, logits, self.ids, self.dgates, self.dlogits)
        return self.dx, self.dup, self.ddown, self.dlogits

    def quantise(self, bits=4):
        """The experts in 4 bits or in 8-bit integers, once; serve() then reads a quarter or half of the weights."""
        p, dev, R = self.problem, self.recv.device, self.recv.shape[0]

        def made(x):
            w = x.weights
            if bits == 4:
                codes = torch.empty((*w.shape[:2], x.in_cols // 2), dtype=torch.uint8, device=dev)
                scales = torch.empty(moe.moe_quant4_weight_scale_bytes(p, x), dtype=torch.uint8, device=dev)
                moe.moe_quant4_weights(p, x, codes, scales)
            else:
                codes, scales = torch.empty(w.shape, dtype=torch.int8, device=dev), torch.empty(w.shape[:2], device=dev)
                moe.moe_quant8_weights(p, x, codes, scales)
            return moe.Experts(x.in_cols, x.out_cols, codes, act=x.act, scales=scales)

        def rows(x):
            if bits == 4:
                return (torch.empty((R, x.in_cols // 2), dtype=torch.uint8, device=dev),
                        torch.empty(moe.moe_quant4_row_scale_bytes(p, x.in_cols), dtype=torch.uint8, device=dev))
            return torch.empty((R, x.in_cols), dtype=torch.int8, device=dev), torch.empty(R, device=dev)
        self.bits, self.small = bits, [(made(x), *rows(x)) for x in (self.up, self.down)]

    def serve(self, x, logits):
        p, lay = self.problem, self.layout
        self.receive(x, logits)
        for (experts, codes, scales), rows, out in zip(self.small, (self.recv, self.hidden), (self.hidden, self.y)):
            if self.bits == 4:
                moe.moe_quant4_rows(p, lay, rows, codes, scales)
                moe.moe_expert_forward4(p, lay, experts, codes, scales, out)
            else:
                moe.moe_quant8_rows(p, rows, codes, scales)
                moe.moe_expert_forward8(p, lay, experts, codes, scales, out)
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
    grads = [g.clone() for g in layer.backward(logits, dout)]
    assert all(bool(torch.isfinite(g.float()).all()) for g in grads)
    print(f"{a.tokens} tokens, hidden {a.hidden}, {a.experts} experts top-{a.topk} of width {a.inter}")
    print(f"forward {step_us(lambda: layer.forward(x, logits)):.0f} us, "
          f"forward and backward {step_us(lambda: (layer.forward(x, logits), layer.backward(logits, dout))):.0f} us")
    off = {}
    for bits in (8, 4):
        layer.quantise(bits)
        off[bits] = float((layer.serve(x, logits).float() - out).norm() / out.norm())
        print(f"{bits}-bit experts: {100 * off[bits]:.1f}% off the bf16 result (2-norm), "
              f"forward {step_us(lambda: layer.serve(x, logits)):.0f} us")
    kept = MoeLayer(a.tokens, a.hidden, a.inter, a.experts, a.topk, kept=True)
    kept.up, kept.down = layer.up, layer.down
    assert torch.equal(kept.forward(x, logits).float(), out)
    far = max(float((g.float() - w.float()).norm() / w.float().norm()) for g, w in zip(kept.backward(logits, dout), grads))
    print(f"pre-activations kept in 8 bits: gradients {100 * far:.1f}% off at most, forward and backward "
          f"{step_us(lambda: (kept.forward(x, logits), kept.backward(logits, dout))):.0f} us")
    for each in (layer, kept):
        assert moe.moe_status(each.workspace) == (moe.MOE_OK, 0)
    assert moe.moe_move_faults() == 0
    return off[4]


if __name__ == "__main__":
    main()
