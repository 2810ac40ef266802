"""Layouts with given rows per expert, and the experts' operators in 64 bits."""
from __future__ import annotations

import numpy as np

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def layout_of_counts(moe, counts, expert_to_rank=None, num_ranks=1):
    """Problem and layout (made by moe_layout) of one-expert tokens with counts[e] rows for expert e, tokens
    in a shuffled order."""
    import torch
    ids = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    np.random.default_rng(len(ids)).shuffle(ids)
    return layout_of_ids(moe, ids[:, None], len(counts), expert_to_rank, num_ranks)


def layout_of_ids(moe, ids, E, expert_to_rank=None, num_ranks=1, hidden=1024):
    import torch
    e2r = None if expert_to_rank is None else torch.tensor(expert_to_rank, dtype=torch.int32, device="cuda")
    prob = moe.Problem(ids.shape[0], hidden, ids.shape[1], E, num_ranks, 1, expert_to_rank=e2r)
    lay, ws = moe.Layout(prob), moe.alloc_workspace(prob)
    moe.moe_layout(prob, torch.from_numpy(np.ascontiguousarray(ids, np.int32)).cuda(), ws, lay)
    assert moe.moe_status(ws) == (moe.MOE_OK, 0)
    return prob, lay


def spans(lay):
    """(e, first row, rows) of every expert."""
    first, count = lay.expert_offset.cpu().tolist(), lay.expert_count.cpu().tolist()
    return [(e, first[e], count[e]) for e in range(len(count))]


def randn(shape, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def guarded(shape, dtype, fill):
    """A tensor of this shape inside a larger buffer, and the bytes behind it."""
    import torch
    n = int(np.prod(shape))
    size = torch.empty((), dtype=dtype).element_size()
    raw = torch.full((n * size + 4096,), fill, dtype=torch.uint8, device="cuda")
    return raw[: n * size].view(dtype).view(shape), raw[n * size:]


def products(lay, rows, weights):
    """rows[r] @ weights[e].T in 64 bits, and the sum of magnitudes of its terms."""
    import torch
    out = torch.zeros((rows.shape[0], weights.shape[1]), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for e, r0, n in spans(lay):
        a, b = rows[r0:r0 + n].double(), weights[e].double()
        out[r0:r0 + n] = a @ b.T
        mag[r0:r0 + n] = a.abs() @ b.abs().T
    return out, mag


def gated(pre):
    import torch
    g, u = pre.double().chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


def close(got, want, slack):
    """|got - want| <= one bf16 rounding of want (2^-8 relative, 2^-133 at the denormal end) + slack."""
    import torch
    d = (got.double() - want).abs()
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -133 + slack
    bad = ~(d <= bound)
    assert not bool(bad.any()), (int(bad.sum()), float(d[bad].max()), got[bad][:4].tolist(), want[bad][:4].tolist())


def sum_slack(mag, terms):
    """fp32 sums of `terms` products with magnitudes summing to mag, in any order, truncated or rounded: at
    most 2^-23 of the running magnitude a term."""
    return mag * (terms + 16) * 2.0 ** -23


def gated_slack(pre, slack):
    """What an error `slack` of pre = (g, u) makes of silu(g) u (|silu'| <= 1.1, |silu(g)| <= |g|), and the fp32
    evaluation itself (expf and a division: 16 roundings)."""
    import torch
    g, u = pre.abs().chunk(2, dim=1)
    dg, du = slack.chunk(2, dim=1)
    return 1.1 * dg * (u + du) + (g + dg) * du + 2.0 ** -20 * g * u


# ---- microscaled 4 bits ----------------------------------------------------------


def scale_value(byte):
    """2^(byte - 127) in 64 bits, exact (made from its bits)."""
    import torch
    return ((byte.long() + (1023 - 127)) << 52).view(torch.float64)


def values4(codes, scales):
    """Values in 64 bits of unpacked codes [n, K] and scale bytes [n, K / 32]."""
    import torch
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    x = scale_value(scales)
    x = torch.where(scales == 255, torch.full_like(x, float("nan")), x)
    return table[codes.long()] * x.repeat_interleave(32, dim=1)


def unpack4(packed):
    import torch
    return torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)


def quantise4(x):
    """(codes [n, K], scale bytes [n, K / 32]) of x [n, K], by search over the grid in 64 bits."""
    import torch
    n, K = x.shape
    b = x.double().view(n, K // 32, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(top)
    _, ex = torch.frexp(torch.where(bad | (top == 0), torch.ones_like(top), top))
    byte = torch.where(top == 0, torch.zeros_like(ex), (ex - 1 + 127 - 2).clamp(min=0))
    v = torch.where(bad[..., None], torch.zeros_like(b), b / scale_value(byte)[..., None])
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    dist = (v.abs().clamp(max=6.0)[..., None] - grid).abs()
    least = dist.amin(-1, keepdim=True)
    near = dist == least
    even = torch.arange(8, device=x.device) % 2 == 0
    code = torch.where(near.sum(-1) > 1, (near & even).to(torch.uint8).argmax(-1), near.to(torch.uint8).argmax(-1))
    sign = torch.signbit(b) & ~bad[..., None]
    code = code.to(torch.uint8) | (sign.to(torch.uint8) << 3)
    return code.view(n, K), torch.where(bad, torch.full_like(byte, 255), byte).to(torch.uint8)


def scale_byte(i, j):
    return (i % 32) * 16 + (i // 32) * 4 + j


def row_scales(lay, scales, K):
    """Scale bytes [R, ceil(K / 128) * 4] of the receive rows, out of their scale blocks."""
    import torch
    groups = -(-K // 128)
    blocks = scales.view(-1, groups, 512)
    R = lay.recv_src.shape[0]
    out = torch.zeros((R, groups * 4), dtype=torch.uint8, device="cuda")
    base = 0
    for e, r0, n in spans(lay):
        i = torch.arange(n, device="cuda")
        for j in range(4):
            out[r0:r0 + n, j::4] = blocks[base + i // 128, :, scale_byte(i % 128, j)]
        base += -(-n // 128)
    return out


def weight_scales(experts, E, scales):
    """Scale bytes [E, W, ceil(K / 128) * 4] of the weights, out of their scale blocks."""
    import torch
    glu = experts.weight_rows != experts.out_cols
    per, N, groups = (64 if glu else 128), experts.out_cols, -(-experts.in_cols // 128)
    blocks = scales.view(E, -(-N // per), groups, 512)
    n = torch.arange(N, device="cuda")
    out = torch.zeros((E, experts.weight_rows, groups * 4), dtype=torch.uint8, device="cuda")
    for half in range(2 if glu else 1):
        for j in range(4):
            out[:, half * N:(half + 1) * N, j::4] = blocks[:, n // per, :, scale_byte(n % per + 64 * half, j)].permute(1, 0, 2)
    return out
