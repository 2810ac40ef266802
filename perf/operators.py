"""The operators on both sides of the row moves of an MoE layer, as cases to time and to compare.

    route             the router's choice: top-k expert ids and gates, and the gradient of the logits
    experts           products grouped by expert over ragged receive rows, forward and backward
    quant4            receive rows quantised to microscaled 4-bit codes, then the grouped product in 4 bits
    combine_backward  gradients of the gate-weighted sum: expert-output rows and gates

Where ``own`` is false, ``run`` computes the plain form in 32-bit torch operations; where it is true it
makes the calls of the library's binding.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
# magnitudes of the eight e2m1 codes
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of one sequence: nothing but latency
        dict(name="route one token", op="route", T=1, k=8, E=256, score="softmax", renorm=True, bias=False, masked=0,
             dtype="f32", grad=False),
        # a decode batch behind a bias that balances the experts' load, a few experts switched off per token
        dict(name="route decode, sigmoid and bias", op="route", T=509, k=8, E=160, score="sigmoid", renorm=True, bias=True,
             masked=9, dtype="bf16", grad=False),
        # the router of a training step over a prefill-sized batch: choice, gates and the logits' gradient
        dict(name="route train", op="route", T=16384, k=8, E=128, score="softmax", renorm=True, bias=False, masked=0,
             dtype="f32", grad=True),
        # gate and up products of a small decode batch: every expert's weights for a row or two each
        dict(name="experts decode, gated", op="experts", T=16, k=8, E=128, cin=7168, cout=2048, act=True, train=False,
             back=False, skew=0.0),
        # gate and up products of a prefill: large ragged groups
        dict(name="experts prefill, gated", op="experts", T=4096, k=8, E=128, cin=7168, cout=2048, act=True, train=False,
             back=False, skew=0.0),
        # down product at sizes that fill no tile, skewed routing: some experts get many rows, some hardly any
        dict(name="experts down, odd and skewed", op="experts", T=1999, k=6, E=40, cin=1416, cout=2568, act=False,
             train=False, back=False, skew=0.6),
        # backward of the down product of a training step, through the gated activation: rows and weights
        dict(name="experts train, backward", op="experts", T=4096, k=8, E=32, cin=2048, cout=7168, act=True, train=True,
             back=True, skew=0.2),
        # backward of a small layer without activation: 16 experts top-2, odd widths
        dict(name="experts backward, small and odd", op="experts", T=301, k=2, E=16, cin=1024, cout=520, act=False,
             train=True, back=True, skew=0.3),
        # the decode batch again with weights in 4 bits: a quarter of the bytes
        dict(name="quant4 decode, gated", op="quant4", T=16, k=8, E=128, cin=7168, cout=2048, act=True, skew=0.0),
        # a prefill in 4 bits on the experts of a few ranks
        dict(name="quant4 prefill, gated", op="quant4", T=4096, k=8, E=32, cin=7168, cout=2048, act=True, skew=0.2),
        # gradient of a small batch's combine
        dict(name="combine backward, small", op="combine_backward", T=131, k=8, E=256, h=7168),
        # gradient of a prefill-sized batch's combine: gigabytes of rows in and out
        dict(name="combine backward, prefill", op="combine_backward", T=16384, k=8, E=128, h=7168),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "experts", "experts", "quant4", "combine_backward"))
    if op == "route":
        E = rng.choice((8, 16, 40, 61, 128, 160, 256, 384, 512))
        k = rng.choice([v for v in (1, 2, 3, 4, 6, 8, 16) if v <= E])
        return dict(op=op, T=_log_int(rng, 1, 16384), k=k, E=E, score=rng.choice(("softmax", "sigmoid")),
                    renorm=rng.random() < 0.7, bias=rng.random() < 0.4, masked=rng.choice((0, 0, E // 8, E - k)),
                    dtype=rng.choice(("f32", "bf16")), grad=rng.random() < 0.5)
    if op == "combine_backward":
        return dict(op=op, T=_log_int(rng, 1, 8192), k=rng.choice((1, 2, 4, 6, 8, 10)), E=rng.choice((16, 64, 128, 256)),
                    h=8 * _log_int(rng, 32, 896))
    E = rng.choice((8, 16, 32, 60, 128))
    k = rng.choice((1, 2, 4, 6, 8))
    wide, most = (32, 7168) if op == "quant4" else (8, 7168)
    cin = wide * _log_int(rng, 256 // wide, most // wide)
    cout = wide * _log_int(rng, 256 // wide, 4096 // wide)
    T = _log_int(rng, 1, 4096)
    while T * k * cin * cout > 2.4e11 or E * cin * cout > 1.9e9:  # no more than the largest listed case
        T, cin = max(1, T * 3 // 4), max(wide, cin * 3 // 4 // wide * wide)
    case = dict(op=op, T=T, k=k, E=E, cin=cin, cout=cout, act=rng.random() < 0.5, skew=rng.choice((0.0, 0.2, 0.5)))
    if op == "experts":
        back = rng.random() < 0.5
        case.update(back=back, train=back or rng.random() < 0.3)
    return case


# ---- what a program has in hand ------------------------------------------------------------------


def _routed(case, gen):
    """k distinct experts per token under a popularity (rank of e)^-skew, in receive order."""
    T, k, E = case["T"], case["k"], case["E"]
    rank = torch.randperm(E, generator=gen, device=DEV).float() + 1
    noise = torch.rand((T, E), generator=gen, device=DEV).clamp_(1e-30, 1 - 1e-7)
    keys = -torch.log(-torch.log(noise)) - case.get("skew", 0.0) * torch.log(rank)
    ids = keys.topk(k, dim=1).indices
    order = torch.sort(ids.reshape(-1), stable=True).indices
    pos = torch.empty(T * k, dtype=torch.int32, device=DEV)
    pos[order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    count = torch.bincount(ids.reshape(-1), minlength=E)
    offset = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offset[1:] = count.cumsum(0)
    return dict(pos=pos.view(T, k), count=count.to(torch.int32), offset=offset, most=int(count.max()))


def _bf16(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(scale)


def _codes4(x):
    """e2m1 codes (values 0..15, one per element) and e8m0 scales of the 32-blocks along the last axis."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    bits = amax.view(torch.int32)
    scale = ((bits >> 23) - 2).clamp(min=0)                 # biased exponent: floor(log2 amax) - 2
    inv = ((254 - scale) << 23).view(torch.float32)         # 2^(127 - scale), exact
    bad = (bits >> 23) == 255
    v = torch.where(bad, torch.zeros_like(b), (b * inv).abs()).clamp(max=6.0)
    # neighbours of the grid meet at 0.25, 0.75, ..., 5; a value half-way goes to the even code
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
    code = code.to(torch.uint8) | ((b < 0).to(torch.uint8) << 3)
    scale = torch.where(bad, torch.full_like(scale, 255), scale)
    return code.flatten(-2), scale.squeeze(-1).to(torch.uint8)


def _packed(codes):
    """Two codes a byte, the even column in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _scale_blocks(scales, glu):
    """Weight scales [N, K/32] in blocks of 128 rows by 4 scales (512 bytes): row r of a block at byte
    (r % 32) * 16 + (r / 32) * 4.  With a gated activation a block holds 64 gate rows, then their 64 up rows."""
    n, g = scales.shape
    if glu:
        half = torch.nn.functional.pad(scales.view(2, n // 2, g), (0, 0, 0, -(n // 2) % 64)).unflatten(1, (-1, 64))
        scales = half.permute(1, 0, 2, 3).reshape(-1, g)
    scales = torch.nn.functional.pad(scales, (0, -g % 4, 0, -scales.shape[0] % 128))
    return scales.view(scales.shape[0] // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    R = T * k
    s = dict(case=case)
    f32 = dict(dtype=torch.float32, device=DEV)
    if op == "route":
        kind = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["logits"] = (1.5 * torch.randn((T, E), generator=gen, device=DEV)).to(kind)
        if case["masked"]:
            off = torch.rand((T, E), generator=gen, device=DEV).topk(case["masked"], dim=1).indices
            s["logits"].scatter_(1, off, -math.inf)
        s["bias"] = 0.3 * torch.randn(E, generator=gen, device=DEV) if case["bias"] else None
        s["dgates"] = torch.randn((T, k), generator=gen, device=DEV)
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        s["gates"] = torch.empty((T, k), **f32)
        s["dlogits"] = torch.empty_like(s["logits"]) if case["grad"] else None
        return s
    s.update(_routed(case, gen))
    if op == "combine_backward":
        h = case["h"]
        s["dout"] = _bf16((T, h), gen)
        s["y"] = _bf16((R, h), gen)
        s["gates"] = torch.softmax(torch.randn((T, k), generator=gen, device=DEV), dim=1)
        s["dy"] = torch.empty_like(s["y"])
        s["dgates"] = torch.empty((T, k), **f32)
        return s
    cin, cout, act = case["cin"], case["cout"], case["act"]
    empty = dict(dtype=torch.bfloat16, device=DEV)
    if op == "quant4":
        wide = 2 * cout if act else cout
        s["rows"] = _bf16((R, cin), gen) * torch.exp(0.7 * torch.randn(cin, generator=gen, device=DEV)).to(torch.bfloat16)
        codes, scales, plain = [], [], []
        for _ in range(E):  # an expert at a time: the 32-bit weights are not kept
            c, x = _codes4(torch.randn((wide, cin), generator=gen, device=DEV) / math.sqrt(cin))
            codes.append(_packed(c))
            scales.append(_scale_blocks(x, act))
            plain.append(x)
        s["wcodes"], s["wblocks"], s["wscales"] = torch.stack(codes), torch.stack(scales), torch.stack(plain)
        s["codes"] = torch.empty((R, cin // 2), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((R // 128 + E, -(-cin // 128), 512), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty((R, cout), **empty)
        return s
    if not case["back"]:
        s["rows"] = _bf16((R, cin), gen)
        s["weights"] = _bf16((E, 2 * cout if act else cout, cin), gen, 1 / math.sqrt(cin))
        s["pre"] = torch.empty((R, 2 * cout), **empty) if act and case["train"] else None
        s["out"] = torch.empty((R, cout), **empty)
        return s
    # backward of a product from cin to cout columns; with act its rows were silu(g) * u of pre = (g, u)
    s["weights"] = _bf16((E, cout, cin), gen, 1 / math.sqrt(cin))
    s["dout"] = _bf16((R, cout), gen)
    s["rows"] = _bf16((R, cin), gen)
    s["pre"] = _bf16((R, 2 * cin), gen) if act else None
    s["drows"] = torch.empty((R, 2 * cin if act else cin), **empty)
    s["dweights"] = torch.empty((E, cout, cin), **empty)
    return s


# ---- the plain forms -----------------------------------------------------------------------------


def _softmax_of(x):
    """exp(x - max) / sum along the last axis; all -inf gives zeros."""
    m = x.amax(-1, keepdim=True)
    z = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = z.sum(-1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(z), z / total)


def _plain_route(s):
    c = s["case"]
    logits = s["logits"].float()
    key = logits if s["bias"] is None else logits + s["bias"]
    key = torch.where(torch.isnan(key), torch.full_like(key, -math.inf), key)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, : c["k"]]
    chosen = logits.gather(1, ids)
    if c["score"] == "softmax":
        p = _softmax_of(chosen) if c["renorm"] else _softmax_of(logits).gather(1, ids)
    else:
        sig = 1 / (1 + torch.exp(-chosen))
        total = sig.sum(1, keepdim=True)
        p = torch.where(total == 0, torch.zeros_like(sig), sig / total) if c["renorm"] else sig
    out = dict(ids=ids.to(torch.int32), gates=p)
    if c["grad"]:
        a = s["dgates"]
        dl = torch.zeros_like(logits)
        if c["score"] == "softmax":
            mean = (p * a).sum(1, keepdim=True)
            if c["renorm"]:
                dl.scatter_(1, ids, p * (a - mean))
            else:
                dl = -_softmax_of(logits) * mean
                dl.scatter_add_(1, ids, p * a)
        elif c["renorm"]:
            dl.scatter_(1, ids, p * (1 - sig) * (a - (p * a).sum(1, keepdim=True)))
        else:
            dl.scatter_(1, ids, a * sig * (1 - sig))
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _padded(s, x):
    """[E, most, ...]: each expert's rows of x in 32 bits, zeros after them."""
    at = torch.arange(s["most"], device=DEV)
    rows = (s["offset"][:-1, None] + at).clamp(max=x.shape[0] - 1)
    return torch.where((at < s["count"][:, None])[..., None], x[rows].float(), torch.zeros((), device=DEV))


def _rows_of(s, padded):
    """The receive rows of a padded product."""
    r = torch.arange(s["case"]["T"] * s["case"]["k"], dtype=torch.int32, device=DEV)
    e = torch.searchsorted(s["offset"][1:], r, right=True)
    return padded[e, r - s["offset"][e]]


def _gated(pre):
    g, u = pre.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _plain_experts(s):
    c = s["case"]
    if not c["back"]:
        pre = _rows_of(s, torch.bmm(_padded(s, s["rows"]), s["weights"].float().transpose(1, 2)))
        out = dict(out=(_gated(pre) if c["act"] else pre).to(torch.bfloat16))
        if s["pre"] is not None:
            out["pre"] = pre.to(torch.bfloat16)
        return out
    dout = _padded(s, s["dout"])
    dweights = torch.bmm(dout.transpose(1, 2), _padded(s, s["rows"])).to(torch.bfloat16)
    drows = _rows_of(s, torch.bmm(dout, s["weights"].float()))
    if c["act"]:
        g, u = s["pre"].float().chunk(2, dim=1)
        sig = 1 / (1 + torch.exp(-g))
        drows = torch.cat((drows * u * sig * (1 + g * (1 - sig)), drows * g * sig), dim=1)
    return dict(drows=drows.to(torch.bfloat16), dweights=dweights)


def _values4(codes, scales):
    """What e2m1 codes (one per element) and e8m0 scales stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    scale = scales.to(torch.int32)                          # 2^(scale - 127); 0 stands for the subnormal 2^-127
    scale = torch.where(scale == 0, torch.full_like(scale, 1 << 22), scale << 23).view(torch.float32)
    scale = torch.where(scales == 255, torch.full_like(scale, math.nan), scale)
    return (table[codes.to(torch.int32)].unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def _plain_quant4(s):
    packed = s["wcodes"]
    weights = _values4(torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2), s["wscales"])
    pre = _rows_of(s, torch.bmm(_padded(s, _values4(*_codes4(s["rows"]))), weights.transpose(1, 2)))
    return (_gated(pre) if s["case"]["act"] else pre).to(torch.bfloat16)


def _plain_combine_backward(s):
    pos = s["pos"].long()
    dout = s["dout"].float()
    dgates = (dout[:, None, :] * s["y"][pos].float()).sum(-1)
    dy = torch.empty_like(s["y"])
    dy[pos.reshape(-1)] = (s["gates"][..., None] * dout[:, None, :]).to(torch.bfloat16).flatten(0, 1)
    return dict(dy=dy, dgates=dgates)


# ---- the library's calls -------------------------------------------------------------------------


def _handles(s):
    """The problem, layout and expert descriptions that a program keeps for a layer."""
    import combine_moe_layout_04_gb300 as moe
    c = s["case"]
    s["problem"] = moe.Problem(c["T"], c.get("h", 1024), c["k"], c["E"], num_ranks=1, ranks_per_host=1)
    if c["op"] == "route":
        score = moe.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else moe.MOE_SCORE_SIGMOID
        s["routing"] = moe.Routing(score=score, renormalise=c["renorm"])
        return moe
    s["layout"] = moe.Layout(s["problem"], DEV)
    s["layout"].expert_count, s["layout"].expert_offset, s["layout"].pos = s["count"], s["offset"], s["pos"]
    if c["op"] == "experts":
        gated = c["act"] and not c["back"]
        s["experts"] = moe.Experts(c["cin"], c["cout"], s["weights"], act=moe.MOE_ACT_SWIGLU if gated else moe.MOE_ACT_NONE)
    elif c["op"] == "quant4":
        s["experts"] = moe.Experts(c["cin"], c["cout"], s["wcodes"], scales=s["wblocks"],
                                   act=moe.MOE_ACT_SWIGLU if c["act"] else moe.MOE_ACT_NONE)
    return moe


def _own(s):
    import combine_moe_layout_04_gb300 as moe
    if "problem" not in s:
        _handles(s)
    c, p = s["case"], s["problem"]
    if c["op"] == "route":
        moe.moe_route(p, s["routing"], s["logits"], s["ids"], s["gates"], bias=s["bias"])
        out = dict(ids=s["ids"], gates=s["gates"])
        if c["grad"]:
            moe.moe_route_backward(p, s["routing"], s["logits"], s["ids"], s["dgates"], s["dlogits"])
            out["dlogits"] = s["dlogits"]
        return out
    if c["op"] == "combine_backward":
        moe.moe_combine_backward(p, s["layout"], s["dout"], s["y"], s["gates"], s["dy"], s["dgates"])
        return dict(dy=s["dy"], dgates=s["dgates"])
    if c["op"] == "quant4":
        moe.moe_quant4_rows(p, s["layout"], s["rows"], s["codes"], s["scales"])
        moe.moe_expert_forward4(p, s["layout"], s["experts"], s["codes"], s["scales"], s["out"])
        return s["out"]
    if not c["back"]:
        moe.moe_expert_forward(p, s["layout"], s["experts"], s["rows"], s["out"], pre=s["pre"])
        return dict(out=s["out"]) if s["pre"] is None else dict(out=s["out"], pre=s["pre"])
    moe.moe_expert_backward_rows(p, s["layout"], s["experts"], s["dout"], s["drows"], pre=s["pre"])
    moe.moe_expert_backward_weights(p, s["layout"], s["experts"], s["rows"], s["dout"], s["dweights"])
    return dict(drows=s["drows"], dweights=s["dweights"])


PLAIN = {"route": _plain_route, "experts": _plain_experts, "quant4": _plain_quant4,
         "combine_backward": _plain_combine_backward}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    R = T * k
    if op == "route":
        size = 4 if case["dtype"] == "f32" else 2
        moved = T * E * size + T * k * 8 + (E * 4 if case["bias"] else 0)
        if case["grad"]:
            moved += T * E * size + T * k * 4
        return dict(bytes=moved, flops=T * E * (6 if case["grad"] else 3))
    if op == "combine_backward":
        return dict(bytes=2 * T * case["h"] + 4 * R * case["h"] + 12 * R, flops=3 * R * case["h"])
    cin, cout, act = case["cin"], case["cout"], case["act"]
    used = E * (1 - (1 - k / E) ** T)  # experts that get a row
    if op == "experts" and case["back"]:
        moved = 2 * R * (cin + cout) + 2 * (used + E) * cin * cout + 2 * R * cin * (4 if act else 1)
        return dict(bytes=moved, flops=4 * R * cin * cout)
    wide = 2 * cout if act else cout
    if op == "quant4":
        return dict(bytes=2 * R * cin + used * wide * cin * 17 / 32 + 2 * R * cout, flops=2 * R * cin * wide)
    moved = 2 * R * cin + 2 * used * wide * cin + 2 * R * cout + (2 * R * wide if act and case["train"] else 0)
    return dict(bytes=moved, flops=2 * R * cin * wide)


# ---- the definitions in 64 bits ------------------------------------------------------------------


def _exact_route(s):
    c, logits = s["case"], s["logits"].double()
    key = s["logits"].float()
    key = key if s["bias"] is None else key + s["bias"]         # the choice is made in 32 bits by definition
    T, E = key.shape
    better = torch.argsort(torch.where(key.isnan(), -math.inf, key), dim=1, descending=True, stable=True)
    taken = torch.zeros((T, E), dtype=torch.bool, device=DEV).scatter_(1, better[:, : c["k"]], True)
    if c["score"] == "softmax":
        seen = logits.masked_fill(~taken, -math.inf) if c["renorm"] else logits
        weight = torch.nan_to_num(torch.softmax(seen, dim=1), nan=0.0)
        slope = None
    else:
        sig = torch.sigmoid(logits)
        norm = (sig * taken).sum(1, keepdim=True) if c["renorm"] else torch.ones((T, 1), dtype=torch.float64, device=DEV)
        weight = torch.where(norm == 0, torch.zeros_like(sig), sig * taken / norm)
        slope = 1 - sig
    out = dict(ids=None, gates=weight.gather(1, better[:, : c["k"]]))
    if c["grad"]:
        a = torch.zeros((T, E), dtype=torch.float64, device=DEV).scatter_(1, better[:, : c["k"]], s["dgates"].double())
        if c["score"] == "softmax" or c["renorm"]:
            d = weight * (a - (weight * a * taken).sum(1, keepdim=True))
        else:
            d = weight * a
        out["dlogits"] = d if slope is None else d * slope
    return out


def _exact_products(s, values=None, weights_of=None):
    """Forward rows, an expert at a time."""
    c, at = s["case"], s["offset"].tolist()
    x = s["rows"].double() if values is None else values
    pre = [x[at[e]:at[e + 1]] @ (s["weights"][e].double() if weights_of is None else weights_of(e)).T
           for e in range(c["E"])]
    return torch.cat(pre)


def _exact_gated(pre):
    half = pre.shape[1] // 2
    return torch.nn.functional.silu(pre[:, :half]) * pre[:, half:]


def _exact_values4(x):
    """Rows rounded to microscaled 4 bits, by distance to the grid."""
    b = x.double().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    exponent = torch.frexp(torch.where(top == 0, torch.ones_like(top), top)).exponent - 3   # floor(log2 top) - 2
    step = ((exponent.long() + 1023) << 52).view(torch.float64)                             # 2^exponent, exact
    v = (b / step).abs().clamp(max=6)
    unit = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0)).double()
    return (torch.round(v / unit) * unit * b.sign() * step).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "combine_backward":
        dy = torch.empty(s["y"].shape, dtype=torch.float64, device=DEV)
        dgates = torch.empty(s["gates"].shape, dtype=torch.float64, device=DEV)
        for j in range(case["k"]):
            rows = s["pos"][:, j].long()
            dgates[:, j] = torch.linalg.vecdot(s["dout"].double(), s["y"][rows].double())
            dy[rows] = s["dout"].double() * s["gates"][:, j, None].double()
        return dict(dy=dy, dgates=dgates)
    if op == "quant4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)

        def weights_of(e):
            p = s["wcodes"][e].int()
            v = torch.empty((p.shape[0], 2 * p.shape[1]), dtype=torch.float64, device=DEV)
            v[:, 0::2], v[:, 1::2] = table[p % 16], table[p // 16]
            return v * torch.exp2(s["wscales"][e].double() - 127).repeat_interleave(32, dim=1)
        pre = _exact_products(s, _exact_values4(s["rows"]), weights_of)
        return _exact_gated(pre) if case["act"] else pre
    if not case["back"]:
        pre = _exact_products(s)
        out = dict(out=_exact_gated(pre) if case["act"] else pre)
        if s["pre"] is not None:
            out["pre"] = pre
        return out
    at, dx, dw = s["offset"].tolist(), [], []
    for e in range(case["E"]):
        d, x = s["dout"][at[e]:at[e + 1]].double(), s["rows"][at[e]:at[e + 1]].double()
        dx.append(d @ s["weights"][e].double())
        dw.append(d.T @ x)
    dx = torch.cat(dx)
    if case["act"]:
        pre = s["pre"].double().requires_grad_(True)
        with torch.enable_grad():
            dx, = torch.autograd.grad(_exact_gated(pre), pre, dx)
    return dict(drows=dx, dweights=torch.stack(dw))
