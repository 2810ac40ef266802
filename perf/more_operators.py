"""More operators of an MoE layer, as cases to time and to compare.

    groups   the router's choice limited to a few groups of experts; scores with a bias for balance
    int8     receive rows quantised to 8-bit integers, then the grouped product in 8-bit integers
    keep     the gated experts' forward product, its pre-activations kept in 8 bits for the way back
    back     the gradient through the activation from what was kept, and the activation made anew

Where ``own`` is false, ``run`` computes the plain form in elementary torch operations; where it is true it
makes the calls of the library's binding.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # one token of one sequence: nothing but latency
        dict(name="groups one token", op="groups", T=1, k=8, E=256, G=8, keep=4, top=2, score="sigmoid", renorm=True, bias=True,
             masked=0, dtype="f32", grad=False),
        # a decode batch whose groups count by their best expert, a few experts switched off per token
        dict(name="groups decode, softmax", op="groups", T=509, k=6, E=160, G=8, keep=3, top=1, score="softmax", renorm=False,
             bias=False, masked=9, dtype="bf16", grad=False),
        # the router of a training step over a prefill-sized batch: choice, gates and the logits' gradient
        dict(name="groups train", op="groups", T=16384, k=8, E=256, G=8, keep=4, top=2, score="sigmoid", renorm=True, bias=True,
             masked=0, dtype="f32", grad=True),
        # one token's down products: eight experts of many, latency and a few megabytes of weights
        dict(name="int8 one token, down", op="int8", T=1, k=8, E=64, cin=2048, cout=7168, act=False, skew=0.0),
        # gate and up products of a small decode batch: every expert's weights for a row or two each
        dict(name="int8 decode, gated", op="int8", T=16, k=8, E=128, cin=7168, cout=2048, act=True, skew=0.0),
        # down products at sizes that fill no tile, skewed routing: some experts get many rows, some hardly any
        dict(name="int8 down, odd and skewed", op="int8", T=1999, k=6, E=40, cin=1424, cout=2568, act=False, skew=0.6),
        # gate and up products of a prefill on the experts of a few ranks: large ragged groups
        dict(name="int8 prefill, gated", op="int8", T=4096, k=8, E=32, cin=7168, cout=2048, act=True, skew=0.2),
        # forward of a small layer's gated products, top-2 of 16, odd widths
        dict(name="keep small and odd", op="keep", T=301, k=2, E=16, cin=1032, cout=520, skew=0.3),
        # forward of a training step: what the way back needs of the products takes half the memory
        dict(name="keep train", op="keep", T=4096, k=8, E=32, cin=7168, cout=2048, skew=0.2),
        # way back of the small layer
        dict(name="back small and odd", op="back", T=301, k=2, E=16, cin=520, cout=1032, skew=0.3),
        # way back of the training step, through the activation
        dict(name="back train", op="back", T=4096, k=8, E=32, cin=2048, cout=7168, skew=0.2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("groups", "int8", "int8", "keep", "back"))
    if op == "groups":
        E, G = rng.choice(((16, 4), (60, 5), (64, 4), (64, 8), (128, 8), (160, 8), (192, 6), (256, 8), (256, 16), (384, 8), (512, 16)))
        k = rng.choice((1, 2, 3, 4, 6, 8))
        keep = max(rng.randint(1, G), -(-k * G // E))
        sigmoid = rng.random() < 0.6
        return dict(op=op, T=_log_int(rng, 1, 16384), k=k, E=E, G=G, keep=keep, top=rng.choice((1, 2)),
                    score="sigmoid" if sigmoid else "softmax", renorm=rng.random() < 0.7, bias=rng.random() < 0.6,
                    masked=rng.choice((0, 0, E // 8)), dtype=rng.choice(("f32", "bf16")), grad=rng.random() < 0.5)
    E = rng.choice((8, 16, 32, 60, 128))
    k = rng.choice((1, 2, 4, 6, 8))
    wide = 16 if op == "int8" else 8
    cin = wide * _log_int(rng, 256 // wide, 7168 // wide)
    cout = 8 * _log_int(rng, 256 // 8, 4096 // 8)
    T = _log_int(rng, 1, 4096)
    while T * k * cin * cout > 2.4e11 or E * cin * cout > 1.9e9:  # no more than the largest listed case
        T, cin = max(1, T * 3 // 4), max(wide, cin * 3 // 4 // wide * wide)
    case = dict(op=op, T=T, k=k, E=E, cin=cin, cout=cout, skew=rng.choice((0.0, 0.2, 0.5)))
    if op == "int8":
        case["act"] = rng.random() < 0.5
    return case


# ---- what a program has in hand ------------------------------------------------------------------


def _routed(case, gen):
    """k distinct experts per token under a popularity (rank of e)^-skew, in receive order."""
    T, k, E = case["T"], case["k"], case["E"]
    rank = torch.randperm(E, generator=gen, device=DEV).float() + 1
    noise = torch.rand((T, E), generator=gen, device=DEV).clamp_(1e-30, 1 - 1e-7)
    keys = -torch.log(-torch.log(noise)) - case["skew"] * torch.log(rank)
    ids = keys.topk(k, dim=1).indices
    count = torch.bincount(ids.reshape(-1), minlength=E)
    offset = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offset[1:] = count.cumsum(0)
    return dict(count=count.to(torch.int32), offset=offset, most=int(count.max()))


def _bf16(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(scale)


def _integers(x):
    """8-bit integers of x (32 bits) and the scale of each of its rows."""
    top = x.abs().amax(-1, keepdim=True)
    # a row so small that 127 / top overflows is scaled up by 2^100 first, exactly
    lift = torch.where(top < 2.0 ** -100, 2.0 ** 100, 1.0)
    codes = torch.round((x * lift) * (127.0 / (top * lift)))
    codes = torch.where(top == 0, torch.zeros_like(codes), codes)
    return codes, torch.where(top == 0, torch.ones_like(top), top / 127.0).squeeze(-1)


def _kept(x):
    """x (32 bits) as e4m3 codes and one e8m0 scale for 32 columns of a row: the least power of two with no value over
    448 of it."""
    cols = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -cols % 32)).unflatten(-1, (-1, 32))
    bits = b.abs().amax(-1, keepdim=True).view(torch.int32)
    scale = (((bits + 0x1fffff) >> 23) - 8).clamp(min=0)    # 448 = 1.75 * 2^8
    inv = ((254 - scale) << 23).view(torch.float32)         # 2^(127 - scale), exact
    codes = (b * inv).to(torch.float8_e4m3fn).flatten(-2)[..., :cols]
    return codes.contiguous(), scale.squeeze(-1).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    R = T * k
    s = dict(case=case)
    if op == "groups":
        kind = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["logits"] = (1.5 * torch.randn((T, E), generator=gen, device=DEV)).to(kind)
        if case["masked"]:
            off = torch.rand((T, E), generator=gen, device=DEV).topk(case["masked"], dim=1).indices
            s["logits"].scatter_(1, off, -math.inf)
        # a balance bias is of the size of the scores' own differences
        s["bias"] = (0.1 if case["score"] == "sigmoid" else 0.3 / E) * torch.randn(E, generator=gen, device=DEV) if case["bias"] else None
        s["dgates"] = torch.randn((T, k), generator=gen, device=DEV)
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        s["gates"] = torch.empty((T, k), device=DEV)
        s["dlogits"] = torch.empty_like(s["logits"]) if case["grad"] else None
        return s
    s.update(_routed(case, gen))
    cin, cout = case["cin"], case["cout"]
    bf16, byte = dict(dtype=torch.bfloat16, device=DEV), dict(dtype=torch.uint8, device=DEV)
    if op == "int8":
        wide = 2 * cout if case["act"] else cout
        s["rows"] = _bf16((R, cin), gen) * torch.exp(0.7 * torch.randn(cin, generator=gen, device=DEV)).to(torch.bfloat16)
        s["weights"] = torch.empty((E, wide, cin), dtype=torch.int8, device=DEV)
        s["wscales"] = torch.empty((E, wide), device=DEV)
        for e in range(E):  # an expert at a time: the 32-bit weights are not kept
            codes, s["wscales"][e] = _integers(torch.randn((wide, cin), generator=gen, device=DEV) / math.sqrt(cin))
            s["weights"][e] = codes.to(torch.int8)
        s["codes"] = torch.empty((R, cin), dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(R, device=DEV)
        s["out"] = torch.empty((R, cout), **bf16)
        return s
    if op == "keep":
        s["rows"] = _bf16((R, cin), gen)
        s["weights"] = _bf16((E, 2 * cout, cin), gen, 1 / math.sqrt(cin))
        s["out"] = torch.empty((R, cout), **bf16)
        s["kept"] = torch.empty((R, 2 * cout), **byte)
        s["scales"] = torch.empty((R, 2, -(-cout // 32)), **byte)
        return s
    # way back of a product from cin to cout columns, whose rows were silu(g) * u of the (g, u) that was kept
    s["weights"] = _bf16((E, cout, cin), gen, 1 / math.sqrt(cin))
    s["dout"] = _bf16((R, cout), gen)
    codes, s["scales"] = _kept(torch.randn((R, 2, cin), generator=gen, device=DEV))
    s["kept"] = codes.view(R, 2 * cin).view(torch.uint8)
    s["drows"] = torch.empty((R, 2 * cin), **bf16)
    s["act"] = torch.empty((R, cin), **bf16)
    return s


# ---- the plain forms -----------------------------------------------------------------------------


def _softmax_of(x):
    """exp(x - max) / sum along the last axis, the sum rounded once to 32 bits; all -inf gives zeros."""
    m = x.amax(-1, keepdim=True)
    z = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = z.double().sum(-1, keepdim=True).float()
    return torch.where(total == 0, torch.zeros_like(z), z / total)


def _scores(c, x):
    return _softmax_of(x) if c["score"] == "softmax" else 1 / (1 + torch.exp(-x))


def _choice(c, x, bias):
    """ids [T, k] of logits x in 32 bits: the largest keys of the groups with the largest values."""
    T, E, G = c["T"], c["E"], c["G"]
    scores = _scores(c, x)
    # an expert with a score of 0 (a logit of -inf, or too low for its exponential) is masked whatever its bias
    key = torch.where(scores == 0, torch.full_like(scores, -math.inf), scores if bias is None else scores + bias)
    best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values[..., : c["top"]]
    value = best[..., 0]
    if best.shape[2] == 2:
        value = value + torch.where(best[..., 1] == -math.inf, torch.zeros_like(value), best[..., 1])
    kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, : c["keep"]]
    on = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, kept, True)
    on = on[..., None].expand(T, G, E // G).reshape(T, E)
    # a masked expert of a group that stays comes before every expert of one that does not
    key = torch.where(on, key.clamp(min=torch.finfo(torch.float32).min), torch.full_like(key, -math.inf))
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, : c["k"]]


def _plain_groups(s):
    c = s["case"]
    x = s["logits"].float()
    ids = _choice(c, x, s["bias"])
    chosen = x.gather(1, ids)
    if c["score"] == "softmax":
        p = _softmax_of(chosen) if c["renorm"] else _softmax_of(x).gather(1, ids)
    else:
        sig = 1 / (1 + torch.exp(-chosen))
        total = sig.sum(1, keepdim=True)
        p = torch.where(total == 0, torch.zeros_like(sig), sig / total) if c["renorm"] else sig
    out = dict(ids=ids.to(torch.int32), gates=p)
    if c["grad"]:
        a = s["dgates"]
        dl = torch.zeros_like(x)
        mean = (p * a).sum(1, keepdim=True)
        if c["score"] == "softmax":
            if c["renorm"]:
                dl.scatter_(1, ids, p * (a - mean))
            else:
                dl = -_softmax_of(x) * mean
                dl.scatter_add_(1, ids, p * a)
        else:
            dl.scatter_(1, ids, p / (1 + torch.exp(chosen)) * (a - mean if c["renorm"] else a))
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _padded(s, x):
    """[E, most, ...]: each expert's rows of x in 32 bits, zeros after them."""
    at = torch.arange(s["most"], device=DEV)
    rows = (s["offset"][:-1, None] + at).clamp(max=x.shape[0] - 1)
    return torch.where((at < s["count"][:, None])[..., None], x[rows].float(), torch.zeros((), device=DEV))


def _expert_of_rows(s):
    r = torch.arange(s["case"]["T"] * s["case"]["k"], dtype=torch.int32, device=DEV)
    return r, torch.searchsorted(s["offset"][1:], r, right=True)


def _rows_of(s, padded):
    """The receive rows of a padded product."""
    r, e = _expert_of_rows(s)
    return padded[e, r - s["offset"][e]]


def _gated(pre):
    g, u = pre.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _plain_int8(s):
    codes, scales = _integers(s["rows"].float())
    sums = _rows_of(s, torch.bmm(_padded(s, codes), s["weights"].float().transpose(1, 2)))
    pre = sums * s["wscales"][_expert_of_rows(s)[1]] * scales[:, None]
    return (_gated(pre) if s["case"]["act"] else pre).to(torch.bfloat16)


def _plain_keep(s):
    pre = _rows_of(s, torch.bmm(_padded(s, s["rows"]), s["weights"].float().transpose(1, 2)))
    codes, scales = _kept(pre.unflatten(1, (2, -1)))
    return dict(out=_gated(pre).to(torch.bfloat16), kept=codes.flatten(1), scales=scales.view(torch.float8_e8m0fnu))


def _values(kept, scales, dtype):
    """What kept codes [R, 2 * cols] and scales [R, 2, cols / 32] stand for, as (g, u)."""
    power = torch.exp2(scales.to(dtype) - 127)              # exact
    codes = kept.view(torch.float8_e4m3fn).to(dtype).view(kept.shape[0], 2, -1)
    return (codes * power.repeat_interleave(32, dim=2)[..., : codes.shape[2]]).unbind(1)


def _plain_back(s):
    drows = _rows_of(s, torch.bmm(_padded(s, s["dout"]), s["weights"].float()))
    g, u = _values(s["kept"], s["scales"], torch.float32)
    sig = 1 / (1 + torch.exp(-g))
    drows = torch.cat((drows * u * sig * (1 + g * (1 - sig)), drows * g * sig), dim=1)
    return dict(drows=drows.to(torch.bfloat16), act=(g * sig * u).to(torch.bfloat16))


# ---- the library's calls -------------------------------------------------------------------------


def _handles(s):
    """The problem, layout and expert descriptions that a program keeps for a layer."""
    import combine_moe_layout_04_gb300 as moe
    c = s["case"]
    s["problem"] = moe.Problem(c["T"], 1024, c["k"], c["E"], num_ranks=1, ranks_per_host=1)
    if c["op"] == "groups":
        score = moe.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else moe.MOE_SCORE_SIGMOID
        s["routing"] = moe.Routing(score=score, renormalise=c["renorm"])
        s["grouping"] = moe.Grouping(c["G"], c["keep"], top=c["top"])
        return
    s["layout"] = moe.Layout(s["problem"], DEV)
    s["layout"].expert_count, s["layout"].expert_offset = s["count"], s["offset"]
    gated = c["op"] == "keep" or c.get("act")
    s["experts"] = moe.Experts(c["cin"], c["cout"], s["weights"], scales=s.get("wscales"),
                               act=moe.MOE_ACT_SWIGLU if gated else moe.MOE_ACT_NONE)


def _own(s):
    import combine_moe_layout_04_gb300 as moe
    if "problem" not in s:
        _handles(s)
    c, p = s["case"], s["problem"]
    if c["op"] == "groups":
        moe.moe_route_groups(p, s["routing"], s["grouping"], s["logits"], s["ids"], s["gates"], bias=s["bias"])
        out = dict(ids=s["ids"], gates=s["gates"])
        if c["grad"]:
            moe.moe_route_backward(p, s["routing"], s["logits"], s["ids"], s["dgates"], s["dlogits"])
            out["dlogits"] = s["dlogits"]
        return out
    if c["op"] == "int8":
        moe.moe_quant8_rows(p, s["rows"], s["codes"], s["scales"])
        moe.moe_expert_forward8(p, s["layout"], s["experts"], s["codes"], s["scales"], s["out"])
        return s["out"]
    if c["op"] == "keep":
        moe.moe_expert_forward_kept(p, s["layout"], s["experts"], s["rows"], s["out"], s["kept"], s["scales"])
        return dict(out=s["out"], kept=s["kept"].view(torch.float8_e4m3fn), scales=s["scales"].view(torch.float8_e8m0fnu))
    moe.moe_expert_backward_kept(p, s["layout"], s["experts"], s["dout"], s["kept"], s["scales"], s["drows"], act=s["act"])
    return dict(drows=s["drows"], act=s["act"])


PLAIN = {"groups": _plain_groups, "int8": _plain_int8, "keep": _plain_keep, "back": _plain_back}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    R = T * k
    if op == "groups":
        size = 4 if case["dtype"] == "f32" else 2
        moved = T * E * size + T * k * 8 + (E * 4 if case["bias"] else 0)
        if case["grad"]:
            moved += T * E * size + T * k * 4
        return dict(bytes=moved, flops=T * E * (8 if case["grad"] else 5))
    cin, cout = case["cin"], case["cout"]
    used = E * (1 - (1 - k / E) ** T)  # experts that get a row
    if op == "int8":
        wide = 2 * cout if case["act"] else cout
        return dict(bytes=2 * R * cin + used * wide * (cin + 4) + 2 * R * cout, flops=2 * R * cin * wide)
    if op == "keep":
        moved = 2 * R * cin + 4 * used * cout * cin + 2 * R * cout + 2 * R * (cout + -(-cout // 32))
        return dict(bytes=moved, flops=4 * R * cin * cout)
    moved = 2 * R * cout + 2 * used * cout * cin + 2 * R * (cin + -(-cin // 32)) + 6 * R * cin
    return dict(bytes=moved, flops=2 * R * cin * cout)


# ---- the definitions in 64 bits ------------------------------------------------------------------


def _largest(v, n):
    """Indexes of the n largest along dimension 1 in falling order, equal ones by index, found one after another."""
    left, ids = torch.ones_like(v, dtype=torch.bool), []
    for _ in range(n):
        best = torch.where(left, v, -math.inf).amax(1, keepdim=True)
        ids.append((left & (v == best)).int().argmax(1, keepdim=True))
        left.scatter_(1, ids[-1], False)
    return torch.cat(ids, dim=1)


def _exact_choice(c, logits, bias):
    """Keys are 32-bit by definition (the softmax's sum rounded once), so the choice is made on those."""
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        z = torch.exp(logits - logits.max(1, keepdim=True).values)
        score = z / z.sum(1, keepdim=True, dtype=torch.float64).float()
    key = (score + bias if bias is not None else score).masked_fill(score == 0, -math.inf).unflatten(1, (c["G"], -1))
    value = key.topk(c["top"], dim=2).values
    value = torch.where(value[..., 0] == -math.inf, -math.inf, value.masked_fill(value == -math.inf, 0).sum(2))
    on = torch.zeros_like(value, dtype=torch.bool).scatter_(1, _largest(value, c["keep"]), True)
    key = torch.where(on[..., None], key.clamp(min=-1e30), -2e30).flatten(1)
    return _largest(key, c["k"])


def _exact_groups(s):
    c, x = s["case"], s["logits"].double()
    ids = _exact_choice(c, s["logits"].float(), s["bias"])
    taken = torch.zeros(x.shape, dtype=torch.bool, device=DEV).scatter_(1, ids, True)
    if c["score"] == "softmax":
        weight = torch.nan_to_num(torch.softmax(x.masked_fill(~taken, -math.inf) if c["renorm"] else x, dim=1), nan=0.0)
        slope = None
    else:
        sig = torch.sigmoid(x)
        norm = (sig * taken).sum(1, keepdim=True) if c["renorm"] else torch.ones((c["T"], 1), dtype=torch.float64, device=DEV)
        weight = torch.where(norm == 0, torch.zeros_like(sig), sig * taken / norm)
        slope = torch.sigmoid(-x)
    out = dict(ids=None, gates=weight.gather(1, ids))
    if c["grad"]:
        a = torch.zeros_like(x).scatter_(1, ids, s["dgates"].double())
        if c["score"] == "softmax" or c["renorm"]:
            d = weight * (a - (weight * a * taken).sum(1, keepdim=True))
        else:
            d = weight * a
        out["dlogits"] = d if slope is None else d * slope
    return out


def _exact_products(s, rows, across=False):
    """Rows against their expert's weights, an expert at a time."""
    at = s["offset"].tolist()
    return torch.cat([rows[at[e]:at[e + 1]].double() @ (s["weights"][e].double() if across else s["weights"][e].double().T)
                      for e in range(s["case"]["E"])])


def _exact_gated(pre):
    half = pre.shape[1] // 2
    return torch.nn.functional.silu(pre[:, :half]) * pre[:, half:]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "groups":
        return _exact_groups(s)
    if op == "int8":
        at, x = s["offset"].tolist(), s["rows"].double()
        step = x.abs().amax(1, keepdim=True) / 127
        pre = _exact_products(s, torch.round(x / step)) * step
        for e in range(case["E"]):
            pre[at[e]:at[e + 1]] *= s["wscales"][e].double()
        return _exact_gated(pre) if case["act"] else pre
    if op == "keep":
        # a code has no value of its own in 64 bits: a sum next to a border may fall to either side of it
        return dict(out=_exact_gated(_exact_products(s, s["rows"])), kept=None, scales=None)
    pre = torch.cat(_values(s["kept"], s["scales"], torch.float64), dim=1).requires_grad_(True)
    with torch.enable_grad():
        act = _exact_gated(pre)
        drows, = torch.autograd.grad(act, pre, _exact_products(s, s["dout"], across=True))
    return dict(drows=drows, act=act.detach())
