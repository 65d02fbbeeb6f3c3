"""The operators around a layer's products as they are measured: the norm that adds to
the residual stream and quantizes, the norm of heads, routing to experts, the gate's
activation quantized between two expert products, and the experts' weighted sum back
onto the residual stream.

Where `own` is false, `run` is the operators' definition in elementary torch
operations; where it is true, `run` makes the library's calls on the same inputs.
`exact` is the definition once more, in 64 bits.  Both forms round once to float32
before values are quantized (a last bit there changes codes); int8 activations are
returned as the values that they stand for.
"""
import math

import torch

own = False

# Sizes: widths 2048, 4096 and 5120, 64 and 128 experts of 1536 and 2048 rows are this
# repository's workloads; the others are generic.
_LISTED = [
    # one decoded token: attention's output joins the stream, the next product's input
    dict(name="norm_one_token", op="norm", tokens=1, width=4096, add=True, y=False, quant=True),
    # a verification batch whose normalised values the router reads too
    dict(name="norm_b7_router", op="norm", tokens=7, width=5120, add=True, y=True, quant=True),
    # a prompt batch: the largest
    dict(name="norm_prompt_4096", op="norm", tokens=4096, width=5120, add=True, y=False, quant=True),
    # queries and keys normed head by head where they lie in the rows of a QKV product
    dict(name="heads_prompt_2049", op="heads", tokens=2049, heads=40, dim=128, gap=1024),
    # one token over 128 experts, the eight best
    dict(name="route_one_token", op="route", tokens=1, experts=128, top_k=8, score="softmax",
         bias=False, groups=1, group_top=1, top_groups=1, renorm=True, scale=1.0),
    # a prompt batch over 64 experts, the weights as the softmax leaves them
    dict(name="route_1024_top4", op="route", tokens=1024, experts=64, top_k=4, score="softmax",
         bias=False, groups=1, group_top=1, top_groups=1, renorm=False, scale=1.0),
    # sigmoid scores with a balancing bias, experts in eight groups of which four stay
    dict(name="route_groups_4099", op="route", tokens=4099, experts=256, top_k=8, score="sigmoid",
         bias=True, groups=8, group_top=2, top_groups=4, renorm=True, scale=2.5),
    # one token's eight experts between gate/up and down product
    dict(name="gated_one_token", op="gated", rows=8, width=1536, act="silu", joined=True),
    # 512 tokens' eight experts
    dict(name="gated_prompt_4096", op="gated", rows=4096, width=1536, act="silu", joined=True),
    # a dense feed-forward's gate and up from two products, an odd count of tokens
    dict(name="gated_dense_gelu", op="gated", rows=777, width=8192, act="gelu", joined=False),
    # three decoded tokens: eight experts' rows onto the stream, then the next norm
    dict(name="combine_b3", op="combine", tokens=3, top_k=8, width=4096, norm=True),
    # a prompt batch of the same
    dict(name="combine_prompt_512", op="combine", tokens=512, top_k=8, width=4096, norm=True),
]

EPS = 1e-6


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "heads", "route", "route", "gated", "combine", "combine"])
    cap = 4096 * 5120 // 2                                   # values of an input
    if op == "heads":
        heads = rng.randint(1, 64)
        dim = rng.choice([64, 128, 128, 256, 4 * rng.randint(1, 160)])
        return dict(op=op, tokens=min(_log(rng, 1, 4000), max(1, cap // (heads * dim))), heads=heads,
                    dim=dim, gap=4 * rng.choice([0, 0, rng.randint(1, 512)]))
    if op == "route":
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        experts = max(groups * rng.choice([2, 4, 5, 8, 16, 16, 32, 33]), 8) if groups > 1 else rng.choice(
            [8, 60, 64, 96, 128, 160, 256, 384, rng.randint(2, 512)])
        kept = rng.randint(1, groups)
        bias = rng.choice([True, False])
        top_k = min(rng.choice([1, 2, 4, 6, 8, 8, 10, 16]), experts // groups * kept)
        return dict(op=op, tokens=_log(rng, 1, 8000), experts=experts, top_k=top_k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=bias, groups=groups,
                    group_top=2 if bias and groups > 1 and rng.random() < 0.7 else 1, top_groups=kept,
                    renorm=rng.choice([True, True, False]), scale=rng.choice([1.0, 1.0, 2.5]))
    width = 32 * rng.choice([64, 128, 160, _log(rng, 1, 512)])
    if op == "norm":
        y = rng.choice([True, False])
        return dict(op=op, tokens=min(_log(rng, 1, 8000), max(1, cap // width)), width=width,
                    add=rng.choice([True, True, False]), y=y, quant=not y or rng.choice([True, False]))
    if op == "gated":
        return dict(op=op, rows=min(_log(rng, 1, 16000), max(1, cap // width)), width=width,
                    act=rng.choice(["silu", "silu", "gelu"]), joined=rng.choice([True, False]))
    top_k = rng.choice([1, 2, 4, 6, 8, 8, 10])
    return dict(op=op, tokens=min(_log(rng, 1, 4000), max(1, cap // (width * top_k))), top_k=top_k,
                width=width, norm=rng.choice([True, True, False]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s, op = dict(case=case), case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=dev)

    if op == "heads":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        s["rows"] = normal(T, H * D + case["gap"])           # the heads, then what lies beside them
        s["gain"] = 1.0 + 0.2 * normal(D)
        s["out"] = empty(T, H, D)
        return s
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        s["logits"] = 1.5 * normal(T, E) + 0.5 * normal(E)
        s["bias"] = 0.1 * normal(E) if case["bias"] else None
        s["ids"], s["weights"] = empty(T, k, dtype=torch.int32), empty(T, k)
        return s
    W = case["width"]
    if op == "gated":
        M = case["rows"]
        gu = 1.5 * normal(M, 2 * W)
        s["gate"], s["up"] = (gu[:, :W], gu[:, W:]) if case["joined"] else (
            gu[:, :W].contiguous(), gu[:, W:].contiguous())
        quant, M_q = True, M
    else:
        T = M_q = case["tokens"]
        # a stream whose channels differ in size, a few of them far out
        s["x"] = normal(T, W) * torch.exp(0.8 * normal(W))
        s["gain"] = 1.0 + 0.2 * normal(W)
        s["h"] = empty(T, W)
        if op == "norm":
            s["add"] = 0.5 * normal(T, W) if case["add"] else None
            s["y"] = empty(T, W) if case["y"] else None
            quant = case["quant"]
        else:
            s["rows"] = normal(T, case["top_k"], W)
            s["weights"] = torch.softmax(normal(T, case["top_k"]), -1)
            quant = case["norm"]
    s["q"] = s["d"] = None
    if quant:
        s["q"], s["d"] = empty(M_q, W, dtype=torch.int8), empty(M_q, W // 32)
        s["value"] = empty(M_q, W)
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _quantized(y):
    """What int8 activations stand for: per 32 values d = max|y| / 127, codes y / d
    rounded to float32 and then half away from zero."""
    b = y.unflatten(-1, (-1, 32))
    d = (b.abs().amax(-1, keepdim=True).double() / 127.0).float()
    r = torch.where(d == 0, 0.0, b.double() / d.double()).float().double()
    q = (torch.sign(r) * torch.floor(r.abs() + 0.5)).clamp(-127, 127)
    return (q.float() * d).flatten(-2)


def _normed(h, gain):
    """64 bits: the result is rounded once, before codes are made of it."""
    t = h.double()
    inv = 1.0 / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)
    return (t * inv * gain.double()).float()


def _route(s):
    c, l = s["case"], s["logits"].double()
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    v = p + s["bias"].double() if c["bias"] else l
    if c["groups"] > 1:
        by = v.unflatten(-1, (c["groups"], -1))
        value = torch.sort(by, dim=-1, descending=True).values[..., :c["group_top"]].sum(-1)
        kept = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        there = torch.zeros_like(value, dtype=torch.bool).scatter_(-1, kept, True)
        v = torch.where(there[..., None], by, -math.inf).flatten(-2)
    ids = torch.sort(v, dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = torch.gather(p, -1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return dict(ids=ids.int(), weights=(c["scale"] * w).float())


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "heads":
        H, D = c["heads"], c["dim"]
        return _normed(s["rows"][:, :H * D].unflatten(-1, (H, D)), s["gain"])
    if op == "route":
        return _route(s)
    if op == "gated":
        g = s["gate"].double()
        if c["act"] == "silu":
            a = g / (1.0 + torch.exp(-g))
        else:
            a = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
        return _quantized((a * s["up"].double()).float())
    if op == "norm":
        h = s["x"] + s["add"] if c["add"] else s["x"]
        y = _normed(h, s["gain"])
        return dict(h=h if c["add"] else None, y=y if c["y"] else None,
                    value=_quantized(y) if c["quant"] else None)
    h = (s["x"].double() + (s["weights"].double()[..., None] * s["rows"].double()).sum(1)).float()
    return dict(h=h, value=_quantized(_normed(h, s["gain"])) if c["norm"] else None)


def _run_own(s):
    import bit_gemv_amd as rf
    c, op = s["case"], s["case"]["op"]
    if op == "heads":
        rf.rfp2_rms_norm(s["rows"], c["tokens"], c["heads"], c["dim"], s["gain"], EPS, s["out"])
        return s["out"]
    if op == "route":
        rf.rfp2_moe_route(s["logits"], c["tokens"], c["experts"], s["bias"],
                          rf.ROUTE_SOFTMAX if c["score"] == "softmax" else rf.ROUTE_SIGMOID,
                          c["groups"], c["group_top"], c["top_groups"], c["top_k"], c["renorm"],
                          c["scale"], s["ids"], s["weights"])
        return dict(ids=s["ids"], weights=s["weights"])
    W = c["width"]
    if op == "gated":
        rf.rfp2_quantize_gated_acts(s["gate"], s["up"], c["rows"], W,
                                    rf.GATE_SILU if c["act"] == "silu" else rf.GATE_GELU,
                                    s["q"], s["d"])
        rf.rfp2_dequantize_acts(s["q"], s["d"], c["rows"], W, s["value"])
        return s["value"]
    T = c["tokens"]
    if op == "norm":
        h = s["h"] if c["add"] else None
        rf.rfp2_add_rms_norm(s["x"], s["add"], T, W, s["gain"], EPS, h, s["y"], s["q"], s["d"])
        y, quant = s["y"], c["quant"]
    else:
        h, y, quant = s["h"], None, c["norm"]
        if c["norm"]:
            rf.rfp2_moe_combine(s["x"], s["rows"], s["weights"], T, c["top_k"], W, h, s["gain"], EPS,
                                None, s["q"], s["d"])
        else:
            rf.rfp2_moe_combine(s["x"], s["rows"], s["weights"], T, c["top_k"], W, h)
    if quant:
        rf.rfp2_dequantize_acts(s["q"], s["d"], T, W, s["value"])
    if op == "norm":
        return dict(h=h, y=y, value=s["value"] if quant else None)
    return dict(h=h, value=s["value"] if quant else None)


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    coded = 1.125 + 1.125 + 4.0                              # written, read back, written out
    if op == "heads":
        n = case["tokens"] * case["heads"] * case["dim"]
        return dict(bytes=8.0 * n, flops=4.0 * n)
    if op == "route":
        return dict(bytes=case["tokens"] * (4.0 * case["experts"] + 8.0 * case["top_k"]),
                    flops=4.0 * case["tokens"] * case["experts"])
    W = case["width"]
    if op == "gated":
        n = case["rows"] * W
        return dict(bytes=n * (8.0 + coded), flops=12.0 * n)
    n = case["tokens"] * W
    if op == "norm":
        return dict(bytes=n * (4.0 + 8.0 * case["add"] + 4.0 * case["y"] + coded * case["quant"]),
                    flops=n * (5.0 + 4.0 * case["quant"]))
    return dict(bytes=n * (4.0 * case["top_k"] + 8.0 + coded * case["norm"]),
                flops=n * (2.0 * case["top_k"] + 9.0 * case["norm"]))


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _stands_for(y):
    """Codes and scales of float32 values, multiplied in 64 bits."""
    b = y.reshape(*y.shape[:-1], -1, 32)
    d = (b.abs().max(-1, keepdim=True).values.double() / 127).float().double()
    r = torch.nan_to_num(b.double() / d).float().double()
    return (torch.trunc(r + torch.copysign(torch.full_like(r, 0.5), r)) * d).reshape(y.shape)


def _unit(h, gain):
    """h over its root mean square, times the gain."""
    h = h.double()
    return h / torch.sqrt(torch.linalg.vecdot(h, h)[..., None] / h.shape[-1] + EPS) * gain.double()


def _before(v):
    """[T][n] -> how many entries of the row come before each: larger ones, and equal ones
    at lower places."""
    n = v.shape[-1]
    place = torch.arange(n, device=v.device)
    a, b = v[:, :, None], v[:, None, :]
    return ((b > a) | ((b == a) & (place[None, :] < place[:, None]))).sum(-1)


def _routed(case, l, bias):
    l = l.double()
    p = torch.softmax(l, -1) if case["score"] == "softmax" else torch.sigmoid(l)
    v = p + bias.double() if case["bias"] else l.clone()
    G, E = case["groups"], case["experts"]
    if G > 1:
        value = sum(x for x in v.view(-1, G, E // G).topk(case["group_top"], -1).values.unbind(-1))
        lost = _before(value) >= case["top_groups"]
        v[lost.repeat_interleave(E // G, -1)] = -math.inf
    rank = _before(v)
    ids = torch.stack([(rank == j).int().argmax(-1) for j in range(case["top_k"])], -1)
    w = p.gather(-1, ids)
    return ids.int(), case["scale"] * (w / w.sum(-1, keepdim=True) if case["renorm"] else w)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "heads":
        return _unit(s["rows"][:, :case["heads"] * case["dim"]].reshape(
            case["tokens"], case["heads"], case["dim"]), s["gain"])
    if op == "route":
        parts = [_routed(case, l, s["bias"]) for l in s["logits"].split(max(1, (1 << 26) // case["experts"] ** 2))]
        return dict(ids=torch.cat([i for i, _ in parts]), weights=torch.cat([w for _, w in parts]))
    if op == "gated":
        g, u = s["gate"].double(), s["up"].double()
        if case["act"] == "silu":
            a = g * torch.sigmoid(g)
        else:
            a = g * torch.sigmoid(math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3))
        return _stands_for((a * u).float())
    if op == "norm":
        h = s["x"] + s["add"] if case["add"] else s["x"]
        y = _unit(h, s["gain"])
        return dict(h=s["x"].double() + s["add"].double() if case["add"] else None,
                    y=y if case["y"] else None, value=_stands_for(y.float()) if case["quant"] else None)
    h = s["x"].double()
    for j in range(case["top_k"]):
        h = h + s["rows"][:, j].double() * s["weights"][:, j, None].double()
    return dict(h=h, value=_stands_for(_unit(h.float(), s["gain"]).float()) if case["norm"] else None)
