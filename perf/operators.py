"""The decode-side attention operators as they are measured: rotary positions,
the paged key/value cache (written quantized, read back) and the attention of
a sequence's newest tokens over that cache.

Where `own` is false, `run` is the operators' definition in elementary torch
operations; where it is true, `run` makes the library's calls on the same
inputs.  `exact` is the definition once more, in 64 bits.

The cache's memory, for pages of P tokens, H key/value heads of D values:
    k        [pages][H][P][D]          float16, or int8 codes
    v        [pages][H][P/8][D][8]     eight tokens interleaved, same type
    k_scale, v_scale  [pages][H][P/8][D/32][8] float32 (int8 codes only)
Token p of sequence s lives in page table[s][p / P] at row p % P.
"""
import math

import torch

own = False

# Sizes are generic: heads of 64, 128 and 256 values, 1 to 16 query heads to a
# key/value head, contexts from a few tokens to 128K.
_LISTED = [
    # one new token's 32 query and 8 key heads, the smallest call of a decode step
    dict(name="rope_one_token", op="rope", tokens=1, heads=40, dim=128, rot=128,
         style="half", factor=1.0, first=1000),
    # a prompt far into a context stretched 16 times, half of each head rotated,
    # neighbouring values paired
    dict(name="rope_prompt_scaled", op="rope", tokens=4096, heads=40, dim=128, rot=64,
         style="interleaved", factor=16.0, first=123457),
    # one decode step of 48 sequences: rotate, quantize into the pages, read back
    dict(name="append_i8_b48", op="append", batch=48, heads=32, kv_heads=8, dim=128,
         page=64, format="i8", min_len=1, max_len=3000, rot=128, style="half",
         factor=1.0),
    # a prompt of 4001 tokens written into half-precision pages and read back
    dict(name="prompt_f16_4001", op="prompt", tokens=4001, heads=16, kv_heads=8, dim=128,
         page=32, format="f16", rot=128, style="half", factor=4.0),
    # an int8 cache read back whole (moving a sequence, or attending densely)
    dict(name="gather_i8_20011", op="gather", tokens=20011, kv_heads=8, dim=128, page=64,
         format="i8"),
    # a short chat turn: one sequence, one head to a key/value head; latency
    dict(name="attn_f16_b1_77", op="attn", batch=1, new=1, heads=8, kv_heads=8, dim=64,
         page=16, format="f16", min_len=77, max_len=77, window=0),
    # one sequence at a few thousand tokens: few rows, split over the length
    dict(name="attn_i8_b1_4097", op="attn", batch=1, new=1, heads=32, kv_heads=8, dim=128,
         page=64, format="i8", min_len=4097, max_len=4097, window=0),
    # an ordinary serving batch with ragged lengths
    dict(name="attn_i8_b24_ragged", op="attn", batch=24, new=1, heads=32, kv_heads=8,
         dim=128, page=64, format="i8", min_len=1, max_len=5000, window=0),
    # a long document, one user
    dict(name="attn_i8_b1_131001", op="attn", batch=1, new=1, heads=64, kv_heads=8,
         dim=128, page=128, format="i8", min_len=131001, max_len=131001, window=0),
    # five drafted tokens verified at once, causal among themselves
    dict(name="attn_f16_b8_verify5", op="attn", batch=8, new=5, heads=64, kv_heads=8,
         dim=128, page=64, format="f16", min_len=900, max_len=9000, window=0),
    # wide heads, one key/value head, a sliding window and the smallest pages
    dict(name="attn_f16_b96_window", op="attn", batch=96, new=1, heads=8, kv_heads=1,
         dim=256, page=16, format="f16", min_len=200, max_len=20000, window=2048),
    # a full batch of long sequences: the largest
    dict(name="attn_i8_b128_8000", op="attn", batch=128, new=1, heads=32, kv_heads=8,
         dim=128, page=64, format="i8", min_len=3000, max_len=8000, window=0),
]


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "prompt", "gather", "attn", "attn", "attn", "attn"])
    dim = rng.choice([32, 64, 96, 128, 128, 192, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    fmt = rng.choice(["f16", "i8"])
    rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
    turn = dict(rot=rot, style=rng.choice(["half", "interleaved"]),
                factor=rng.choice([1.0, 4.0, 32.0]))
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 3000), heads=rng.randint(1, 48), dim=dim,
                    first=_log(rng, 1, 1000000), **turn)
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if op == "append":
        hi = _log(rng, 2, 4000)
        return dict(op=op, batch=_log(rng, 1, 200), heads=kv * group, kv_heads=kv, dim=dim,
                    page=page, format=fmt, min_len=1, max_len=hi, **turn)
    if op == "prompt":
        return dict(op=op, tokens=_log(rng, 2, 4000), heads=kv * min(group, 4), kv_heads=kv,
                    dim=dim, page=page, format=fmt, **turn)
    if op == "gather":
        return dict(op=op, tokens=_log(rng, 1, 20000), kv_heads=kv, dim=dim, page=page,
                    format=fmt)
    # batch * longest * kv_heads * dim stays below a quarter of the largest listed case
    cap = 128 * 8000 * 8 * 128 // 4
    batch = _log(rng, 1, 160)
    hi = min(_log(rng, 1, 100000), max(1, cap // (batch * kv * dim)))
    return dict(op=op, batch=batch, new=rng.choice([1, 1, 1, 2, 4, 8]), heads=kv * group,
                kv_heads=kv, dim=dim, page=page, format=fmt,
                min_len=rng.choice([0, 1, hi]) if hi > 1 else hi, max_len=hi,
                window=rng.choice([0, 0, _log(rng, 1, 5000)]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lens(case):
    """The sequences' lengths: spread over the case's range, the first the longest."""
    lo, hi, n = case["min_len"], case["max_len"], case["batch"]
    return [hi - int((hi - lo) * ((0.6180339887 * b) % 1.0)) for b in range(n)]


def _freqs(rot, factor, device):
    """Angle a position: base 10000; a factor over 1 slows the frequencies that turn
    less than once over 4096 tokens by the factor, those over 32 turns not at all."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=device), -2.0 * i / rot)
    g = ((4096.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return (1 - g) * f / factor + g * f


def _mscale(factor):
    return 1.0 if factor <= 1.0 else 0.1 * math.log(factor) + 1.0


def _half_away(x):
    return torch.sign(x) * torch.floor(x.abs() + 0.5)


def _quantize(x):
    """int8 codes and one float32 scale per 32 values: d = max|x| / 127, x / d rounded
    to float32 and then half away from zero."""
    b = x.unflatten(-1, (-1, 32))
    d = (b.abs().amax(-1).double() / 127.0).float()
    r = torch.where(d[..., None] == 0, 0.0, b.double() / d[..., None].double()).float()
    return _half_away(r.double()).clamp(-127, 127).to(torch.int8).flatten(-2), d


def _interleave(x):
    """[.., P, n] -> [.., P/8, n, 8]"""
    return x.unflatten(-2, (-1, 8)).transpose(-1, -2).contiguous()


def _cache(case, seqs, lens, g, dev, empty=False):
    """A cache whose sequences hold `lens` tokens in pages scattered over the memory.
    What no token was written to holds NaN, and table entries past the end are -1."""
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    need = [-(-n // P) for n in lens]
    width = max(max(need), 1)
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    used = torch.arange(width, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=dev)
    table[used] = order[:sum(need)]
    gain = torch.exp(0.4 * torch.randn(H, 1, D, generator=g, device=dev))
    i8 = case["format"] == "i8"
    kind = torch.int8 if i8 else torch.float16
    k = torch.empty(pages, H, P, D, dtype=kind, device=dev)
    v = torch.empty(pages, H, P // 8, D, 8, dtype=kind, device=dev)
    ks = vs = None
    if i8:
        ks = torch.empty(pages, H, P // 8, D // 32, 8, device=dev)
        vs = torch.empty_like(ks)
    # the tokens that page j of the memory holds
    fill = torch.zeros(pages, dtype=torch.int64, device=dev)
    left = torch.tensor(lens, device=dev)[:, None] - P * torch.arange(width, device=dev)[None, :]
    fill[table[used].long()] = left.clamp(0, P)[used]
    if empty:
        fill.zero_()
    step = max(1, (1 << 27) // (H * P * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        off = torch.arange(P, device=dev)[None, None, :, None] >= fill[at:at + n, None, None, None]
        x = torch.randn(n, H, P, D, generator=g, device=dev) * gain
        y = torch.randn(n, H, P, D, generator=g, device=dev)
        if i8:
            (kc, kd), (vc, vd) = _quantize(x), _quantize(y)
            kd, vd = (t.masked_fill(off, float("nan")) for t in (kd, vd))
            k[at:at + n], ks[at:at + n] = kc, _interleave(kd)
            v[at:at + n], vs[at:at + n] = _interleave(vc), _interleave(vd)
        else:
            k[at:at + n] = x.masked_fill(off, float("nan")).half()
            v[at:at + n] = _interleave(y.masked_fill(off, float("nan")).half())
    s = dict(k=k, v=v, ks=ks, vs=vs, table=table)
    if own:
        import bit_gemv_amd as rf
        s["cache"] = rf.KvCache(k, v, ks, vs, table)
    return s


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, D = case["op"], case["dim"]
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if op == "rope":
        T, H = case["tokens"], case["heads"]
        s["x"] = normal(T, H, D)
        s["pos"] = case["first"] + torch.arange(T, dtype=torch.int32, device=dev)
        s["y"] = torch.empty_like(s["x"])
    elif op in ("append", "prompt"):
        Hq, H = case["heads"], case["kv_heads"]
        if op == "append":
            T, lens = case["batch"], _lens(case)
            seq, pos = torch.arange(T), torch.tensor(lens) - 1
        else:
            T, lens = case["tokens"], [case["tokens"]]
            seq, pos = torch.zeros(T), torch.arange(T)
        s.update(_cache(case, len(lens), lens, g, dev, empty=True))
        s["seq"], s["pos"] = (t.to(torch.int32).to(dev) for t in (seq, pos))
        s["qkv"] = normal(T, (Hq + 2 * H) * D)     # one product's rows: q, k, v side by side
        s["q_out"] = torch.empty(T, Hq, D, device=dev)
        s["k_out"], s["v_out"] = (torch.empty(T, H, D, device=dev) for _ in range(2))
    elif op == "gather":
        T = case["tokens"]
        s.update(_cache(case, 1, [T], g, dev))
        s["seq"] = torch.zeros(T, dtype=torch.int32, device=dev)
        s["pos"] = torch.arange(T, dtype=torch.int32, device=dev)
        s["k_out"], s["v_out"] = (torch.empty(T, case["kv_heads"], D, device=dev) for _ in range(2))
    else:
        lens = _lens(case)
        s.update(_cache(case, len(lens), lens, g, dev))
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"] = 1.5 * normal(len(lens), case["new"], case["heads"], D)
        s["y"] = torch.empty_like(s["q"])
        if own:
            import bit_gemv_amd as rf
            n = rf.rfp2_paged_attn_workspace_bytes(s["cache"], len(lens), case["new"],
                                                   case["heads"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
    if "rot" in case:
        s["freqs"] = _freqs(case["rot"], case["factor"], dev)
        s["mscale"] = _mscale(case["factor"])
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _rope(x, pos, s):
    """x [T][H][D]: angles of far positions and values that are rounded to codes
    afterwards need 64 bits; one rounding at the end."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    a = pos.double()[:, None] * s["freqs"]
    c, n = (s["mscale"] * torch.cos(a))[:, None], (s["mscale"] * torch.sin(a))[:, None]
    t = x[..., :rot].double()
    if s["case"]["style"] == "half":
        a, b = t[..., :half], t[..., half:]
        r = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        r = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([r.float(), x[..., rot:]], -1)


def _write(s, k, v, page, row):
    if s["ks"] is None:
        s["k"][page, :, row] = k.half()
        s["v"][page, :, row // 8, :, row % 8] = v.half()
    else:
        s["k"][page, :, row], s["ks"][page, :, row // 8, :, row % 8] = _quantize(k)
        s["v"][page, :, row // 8, :, row % 8], s["vs"][page, :, row // 8, :, row % 8] = _quantize(v)


def _scaled(x, d):
    return x.float() if d is None else (x.float().unflatten(-1, (-1, 32)) * d[..., None]).flatten(-2)


def _read(s, page, row):
    d = (None, None) if s["ks"] is None else tuple(
        t[page, :, row // 8, :, row % 8] for t in (s["ks"], s["vs"]))
    return _scaled(s["k"][page, :, row], d[0]), _scaled(s["v"][page, :, row // 8, :, row % 8], d[1])


def _attn(s):
    case = s["case"]
    B, T, Hq, D = s["q"].shape
    H, P = case["kv_heads"], case["page"]
    at = s["table"].clamp(min=0).long()
    L = at.shape[1] * P

    def tokens(x, inner):      # [B][width][H][P/8][inner][8] -> [B][H][L][inner]
        return x.transpose(-1, -2).permute(0, 2, 1, 3, 4, 5).reshape(B, H, L, inner)

    k = s["k"][at].permute(0, 2, 1, 3, 4).reshape(B, H, L, D)
    v = tokens(s["v"][at], D)
    kd, vd = (None, None) if s["ks"] is None else (tokens(t[at], D // 32) for t in (s["ks"], s["vs"]))
    there = (torch.arange(L, device=at.device) < s["lens"][:, None])[:, None, :, None]
    k, v = (torch.where(there, _scaled(x, d), 0.0) for x, d in ((k, kd), (v, vd)))
    q = s["q"].view(B, T, H, Hq // H, D).transpose(1, 2).reshape(B, H, -1, D)
    x = (q @ k.transpose(-1, -2)) * D ** -0.5
    mine = (s["lens"][:, None] - T + torch.arange(T, device=at.device))[:, None, :, None, None]
    pos = torch.arange(L, device=at.device)
    seen = pos <= mine
    if case["window"]:
        seen = seen & (pos > mine - case["window"])
    x = torch.where(seen, x.view(B, H, T, Hq // H, L), -math.inf)
    any_ = seen.any(-1, keepdim=True)
    p = torch.where(seen, torch.exp(x - torch.where(any_, x.amax(-1, keepdim=True), 0.0)), 0.0)
    o = (p.view(B, H, -1, L) @ v).view(B, H, T, -1, D) / torch.where(any_, p.sum(-1, keepdim=True), 1.0)
    return o.transpose(1, 2).reshape(B, T, Hq, D)


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        return _rope(s["x"], s["pos"], s)
    if op == "attn":
        return _attn(s)
    page, row = s["table"][s["seq"].long(), s["pos"].long() // case["page"]].long(), s["pos"].long() % case["page"]
    if op == "gather":
        k, v = _read(s, page, row)
        return dict(k=k, v=v)
    Hq, H, D = case["heads"], case["kv_heads"], case["dim"]
    q, k, v = (t.unflatten(-1, (-1, D)) for t in s["qkv"].split([Hq * D, H * D, H * D], -1))
    _write(s, _rope(k, s["pos"], s), v, page, row)
    k, v = _read(s, page, row)
    return dict(q=_rope(q, s["pos"], s), k=k, v=v)


def _run_own(s):
    import bit_gemv_amd as rf
    case, op, D = s["case"], s["case"]["op"], s["case"]["dim"]
    if op == "attn":
        rf.rfp2_paged_attn(s["cache"], s["q"], case["batch"], case["new"], case["heads"], s["lens"],
                           D ** -0.5, s["y"], window=case["window"], workspace=s["ws"])
        return s["y"]
    if op == "gather":
        rf.rfp2_kv_read(s["cache"], case["tokens"], s["seq"], s["pos"], s["k_out"], s["v_out"])
        return dict(k=s["k_out"], v=s["v_out"])
    turn = (s["freqs"], case["rot"], rf.ROPE_HALF if case["style"] == "half" else rf.ROPE_INTERLEAVED,
            s["mscale"])
    if op == "rope":
        rf.rfp2_rope(s["x"], case["tokens"], case["heads"], D, s["pos"], *turn, s["y"])
        return s["y"]
    Hq, H, T = case["heads"], case["kv_heads"], s["qkv"].shape[0]
    q, k, v = s["qkv"].split([Hq * D, H * D, H * D], -1)
    rf.rfp2_rope_kv_write(s["cache"], q, k, v, T, Hq, s["seq"], s["pos"], *turn, s["q_out"])
    rf.rfp2_kv_read(s["cache"], T, s["seq"], s["pos"], s["k_out"], s["v_out"])
    return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, D = case["op"], case["dim"]
    value = 1.125 if case.get("format") == "i8" else 2.0     # bytes a cached value
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return dict(bytes=8.0 * n * D, flops=3.0 * n * case["rot"])
    if op == "gather":
        n = case["tokens"] * case["kv_heads"] * D * 2
        return dict(bytes=n * (value + 4.0), flops=float(n))
    if op in ("append", "prompt"):
        T = case["batch"] if op == "append" else case["tokens"]
        q, kv = T * case["heads"] * D, T * case["kv_heads"] * D * 2
        return dict(bytes=8.0 * q + kv * (4.0 + value + value + 4.0), flops=3.0 * q + 4.0 * kv)
    T, w, seen, read = case["new"], case["window"], 0, 0
    for n in _lens(case):
        for t in range(T):
            at = n - T + t + 1                                # tokens up to and with this one
            seen += max(0, min(at, w) if w else at)
        read += min(n, w + T - 1) if w else n
    return dict(bytes=read * case["kv_heads"] * D * 2 * value + 8.0 * case["batch"] * T * case["heads"] * D,
                flops=4.0 * seen * case["heads"] * D)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _turned(x, case, s):
    """Each pair as a complex number times m e^(i a)."""
    rot = case["rot"]
    z = torch.polar(torch.tensor(s["mscale"], dtype=torch.float64, device=x.device),
                    s["pos"].double()[:, None] * s["freqs"][None])[:, None, :]
    y = x.double().clone()
    if case["style"] == "half":
        r = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = r.real, r.imag
    else:
        r = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * z
        y[..., 0:rot:2], y[..., 1:rot:2] = r.real, r.imag
    return y


def _held(x, case):
    """What the cache stands for after float32 values x were written."""
    x = x.float()
    if case["format"] == "f16":
        return x.half().double()
    b = x.reshape(*x.shape[:-1], -1, 32)
    d = (b.abs().max(-1, keepdim=True).values.double() / 127).float().double()
    r = torch.nan_to_num(b.double() / d).float().double()
    return (torch.trunc(r + torch.copysign(torch.full_like(r, 0.5), r)) * d).reshape(x.shape)


def _tokens_of(s, case, b, n):
    """The first n cached tokens of sequence b, [n][H][D] each, page after page."""
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    pages = s["table"][b, :-(-n // P)].long()
    got = []
    for x, d, wide in ((s["k"], s["ks"], False), (s["v"], s["vs"], True)):
        x = x[pages]
        x = (x.permute(0, 2, 4, 1, 3) if wide else x.permute(0, 2, 1, 3)).reshape(-1, H, D)[:n].double()
        if d is not None:
            d = d[pages].permute(0, 2, 4, 1, 3).reshape(-1, H, D // 32)[:n].double()
            x = x * d.repeat_interleave(32, -1)
        got.append(x)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["dim"]
    if op == "rope":
        return _turned(s["x"], case, s)
    if op == "gather":
        k, v = _tokens_of(s, case, 0, case["tokens"])
        return dict(k=k, v=v)
    Hq, H = case["heads"], case["kv_heads"]
    if op in ("append", "prompt"):
        x = s["qkv"].reshape(len(s["pos"]), Hq + 2 * H, D)
        return dict(q=_turned(x[:, :Hq], case, s), k=_held(_turned(x[:, Hq:Hq + H], case, s), case),
                    v=_held(x[:, Hq + H:], case))
    T, out = case["new"], torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        k, v = _tokens_of(s, case, b, n)
        k, v = k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous()
        for t in range(max(0, T - n), T):
            hi = n - T + t + 1
            lo = max(0, hi - case["window"]) if case["window"] else 0
            q = s["q"][b, t].double().view(H, Hq // H, D)
            w = torch.softmax((k[:, None, lo:hi] * q[:, :, None]).sum(-1) / math.sqrt(D), -1)
            out[b, t] = (w[..., None] * v[:, None, lo:hi]).sum(-2).view(Hq, D)
    return out
