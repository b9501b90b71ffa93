"""Cases and plain forms of the operators around the products of a decode step.

A step of a model with 4-bit weights and a paged key-value cache does three
things beside its products and its attention. It turns queries and keys by
their positions (``rope``), writes the turned keys and the values into the
cache's pages (``append``), and, where a layer has many experts, picks a few of
them for each token (``route``) and multiplies with their 4-bit weights only
(``moe``).

Experts' weights: E2M1 pairs, low nibble = even element, [experts][rows][k / 2],
with E8M0 scales per 32 along k (mxfp4), or E4M3FN scales per 16 and one
32-bit factor per expert (nvfp4). Rows of the first product: the gate's, then
the up projection's.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BITS = {"bf16": 16.0, "mxfp8": 8.25, "mxfp4": 4.25}  # of a cache's element, scales included
WEIGHT_BITS = {"mxfp4": 4.25, "nvfp4": 4.5}


def _rope(name, tokens, heads, dim, rot, layout="half", scaling="none", far=4096, src="bf16", inplace=False):
    c = {"op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rot": rot, "layout": layout, "scaling": scaling,
         "far": far, "src": src, "inplace": inplace}
    return dict(c, name=name) if name else c


def _append(name, fmt, page, seqs, length, new, heads, kv, dim, rot, layout="half", scaling="none", src="bf16"):
    c = {"op": "append", "fmt": fmt, "page": page, "seqs": seqs, "length": length, "new": new, "heads": heads, "kv": kv,
         "dim": dim, "rot": rot, "layout": layout, "scaling": scaling, "src": src}
    return dict(c, name=name) if name else c


def _route(name, tokens, hidden, experts, top, normalize=True, bias=False):
    c = {"op": "route", "tokens": tokens, "hidden": hidden, "experts": experts, "top": top, "normalize": normalize,
         "bias": bias}
    return dict(c, name=name) if name else c


def _moe(name, fmt, tokens, hidden, inter, experts, top, normalize=True, bias=False):
    c = {"op": "moe", "fmt": fmt, "tokens": tokens, "hidden": hidden, "inter": inter, "experts": experts, "top": top,
         "normalize": normalize, "bias": bias}
    return dict(c, name=name) if name else c


def listed():
    return [
        # queries and keys of a small batch's step, as views of the fused projection: latency
        _rope("rope step", 16, 40, 128, 128),
        # half of an odd head turned, interleaved pairs, 32-bit activations, in place
        _rope("rope part", 1531, 12, 96, 48, layout="interleaved", scaling="bands", far=100_000, src="f32", inplace=True),
        # long documents far behind the trained length: bandwidth
        _rope("rope prompt", 16384, 40, 128, 128, scaling="yarn", far=1_000_000),
        # one step of a serving batch: one new token per sequence
        _append("append step", "mxfp8", 64, 32, 2048, 1, 32, 8, 128, 128),
        # the last tokens of one very long document, one key-value head, a quarter of the head turned, 32-bit source
        _append("append far", "bf16", 128, 1, 262144, 64, 8, 1, 64, 16, layout="interleaved", scaling="linear", src="f32"),
        # four prompts of mixed length at once
        _append("append prompts", "mxfp8", 64, 4, 8192, 4096, 32, 8, 128, 128, scaling="ntk"),
        # one user's token: which of 128 experts
        _route("route one", 1, 4096, 128, 8),
        # a prompt's tokens, odd in number, a bias, probabilities as they are
        _route("route prompt", 1999, 2048, 64, 6, normalize=False, bias=True),
        # one user's token through a whole layer: the eight experts' weights
        _moe("moe one", "mxfp4", 1, 4096, 1536, 64, 8),
        # a few tokens, odd widths, nvfp4
        _moe("moe few", "nvfp4", 7, 1120, 736, 32, 4, normalize=False),
        # a serving batch: nearly every expert has a token or more
        _moe("moe batch", "mxfp4", 64, 2048, 1408, 64, 6, bias=True),
        # a large batch on a large layer: 1.3 GB of weights, 16 tokens for an expert
        _moe("moe large", "mxfp4", 256, 4096, 1536, 128, 8),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "append", "append", "append", "route", "moe", "moe", "moe"))
    layout = rng.choice(("half", "interleaved"))
    scaling = rng.choice(("none", "linear", "ntk", "bands", "yarn"))
    src = rng.choice(("bf16", "f32"))
    if op == "rope":
        dim = rng.choice((32, 64, 96, 128, 192, 256))
        heads = rng.randrange(1, 49)
        return _rope("", _spread(rng, 1, min(65536, 40_000_000 // (heads * dim))), heads, dim,
                     rng.choice([r for r in (16, 32, 48, 64, 96, 128, 192, 256) if r <= dim] + [dim, dim]), layout, scaling,
                     _spread(rng, 100, 1_000_000), src, rng.random() < 0.3)
    if op == "append":
        dim = rng.choice((64, 96, 128, 192, 256))
        kv = rng.choice((1, 2, 3, 4, 8))
        seqs = _spread(rng, 1, 128)
        new = rng.choice((1, 1, _spread(rng, 2, max(2, 8192 // seqs))))
        return _append("", rng.choice(("bf16", "mxfp8", "mxfp4")), rng.choice((16, 32, 64, 128, 256)), seqs,
                       new + _spread(rng, 1, 65536 // seqs), new, kv * rng.choice((1, 2, 4, 7, 8)), kv, dim,
                       rng.choice([r for r in (16, 32, 48, 64, 96, 128, 192, 256) if r <= dim] + [dim, dim]), layout,
                       scaling, src)
    experts = _spread(rng, 2, 256)
    top = rng.randrange(1, min(experts, 10) + 1)
    hidden = 32 * _spread(rng, 4, 160)
    more = dict(normalize=rng.random() < 0.6, bias=rng.random() < 0.3)
    if op == "route":
        return _route("", _spread(rng, 1, 4096), hidden, experts, top, **more)
    inter = 32 * _spread(rng, 1, max(1, min(128, 800_000_000 // (32 * hidden * experts))))
    tokens = _spread(rng, 1, 256)
    return _moe("", rng.choice(("mxfp4", "nvfp4")), tokens, hidden, inter, experts, top, **more)


# ---------------------------------------------------------------- what a case's sequences are (the same for every seed)

def _lengths(c):
    """(tokens in each sequence after the pass, how many of them are new): the
    first is the longest, the others spread over 1/30 to 1 of it."""
    r = random.Random("%d %d %d" % (c["seqs"], c["length"], c["new"]))
    f = [1.0] + [math.exp(r.uniform(math.log(1 / 30), 0.0)) for _ in range(c["seqs"] - 1)]
    lens = [max(1, int(c["length"] * x)) for x in f]
    g = [1.0] + [math.exp(r.uniform(math.log(1 / 30), 0.0)) for _ in range(c["seqs"] - 1)]
    return lens, [max(1, min(n, int(c["new"] * x))) for n, x in zip(lens, g)]


def _active(c):
    """How many experts a batch needs, were its choices even and independent."""
    return c["experts"] * (1.0 - (1.0 - c["top"] / c["experts"]) ** c["tokens"])


def work(case):
    c = case
    if c["op"] in ("rope", "append"):
        size = 4 if c["src"] == "f32" else 2
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 2.0 * n * size + 4.0 * c["tokens"], "flops": 3.0 * c["tokens"] * c["heads"] * c["rot"]}
    if c["op"] == "append":
        t = sum(_lengths(c)[1])
        q, k = t * c["heads"] * c["dim"], t * c["kv"] * c["dim"]
        return {"bytes": q * (size + 2) + 2 * k * (size + BITS[c["fmt"]] / 8),
                "flops": 3.0 * t * (c["heads"] + c["kv"]) * c["rot"] + 2.0 * k}
    t, h, e = c["tokens"], c["hidden"], c["experts"]
    route = {"bytes": 2.0 * (t + e) * h + 8.0 * t * c["top"], "flops": 2.0 * t * e * h}
    if c["op"] == "route":
        return route
    each = 3.0 * h * c["inter"] * WEIGHT_BITS[c["fmt"]] / 8
    return {"bytes": route["bytes"] + 2.0 * t * h + _active(c) * each,
            "flops": route["flops"] + 6.0 * t * c["top"] * h * c["inter"]}


# ---------------------------------------------------------------- inputs

# what a scaled rotation is made for: four times the length that the model was trained on
SCALE, TRAINED, BASE = 4.0, 8192, 10000.0


def _frequencies(c):
    """Radians per position of each pair, in 64 bits, and the factor on cosine and sine."""
    r, base, factor = c["rot"], BASE, 1.0
    if c["scaling"] == "ntk":
        base = BASE * SCALE ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if c["scaling"] == "linear":
        f = [x / SCALE for x in f]
    elif c["scaling"] == "bands":  # long waves are stretched, short ones are not, a band between them in part
        lo, hi = 1.0, 4.0
        part = [min(1.0, max(0.0, (TRAINED * x / (2 * math.pi) - lo) / (hi - lo))) for x in f]
        f = [x * p + x / SCALE * (1 - p) for x, p in zip(f, part)]
    elif c["scaling"] == "yarn":  # a ramp over the pairs between 32 and 1 turns in the trained length
        at = [r * math.log(TRAINED / (turns * 2 * math.pi)) / (2 * math.log(BASE)) for turns in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
        part = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(r // 2)]
        f = [x * (1 - p) + x / SCALE * p for x, p in zip(f, part)]
        factor = 0.1 * math.log(SCALE) + 1.0
    return f, factor


def _rope_handle(c):
    import bit_block_quantized_nibble_amd as qbn

    more = {"none": {}, "linear": dict(scale=SCALE), "ntk": dict(scale=SCALE), "bands": dict(scale=SCALE, original=TRAINED),
            "yarn": dict(scale=SCALE, original=TRAINED)}[c["scaling"]]
    return qbn.Rope.make(c["rot"], base=BASE, scaling=c["scaling"], layout=c["layout"], device="cuda:0", **more)


def _pairs(dev):
    """The two values of each byte of E2M1 codes."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=dev)
    b = torch.arange(256, device=dev)
    return torch.stack((v[b % 16], v[b // 16]), -1).contiguous()


def _prepare_rope(c, g, dev):
    dt = torch.float32 if c["src"] == "f32" else torch.bfloat16
    wide = c["heads"] + 2  # a view of a fused projection's output
    x = torch.randn(c["tokens"], wide, c["dim"], generator=g, device=dev, dtype=torch.float32).to(dt)[:, :c["heads"]]
    # runs of consecutive positions, as packed sequences have them
    starts = torch.randint(0, max(1, c["far"] - c["tokens"]), (8,), generator=g, device=dev)
    t = torch.arange(c["tokens"], device=dev)
    pos = (starts[t * 8 // c["tokens"]] + t).to(torch.int32)
    f, factor = _frequencies(c)
    s = {"x": x, "pos": pos, "freq": torch.tensor(f, dtype=torch.float64, device=dev), "factor": factor}
    if c["inplace"]:  # the pass turns a buffer that it has just filled
        s["buffer"] = torch.empty_like(x, memory_format=torch.contiguous_format)
    return s


def _prepare_append(c, g, dev):
    lens, new = _lengths(c)
    need = sum(-(-n // c["page"]) for n in lens)
    pages = need + need // 16 + 1
    shape = (1, pages, c["kv"], c["page"], c["dim"])
    s = {}
    for part in ("k", "v"):  # pages in use: any content, none of it NaN
        if c["fmt"] == "bf16":
            s[part] = torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)
            s[part + "s"] = None
            continue
        width = c["dim"] // (2 if c["fmt"] == "mxfp4" else 1)
        code = torch.randint(0, 255 if c["fmt"] == "mxfp4" else 126, shape[:-1] + (width,), generator=g, device=dev)
        s[part] = code.to(torch.uint8)
        mid = 126 if c["fmt"] == "mxfp4" else 119  # of the new tokens' size
        scale = torch.randint(mid - 1, mid + 2, (1, pages, c["kv"], c["dim"] // 32, c["page"]), generator=g, device=dev)
        s[part + "s"] = scale.to(torch.uint8)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    width = -(-max(lens) // c["page"]) + 2  # rows have room to spare
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32, device=dev)
    cu, at = [0], 0
    for b, (n, t) in enumerate(zip(lens, new)):
        k = -(-n // c["page"])
        table[b, :k] = order[at:at + k]
        at += k
        cu.append(cu[-1] + t)
    s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    dt = torch.float32 if c["src"] == "f32" else torch.bfloat16
    x = torch.randn(cu[-1], c["heads"] + 2 * c["kv"], c["dim"], generator=g, device=dev, dtype=torch.float32).to(dt)
    s["q"], s["newk"], s["newv"] = x.split((c["heads"], c["kv"], c["kv"]), 1)
    f, factor = _frequencies(c)
    s["freq"], s["factor"] = torch.tensor(f, dtype=torch.float64, device=dev), factor
    if c["fmt"] == "mxfp4":
        s["pairs"] = _pairs(dev).to(torch.bfloat16)
    return s


def _prepare_route(c, g, dev):
    s = {"x": torch.randn(c["tokens"], c["hidden"], generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)}
    router = torch.randn(c["experts"], c["hidden"], generator=g, device=dev, dtype=torch.float32)
    s["router"] = (router * 1.5 * c["hidden"] ** -0.5).to(torch.bfloat16)  # uneven choices, as trained routers make them
    s["bias"] = None
    if c["bias"]:
        s["bias"] = torch.randn(c["experts"], generator=g, device=dev, dtype=torch.float32) * 0.5
    return s


def _weights(c, rows, k, g, dev):
    """(codes, scales, factor per expert or None) whose products keep the size of what goes in."""
    e = c["experts"]
    codes = torch.randint(-2 ** 31, 2 ** 31, (e, rows, k // 8), generator=g, device=dev, dtype=torch.int32)
    codes = codes.view(torch.uint8).reshape(e, rows, k // 2)
    if c["fmt"] == "mxfp4":
        mid = 127 - int(round(0.5 * math.log2(k))) - 1
        scales = torch.randint(mid - 1, mid + 2, (e, rows, k // 32), generator=g, device=dev, dtype=torch.int16)
        return codes, scales.to(torch.uint8), None
    scales = torch.randint(0x28, 0x41, (e, rows, k // 16), generator=g, device=dev, dtype=torch.int16).to(torch.uint8)
    factor = torch.rand(e, generator=g, device=dev, dtype=torch.float32) * 0.2 + 0.4
    return codes, scales, factor * k ** -0.5


def _prepare_moe(c, g, dev):
    s = _prepare_route(c, g, dev)
    s["w13"], s["s13"], s["f13"] = _weights(c, 2 * c["inter"], c["hidden"], g, dev)
    s["w2"], s["s2"], s["f2"] = _weights(c, c["hidden"], c["inter"], g, dev)
    s["pairs"] = _pairs(dev)
    return s


def prepare(case, seed):
    c, dev = case, torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"rope": _prepare_rope, "append": _prepare_append, "route": _prepare_route, "moe": _prepare_moe}[c["op"]](c, g, dev)
    s["case"] = dict(c)
    if own:
        import bit_block_quantized_nibble_amd as qbn

        if c["op"] in ("rope", "append"):
            s["rope"] = _rope_handle(c)
        if c["op"] == "append":
            s["cache"] = qbn.KVCache(c["fmt"], s["k"], s["v"], s["ks"], s["vs"])
        if c["op"] == "route":
            s["router_of"] = qbn.MoERouter(s["router"], c["top"], bias=s["bias"], normalize=c["normalize"])
        if c["op"] == "moe":
            router = qbn.MoERouter(s["router"], c["top"], bias=s["bias"], normalize=c["normalize"])
            s["layer"] = qbn.MoE(c["fmt"], router, s["w13"], s["s13"], s["w2"], s["s2"], w13_scale2=s["f13"], w2_scale2=s["f2"])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return {"rope": _run_rope, "append": _run_append, "route": _run_route, "moe": _run_moe}[state["case"]["op"]](state)


def _turn(c, x, pos, freq, factor):
    """x [tokens][heads][dim] in 32 bits, its first `rot` elements of each head
    turned by pos * freq; angles in 64 bits (far positions)."""
    angle = pos.double()[:, None] * freq
    cos, sin = (torch.cos(angle) * factor).float()[:, None], (torch.sin(angle) * factor).float()[:, None]
    part = x[..., :c["rot"]]
    if c["layout"] == "half":
        a, b = part.chunk(2, -1)
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., c["rot"]:]), -1)


def _run_rope(s):
    c = s["case"]
    if c["inplace"]:
        s["buffer"].copy_(s["x"])
    if own:
        import bit_block_quantized_nibble_amd as qbn

        if c["inplace"]:
            return qbn.rope(s["buffer"], s["pos"], s["rope"], out=s["buffer"])
        return qbn.rope(s["x"], s["pos"], s["rope"])
    x = s["buffer"] if c["inplace"] else s["x"]
    out = _turn(c, x.float(), s["pos"], s["freq"], s["factor"]).to(x.dtype)
    if c["inplace"]:
        return s["buffer"].copy_(out)
    return out


def _held(s):
    """The cache's content as the values it stands for: E4M3FN and E8M0 as
    views, E2M1 pairs by a table."""
    fmt = s["case"]["fmt"]
    if fmt == "bf16":
        return {"k": s["k"], "v": s["v"]}
    d = {"ks": s["ks"].view(torch.float8_e8m0fnu), "vs": s["vs"].view(torch.float8_e8m0fnu)}
    if fmt == "mxfp8":
        d["k"], d["v"] = s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
    else:
        pairs = s["pairs"].view(torch.int32).reshape(-1)
        d["k"] = pairs.index_select(0, s["k"].reshape(-1).int()).view(torch.bfloat16)
        d["v"] = pairs.index_select(0, s["v"].reshape(-1).int()).view(torch.bfloat16)
    return d


def _encode(x, fmt):
    """x (32-bit, [..., D]) -> (elements, E8M0 bytes [..., D / 32]): exponent
    floor(log2 of the largest magnitude) - emax per 32, elements rounded to
    nearest even and saturated."""
    b = x.reshape(x.shape[:-1] + (-1, 32))
    top = b.abs().amax(-1)
    e = ((top.view(torch.int32) >> 23) - 127 - (8 if fmt == "mxfp8" else 2)).clamp(-127, 127)
    y = torch.ldexp(b.double(), -e.double().unsqueeze(-1)).float()
    scales = (e + 127).to(torch.uint8)
    if fmt == "mxfp8":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape), scales
    m = y.abs()
    code = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _run_append(s):
    if own:
        import bit_block_quantized_nibble_amd as qbn

        q = qbn.kv_append_rope(s["cache"], s["q"], s["newk"], s["newv"], s["table"], s["lens"], s["rope"], s["cu"])
        return dict(_held(s), q=q)
    c, ps = s["case"], s["case"]["page"]
    t = torch.arange(s["newk"].shape[0], device=s["k"].device)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = s["lens"].long()[b] - (s["cu"].long()[b + 1] - t)
    page, slot = s["table"].long()[b, pos // ps], pos % ps
    q = _turn(c, s["q"].float(), pos, s["freq"], s["factor"]).to(torch.bfloat16)
    k = _turn(c, s["newk"].float(), pos, s["freq"], s["factor"])
    for part, scale, x in ((s["k"], s["ks"], k), (s["v"], s["vs"], s["newv"].float())):
        if c["fmt"] == "bf16":
            part[0, page, :, slot] = x.to(torch.bfloat16)
        else:
            part[0, page, :, slot], scale[0, page, :, :, slot] = _encode(x, c["fmt"])
    return dict(_held(s), q=q)


def _routed(c, x, router, bias):
    """The top experts of each token, best first, equal ones by their number, and
    their weights. In 64 bits: which expert comes next may hang on the last bit."""
    logits = x.double() @ router.double().t()
    if bias is not None:
        logits = logits + bias.double()
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    best, ids = best[:, :c["top"]], ids[:, :c["top"]]
    weights = torch.softmax(best if c["normalize"] else logits, -1)
    return ids, (weights if c["normalize"] else weights.gather(1, ids)).float()


def _run_route(s):
    c = s["case"]
    if own:
        import bit_block_quantized_nibble_amd as qbn

        ids, weights = qbn.moe_route(s["router_of"], s["x"])
    else:
        ids, weights = _routed(c, s["x"], s["router"], s["bias"])
        ids = ids.int()
    return {"ids": ids, "weights": weights}


def _values(s, codes, scales, factor):
    """Weights [..., rows, k / 2] in 32 bits."""
    w = s["pairs"].index_select(0, codes.reshape(-1).int()).reshape(codes.shape[:-1] + (-1,))
    if s["case"]["fmt"] == "mxfp4":
        each, scale = 32, scales.view(torch.float8_e8m0fnu).float()
    else:
        each, scale = 16, scales.view(torch.float8_e4m3fn).float()
    w = (w.reshape(w.shape[:-1] + (-1, each)) * scale.unsqueeze(-1)).reshape(w.shape)
    return w if factor is None else w * factor[:, None, None]


def _run_moe(s):
    c = s["case"]
    if own:
        import bit_block_quantized_nibble_amd as qbn

        out, ids, weights = qbn.moe(s["layer"], s["x"])
        return {"out": out, "ids": ids, "weights": weights}
    ids, weights = _routed(c, s["x"], s["router"], s["bias"])
    n, x = c["tokens"], s["x"].float()
    few = n * c["top"] <= c["experts"]
    pick = ids.reshape(-1) if few else slice(None)  # the chosen experts' weights alone, or all of them
    of = lambda f: None if f is None else f[pick]  # noqa: E731
    w = _values(s, s["w13"][pick], s["s13"][pick], of(s["f13"]))
    rows = x.repeat_interleave(c["top"], 0)[:, None] if few else x.expand(c["experts"], -1, -1)
    gate, up = torch.bmm(rows, w.transpose(1, 2)).chunk(2, -1)
    del w
    h = gate * torch.sigmoid(gate) * up
    w = _values(s, s["w2"][pick], s["s2"][pick], of(s["f2"]))
    y = torch.bmm(h, w.transpose(1, 2))
    del w
    if few:
        out = (y.reshape(n, c["top"], -1) * weights.unsqueeze(-1)).sum(1)
    else:
        out = (y[ids, torch.arange(n, device=ids.device)[:, None]] * weights.unsqueeze(-1)).sum(1)
    return {"out": out.to(torch.bfloat16), "ids": ids.int(), "weights": weights}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _exact_turn(c, x, pos):
    """x [tokens][heads][dim] as complex numbers times factor * exp(i * angle)."""
    f, factor = _frequencies(c)
    f = torch.tensor(f, dtype=torch.float64, device=x.device)
    spin = torch.polar(torch.full_like(f, factor).expand(pos.shape[0], -1).contiguous(), torch.outer(pos.double(), f))
    y = x.double().clone()
    n = c["rot"] // 2
    i = torch.arange(n, device=x.device)
    re, im = (i, i + n) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(y[..., re], y[..., im]) * spin[:, None]
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_append(c, seed):
    """Nearest values by search over every finite code, ties to the even code."""
    s = prepare(c, seed)
    lens, new = _lengths(c)
    ps, dev = c["page"], s["k"].device
    got = {name: x.double().reshape(s[name].shape[:-1] + (-1,)).clone() for name, x in _held(s).items()}
    if c["fmt"] == "mxfp4":
        grid, most = list(E2M1), 2
    else:
        grid = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                for e in range(16) for m in range(8)][:127]
        most = 8
    grid = torch.tensor(grid, dtype=torch.float64, device=dev)
    at, qs = 0, []
    for b, (n, t) in enumerate(zip(lens, new)):
        pos = torch.arange(n - t, n, device=dev)
        page, slot = s["table"][b].long()[pos // ps], pos % ps
        qs.append(_exact_turn(c, s["q"][at:at + t], pos))
        for part in ("k", "v"):
            x = s["new" + part][at:at + t]
            x = _exact_turn(c, x, pos) if part == "k" else x.double()
            if c["fmt"] == "bf16":
                got[part][0, page, :, slot] = x
                continue
            y = x.reshape(t, c["kv"], -1, 32)
            top = y.abs().amax(-1)
            e = torch.where(top == 0, -127, torch.frexp(top)[1] - 1 - most).clamp(-127, 127).double()
            y = y / torch.pow(2.0, e)[..., None]
            m = y.abs().clamp(max=float(grid[-1]))
            hi = torch.searchsorted(grid, m).clamp(max=grid.numel() - 1)
            lo = (hi - 1).clamp(min=0)
            up, down = grid[hi] - m, m - grid[lo]
            pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            got[part][0, page, :, slot] = torch.copysign(grid[pick], y).reshape(t, c["kv"], -1)
            got[part + "s"][0, page, :, :, slot] = torch.pow(2.0, e)
        at += t
    got = {k: (x.reshape(-1) if c["fmt"] == "mxfp4" and k in ("k", "v") else x) for k, x in got.items()}
    return dict(got, q=torch.cat(qs))


def _exact_route(c, s):
    """The best experts one rank at a time, and their shares."""
    logits = (s["x"].double()[:, None] * s["router"].double()).sum(-1) if c["tokens"] < 8 else \
        torch.stack([s["x"].double() @ r for r in s["router"].double()], 1)
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    left, ids, val = logits.clone(), [], []
    for _ in range(c["top"]):
        top = left.amax(-1, keepdim=True)
        i = (left == top).int().argmax(-1, keepdim=True)
        ids.append(i)
        val.append(top)
        left.scatter_(1, i, -math.inf)
    ids, val = torch.cat(ids, 1), torch.cat(val, 1)
    total = torch.logsumexp(val if c["normalize"] else logits, -1, keepdim=True)
    return ids, torch.exp(val - total)


def _exact_rows(c, codes, scales, factor):
    """One expert's weights [rows][k] in 64 bits, from the bit fields."""
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    sign, e, m = x >> 3, (x >> 1) & 3, x & 1
    v = torch.where(e == 0, m.double() / 2, (1 + m.double() / 2) * torch.pow(2.0, e.double() - 1))
    v = torch.where(sign == 1, -v, v)
    b = scales.int()
    if c["fmt"] == "mxfp4":
        return v * torch.pow(2.0, b.double() - 127).repeat_interleave(32, -1)
    e, m = (b >> 3) & 15, (b & 7).double() / 8
    w = torch.where(e == 0, m * 2.0 ** -6, (1 + m) * torch.pow(2.0, e.double() - 7))
    return v * w.repeat_interleave(16, -1) * factor.double()


def _exact_moe(c, seed):
    s = prepare(c, seed)
    ids, weights = _exact_route(c, s)
    out = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device=ids.device)
    for e in range(c["experts"]):
        token, rank = (ids == e).nonzero(as_tuple=True)
        if not token.numel():
            continue
        w = _exact_rows(c, s["w13"][e], s["s13"][e], None if s["f13"] is None else s["f13"][e])
        g, u = (s["x"][token].double() @ w.t()).split(c["inter"], -1)
        w = _exact_rows(c, s["w2"][e], s["s2"][e], None if s["f2"] is None else s["f2"][e])
        out.index_add_(0, token, (g / (1 + torch.exp(-g)) * u) @ w.t() * weights[token, rank, None])
    return {"out": out, "ids": ids.int(), "weights": weights}


def exact(case, seed):
    c = case
    if c["op"] == "rope":
        s = prepare(c, seed)
        return _exact_turn(c, s["x"], s["pos"])
    if c["op"] == "append":
        return _exact_append(c, seed)
    if c["op"] == "route":
        ids, weights = _exact_route(c, prepare(c, seed))
        return {"ids": ids.int(), "weights": weights}
    return _exact_moe(c, seed)
