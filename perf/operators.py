"""Cases and plain forms of the paged key-value cache operators.

A decode step of a model with 4-bit weights streams two things: the weights
and the key-value cache. These cases cover the second: writing new tokens
into a paged cache (``append``), attention of one new token per sequence over
it (``decode``), causal attention of chunks of new tokens with a sliding window
and a few first tokens that stay visible (``prefill``), and the page
bookkeeping between steps (``pages``: free, fork, reserve, compact).

A cache holds, per layer and page, K and V elements [heads][page][head_dim]
(bfloat16, E4M3FN or E2M1 pairs, low nibble = even element) and, for the last
two, E8M0 scales [heads][head_dim / 32][page], one per 32 elements of a token.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BITS = {"bf16": 16.0, "mxfp8": 8.25, "mxfp4": 4.25}  # per element, scales included


def _case(name, op, fmt, page, seqs, length, new, heads, kv, dim, window=0, sinks=0, ragged=True, layers=1, forks=0,
          gone=0, src="bf16"):
    c = {"op": op, "fmt": fmt, "page": page, "seqs": seqs, "length": length, "new": new, "heads": heads, "kv": kv,
         "dim": dim, "window": window, "sinks": sinks, "ragged": ragged, "layers": layers, "forks": forks,
         "gone": gone, "src": src}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step's new tokens of a small batch: latency
        _case("append step", "append", "mxfp8", 16, 16, 700, 1, 8, 8, 128),
        # the prompts of four requests, at the 4-bit layout
        _case("append prompts", "append", "mxfp4", 64, 4, 8192, 4096, 8, 8, 128),
        # one user, a short chat, unquantized cache: the smallest attention call
        _case("decode one short", "decode", "bf16", 16, 1, 129, 1, 32, 8, 128, ragged=False),
        # an ordinary serving batch with mixed lengths
        _case("decode batch", "decode", "mxfp8", 64, 32, 4096, 1, 32, 8, 128),
        # two users with very long documents at 4 bits: bandwidth
        _case("decode long", "decode", "mxfp4", 128, 2, 131072, 1, 64, 8, 128),
        # streaming chats: a window and four sinks, one key-value head, head size 64
        _case("decode window", "decode", "mxfp4", 32, 64, 32768, 1, 8, 1, 64, window=4096, sinks=4),
        # a whole prompt, causal, unquantized cache
        _case("prefill prompt", "prefill", "bf16", 64, 1, 4096, 4096, 32, 8, 128, ragged=False),
        # short and odd chunks on contexts of mixed length, head size 96
        _case("prefill chunks", "prefill", "mxfp8", 16, 5, 1531, 341, 12, 4, 96),
        # a long document in one chunk: window and sinks, 4-bit cache
        _case("prefill window", "prefill", "mxfp4", 128, 1, 16384, 8192, 32, 8, 128, window=2048, sinks=16,
              ragged=False),
        # a beam search's turn: 4 requests leave, 12 beams fork, every sequence takes a token, the pool is packed
        _case("pages small", "pages", "bf16", 16, 24, 300, 1, 2, 2, 64, layers=2, forks=12, gone=4),
        # a busy server's turn: half of the requests leave at once, and their pages are packed
        _case("pages large", "pages", "mxfp8", 32, 96, 4000, 16, 8, 8, 128, layers=4, forks=24, gone=48),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "prefill", "prefill", "pages"))
    fmt = rng.choice(("bf16", "mxfp8") if op == "pages" else ("bf16", "mxfp8", "mxfp4"))
    page = rng.choice((16, 32, 64, 128))
    dim = rng.choice((64, 96, 128, 192, 256))
    kv = rng.choice((1, 2, 3, 4, 8))
    heads = kv * rng.choice((1, 2, 3, 4, 7, 8, 16))
    if op == "append":
        seqs = _spread(rng, 1, 64)
        new = rng.choice((1, 1, _spread(rng, 2, max(2, 8192 // seqs))))
        return _case("", op, fmt, page, seqs, new + _spread(rng, 1, 4096), new, kv, kv, dim,
                     src=rng.choice(("bf16", "f32")))
    if op == "decode":
        seqs = _spread(rng, 1, 128)
        length = _spread(rng, 1, min(131072, 100_000_000 // (seqs * kv * dim)))
        window = rng.choice((0, 0, _spread(rng, 1, 8192)))
        return _case("", op, fmt, page, seqs, length, 1, heads, kv, dim, window=window,
                     sinks=rng.choice((0, 1, 4, 33)) if window else 0)
    if op == "prefill":
        heads = min(heads, 32 // kv * kv)
        seqs = _spread(rng, 1, 12)
        length = _spread(rng, 1, 8192)
        new = _spread(rng, 1, max(1, min(length, 250_000_000 // (seqs * heads * length))))
        window = rng.choice((0, 0, _spread(rng, 1, 4096)))
        return _case("", op, fmt, page, seqs, length, new, heads, kv, dim, window=window,
                     sinks=rng.choice((0, 1, 4, 33)) if window else 0)
    seqs = _spread(rng, 4, 96)
    gone = rng.randrange(1, seqs // 2 + 1)
    return _case("", op, fmt, page, seqs, _spread(rng, 16, 2000), rng.choice((1, 5, 40)), kv, kv, dim,
                 layers=rng.choice((1, 2, 3)), forks=rng.randrange(1, seqs + 1), gone=gone)


# ---------------------------------------------------------------- what a case's sequences are (the same for every seed)

def _lengths(c):
    """(tokens in each sequence after the pass, how many of them are new): the
    first is the longest, the others of a ragged batch spread over 1/30 to 1."""
    r = random.Random("%d %d %d" % (c["seqs"], c["length"], c["new"]))
    f = [1.0] + [math.exp(r.uniform(math.log(1 / 30), 0.0)) if c["ragged"] else 1.0 for _ in range(c["seqs"] - 1)]
    lens = [max(1, int(c["length"] * x)) for x in f]
    g = [1.0] + [math.exp(r.uniform(math.log(1 / 30), 0.0)) if c["ragged"] else 1.0 for _ in range(c["seqs"] - 1)]
    return lens, [max(1, min(n, int(c["new"] * x))) for n, x in zip(lens, g)]


def _pages_plan(c):
    """The pages case: lengths of the sequences at hand, who leaves, who is
    forked into which empty row, and the room that each sequence takes."""
    r = random.Random("pages %d %d %d" % (c["seqs"], c["length"], c["forks"]))
    lens = [max(1, int(c["length"] * math.exp(r.uniform(math.log(1 / 8), 0.0)))) for _ in range(c["seqs"])]
    order = list(range(c["seqs"]))
    r.shuffle(order)
    gone, stay = sorted(order[:c["gone"]]), sorted(order[c["gone"]:])
    parents = [r.choice(stay) for _ in range(c["forks"])]
    children = list(range(c["seqs"], c["seqs"] + c["forks"]))
    takers = stay + children
    return lens, gone, parents, children, takers


def _visible(c, pos):
    """How many tokens a query at position pos sees."""
    if not c["window"] or pos + 1 <= c["window"]:
        return pos + 1
    return c["window"] + min(c["sinks"], pos + 1 - c["window"])


def work(case):
    c = case
    each = BITS[c["fmt"]] / 8
    if c["op"] == "append":
        n = sum(_lengths(c)[1]) * c["kv"] * c["dim"] * 2
        return {"bytes": n * ((4 if c["src"] == "f32" else 2) + each), "flops": 2.0 * n}
    if c["op"] == "pages":
        lens, gone, parents, children, takers = _pages_plan(c)
        ps = c["page"]
        full = lambda n: -(-n // ps)  # noqa: E731
        kids = [lens[p] for p in parents]
        stay = [lens[s] for s in range(c["seqs"]) if s not in gone]
        live = sum(full(n + c["new"]) for n in stay)
        live += sum(full(n + c["new"]) - n // ps for n in kids)
        before = sum(full(n) for n in lens)
        moved = max(0, min(live, int(before * (1 - live / max(before, live)))))  # what stands above the packed end, on average
        copied = sum(1 for n in kids if n % ps)
        payload = (moved + copied) * c["layers"] * c["kv"] * ps * c["dim"] * 2 * each
        width = full(max(lens) + c["new"]) + 2
        rows = c["seqs"] + c["forks"]
        return {"bytes": 2 * payload + 8.0 * rows * width + 8.0 * _pool_pages(c), "flops": 1.0 * rows * width}
    lens, new = _lengths(c)
    q = sum(new) * c["heads"] * c["dim"]
    pairs = keys = 0
    for n, t in zip(lens, new):
        seen = [_visible(c, p) for p in range(n - t, n)]
        pairs += sum(seen)
        keys += n if not c["window"] else min(n, c["window"] + t - 1 + min(c["sinks"], max(0, n - c["window"] - t + 1)))
    return {"bytes": 4.0 * q + 4.0 * sum(new) * c["heads"] + keys * c["kv"] * c["dim"] * 2 * each,
            "flops": 4.0 * c["dim"] * c["heads"] * pairs}


def _pool_pages(c):
    if c["op"] == "pages":
        lens, _, parents, _, takers = _pages_plan(c)
        need = sum(-(-n // c["page"]) for n in lens) + len(takers) * (2 + -(-c["new"] // c["page"]))
    else:
        need = sum(-(-n // c["page"]) for n in _lengths(c)[0])
    return need + need // 16 + 1


# ---------------------------------------------------------------- inputs

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
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _pool(c, pages, g, dev):
    """K (or V) of a cache in use: elements and scales of every page."""
    shape = (c["layers"], pages, c["kv"], c["page"], c["dim"])
    n = math.prod(shape)
    pad = -n % 32
    x = torch.randn(n + pad, generator=g, device=dev, dtype=torch.float32)[:n].reshape(shape)
    if c["fmt"] == "bf16":
        return x.to(torch.bfloat16), None
    parts = [_encode(x[:, i:i + 2048], c["fmt"]) for i in range(0, pages, 2048)]
    return (torch.cat([p[0] for p in parts], 1),
            torch.cat([p[1] for p in parts], 1).transpose(-1, -2).contiguous())


def prepare(case, seed):
    c, dev = case, torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    pages = _pool_pages(c)
    s = {"case": dict(c)}
    s["k"], s["ks"] = _pool(c, pages, g, dev)
    s["v"], s["vs"] = _pool(c, pages, g, dev)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu().tolist()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if c["op"] == "pages":
        lens, gone, parents, children, takers = _pages_plan(c)
        lens = lens + [0] * len(children)
        after = c["new"]
    else:
        lens, new = _lengths(c)
        after = 0
    width = -(-(max(lens) + after) // c["page"]) + 2  # rows have room to spare
    rows, at = [], 0
    for n in lens:
        k = -(-n // c["page"])
        rows.append(order[at:at + k] + [-1] * (width - k))
        at += k
    s["table"], s["lens"] = ints(rows), ints(lens)
    if c["op"] == "pages":
        refs = [0] * pages
        for p in order[:at]:
            refs[p] = 1
        s["refs"] = ints(refs)
        s["gone"], s["parents"], s["children"], s["takers"] = ints(gone), ints(parents), ints(children), ints(takers)
        s["take"] = ints([c["new"]] * len(takers))
    else:
        cu = [0]
        for t in new:
            cu.append(cu[-1] + t)
        s["cu"], s["most"] = ints(cu), max(new)
        total, dt = cu[-1], torch.float32 if c["src"] == "f32" else torch.bfloat16
        wide = c["heads"] + 2 * c["kv"]  # q, k and v are views of one fused projection's output
        x = torch.randn(total, wide, c["dim"], generator=g, device=dev, dtype=torch.float32)
        x[:, :c["heads"]] *= 2.0  # attention in earnest is not flat
        x = x.to(dt)
        if c["op"] == "append":
            s["newk"], s["newv"] = x[:, c["heads"]:c["heads"] + c["kv"]], x[:, c["heads"] + c["kv"]:]
        else:
            s["q"] = x[:, :c["heads"]]
    if c["fmt"] == "mxfp4":
        lo = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=dev)
        b = torch.arange(256, device=dev)
        s["pairs"] = torch.stack((lo[b % 16], lo[b // 16]), -1).to(torch.bfloat16).contiguous()
    if own:
        import bit_block_quantized_nibble_amd as qbn

        s["cache"] = qbn.KVCache(c["fmt"], s["k"], s["v"], s["ks"], s["vs"])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if state["case"]["op"] == "append":
        return _run_append(state)
    if state["case"]["op"] == "pages":
        return _run_pages(state)
    return _run_decode(state) if state["case"]["op"] == "decode" else _run_prefill(state)


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


def _run_append(s):
    if own:
        import bit_block_quantized_nibble_amd as qbn

        qbn.kv_append(s["cache"], s["newk"], s["newv"], s["table"], s["lens"], s["cu"])
        return _held(s)
    c, ps = s["case"], s["case"]["page"]
    t = torch.arange(s["newk"].shape[0], device=s["k"].device)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = s["lens"].long()[b] - (s["cu"].long()[b + 1] - t)
    page, slot = s["table"].long()[b, pos // ps], pos % ps
    for part, scale, x in ((s["k"], s["ks"], s["newk"]), (s["v"], s["vs"], s["newv"])):
        if c["fmt"] == "bf16":
            part[0, page, :, slot] = x.to(torch.bfloat16)
        else:
            part[0, page, :, slot], scale[0, page, :, :, slot] = _encode(x.float(), c["fmt"])
    return _held(s)


def _values(s, elements, scales):
    """Gathered pages (elements [..., page, D or D / 2]) as 32-bit values."""
    fmt = s["case"]["fmt"]
    if fmt == "bf16":
        return elements.float()
    if fmt == "mxfp8":
        x = elements.view(torch.float8_e4m3fn).float()
    else:
        x = s["pairs"].float()[elements.long()].flatten(-2)
    w = scales.view(torch.float8_e8m0fnu).float().transpose(-1, -2)
    return (x.reshape(x.shape[:-1] + (-1, 32)) * w.unsqueeze(-1)).reshape(x.shape)


def _gathered(s):
    """K and V of every sequence, padded to the longest: [seqs][kv][tokens][D]."""
    idx = s["table"].long()
    idx = idx[:, :-(-s["case"]["length"] // s["case"]["page"])].clamp(min=0)
    flat = lambda x: x.permute(0, 2, 1, 3, 4).flatten(2, 3)  # noqa: E731
    k = _values(s, s["k"][0][idx], None if s["ks"] is None else s["ks"][0][idx])
    v = _values(s, s["v"][0][idx], None if s["vs"] is None else s["vs"][0][idx])
    return flat(k), flat(v)


def _softmax_product(scores, seen, v):
    """(sum over the visible of softmax * v, log of the sum of exp); a row that
    sees nothing gives 0 and -inf."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (top + torch.log(total)).squeeze(-1)


def _run_decode(s):
    c = s["case"]
    if own:
        import bit_block_quantized_nibble_amd as qbn

        out, lse = qbn.kv_attention_decode(s["cache"], s["q"], s["table"], s["lens"], window=c["window"],
                                           sinks=c["sinks"])
        return {"out": out, "lse": lse}
    k, v = _gathered(s)
    n = s["q"].shape[0]
    q = s["q"].float().reshape(n, c["kv"], -1, c["dim"])
    j = torch.arange(k.shape[2], device=k.device)
    last = s["lens"].long()[:, None] - 1
    seen = j[None] <= last
    if c["window"]:
        seen = seen & ((j[None] > last - c["window"]) | (j[None] < c["sinks"]))
    o, lse = _softmax_product(torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(c["dim"]), seen[:, None, None], v)
    return {"out": o.reshape(n, c["heads"], c["dim"]).to(torch.bfloat16), "lse": lse.reshape(n, c["heads"])}


def _run_prefill(s):
    c = s["case"]
    if own:
        import bit_block_quantized_nibble_amd as qbn

        out, lse = qbn.kv_attention_prefill(s["cache"], s["q"], s["cu"], s["table"], s["lens"], window=c["window"],
                                            sinks=c["sinks"])
        return {"out": out, "lse": lse}
    k, v = _gathered(s)
    cu, lens = s["cu"].long(), s["lens"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(s["most"], device=k.device)
    live = i[None] < new[:, None]
    row = torch.where(live, cu[:-1, None] + i[None], 0)
    pos = (lens - new)[:, None] + i[None]
    q = s["q"].float()[row].reshape(c["seqs"], s["most"], c["kv"], -1, c["dim"]).permute(0, 2, 3, 1, 4)
    j = torch.arange(k.shape[2], device=k.device)
    seen = (j <= pos[..., None]) & live[..., None]
    if c["window"]:
        seen = seen & ((j > pos[..., None] - c["window"]) | (j < c["sinks"]))
    # the heads of one key-value head share one product: rows are (head, query)
    scores = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)) / math.sqrt(c["dim"])
    seen = seen[:, None].expand(-1, c["heads"] // c["kv"], -1, -1).flatten(1, 2)[:, None]
    o, lse = _softmax_product(scores, seen, v)
    b = torch.searchsorted(cu[1:], torch.arange(s["q"].shape[0], device=k.device), right=True)
    at = torch.arange(s["q"].shape[0], device=k.device) - cu[b]
    o = o.reshape(c["seqs"], c["heads"], s["most"], c["dim"])[b, :, at]
    lse = lse.reshape(c["seqs"], c["heads"], s["most"])[b, :, at]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _run_pages(s):
    if own:
        import bit_block_quantized_nibble_amd as qbn

        pool = qbn.KVPool(s["table"], s["lens"], s["refs"], s["case"]["page"])
        after = qbn.KVPool.like(pool)  # the tables of the step before stay as they are
        qbn.kv_free(pool, s["gone"], out=after)
        forked = qbn.kv_fork(s["cache"], after, s["parents"], s["children"])
        got = qbn.kv_reserve(after, s["takers"], s["take"])
        live = qbn.kv_compact(s["cache"], after)
        return dict(_held(s), table=after.table, lens=after.lens, refs=after.refs, forked=forked, got=got, live=live)
    ps = s["case"]["page"]
    table, lens, refs = s["table"].long(), s["lens"].long(), s["refs"].long()
    col = torch.arange(table.shape[1], device=table.device)[None]
    parts = [x for x in (s["k"], s["v"], s["ks"], s["vs"]) if x is not None]
    # free: their pages lose a reference each
    gone = s["gone"].long()
    old = table[gone]
    refs.index_add_(0, old[old >= 0], torch.full_like(old[old >= 0], -1))
    table[gone], lens[gone] = -1, 0
    # fork: whole pages are shared, a last page that is not full is copied to the lowest free page
    par, kid = s["parents"].long(), s["children"].long()
    n = lens[par]
    rows = torch.where(col < n[:, None] // ps, table[par], -1)
    free = (refs == 0).nonzero()[:, 0]
    refs.index_add_(0, rows[rows >= 0], torch.ones_like(rows[rows >= 0]))
    tail = (n % ps > 0).nonzero()[:, 0]
    new = free[:tail.shape[0]]
    src = table[par[tail], n[tail] // ps]
    rows[tail, n[tail] // ps] = new
    refs[new] = 1
    table[kid], lens[kid] = rows, n
    for x in parts:
        x[:, new] = x[:, src]
    # reserve: the lowest free pages, in the order of the requests
    who, take = s["takers"].long(), s["take"].long()
    have, want = -(-lens[who] // ps), -(-(lens[who] + take) // ps)
    i = torch.repeat_interleave(torch.arange(who.shape[0], device=who.device), want - have)
    first = torch.cumsum(want - have, 0) - (want - have)
    j = torch.arange(i.shape[0], device=i.device) - first[i]
    new = (refs == 0).nonzero()[:i.shape[0], 0]
    table[who[i], have[i] + j] = new
    refs[new] = 1
    lens[who] = lens[who] + take
    # compact: live pages beyond the number of live pages move into the holes below it, in order
    used = refs > 0
    live = used.sum()
    over = torch.arange(refs.shape[0], device=refs.device) >= live
    src, dst = (used & over).nonzero()[:, 0], (~used & ~over).nonzero()[:, 0]
    to = torch.arange(refs.shape[0], device=refs.device)
    to[src] = dst
    table = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    refs[dst] = refs[src]
    refs[src] = 0
    for x in parts:
        x[:, dst] = x[:, src]
    ok = torch.full((1,), -1, dtype=torch.int32, device=table.device)
    return dict(_held(s), table=table.int(), lens=lens.int(), refs=refs.int(), forked=ok, got=ok.clone(),
                live=live.int().reshape(1))


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _exact_rows(c, s, b, n, which):
    """K or V of sequence b in 64 bits: [kv][n][D], element by element from the
    bit fields."""
    ps = c["page"]
    pages = s["table"][b, :-(-n // ps)].long()
    x = s[which][0].index_select(0, pages).transpose(0, 1).flatten(1, 2)[:, :n]
    if c["fmt"] == "bf16":
        return x.double()
    w = s[which + "s"][0].index_select(0, pages).permute(1, 0, 3, 2).flatten(1, 2)[:, :n]
    w = torch.pow(2.0, w.double() - 127.0).repeat_interleave(32, -1)
    x = x.int()
    if c["fmt"] == "mxfp4":
        x = torch.stack((x & 15, x >> 4), -1).flatten(-2)
        sign, e, m, bias, mb = x >> 3, (x >> 1) & 3, x & 1, 1, 1
    else:
        sign, e, m, bias, mb = x >> 7, (x >> 3) & 15, x & 7, 7, 3
    frac = m.double() / (1 << mb)
    val = torch.where(e == 0, frac * 2.0 ** (1 - bias), (1 + frac) * torch.pow(2.0, e.double() - bias))
    return torch.where(sign == 1, -val, val) * w


def _exact_attention(c, seed):
    s = prepare(c, seed)
    lens, new = _lengths(c)
    rep = c["heads"] // c["kv"]
    outs, lses, at = [], [], 0
    for b, (n, t) in enumerate(zip(lens, new)):
        k, v = _exact_rows(c, s, b, n, "k"), _exact_rows(c, s, b, n, "v")
        q = s["q"][at:at + t].double().transpose(0, 1)
        at += t
        o, l = [], []
        key = torch.arange(n, device=k.device)
        step = max(1, (1 << 28) // n)
        for h in range(c["heads"]):
            oh, lh = [], []
            for r in range(0, t, step):
                pos = torch.arange(n - t + r, n - t + min(t, r + step), device=k.device)[:, None]
                hide = key > pos
                if c["window"]:
                    hide = hide | ((key + c["window"] <= pos) & (key >= c["sinks"]))
                x = (q[h, r:r + step] @ k[h // rep].t()) * c["dim"] ** -0.5
                x = x.masked_fill(hide, -math.inf)
                lh.append(torch.logsumexp(x, -1))
                oh.append(torch.softmax(x, -1) @ v[h // rep])
            o.append(torch.cat(oh))
            l.append(torch.cat(lh))
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(l, 1))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_append(c, seed):
    """Nearest values by search over every finite code, ties to the even code."""
    s = prepare(c, seed)
    lens, new = _lengths(c)
    ps, dev = c["page"], s["k"].device
    got = _held(s)
    got = {name: x.double().reshape(s[name].shape[:-1] + (-1,)).clone() for name, x in got.items()}
    if c["fmt"] == "mxfp4":
        grid, most = list(E2M1), 2
    else:
        grid = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                for e in range(16) for m in range(8)][:127]
        most = 8
    grid = torch.tensor(grid, dtype=torch.float64, device=dev)
    at = 0
    for b, (n, t) in enumerate(zip(lens, new)):
        pos = torch.arange(n - t, n, device=dev)
        page, slot = s["table"][b].long()[pos // ps], pos % ps
        for part in ("k", "v"):
            x = s["new" + part][at:at + t].double()
            if c["fmt"] == "bf16":
                got[part][0, page, :, slot] = x
                continue
            y = x.reshape(t, c["kv"], -1, 32)
            e = torch.frexp(y.abs().amax(-1))[1] - 1 - most  # of 0: any, its elements are 0
            e = torch.where(y.abs().amax(-1) == 0, -127, e).clamp(-127, 127).double()
            y = y / torch.pow(2.0, e)[..., None]
            m = y.abs().clamp(max=float(grid[-1]))
            hi = torch.searchsorted(grid, m).clamp(max=grid.numel() - 1)
            lo = (hi - 1).clamp(min=0)
            up, down = grid[hi] - m, m - grid[lo]
            pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            got[part][0, page, :, slot] = torch.copysign(grid[pick], y).reshape(t, c["kv"], -1)
            got[part + "s"][0, page, :, :, slot] = torch.pow(2.0, e)
        at += t
    return {k: (x.reshape(-1) if c["fmt"] == "mxfp4" and k in ("k", "v") else x) for k, x in got.items()}


def _exact_pages(c, seed):
    """The turn by its definition, one sequence and one page at a time."""
    s = prepare(c, seed)
    ps = c["page"]
    rows, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    held = {i: i for i in range(len(refs))}  # page -> the page whose first content it has

    def lowest():
        p = refs.index(0)
        refs[p] = 1
        return p

    for b in s["gone"].tolist():
        for p in rows[b]:
            if p >= 0:
                refs[p] -= 1
        rows[b], lens[b] = [-1] * len(rows[b]), 0
    made = []
    for a, b in zip(s["parents"].tolist(), s["children"].tolist()):
        rows[b], lens[b] = list(rows[a]), lens[a]
        for i, p in enumerate(rows[b]):
            if i < lens[a] // ps:
                refs[p] += 1
            elif i == lens[a] // ps and lens[a] % ps:
                made.append((b, i, p))
                rows[b][i] = -1
            else:
                rows[b][i] = -1
    for b, i, p in made:
        rows[b][i] = lowest()
        held[rows[b][i]] = held[p]
    for b, t in zip(s["takers"].tolist(), s["take"].tolist()):
        for i in range(-(-lens[b] // ps), -(-(lens[b] + t) // ps)):
            rows[b][i] = lowest()
        lens[b] += t
    live = sum(r > 0 for r in refs)
    holes = [p for p in range(live) if refs[p] == 0]
    to = dict(zip([p for p in range(live, len(refs)) if refs[p] > 0], holes))
    for p, h in to.items():
        held[h] = held[p]
    order = torch.tensor([held[p] for p in range(len(refs))], device=s["k"].device)
    d = {name: x.double()[:, order] for name, x in _held(s).items()}
    return dict(d, table=None, lens=None, refs=None, forked=None, got=None, live=None)


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, seed)
    if case["op"] == "pages":
        return _exact_pages(case, seed)
    return _exact_attention(case, seed)
