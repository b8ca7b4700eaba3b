"""Eviction from the Full KV Pool by accumulated attention weight: cases, plain forms and
values in 64 bits, for measuring the library's kernels.

Four operators, in the order in which a server that bounds its caches calls them:

  prompt   the attention weight that a prompt's last queries put on every cached key, summed
           over the queries and the query heads of a KV head, added to what was there
  select   the positions of a budget that stay: the first ones, the newest ones, and of the
           rest those with the largest weight (each one's or its neighbours')
  compact  the rows of K and V that stay, moved into pages of their own, their weights beside
  weigh    decode attention that also adds the step's weight on every key

Sizes are this library's own: 32 query heads over 4 KV heads (and the small 16 over 2), head
size 128, 64-token pages, contexts of 2K to 1M tokens.
"""
import math
import random

import torch

own = False

D, PAGE = 128, 64
SCALE = D ** -0.5
DEV = "cuda"


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # a small model's step of four short conversations
        dict(name="weigh few", op="weigh", layer="full", b=4, t=1, lo=1000, hi=2048, hq=16, hkv=2, prev=True, decay=1.0, lens=1),
        # one decode step of 32 sequences of 8K to 64K tokens
        dict(name="weigh decode", op="weigh", layer="full", b=32, t=1, lo=8192, hi=65536, hq=32, hkv=4, prev=True, decay=1.0, lens=2),
        # four tokens to verify for each of 16 sequences, older weights fading
        dict(name="weigh verify", op="weigh", layer="full", b=16, t=4, lo=3001, hi=20000, hq=32, hkv=4, prev=True, decay=0.97, lens=3),
        # a step over an FP8 layer
        dict(name="weigh fp8", op="weigh", layer="e4m3", b=8, t=1, lo=8192, hi=65536, hq=32, hkv=4, prev=True, decay=1.0, lens=4),
        # two short prompts, the last 16 tokens' queries
        dict(name="prompt small", op="prompt", r=2, lo=300, hi=900, rows=200, window=16, hq=16, hkv=2, prev=False, decay=1.0, lens=5),
        # eight prompts of 16K to 128K tokens at their last chunks
        dict(name="prompt chunks", op="prompt", r=8, lo=16384, hi=131072, rows=2048, window=32, hq=32, hkv=4, prev=False, decay=1.0, lens=6),
        # one long document, more queries, on top of earlier chunks' weights
        dict(name="prompt long", op="prompt", r=1, lo=262144, hi=262144, rows=8192, window=64, hq=32, hkv=4, prev=True, decay=0.5, lens=7),
        # a short cache that has grown a little past its budget
        dict(name="select few", op="select", r=4, h=2, lo=600, hi=2048, budget=512, sinks=4, recent=128, reach=0, lens=8),
        # prompts of 8K to 64K tokens cut to 4096, neighbours kept together
        dict(name="select batch", op="select", r=32, h=4, lo=8192, hi=65536, budget=4096, sinks=4, recent=64, reach=3, lens=9),
        # the longest contexts
        dict(name="select long", op="select", r=4, h=4, lo=262144, hi=1000000, budget=16384, sinks=16, recent=512, reach=0, lens=10),
        # what stays of 16 sequences, 4096 tokens each, a choice for each head
        dict(name="compact batch", op="compact", layer="full", r=16, h=4, lo=6000, hi=16000, budget=4096, hkv=4, lens=11),
        # the same for an FP8 layer, one choice for all heads
        dict(name="compact fp8", op="compact", layer="e5m2", r=8, h=1, lo=3000, hi=9000, budget=2000, hkv=4, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["weigh", "weigh", "prompt", "select", "compact"])
    hq, hkv = rng.choice([(32, 4), (32, 4), (16, 2), (16, 4), (8, 8)])
    lens = rng.randrange(100, 1 << 30)
    if op == "weigh":
        t = rng.choice([1, 1, 1, 2, 3, 4])
        b = _log(rng, 1, 48)
        hi = _log(rng, 100, min(200000, 1000000 // (b * t) * 4 // max(4, hkv)))
        return dict(op=op, layer=rng.choice(["full", "full", "e4m3", "e5m2"]), b=b, t=t, lo=max(0, hi // rng.choice([1, 3, 20])), hi=hi,
                    hq=hq, hkv=hkv, prev=rng.random() < 0.7, decay=rng.choice([1.0, 0.9, 0.999]), lens=lens)
    if op == "prompt":
        r = _log(rng, 1, 16)
        hi = _log(rng, 60, 400000 // r * 4 // max(4, hkv))
        return dict(op=op, r=r, lo=max(1, hi // rng.choice([1, 2, 10])), hi=hi, rows=_log(rng, 1, 2000), window=rng.choice([1, 8, 16, 32, 33, 64]),
                    hq=hq, hkv=hkv, prev=rng.random() < 0.5, decay=rng.choice([1.0, 0.9, 0.5]), lens=lens)
    r = _log(rng, 1, 32)
    if op == "select":
        hi = _log(rng, 50, min(1000000, 2400000 // r))
        budget = max(1, int(hi * rng.choice([0.05, 0.2, 0.5, 1.1])))
        sinks, recent = rng.choice([(0, 0), (4, min(64, budget // 2)), (1, budget // 3)])
        sinks = min(sinks, budget - recent)
        return dict(op=op, r=r, h=rng.choice([1, 2, 4, 8]), lo=max(0, hi // rng.choice([1, 2, 8])), hi=hi, budget=budget, sinks=sinks,
                    recent=recent, reach=rng.choice([0, 0, 1, 3, 7]), lens=lens)
    hi = _log(rng, 100, min(60000, 250000 // r))
    return dict(op=op, layer=rng.choice(["full", "full", "e4m3", "e5m2"]), r=r, h=rng.choice([1, hkv]), lo=max(1, hi // rng.choice([1, 2, 4])),
                hi=hi, budget=max(1, min(4096, int(hi * rng.choice([0.1, 0.25, 0.5])))), hkv=hkv, lens=lens)


def _lengths(c):
    """The token counts of a case: they follow from the case alone."""
    rng = random.Random(c["lens"])
    n = [rng.randint(c["lo"], c["hi"]) for _ in range(c["b"] if c["op"] == "weigh" else c["r"])]
    if c["op"] == "prompt":  # new rows of each request: most of a chunk, or a short last one
        return n, [min(x, max(1, c["rows"] // rng.choice([1, 1, 2, 50]))) for x in n]
    return n


def _stride(n):
    return (max(n) + 4 + 3) // 4 * 4


def work(case):
    c = case
    if c["op"] == "weigh":
        n = _lengths(c)
        keys = sum(n) + len(n) * c["t"]
        pairs = sum(c["t"] * x + c["t"] * (c["t"] + 1) // 2 for x in n)
        row = 2 * (D * 2 if c["layer"] == "full" else D + 4) * c["hkv"]
        return {"bytes": sum(n) * row + len(n) * c["t"] * 4 * D * (c["hq"] + c["hkv"]) + 4 * c["hkv"] * (keys + (sum(n) if c["prev"] else 0)),
                "flops": 4 * pairs * c["hq"] * D}
    if c["op"] == "prompt":
        n, m = _lengths(c)
        t = [min(c["window"], x) for x in m]
        pairs = sum(k * x - k * (k - 1) // 2 for k, x in zip(t, n))
        old = sum(x - k for x, k in zip(n, m)) if c["prev"] else 0
        return {"bytes": c["hkv"] * (sum(n) * (2 * D + 4) + 4 * old) + sum(t) * c["hq"] * 2 * D, "flops": 2 * pairs * c["hq"] * D}
    n = _lengths(c)
    kept = sum(min(x, c["budget"]) for x in n)
    if c["op"] == "select":
        return {"bytes": 4 * c["h"] * (sum(n) + c["r"] * c["budget"]), "flops": c["h"] * sum(n)}
    row = 2 * (D * 2 if c["layer"] == "full" else D + 4)
    return {"bytes": kept * c["hkv"] * (2 * row + 8) + 4 * kept * c["h"], "flops": kept}


# ----------------------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).bfloat16()


def _perm16():
    return torch.tensor([4 * ((l % 8) // 2) + l % 2 + 2 * (l // 8) for l in range(16)], device=DEV)


def _k_place():
    """Stored byte of each dimension of a K row of an FP8 layer."""
    return 16 * (torch.arange(D, device=DEV) // 16) + _perm16().repeat(D // 16)


def _v_place():
    """Stored byte of each key of a V page's row (a dimension) of an FP8 layer."""
    return 16 * (torch.arange(PAGE, device=DEV) // 16) + _perm16().repeat(PAGE // 16)


def _codes(x, kind):
    t, top = (torch.float8_e4m3fn, 448.0) if kind == "e4m3" else (torch.float8_e5m2, 57344.0)
    scale = x.float().abs().amax(-1) / top
    return (x.float() / scale[..., None]).clamp(-top, top).to(t).view(torch.uint8), scale


def _layer(c, nb, g):
    """A full layer's K and V: bf16 pages, or FP8 codes and scales of such pages."""
    hkv = c["hkv"]
    if c["layer"] == "full":
        return _randn(g, nb, hkv, PAGE, D), _randn(g, nb, hkv, PAGE, D)
    cb = nb * hkv * PAGE * D
    kp, vp = (torch.empty(nb * hkv * PAGE * (D + 4), dtype=torch.uint8, device=DEV) for _ in range(2))
    for lo in range(0, nb, 4096):
        hi = min(nb, lo + 4096)
        for buf, is_v in ((kp, False), (vp, True)):
            code, scale = _codes(_randn(g, hi - lo, hkv, PAGE, D), c["layer"])
            if is_v:
                buf[:cb].view(nb, hkv, D, PAGE)[lo:hi, :, :, _v_place()] = code.transpose(-1, -2)
            else:
                buf[:cb].view(nb, hkv, PAGE, D)[lo:hi, :, :, _k_place()] = code
            buf[cb:].view(torch.float32).view(nb, hkv, PAGE)[lo:hi] = scale
    return kp, vp


def _tables(n, width, g):
    """Pages of n[i] tokens each, at random places; -1 behind them."""
    pages = [(x + PAGE - 1) // PAGE for x in n]
    ids = torch.randperm(sum(pages), generator=g, device=DEV).int()
    tables = torch.full((len(n), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, p in enumerate(pages):
        tables[i, :p] = ids[at:at + p]
        at += p
    return tables, sum(pages)


def _weights(g, *shape):
    """Accumulated weights as softmax leaves them: a long tail, and keys that got none."""
    x = torch.randn(shape, generator=g, device=DEV).mul_(2.5).exp_().mul_(1e-4)
    return x.mul_(torch.rand(shape, generator=g, device=DEV) > 0.05)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = {"c": c}
    if own:
        import full_attention_kv_gb300 as hsa
        s["hsa"], s["err"] = hsa, i32([0])
    order = random.Random(seed)
    if c["op"] == "weigh":
        n, b, t, hq, hkv = _lengths(c), c["b"], c["t"], c["hq"], c["hkv"]
        s["n"], s["stride"] = n, _stride(n)
        s["tables"], s["nb"] = _tables([x + t for x in n], (max(n) + t + PAGE - 1) // PAGE, g)
        s["kp"], s["vp"] = _layer(c, s["nb"], g)
        # queries that are sharper than noise, as trained ones are
        s["q"] = (torch.randn(b, t, hq, D, generator=g, device=DEV) * 2).bfloat16()
        s["k"], s["v"] = _randn(g, b, t, hkv, D), _randn(g, b, t, hkv, D)
        s["cached"] = i32(n)
        s["prev"] = _weights(g, b, hkv, s["stride"]) if c["prev"] else None
        s["w"], s["out"] = torch.zeros(b, hkv, s["stride"], device=DEV), torch.empty_like(s["q"])
        if own:
            s["pool"] = hsa.DualPool([True], [s["kp"]], [s["vp"]], s["tables"], i32([0] * b), hq, kv_fp8=[c["layer"] if c["layer"] != "full" else None],
                                     Hkv=hkv, d=D, num_blocks=s["nb"])
            s["ws"] = hsa.decode_weights_workspace(s["pool"], b, t, s["stride"])
        return s
    if c["op"] == "prompt":
        (n, m), r, hq, hkv = _lengths(c), c["r"], c["hq"], c["hkv"]
        s["n"], s["m"], s["stride"] = n, m, _stride(n)
        seq = order.sample(range(r), r)  # request i is sequence seq[i]
        tables, s["nb"] = _tables(n, (max(n) + PAGE - 1) // PAGE, g)
        s["tables"] = torch.empty_like(tables)
        s["tables"][seq] = tables
        s["kp"] = _randn(g, s["nb"], hkv, PAGE, D)
        s["q"] = (torch.randn(sum(m), hq, D, generator=g, device=DEV) * 2).bfloat16()
        s["cu"] = i32([sum(m[:i]) for i in range(r + 1)])
        s["len"], s["seq"], s["at"] = i32(n), i32(seq), seq
        s["prev"] = _weights(g, r, hkv, s["stride"]) if c["prev"] else None
        s["w"] = torch.zeros(r, hkv, s["stride"], device=DEV)
        if own:
            s["pool"] = hsa.DualPool([True], [s["kp"]], [s["kp"]], s["tables"], i32([0] * r), hq)
            s["ws"] = hsa.prefill_weights_workspace(s["pool"], r, c["window"])
        return s
    n, r = _lengths(c), c["r"]
    s["n"], s["stride"] = n, _stride(n)
    seq = order.sample(range(r), r)
    s["at"], s["seq"], s["len"] = seq, i32(seq), i32(n)
    if c["op"] == "select":
        s["w"] = _weights(g, r, c["h"], s["stride"])
        s["keep"] = torch.empty(r, c["h"], c["budget"], dtype=torch.int32, device=DEV)
        s["new"] = torch.empty(r, dtype=torch.int32, device=DEV)
        return s
    kept = [min(x, c["budget"]) for x in n]
    dst = [(k + PAGE - 1) // PAGE for k in kept]
    tables, nb = _tables(n, (max(n) + PAGE - 1) // PAGE, g)
    s["tables"] = torch.empty_like(tables)
    s["tables"][seq] = tables
    s["nb"] = nb + sum(dst)
    s["kp"], s["vp"] = _layer(c, s["nb"], g)
    # pages of their own for what stays, in no order
    free = torch.randperm(sum(dst), generator=g, device=DEV).int() + nb
    s["dst"] = torch.full((r, max(dst)), -1, dtype=torch.int32, device=DEV)
    for i, p in enumerate(dst):
        s["dst"][i, :p] = free[sum(dst[:i]):sum(dst[:i]) + p]
    s["keep"] = torch.full((r, c["h"], c["budget"]), -1, dtype=torch.int32, device=DEV)
    for i in range(r):
        pick = torch.rand(c["h"], n[i], generator=g, device=DEV).argsort(-1)[:, :kept[i]].sort(-1).values
        s["keep"][i, :, :kept[i]] = pick.int()
    s["new"], s["kept"] = i32(kept), kept
    s["w"] = _weights(g, r, c["hkv"], s["stride"])
    s["w_out"] = torch.zeros_like(s["w"])
    if own:
        s["pool"] = hsa.DualPool([True], [s["kp"]], [s["vp"]], s["tables"], i32([0] * r), c["hkv"] * 8,
                                 kv_fp8=[c["layer"] if c["layer"] != "full" else None], Hkv=c["hkv"], d=D, num_blocks=s["nb"])
    return s


# ------------------------------------------------------------------------ plain forms

def _rows(s, name, blocks, n, dtype):
    """[hkv, n, D] values of a sequence's first n tokens in a layer's pages."""
    c, buf = s["c"], s[name]
    if c.get("layer", "full") == "full":
        return buf[blocks].to(dtype).transpose(0, 1).reshape(c["hkv"], -1, D)[:, :n]
    nb, hkv = s["nb"], c["hkv"]
    cb = nb * hkv * PAGE * D
    t = torch.float8_e4m3fn if c["layer"] == "e4m3" else torch.float8_e5m2
    scale = buf[cb:].view(torch.float32).view(nb, hkv, PAGE)[blocks].to(dtype)
    if name == "kp":
        code = buf[:cb].view(nb, hkv, PAGE, D)[blocks][..., _k_place()]
    else:
        code = buf[:cb].view(nb, hkv, D, PAGE)[blocks][..., _v_place()].transpose(-1, -2).contiguous()
    x = code.view(t).to(dtype) * scale[..., None]
    return x.transpose(0, 1).reshape(hkv, -1, D)[:, :n]


def _softmax(x):
    x = (x - x.amax(-1, keepdim=True)).exp_()
    return x.div_(x.sum(-1, keepdim=True))


def _weigh_plain(s):
    c = s["c"]
    t, hkv, per = c["t"], c["hkv"], c["hq"] // c["hkv"]
    for i, n in enumerate(s["n"]):
        blocks = s["tables"][i, :(n + PAGE - 1) // PAGE].long()
        k = torch.cat((_rows(s, "kp", blocks, n, torch.float32), s["k"][i].float().transpose(0, 1)), 1)
        v = torch.cat((_rows(s, "vp", blocks, n, torch.float32), s["v"][i].float().transpose(0, 1)), 1)
        q = s["q"][i].float().view(t, hkv, per, D).transpose(0, 1).reshape(hkv, t * per, D)
        x = (q @ k.transpose(-1, -2)).mul_(SCALE)
        step = torch.arange(t, device=DEV).repeat_interleave(per)
        x.masked_fill_(torch.arange(n + t, device=DEV) > n + step[:, None], -math.inf)
        p = _softmax(x)
        s["out"][i] = (p @ v).view(hkv, t, per, D).transpose(0, 1).reshape(t, c["hq"], D).bfloat16()
        w = p.sum(1)
        if c["prev"]:
            w[:, :n] += c["decay"] * s["prev"][i, :, :n]
        s["w"][i, :, :n + t] = w
    return {"out": s["out"], "w": s["w"]}


def _prompt_plain(s):
    c = s["c"]
    hkv, per = c["hkv"], c["hq"] // c["hkv"]
    last = 0
    for n, m, at in zip(s["n"], s["m"], s["at"]):
        last += m
        t = min(c["window"], m)
        k = _rows(s, "kp", s["tables"][at, :(n + PAGE - 1) // PAGE].long(), n, torch.float32)
        q = s["q"][last - t:last].float().view(t, hkv, per, D).transpose(0, 1).reshape(hkv, t * per, D)
        x = (q @ k.transpose(-1, -2)).mul_(SCALE)
        step = torch.arange(t, device=DEV).repeat_interleave(per)
        x.masked_fill_(torch.arange(n, device=DEV) > n - t + step[:, None], -math.inf)
        w = _softmax(x).sum(1)
        if c["prev"]:
            w[:, :n - m] += c["decay"] * s["prev"][at, :, :n - m]
        s["w"][at, :, :n] = w
    return s["w"]


def _select_plain(s):
    c, keep = s["c"], s["keep"]
    keep.fill_(-1)
    for i, n in enumerate(s["n"]):
        if n <= c["budget"]:
            keep[i, :, :n] = torch.arange(n, dtype=torch.int32, device=DEV)
            continue
        x = s["w"][s["at"][i], :, :n]
        best = x.clone()
        for d in range(1, c["reach"] + 1):
            best[:, d:] = torch.maximum(best[:, d:], x[:, :-d])
            best[:, :-d] = torch.maximum(best[:, :-d], x[:, d:])
        best[:, :c["sinks"]] = math.inf
        best[:, n - c["recent"]:] = math.inf
        order = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["budget"]]
        keep[i] = order.sort(-1).values.int()
    torch.clamp(s["len"], max=c["budget"], out=s["new"])
    return {"keep": keep, "new_len": s["new"]}


def _compact_plain(s):
    c = s["c"]
    nb, hkv = s["nb"], c["hkv"]
    heads = torch.arange(hkv, device=DEV)[:, None]
    for i, n in enumerate(s["kept"]):
        at = s["at"][i]
        pos = s["keep"][i, :, :n].long().expand(hkv, n)
        to = torch.arange(n, device=DEV)
        b0, o0 = s["tables"][at][pos // PAGE].long(), pos % PAGE
        b1, o1 = s["dst"][i][to // PAGE].long(), to % PAGE
        if c["layer"] == "full":
            for buf in (s["kp"], s["vp"]):
                buf[b1, heads, o1] = buf[b0, heads, o0]
        else:
            cb = nb * hkv * PAGE * D
            k = s["kp"][:cb].view(nb, hkv, PAGE, D)
            k[b1, heads, o1] = k[b0, heads, o0]
            v = s["vp"][:cb].view(nb, hkv, D, PAGE)
            place = _v_place()
            v[b1, heads, :, place[o1]] = v[b0, heads, :, place[o0]]
            for buf in (s["kp"], s["vp"]):
                sc = buf[cb:].view(torch.float32).view(nb, hkv, PAGE)
                sc[b1, heads, o1] = sc[b0, heads, o0]
        s["w_out"][at, :, :n] = s["w"][at].gather(1, pos)


def _pools(s):
    """The layer's buffers; an FP8 layer's as the values of its codes, in stored order, and the scales."""
    if s["c"]["layer"] == "full":
        return {"k_pool": s["kp"], "v_pool": s["vp"]}
    cb = s["nb"] * s["c"]["hkv"] * PAGE * D
    t = torch.float8_e4m3fn if s["c"]["layer"] == "e4m3" else torch.float8_e5m2
    return {"k_codes": s["kp"][:cb].view(t), "k_scales": s["kp"][cb:].view(torch.float32),
            "v_codes": s["vp"][:cb].view(t), "v_scales": s["vp"][cb:].view(torch.float32)}


def run(state):
    s = state
    c = s["c"]
    if c["op"] == "weigh":
        if not own:
            return _weigh_plain(s)
        s["hsa"].hsa_decode_attn_weights(s["pool"], 0, s["q"], s["k"], s["v"], s["cached"], SCALE, s["w"], w_prev=s["prev"],
                                         decay=c["decay"], out=s["out"], workspace=s["ws"], dev_err=s["err"])
        return {"out": s["out"], "w": s["w"]}
    if c["op"] == "prompt":
        if not own:
            return _prompt_plain(s)
        return s["hsa"].hsa_prefill_weights(s["pool"], 0, s["q"], s["cu"], s["len"], s["seq"], c["window"], SCALE, s["w"],
                                            w_prev=s["prev"], decay=c["decay"], workspace=s["ws"], dev_err=s["err"])
    if c["op"] == "select":
        if not own:
            return _select_plain(s)
        s["hsa"].hsa_kv_select(s["w"], s["len"], s["seq"], c["budget"], sinks=c["sinks"], recent=c["recent"], reach=c["reach"],
                               keep=s["keep"], new_len=s["new"], dev_err=s["err"])
        return {"keep": s["keep"], "new_len": s["new"]}
    if own:
        s["hsa"].hsa_kv_compact(s["pool"], 0, s["keep"], s["new"], s["seq"], s["dst"], w=s["w"], w_dst=s["w_out"], dev_err=s["err"])
    else:
        _compact_plain(s)
    return {**_pools(s), "w": s["w_out"]}


# ------------------------------------------------------------------- values in 64 bits

def _exact_rows(s, name, table, h, lo, hi):
    """Tokens lo .. hi - 1 of one KV head, [hi - lo, D] float64, token by token."""
    c, buf = s["c"], s[name]
    at = torch.arange(lo, hi, device=DEV)
    blk, off = table[at // PAGE].long(), at % PAGE
    if c.get("layer", "full") == "full":
        return buf[blk, h, off].double()
    nb, hkv = s["nb"], c["hkv"]
    t = torch.float8_e4m3fn if c["layer"] == "e4m3" else torch.float8_e5m2
    page = blk * hkv + h
    d = torch.arange(D, device=DEV)
    perm = 4 * ((d % 16 % 8) // 2) + d % 2 + 2 * (d % 16 // 8)
    if name == "kp":
        byte = ((page * PAGE + off) * D)[:, None] + 16 * (d // 16) + perm
    else:
        o = off % 16
        key = 16 * (off // 16) + 4 * ((o % 8) // 2) + o % 2 + 2 * (o // 8)
        byte = (page[:, None] * D + d) * PAGE + key[:, None]
    scale = buf[nb * hkv * PAGE * D:].view(torch.float32)[page * PAGE + off]
    return buf[byte].view(t).double() * scale.double()[:, None]


def _exact_attend(q, k, first):
    """Rows q [rows, D] whose keys are 0 .. first[row]: the weights [rows, n] in 64 bits."""
    x = q.double() @ k.T / math.sqrt(D)
    x = x.masked_fill(torch.arange(k.shape[0], device=DEV) > first[:, None], -math.inf)
    return torch.softmax(x, -1)


def exact(case, seed):
    global own
    c, was = case, own
    own = False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "weigh":
        t, per = c["t"], c["hq"] // c["hkv"]
        out, w = s["out"].double(), s["w"].double()
        for i, n in enumerate(s["n"]):
            for h in range(c["hkv"]):
                k = torch.cat((_exact_rows(s, "kp", s["tables"][i], h, 0, n), s["k"][i, :, h].double()))
                v = torch.cat((_exact_rows(s, "vp", s["tables"][i], h, 0, n), s["v"][i, :, h].double()))
                q = s["q"][i, :, h * per:(h + 1) * per].reshape(t * per, D)
                p = _exact_attend(q, k, n + torch.arange(t * per, device=DEV) // per)
                out[i, :, h * per:(h + 1) * per] = (p @ v).view(t, per, D)
                w[i, h, :n + t] = p.sum(0)
                if c["prev"]:
                    w[i, h, :n] += c["decay"] * s["prev"][i, h, :n].double()
        return {"out": out, "w": w}
    if c["op"] == "prompt":
        per, w, last = c["hq"] // c["hkv"], s["w"].double(), 0
        for n, m, at in zip(s["n"], s["m"], s["at"]):
            last += m
            t = min(c["window"], m)
            for h in range(c["hkv"]):
                k = _exact_rows(s, "kp", s["tables"][at], h, 0, n)
                for lo in range(0, t, 16):
                    hi = min(t, lo + 16)
                    q = s["q"][last - t + lo:last - t + hi, h * per:(h + 1) * per].reshape(-1, D)
                    w[at, h, :n] += _exact_attend(q, k, n - t + lo + torch.arange((hi - lo) * per, device=DEV) // per).sum(0)
                if c["prev"]:
                    w[at, h, :n - m] += c["decay"] * s["prev"][at, h, :n - m].double()
        return w
    if c["op"] == "select":
        keep = torch.full((c["r"], c["h"], c["budget"]), -1, dtype=torch.int32, device=DEV)
        for i, n in enumerate(s["n"]):
            for h in range(c["h"]):
                if n <= c["budget"]:
                    keep[i, h, :n] = torch.arange(n, dtype=torch.int32, device=DEV)
                    continue
                x = s["w"][s["at"][i], h, :n].double()
                pad = torch.full((c["reach"],), -math.inf, dtype=torch.float64, device=DEV)
                x = torch.cat((pad, x, pad)).unfold(0, 2 * c["reach"] + 1, 1).amax(-1)
                lo, hi = c["sinks"], n - c["recent"]
                left = c["budget"] - c["sinks"] - c["recent"]
                stays = torch.ones(n, dtype=torch.bool, device=DEV)
                mid = x[lo:hi]
                if left > 0:  # above the last kept value, and as many equal ones as fit, from the left
                    edge = mid.sort(descending=True).values[left - 1]
                    over = mid > edge
                    equal = mid == edge
                    stays[lo:hi] = over | (equal & (equal.cumsum(0) <= left - over.sum()))
                else:
                    stays[lo:hi] = False
                keep[i, h] = stays.nonzero()[:, 0].int()
        return {"keep": keep, "new_len": torch.tensor([min(x, c["budget"]) for x in s["n"]], dtype=torch.int32, device=DEV)}
    # a move: every stored value in its new place, one head's page at a time
    nb, hkv = s["nb"], c["hkv"]
    got = {k: (v if v.dtype.itemsize == 1 else v.double()) for k, v in _pools(s).items()}
    w = s["w_out"].double()
    cb = nb * hkv * PAGE * D
    d = torch.arange(D, device=DEV)
    for i, n in enumerate(s["kept"]):
        at = s["at"][i]
        for h in range(hkv):
            src = s["keep"][i, h if c["h"] > 1 else 0, :n].long()
            dst = torch.arange(n, device=DEV)
            b0, b1 = s["tables"][at][src // PAGE].long(), s["dst"][i][dst // PAGE].long()
            w[at, h, :n] = s["w"][at, h, src].double()
            if c["layer"] == "full":
                got["k_pool"][b1, h, dst % PAGE] = s["kp"][b0, h, src % PAGE].double()
                got["v_pool"][b1, h, dst % PAGE] = s["vp"][b0, h, src % PAGE].double()
                continue
            p0, p1 = b0 * hkv + h, b1 * hkv + h
            r0, r1 = p0 * PAGE + src % PAGE, p1 * PAGE + dst % PAGE
            got["k_scales"][r1] = s["kp"][cb:].view(torch.float32)[r0].double()
            got["v_scales"][r1] = s["vp"][cb:].view(torch.float32)[r0].double()
            kc, vc = s["kp"][:cb], s["vp"][:cb]
            kc.view(-1, D)[r1] = kc.view(-1, D)[r0]
            byte = [16 * (x % PAGE // 16) + 4 * ((x % 8) // 2) + x % 2 + 2 * (x % 16 // 8) for x in (src, dst)]
            vc[(p1[:, None] * D + d) * PAGE + byte[1][:, None]] = vc[(p0[:, None] * D + d) * PAGE + byte[0][:, None]]
    return {**got, "w": w}
