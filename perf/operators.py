"""Rotary positions, the rotating KV append and shared-prefix decode attention: cases,
plain forms and values in 64 bits, for measuring the library's kernels.

Three operators of the dual KV pool's attention path:

  rope     the query and key heads of n tokens turned by their positions on one or
           several axes (time, height, width), pairs split in halves or interleaved
  append   the same rotation on the way into a layer of the pool: pages of a full layer
           (bf16, or FP8 codes with a scale a row) or the ring of a sliding layer
  shared   decode attention of a batch whose groups of sequences share their first pages

Sizes are this library's own: 32 query heads over 4 KV heads (and the small 16 over 2),
head size 128, 64-token pages, a window of 128.
"""
import math
import random

import torch

own = False

D, PAGE, W = 128, 64, 128
BASE = 1.0e6
DEV = "cuda"


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token for each of 32 sequences, before a sliding layer's attention
        dict(name="rope step", op="rope", n=32, hq=32, hkv=4, rot=128, axes=1, pairs="half", fused=True, lens=1),
        # a small model's text, half of each head rotated, pairs side by side
        dict(name="rope partial", op="rope", n=1777, hq=16, hkv=2, rot=64, axes=1, pairs="interleaved", fused=False, lens=2),
        # a long prompt with images and video, q and k taken out of the QKV projection's rows
        dict(name="rope video", op="rope", n=20011, hq=32, hkv=4, rot=128, axes=3, pairs="half", fused=True, lens=3),
        # one decode step of 32 sequences into a full layer
        dict(name="append step", op="append", layer="full", r=32, lo=1, hi=1, hq=32, hkv=4, rot=128, axes=1, pairs="half", fused=True, lens=4),
        # prompts of odd lengths into a sliding layer: only the last 128 tokens of each stay
        dict(name="append ring", op="append", layer="ring", r=9, lo=1, hi=1500, hq=32, hkv=4, rot=128, axes=1, pairs="half", fused=True, lens=5),
        # chunks of prompts with images into an FP8 layer
        dict(name="append fp8", op="append", layer="e4m3", r=4, lo=700, hi=2500, hq=32, hkv=4, rot=128, axes=3, pairs="half", fused=True, lens=6),
        # eight chunks of 2K to 8K tokens into a full layer
        dict(name="append chunks", op="append", layer="full", r=8, lo=2048, hi=8192, hq=32, hkv=4, rot=128, axes=1, pairs="half", fused=True, lens=7),
        # a handful of samples of one short prompt
        dict(name="shared few", op="shared", b=4, t=1, groups=1, plo=2048, phi=2048, slo=1, shi=200, hq=16, hkv=2, lens=8),
        # 32 conversations on one long system prompt
        dict(name="shared decode", op="shared", b=32, t=1, groups=1, plo=32768, phi=32768, slo=64, shi=4096, hq=32, hkv=4, lens=9),
        # three prompts' candidates, four tokens to verify for each sequence
        dict(name="shared verify", op="shared", b=48, t=4, groups=3, plo=5000, phi=17000, slo=0, shi=1000, hq=32, hkv=4, lens=10),
        # many questions on one document
        dict(name="shared document", op="shared", b=128, t=1, groups=1, plo=65600, phi=65600, slo=1, shi=1024, hq=32, hkv=4, lens=11),
        # pairs and triples, each on a document of its own
        dict(name="shared pairs", op="shared", b=32, t=1, groups=12, plo=1000, phi=40000, slo=0, shi=600, hq=32, hkv=4, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice([(32, 4), (32, 4), (16, 2), (16, 4), (8, 8)])
    lens = rng.randrange(100, 1 << 30)
    op = rng.choice(["rope", "append", "shared", "shared"])
    turn = dict(rot=rng.choice([128, 128, 64, 96, 32]), axes=rng.choice([1, 1, 2, 3]),
                pairs=rng.choice(["half", "half", "interleaved"]), fused=rng.random() < 0.6)
    if op == "rope":
        return dict(op=op, n=_log(rng, 1, 20000), hq=hq, hkv=hkv, lens=lens, **turn)
    if op == "append":
        layer = rng.choice(["full", "full", "ring", "e4m3", "e5m2"])
        r = _log(rng, 1, 32)
        hi = _log(rng, 1, (6000 if layer in ("e4m3", "e5m2") else 30000) // r)
        return dict(op=op, layer=layer, r=r, lo=max(1, hi // rng.choice([1, 2, 10])), hi=hi, hq=hq, hkv=hkv, lens=lens, **turn)
    t = rng.choice([1, 1, 1, 2, 3, 4])
    b = _log(rng, 2, 128 // t)
    groups = rng.choice([1, 1, max(1, b // 2), max(1, b // 7)])
    phi = _log(rng, 500, min(64000, 110000 // groups))
    return dict(op=op, b=b, t=t, groups=groups, plo=max(1, phi // rng.choice([1, 1, 4])), phi=phi,
                slo=rng.choice([0, 1, 64]), shi=_log(rng, 64, 1000), hq=hq, hkv=hkv, lens=lens)


def _lengths(c):
    """The token counts of a case: they follow from the case alone."""
    rng = random.Random(c["lens"])
    if c["op"] == "append":
        return [rng.randint(c["lo"], c["hi"]) for _ in range(c["r"])], [rng.randint(0, 60000) for _ in range(c["r"])]
    cut = sorted(rng.sample(range(1, c["b"]), c["groups"] - 1)) if c["groups"] > 1 else []
    cu = [0] + cut + [c["b"]]
    prefix = [rng.randint(c["plo"], c["phi"]) for _ in range(c["groups"])]
    suffix = [rng.randint(c["slo"], c["shi"]) for _ in range(c["b"])]
    return cu, prefix, suffix


def work(case):
    c = case
    qb, kb = c["hq"] * D * 2, c["hkv"] * D * 2
    if c["op"] == "rope":
        pairs = c["n"] * (c["hq"] + c["hkv"]) * c["rot"] / 2
        return {"bytes": c["n"] * (2 * (qb + kb) + 4 * c["axes"]), "flops": 6 * pairs}
    if c["op"] == "append":
        new, _ = _lengths(c)
        n = sum(new)
        kept = sum(min(x, W) for x in new) if c["layer"] == "ring" else n
        row = c["hkv"] * (D + 4) if c["layer"] in ("e4m3", "e5m2") else kb
        vread = kept * kb  # values that the ring drops need not be read
        return {"bytes": n * (2 * qb + 2 * kb + 4 * c["axes"]) + vread + 2 * kept * row,
                "flops": 6 * n * (c["hq"] + c["hkv"]) * c["rot"] / 2}
    cu, prefix, suffix = _lengths(c)
    keys = pairs = 0
    for g, p in enumerate(prefix):
        keys += p // PAGE * PAGE
        for s in suffix[cu[g]:cu[g + 1]]:
            keys += p % PAGE + s + c["t"]
            pairs += c["t"] * (p + s) + c["t"] * (c["t"] + 1) // 2
    return {"bytes": keys * 2 * kb + 2 * c["b"] * c["t"] * qb, "flops": 4 * pairs * c["hq"] * D}


# ----------------------------------------------------------------------------- inputs

def _inv_freq(c):
    return [BASE ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)]


def _axis_of_pair(c):
    """One axis: all pairs on it.  Two and three: sections of the pairs, the first axis
    (time) on the fast ones, as the pairs go."""
    h = c["rot"] // 2
    if c["axes"] == 1:
        return [0] * h
    a = h // 4
    cut = [a, h] if c["axes"] == 2 else [a, a + (h - a) // 2, h]
    return [next(k for k, e in enumerate(cut) if i < e) for i in range(h)]


def _positions(c, start, g):
    """[axes, n] int32.  Several axes: text whose axes agree, and grids of height x width
    whose time stands still or goes on with the frame."""
    n = len(start)
    pos = torch.tensor(start, dtype=torch.int32, device=DEV).repeat(c["axes"], 1)
    if c["axes"] > 1:
        i = torch.arange(n, device=DEV)
        image = (i // 640) % 3 != 0
        at = i % 640
        grid = [at // 320, (at % 320) // 20, at % 20]
        base = pos[0].long() - at
        for a in range(c["axes"]):
            pos[a] = torch.where(image, base + grid[a], pos[a].long()).int()
    return pos


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).bfloat16()


def _heads(c, n, g):
    """q, k, v of n tokens: slices of the QKV projection's rows, or tensors of their own."""
    hq, hkv = c["hq"], c["hkv"]
    if c["fused"]:
        qkv = _randn(g, n, hq + 2 * hkv, D)
        return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    return _randn(g, n, hq, D), _randn(g, n, hkv, D), _randn(g, n, hkv, D)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = {"c": c}
    if c["op"] == "rope":
        s["q"], s["k"], _ = _heads(c, c["n"], g)
        first = random.Random(seed).randint(0, 100000)
        s["pos"] = _positions(c, list(range(first, first + c["n"])), g)
        if c["n"] <= 64:  # a decode step: every token is at a position of its own
            s["pos"] = torch.randint(0, 130000, (1, c["n"]), generator=g, device=DEV, dtype=torch.int32).repeat(c["axes"], 1)
        s["inv"] = torch.tensor(_inv_freq(c), dtype=torch.float64, device=DEV)
        s["axis"] = torch.tensor(_axis_of_pair(c), device=DEV)
        s["q_out"] = torch.empty(c["n"], c["hq"], D, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty(c["n"], c["hkv"], D, dtype=torch.bfloat16, device=DEV)
        if own:
            import full_attention_kv_gb300 as hsa
            s["hsa"] = hsa
            s["rope"] = hsa.Rope(c["rot"], inv_freq=_inv_freq(c), axis_of_pair=_axis_of_pair(c), interleaved=c["pairs"] == "interleaved")
        return s
    if c["op"] == "append":
        new, start = _lengths(c)
        n, r = sum(new), c["r"]
        s["q"], s["k"], s["v"] = _heads(c, n, g)
        cache = [a + i for a, k in zip(start, new) for i in range(k)]
        s["pos"] = _positions(c, cache, g)
        s["cu"], s["seq"], s["start"] = i32([sum(new[:i]) for i in range(r + 1)]), i32(random.Random(seed).sample(range(r), r)), i32(start)
        s["inv"] = torch.tensor(_inv_freq(c), dtype=torch.float64, device=DEV)
        s["axis"] = torch.tensor(_axis_of_pair(c), device=DEV)
        # pages of the tokens that are appended; the earlier ones are not looked at
        first = [a // PAGE for a in start]
        last = [(a + k - 1) // PAGE for a, k in zip(start, new)]
        s["nb"] = sum(b - a + 1 for a, b in zip(first, last))
        ids = torch.randperm(s["nb"], generator=g, device=DEV).int()
        s["tables"] = torch.full((r, max(last) + 1), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, q in enumerate(s["seq"].tolist()):
            k = last[i] - first[i] + 1
            s["tables"][q, first[i]:last[i] + 1] = ids[at:at + k]
            at += k
        s["rows"] = torch.randperm(r, generator=g, device=DEV).int()
        hkv = c["hkv"]
        if c["layer"] == "ring":
            s["kp"], s["vp"] = _randn(g, r, hkv, W, D), _randn(g, r, hkv, W, D)
        elif c["layer"] == "full":
            s["kp"], s["vp"] = _randn(g, s["nb"], hkv, PAGE, D), _randn(g, s["nb"], hkv, PAGE, D)
        else:
            size = s["nb"] * hkv * PAGE * (D + 4)
            s["kp"], s["vp"] = (torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in range(2))
        s["q_out"] = torch.empty(n, c["hq"], D, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty(n, hkv, D, dtype=torch.bfloat16, device=DEV)
        if own:
            import full_attention_kv_gb300 as hsa
            s["hsa"] = hsa
            s["rope"] = hsa.Rope(c["rot"], inv_freq=_inv_freq(c), axis_of_pair=_axis_of_pair(c), interleaved=c["pairs"] == "interleaved")
            fp8 = c["layer"] if c["layer"] in ("e4m3", "e5m2") else False
            s["pool"] = hsa.DualPool([c["layer"] != "ring"], [s["kp"]], [s["vp"]], s["tables"], s["rows"], c["hq"], W=W, page=PAGE,
                                     kv_fp8=[fp8], Hkv=hkv, d=D, num_blocks=s["nb"])
            s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    cu, prefix, suffix = _lengths(c)
    b, t, hq, hkv = c["b"], c["t"], c["hq"], c["hkv"]
    cached = [prefix[k] + suffix[i] for k in range(c["groups"]) for i in range(cu[k], cu[k + 1])]
    # a group's whole shared pages are held once; what follows is each sequence's own
    whole = [p // PAGE for p in prefix]
    pages = [(n + t + PAGE - 1) // PAGE for n in cached]
    nb = sum(whole) + sum(pages[i] - whole[k] for k in range(c["groups"]) for i in range(cu[k], cu[k + 1]))
    ids = torch.randperm(nb, generator=g, device=DEV).int()
    tables = torch.full((b, max(pages)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for k in range(c["groups"]):
        tables[cu[k]:cu[k + 1], :whole[k]] = ids[at:at + whole[k]]
        at += whole[k]
        for i in range(cu[k], cu[k + 1]):
            m = pages[i] - whole[k]
            tables[i, whole[k]:pages[i]] = ids[at:at + m]
            at += m
    s["kp"], s["vp"] = _randn(g, nb, hkv, PAGE, D), _randn(g, nb, hkv, PAGE, D)
    # queries that are sharper than noise, as trained ones are
    s["q"] = (torch.randn(b, t, hq, D, generator=g, device=DEV) * 2).bfloat16()
    s["k"], s["v"] = _randn(g, b, t, hkv, D), _randn(g, b, t, hkv, D)
    s["tables"], s["cached"], s["cu"], s["shared"] = tables, i32(cached), i32(cu), i32(prefix)
    s["sizes"] = (cu, prefix, cached)
    # the plain form's view: the padded member list of each group
    most = max(cu[k + 1] - cu[k] for k in range(c["groups"]))
    s["member"] = torch.tensor([[min(cu[k] + j, cu[k + 1] - 1) for j in range(most)] for k in range(c["groups"])], device=DEV)
    s["group"] = torch.tensor([k for k in range(c["groups"]) for _ in range(cu[k], cu[k + 1])], device=DEV)
    s["slot"] = torch.tensor([i - cu[k] for k in range(c["groups"]) for i in range(cu[k], cu[k + 1])], device=DEV)
    s["whole"] = torch.tensor(whole, device=DEV)
    s["tail"] = max(0, max((cached[i] + PAGE - 1) // PAGE - whole[k] for k in range(c["groups"]) for i in range(cu[k], cu[k + 1])))
    s["out"] = torch.empty_like(s["q"])
    if own:
        import full_attention_kv_gb300 as hsa
        s["hsa"] = hsa
        rows = torch.zeros(b, dtype=torch.int32, device=DEV)
        s["pool"] = hsa.DualPool([True], [s["kp"]], [s["vp"]], tables, rows, hq, W=W, page=PAGE)
        s["ws"] = hsa.decode_shared_workspace(s["pool"], b, t, c["groups"])
        s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------------ plain forms

def _turn(x, pos, inv, axis, pairs, rot):
    """x [n, heads, D] in 32 bits, its first `rot` values turned.  Angles in 64 bits:
    far positions lose too much in 32."""
    angle = pos[axis].T.double() * inv
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    y = x.clone()
    if pairs == "half":
        a, b = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        a, b = slice(0, rot, 2), slice(1, rot, 2)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _perm16():
    return torch.tensor([4 * ((l % 8) // 2) + l % 2 + 2 * (l // 8) for l in range(16)], device=DEV)


def _codes(x, kind):
    """Rows of 32-bit values as FP8 codes (bytes) and a scale each."""
    t, top = (torch.float8_e4m3fn, 448.0) if kind == "e4m3" else (torch.float8_e5m2, 57344.0)
    scale = x.abs().amax(-1) / top
    y = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x)).clamp(-top, top)
    return y.to(t).view(torch.uint8), scale


def _append_plain(s, k32):
    c, n = s["c"], s["q"].shape[0]
    counts = (s["cu"][1:] - s["cu"][:-1]).long()
    r = torch.repeat_interleave(torch.arange(c["r"], device=DEV), counts, output_size=n)
    i = torch.arange(n, device=DEV) - s["cu"][r]
    at, seq = (s["start"][r] + i).long(), s["seq"][r].long()
    if c["layer"] == "ring":
        keep = (i >= counts[r] - W).nonzero()[:, 0]
        row, slot = s["rows"][seq[keep]].long(), at[keep] % W
        s["kp"][row, :, slot] = k32[keep].bfloat16()
        s["vp"][row, :, slot] = s["v"][keep]
        return s["kp"], s["vp"]
    block, off = s["tables"][seq, at // PAGE].long(), at % PAGE
    if c["layer"] == "full":
        s["kp"][block, :, off] = k32.bfloat16()
        s["vp"][block, :, off] = s["v"]
        return s["kp"], s["vp"]
    nb, hkv, cb = s["nb"], c["hkv"], s["nb"] * c["hkv"] * PAGE * D
    place = (16 * (torch.arange(D, device=DEV) // 16) + _perm16().repeat(D // 16))
    kc, ks = _codes(k32, c["layer"])
    vc, vs = _codes(s["v"].float(), c["layer"])
    stored = torch.empty_like(kc)
    stored[..., place] = kc
    s["kp"][:cb].view(nb, hkv, PAGE, D)[block, :, off] = stored
    s["kp"][cb:].view(torch.float32).view(nb, hkv, PAGE)[block, :, off] = ks
    byte = 16 * (off // 16) + _perm16()[off % 16]
    s["vp"][:cb].view(nb, hkv, D, PAGE)[block, :, :, byte] = vc
    s["vp"][cb:].view(torch.float32).view(nb, hkv, PAGE)[block, :, off] = vs
    return s["kp"], s["vp"]


def _shared_plain(s):
    c = s["c"]
    b, t, hq, hkv = c["b"], c["t"], c["hq"], c["hkv"]
    per, scale = hq // hkv, D ** -0.5
    groups, most = s["member"].shape
    # [b, hkv, t * per, D]
    q = s["q"].float().view(b, t, hkv, per, D).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * per, D)
    step = torch.arange(t, device=DEV).repeat_interleave(per)
    # the shared pages, once for a group
    wide = int(s["tables"].shape[1]) - 1
    np_ = max(p // PAGE for p in s["sizes"][1])
    page = s["tables"][s["member"][:, 0]][:, :np_].long()
    page = torch.where(torch.arange(np_, device=DEV) < s["whole"][:, None], page, torch.zeros_like(page))
    ks = s["kp"][page].float().permute(0, 2, 1, 3, 4).reshape(groups, hkv, np_ * PAGE, D)
    vs = s["vp"][page].float().permute(0, 2, 1, 3, 4).reshape(groups, hkv, np_ * PAGE, D)
    qg = q[s["member"]].permute(0, 2, 1, 3, 4).reshape(groups, hkv, most * t * per, D)
    s1 = (qg @ ks.transpose(-1, -2)).mul_(scale)
    seen = torch.arange(np_ * PAGE, device=DEV) < (s["whole"] * PAGE)[:, None]
    s1.masked_fill_(~seen[:, None, None], -math.inf)
    m1 = s1.amax(-1) if np_ else torch.full(s1.shape[:-1], -math.inf, device=DEV)
    p1 = s1.sub_(torch.where(m1 > -math.inf, m1, 0)[..., None]).exp_()
    l1, o1 = p1.sum(-1), p1 @ vs
    back = lambda x: x.reshape(groups, hkv, most, t * per, -1).permute(0, 2, 1, 3, 4)[s["group"], s["slot"]]  # noqa: E731
    m1, l1, o1 = back(m1)[..., 0], back(l1)[..., 0], back(o1)
    # each sequence's own pages
    first = s["whole"][s["group"]]
    at = first[:, None] + torch.arange(s["tail"], device=DEV)
    page = s["tables"].gather(1, at.clamp(max=wide)).long().clamp(min=0)
    ku = s["kp"][page].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, s["tail"] * PAGE, D)
    vu = s["vp"][page].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, s["tail"] * PAGE, D)
    s2 = (q @ ku.transpose(-1, -2)) * scale
    where = first[:, None] * PAGE + torch.arange(s["tail"] * PAGE, device=DEV)
    s2 = s2.masked_fill((where >= s["cached"][:, None])[:, None, None], -math.inf)
    kn, vn = s["k"].float().permute(0, 2, 1, 3), s["v"].float().permute(0, 2, 1, 3)
    s3 = (q @ kn.transpose(-1, -2)) * scale
    s3 = s3.masked_fill(torch.arange(t, device=DEV) > step[:, None], -math.inf)
    s23, v23 = torch.cat((s2, s3), -1), torch.cat((vu, vn), -2)
    m2 = s23.amax(-1)
    p2 = (s23 - m2[..., None]).exp()
    l2, o2 = p2.sum(-1), p2 @ v23
    m = torch.maximum(m1, m2)
    a1, a2 = (m1 - m).exp(), (m2 - m).exp()
    o = (o1 * a1[..., None] + o2 * a2[..., None]) / (l1 * a1 + l2 * a2)[..., None]
    return o.view(b, hkv, t, per, D).permute(0, 2, 1, 3, 4).reshape(b, t, hq, D).bfloat16()


def _fp8_views(s):
    """The FP8 layer's buffers as the values of their codes, in stored order, and the scales."""
    cb = s["nb"] * s["c"]["hkv"] * PAGE * D
    t = torch.float8_e4m3fn if s["c"]["layer"] == "e4m3" else torch.float8_e5m2
    return {"k_codes": s["kp"][:cb].view(t), "k_scales": s["kp"][cb:].view(torch.float32),
            "v_codes": s["vp"][:cb].view(t), "v_scales": s["vp"][cb:].view(torch.float32)}


def run(state):
    s = state
    c = s["c"]
    if c["op"] == "rope":
        if own:
            s["hsa"].hsa_rope(s["rope"], s["q"], s["k"], s["pos"], q_out=s["q_out"], k_out=s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        return {n: _turn(s[n], s["pos"], s["inv"], s["axis"], c["pairs"], c["rot"]).bfloat16() for n in ("q", "k")}
    if c["op"] == "append":
        if own:
            s["hsa"].hsa_rope_kv_append(s["pool"], 0, s["rope"], s["q"], s["k"], s["v"], s["cu"], s["seq"], s["start"], positions=s["pos"],
                                        q_out=s["q_out"], k_out=s["k_out"], dev_err=s["err"])
            got = {"q": s["q_out"], "k": s["k_out"]}
        else:
            q32, k32 = (_turn(s[n], s["pos"], s["inv"], s["axis"], c["pairs"], c["rot"]) for n in ("q", "k"))
            got = {"q": q32.bfloat16(), "k": k32.bfloat16()}
            _append_plain(s, k32)
        if c["layer"] in ("e4m3", "e5m2"):
            return {**got, **_fp8_views(s)}
        return {**got, "k_pool": s["kp"], "v_pool": s["vp"]}
    if own:
        s["hsa"].hsa_decode_attn_shared(s["pool"], 0, s["q"], s["k"], s["v"], s["cached"], s["cu"], s["shared"], D ** -0.5, out=s["out"],
                                        workspace=s["ws"], dev_err=s["err"])
        return s["out"]
    return _shared_plain(s)


# ------------------------------------------------------------------- values in 64 bits

def _exact_turn(x, pos, c):
    """Pair i of a head is the complex number x[a_i] + i x[b_i], times exp(i angle)."""
    h = c["rot"] // 2
    inv = torch.tensor([BASE ** (-2.0 * i / c["rot"]) for i in range(h)], dtype=torch.float64, device=DEV)
    angle = torch.stack([pos[a].double() for a in _axis_of_pair(c)], 1) * inv
    x = x.double()
    head = x[..., :c["rot"]]
    two = head.unflatten(-1, (2, h)).transpose(-1, -2) if c["pairs"] == "half" else head.unflatten(-1, (h, 2))
    z = torch.view_as_complex(two.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    two = torch.view_as_real(z)
    head = (two.transpose(-1, -2) if c["pairs"] == "half" else two).flatten(-2)
    return torch.cat((head, x[..., c["rot"]:]), -1)


def exact(case, seed):
    global own
    c, was = case, own
    own = False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "rope":
        return {n: _exact_turn(s[n], s["pos"], c) for n in ("q", "k")}
    if c["op"] == "append":
        q, k, v = _exact_turn(s["q"], s["pos"], c), _exact_turn(s["k"], s["pos"], c), s["v"].double()
        got = {"q": q, "k": k}
        cu, seq, start = s["cu"].tolist(), s["seq"].tolist(), s["start"].tolist()
        if c["layer"] in ("full", "ring"):
            kp, vp = s["kp"].double(), s["vp"].double()
            for r in range(c["r"]):
                for lo in range(cu[r], cu[r + 1], 4096):
                    i = torch.arange(lo, min(lo + 4096, cu[r + 1]), device=DEV)
                    at = start[r] + i - cu[r]
                    if c["layer"] == "ring":
                        i, at = i[i >= cu[r + 1] - W], at[i >= cu[r + 1] - W]
                        kp[int(s["rows"][seq[r]]), :, at % W] = k[i].transpose(0, 1)
                        vp[int(s["rows"][seq[r]]), :, at % W] = v[i].transpose(0, 1)
                    else:
                        blk = s["tables"][seq[r]][at // PAGE].long()
                        kp[blk, :, at % PAGE] = k[i]
                        vp[blk, :, at % PAGE] = v[i]
            return {**got, "k_pool": kp, "v_pool": vp}
        # scales alone: a code is the nearest of a grid, which 64 bits do not make finer
        top = 448.0 if c["layer"] == "e4m3" else 57344.0
        for name, x in (("k_scales", k), ("v_scales", v)):
            sc = torch.zeros(s["nb"], c["hkv"], PAGE, dtype=torch.float64, device=DEV)
            for r in range(c["r"]):
                at = start[r] + torch.arange(cu[r + 1] - cu[r], device=DEV)
                sc[s["tables"][seq[r]][at // PAGE].long(), :, at % PAGE] = x[cu[r]:cu[r + 1]].abs().amax(-1) / top
            got[name] = sc.flatten()
        return {**got, "k_codes": None, "v_codes": None}
    cu, prefix, cached = s["sizes"]
    per = c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for i in range(c["b"]):
        n = cached[i]
        blk = s["tables"][i, :(n + PAGE - 1) // PAGE].long()
        for h in range(c["hkv"]):
            k = torch.cat((s["kp"][blk, h].reshape(-1, D)[:n], s["k"][i, :, h])).double()
            v = torch.cat((s["vp"][blk, h].reshape(-1, D)[:n], s["v"][i, :, h])).double()
            for j in range(c["t"]):
                x = s["q"][i, j, h * per:(h + 1) * per].double() @ k[:n + j + 1].T / math.sqrt(D)
                out[i, j, h * per:(h + 1) * per] = torch.softmax(x, -1) @ v[:n + j + 1]
    return out
