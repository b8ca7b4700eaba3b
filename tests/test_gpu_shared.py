"""Decode attention over shared prefixes on the GPU, against softmax in 64 bits.

Limits.  A probability is rounded to bf16 once (at most 2^-8 of itself) and so is the
output; a row's sum may take unrounded probabilities.  So a value is off by at most
2^-8 (2 |o| + A), A = sum p |v| / sum p, plus 2^-10 A for fp32 scores (128 products of
bf16 values summed in fp32, below 2^-17 of sum |q k| each way).  Over many values of
zero-mean V the errors are independent: their root mean square, each rounding uniform
with at most 2^-8 / sqrt(3), is below sqrt(2 / 3) 2^-8 of the output's, so 2^-8 holds a
sequence's outputs -- a limit that one lost or doubled key of thousands exceeds."""
import pytest
import torch

import rope_ref

pytestmark = pytest.mark.gpu

D, PAGE, W = 128, 64, 128
SCALE = D ** -0.5


def _hsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import full_attention_kv_gb300 as hsa
    hsa.lib()
    return hsa


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """Pages of a batch whose groups share whole pages; everything else is each one's own."""

    def __init__(self, hsa, members, shared, own, T, hq, hkv, seed=1, sharp=2.0):
        g = _gen(seed)
        self.hsa, self.T, self.hq, self.hkv = hsa, T, hq, hkv
        self.B = sum(members)
        self.members, self.shared = members, shared
        group = [k for k, m in enumerate(members) for _ in range(m)]
        self.cached = [max(0, shared[k] + own[i % len(own)]) for i, k in enumerate(group)]
        whole = [max(0, s) // PAGE for s in shared]
        pages = [(c + T + PAGE - 1) // PAGE for c in self.cached]
        width = max(max(pages), max(whole)) + 1
        nb = sum(whole) + sum(max(0, p - whole[k]) for p, k in zip(pages, group)) + 2
        ids = torch.randperm(nb, generator=g, device="cuda").int().tolist()
        first = {}
        table = [[-1] * width for _ in range(self.B)]
        for i, k in enumerate(group):
            if k not in first:
                first[k] = [ids.pop() for _ in range(whole[k])]
            row = first[k] + [ids.pop() for _ in range(max(0, pages[i] - whole[k]))]
            table[i][:len(row)] = row
        self.spare = ids.pop()
        self.kp = torch.randn(nb, hkv, PAGE, D, generator=g, device="cuda").bfloat16()
        self.vp = torch.randn(nb, hkv, PAGE, D, generator=g, device="cuda").bfloat16()
        self.q = (torch.randn(self.B, T, hq, D, generator=g, device="cuda") * sharp).bfloat16()
        self.k = torch.randn(self.B, T, hkv, D, generator=g, device="cuda").bfloat16()
        self.v = torch.randn(self.B, T, hkv, D, generator=g, device="cuda").bfloat16()
        self.table = _i32(table)
        self.cl = _i32(self.cached)
        self.cu = _i32([sum(members[:i]) for i in range(len(members) + 1)])
        self.sl = _i32(shared)
        self.pool = hsa.DualPool([True], [self.kp], [self.vp], self.table,
                                 torch.zeros(self.B, dtype=torch.int32, device="cuda"), hq)
        self.ws = hsa.decode_shared_workspace(self.pool, self.B, T, len(members))
        self.err = _i32([0])

    def run(self, **kw):
        kw = dict(dict(workspace=self.ws, dev_err=self.err), **kw)
        return self.hsa.hsa_decode_attn_shared(self.pool, 0, self.q, self.k, self.v, self.cl, self.cu,
                                               self.sl, SCALE, **kw)

    def check(self, out, gone=()):
        """gone: physical blocks whose keys are absent."""
        per = self.hq // self.hkv
        nb = self.kp.shape[0]
        for i in range(self.B):
            n = self.cached[i]
            blk = self.table[i, :(n + PAGE - 1) // PAGE].long()
            there = torch.tensor([0 <= int(b) < nb and int(b) not in gone for b in blk], device="cuda",
                                 dtype=torch.bool).repeat_interleave(PAGE)[:n]
            safe = blk.clamp(0, nb - 1)
            k = torch.cat((self.kp[safe].permute(1, 0, 2, 3).reshape(self.hkv, -1, D)[:, :n][:, there],
                           self.k[i].transpose(0, 1)), 1).double()
            v = torch.cat((self.vp[safe].permute(1, 0, 2, 3).reshape(self.hkv, -1, D)[:, :n][:, there],
                           self.v[i].transpose(0, 1)), 1).double()
            m = k.shape[1] - self.T
            q = self.q[i].double().view(self.T, self.hkv, per, D).transpose(0, 1)  # [hkv, T, per, D]
            s = torch.einsum("htgd,hnd->htgn", q, k) * SCALE
            late = torch.arange(k.shape[1], device="cuda") - m > torch.arange(self.T, device="cuda")[:, None]
            p = torch.softmax(s.masked_fill(late[None, :, None], float("-inf")), -1)
            ref = torch.einsum("htgn,hnd->htgd", p, v)
            mag = torch.einsum("htgn,hnd->htgd", p, v.abs())
            got = out[i].double().view(self.T, self.hkv, per, D).transpose(0, 1)
            err = (got - ref).abs()
            lim = 2.0 ** -8 * (2 * ref.abs() + mag) + 2.0 ** -10 * mag
            assert bool((err <= lim).all()), "sequence %d: %g over" % (i, float((err - lim).max()))
            rel = float(err.norm() / ref.norm())
            assert rel <= 2.0 ** -8, "sequence %d of %d cached: %g" % (i, n, rel)


CASES = {
    # members of each group, shared lengths, own lengths (cycled), T, Hq, Hkv
    "one page": ([3], [64], [0, 1, 63], 1, 16, 2),
    "a page and a part": ([4], [130], [0, 1, 62, 70], 1, 32, 4),
    "less than a page": ([3], [63], [0, 5, 200], 1, 16, 2),
    "nothing shared": ([2, 2], [0, 0], [0, 1, 65, 300], 2, 16, 2),
    "odd pages": ([2, 5], [320, 192], [0, 129, 64], 1, 16, 4),
    "singles": ([1, 1, 1], [1000, 64, 129], [3, 0, 64], 1, 32, 4),
    "empty groups": ([0, 2, 0, 0, 3, 0], [500, 640, 64, 0, 200, 9], [10, 0], 1, 16, 2),
    "members that hold less": ([4, 2], [640, 300], [-640, -600, -1, 0, -129, -236], 1, 16, 2),
    "verify": ([9, 2], [700, 2000], [0, 33, 128], 4, 32, 4),
    "three tokens": ([25, 1, 7], [600, 500, 1111], [0, 1, 63, 64, 65], 3, 32, 4),
    "two tokens, pairs of heads": ([70], [400], [7, 0], 2, 8, 4),
    "one head each": ([150, 20], [256, 300], [0, 64, 31], 1, 8, 8),
    "many rows": ([90], [2500], [0, 1, 100, 64], 1, 32, 4),
    "many groups": ([1, 2] * 20 + [0, 3] * 10, [100 + 37 * i for i in range(60)], [0, 10, 70], 1, 16, 2),
    "long": ([3], [20000], [1, 700, 64], 1, 32, 4),
    "long tails": ([2, 1], [128, 640], [9000, 5, 3000], 1, 16, 2),
    "a batch of one": ([1], [5000], [17], 4, 16, 2),
}


@pytest.mark.parametrize("name", CASES)
def test_shared_matches_softmax(name):
    hsa = _hsa()
    c = Case(hsa, *CASES[name], seed=len(name))
    out = c.run()
    assert int(c.err) == 0
    c.check(out)
    # the workspace is as it has to be for the next call, and the result the same
    again = c.run()
    assert torch.equal(out, again)


@pytest.mark.parametrize("max_ctas", [1, 2, 7, 40])
@pytest.mark.parametrize("name", ["odd pages", "three tokens", "many groups", "members that hold less"])
def test_shared_on_few_ctas(name, max_ctas):
    """A CTA that crosses many units, groups and sequences."""
    hsa = _hsa()
    c = Case(hsa, *CASES[name], seed=3)
    c.check(c.run(max_ctas=max_ctas))
    assert int(c.err) == 0


def test_shared_peaked_scores():
    """One key far above the others, in a shared page, an own page or among the new tokens:
    the running maximum is raised late, early and across the merge."""
    hsa = _hsa()
    c = Case(hsa, [6], [1500], [0, 40, 90], 2, 16, 2, seed=9, sharp=0.2)
    first = c.table[0, :1500 // PAGE].long()
    with torch.no_grad():
        for i, where in enumerate([3, 700, 1471, None, None, None]):
            for h in range(2):
                key = c.q[i, 0, 8 * h].float() * 8
                if where is not None:
                    c.kp[first[where // PAGE], h, where % PAGE] = key.bfloat16()
                elif i == 3:
                    c.k[i, 0, h] = key.bfloat16()
                else:
                    at = c.cached[i] - 1
                    c.kp[int(c.table[i, at // PAGE]), h, at % PAGE] = key.bfloat16()
    c.q.mul_(20)
    c.check(c.run())


def test_shared_scores_that_leap():
    """Scores that rise by hundreds from page to page, and fall back: P is never out of
    range, and the maximum of the pages before is given up in time."""
    hsa = _hsa()
    for order in (1, -1):
        c = Case(hsa, [3], [64 * 30], [20], 1, 16, 2, seed=21, sharp=0.0)
        c.q[:] = torch.randn(1, generator=_gen(22), device="cuda").bfloat16().abs() + 1
        for i in range(30):
            level = torch.tensor(float(abs((i * order) % 30 - 7) * 2), device="cuda")
            blk = int(c.table[0, i])
            c.kp[blk] = (torch.randn(2, PAGE, D, generator=_gen(100 + i), device="cuda") * 0.05 + level / 2).bfloat16()
        c.check(c.run())


def test_shared_rows_past_the_end_may_be_nan():
    """Rows of a sequence's last page past its length hold NaN and infinities."""
    hsa = _hsa()
    c = Case(hsa, [4], [200], [1, 50, 63, 129], 1, 32, 4, seed=5)
    for i, n in enumerate(c.cached):
        if n % PAGE:
            blk = int(c.table[i, n // PAGE])
            c.kp[blk, :, n % PAGE:] = float("nan")
            c.vp[blk, :, n % PAGE:] = float("inf")
            c.vp[blk, :, n % PAGE + 1:] = float("nan")
    c.check(c.run())


def test_shared_appends_like_the_append():
    hsa = _hsa()
    for name in ("a page and a part", "three tokens", "members that hold less"):
        c = Case(hsa, *CASES[name], seed=6)
        if name == "members that hold less":  # there the new rows would land in shared pages
            c = Case(hsa, [4, 2], [640, 300], [1, 0, 63, 64], 2, 16, 2, seed=6)
        k0, v0 = c.kp.clone(), c.vp.clone()
        want = c.run()
        assert torch.equal(c.kp, k0) and torch.equal(c.vp, v0)
        got = c.run(append=True)
        assert torch.equal(got, want)
        ref = hsa.DualPool([True], [k0], [v0], c.table, c.pool.ring_row, c.hq)
        T = c.T
        hsa.hsa_kv_append(ref, 0, c.k.view(-1, c.hkv, D), c.v.view(-1, c.hkv, D),
                          _i32([T * i for i in range(c.B + 1)]), _i32(list(range(c.B))), c.cl)
        assert torch.equal(c.kp, k0) and torch.equal(c.vp, v0)
        assert int(c.err) == 0


def test_shared_workspace_serves_the_plain_call():
    """One workspace, the calls in turn: each leaves it as the other wants it."""
    hsa = _hsa()
    c = Case(hsa, *CASES["long tails"], seed=14)
    ws = hsa.decode_workspace(c.pool, c.B, c.T)
    want = hsa.hsa_decode_attn(c.pool, 0, c.q, c.k, c.v, c.cl, SCALE, workspace=ws)
    first = c.run()
    for _ in range(3):
        plain = hsa.hsa_decode_attn(c.pool, 0, c.q, c.k, c.v, c.cl, SCALE, workspace=c.ws)
        assert torch.equal(plain, want)
        assert torch.equal(c.run(), first)
    c.check(first)


def test_shared_offsets_out_of_order_share_nothing():
    hsa = _hsa()
    for bad in ([0, 3, 2, 5], [1, 2, 3, 5], [0, 2, 3, 4], [0, -1, 3, 5], [0, 9, 3, 5]):
        c = Case(hsa, [2, 1, 2], [640, 300, 129], [5, 70], 1, 16, 2, seed=7)
        c.cu = _i32(bad)
        out = c.run()
        assert int(c.err) == hsa.HSA_DEVERR_BAD_LEN
        c.check(out)


def test_shared_lengths_out_of_range():
    hsa = _hsa()
    c = Case(hsa, [2, 1, 2], [640, 300, 129], [5, 70], 1, 16, 2, seed=8)
    c.sl = _i32([640, -5, -2 ** 31])
    out = c.run()
    assert int(c.err) == hsa.HSA_DEVERR_BAD_LEN
    c.check(out)
    # past the block table: a single sequence, so that its own row is what is shared
    c = Case(hsa, [1], [640], [5], 1, 16, 2, seed=8)
    c.sl = _i32([2 ** 31 - 1])
    out = c.run()
    assert int(c.err) & hsa.HSA_DEVERR_BAD_PAGE
    c.check(out)
    # a cached length far past the block table: its pages, and the flag
    c = Case(hsa, [1, 1], [640, 64], [5, 700], 2, 16, 2, seed=8)
    width = c.table.shape[1]
    c.table[:] = torch.arange(width, dtype=torch.int32, device="cuda") % c.kp.shape[0]
    c.cl = _i32([2 ** 31 - 1, c.cached[1]])
    out = c.run()
    assert int(c.err) == hsa.HSA_DEVERR_BAD_PAGE
    c.cached[0] = width * PAGE
    c.check(out)
    # negative cached lengths count as none
    c = Case(hsa, [2], [0], [0], 1, 16, 2, seed=8)
    c.cl = _i32([-7, 0])
    c.check(c.run())


def test_shared_bad_blocks_are_absent():
    """Entries outside the pool, among the shared pages and a sequence's own."""
    hsa = _hsa()
    c = Case(hsa, [3, 2], [640, 450], [5, 130], 1, 16, 2, seed=10)
    c.table[:3, 4] = -1
    c.table[:3, 9] = c.kp.shape[0]
    c.table[3:, 6] = 10 ** 9          # page 6 is the last shared one of an odd count
    c.table[1, 11] = -3
    out = c.run()
    assert int(c.err) == hsa.HSA_DEVERR_BAD_BLOCK
    c.check(out)


def test_shared_on_other_layers_is_the_plain_call():
    hsa = _hsa()
    g = _gen(11)
    B, hq, hkv = 5, 16, 2
    table = _i32([[0, 1, 2], [0, 1, 3], [0, 1, 4], [5, 6, 7], [5, 6, 8]])
    rows = _i32([4, 2, 0, 1, 3])
    q = torch.randn(B, 1, hq, D, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(B, 1, hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    cl = _i32([130, 150, 128, 129, 190])
    cu, sl = _i32([0, 3, 5]), _i32([128, 128])
    for full, fp8 in (([False], False), ([True], "e4m3"), ([True], "e5m2")):
        pool = hsa.DualPool.allocate(full, 9, 5, table, rows, hq, hkv, kv_fp8=fp8)
        kk, vv = (torch.randn(9 * 64, hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        hsa.hsa_kv_append(pool, 0, kk[:558], vv[:558], _i32([0, 190, 380, 558]), _i32([0, 3, 4]), _i32([0, 0, 0]))
        want = hsa.hsa_decode_attn(pool, 0, q, k, v, cl, SCALE)
        ws = hsa.decode_shared_workspace(pool, B, 1, 2)
        assert torch.equal(hsa.hsa_decode_attn_shared(pool, 0, q, k, v, cl, cu, sl, SCALE, workspace=ws), want)
    # no groups: the plain call, on a full layer too
    c = Case(hsa, [3], [300], [4], 1, hq, hkv)
    plain = hsa.hsa_decode_attn(c.pool, 0, c.q, c.k, c.v, c.cl, SCALE)
    got = hsa.hsa_decode_attn_shared(c.pool, 0, c.q, c.k, c.v, c.cl, _i32([0]), c.sl[:0], SCALE, workspace=c.ws)
    assert torch.equal(got, plain)
    # and none of the batch
    assert hsa.hsa_decode_attn_shared(c.pool, 0, c.q[:0], c.k[:0], c.v[:0], c.cl[:0], _i32([0]), c.sl[:0],
                                      SCALE).shape[0] == 0


def test_shared_in_a_graph_and_on_two_streams():
    hsa = _hsa()
    a = Case(hsa, *CASES["verify"], seed=12)
    b = Case(hsa, *CASES["many rows"], seed=13)
    want = a.run(), b.run()
    torch.cuda.synchronize()
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for c, o, s in zip((a, b), outs, streams):
            with torch.cuda.stream(s):
                c.run(out=o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    # a captured call whose lengths and groups change between replays
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(out=outs[0])
    outs[0].zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0])
    a.sl.copy_(_i32([64, 1999]))
    a.cached = [max(0, n - 9) for n in a.cached]
    a.cl.copy_(_i32(a.cached))
    graph.replay()
    torch.cuda.synchronize()
    a.check(outs[0])
    assert int(a.err) == 0


def test_a_run_of_the_operators_together():
    """A prompt of text and an image into a full and a sliding layer, then decode steps of
    five samples of it: rotation, append and shared-prefix attention, step after step,
    against a plain loop that keeps rotated keys in 64 bits."""
    hsa = _hsa()
    g = _gen(20)
    hq, hkv, B, P, steps = 16, 2, 5, 333, 3
    per = hq // hkv
    rope = hsa.Rope(128, base=10000.0, sections=(16, 24, 24))
    inv, ax = list(rope._inv), list(rope._axis)
    whole = P // PAGE
    table = torch.full((B, 8), -1, dtype=torch.int32)
    table[:, :whole] = torch.arange(whole)
    for i in range(B):
        table[i, whole:whole + 2] = torch.tensor([whole + 2 * i, whole + 2 * i + 1])
    pool = hsa.DualPool.allocate([True, False], whole + 2 * B, B, table.cuda(), _i32(list(range(B))), hq, hkv)
    pos = torch.arange(P).repeat(3, 1)
    pos[1, 50:114] = 50 + torch.arange(64) // 8
    pos[2, 50:114] = 50 + torch.arange(64) % 8
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    err = _i32([0])

    def turned(x, p):
        cos, sin = rope_ref.angles(p.tolist(), inv, ax)
        return rope_ref.turn(x, cos, sin, 128, False)[0].cuda()

    def attend(q, keys, vals, window):
        """q [rows, hq, D] at positions n - rows .. n - 1, keys [n, hkv, D], in 64 bits."""
        n, rows = keys.shape[0], q.shape[0]
        s = torch.einsum("rhgd,nhd->hrgn", q.view(rows, hkv, per, D), keys) * SCALE
        at = torch.arange(n - rows, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")
        hide = (key > at) | (key <= at - window)
        p = torch.softmax(s.masked_fill(hide[None, :, None], float("-inf")), -1)
        return torch.einsum("hrgn,nhd->rhgd", p, vals).reshape(rows, hq, D)

    # Rotated q and k are rounded to bf16 before the attention: a score is off by at most
    # 2 * 2^-8 of sum |q_i k_i| scale, here below 0.06 typically far less; outputs of
    # unit-scale values: the limits below hold a wrong position, page or merge, whose
    # error is of the outputs' own size.
    def near(got, ref):
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel <= 0.02, rel

    keys, vals = [[], []], [[], []]
    for layer in range(2):
        window = 10 ** 6 if layer == 0 else W
        qkv = bf(P, hq + 2 * hkv, D)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        pd = pos.int().cuda().contiguous()
        cu, seq, zero = _i32([0, P]), _i32([0]), _i32([0])
        q64, k64, v64 = turned(q, pos), turned(k, pos), v.double()
        if layer == 0:
            qo, ko = hsa.hsa_rope_kv_append(pool, 0, rope, q, k, v, cu, seq, zero, positions=pd, dev_err=err)
        else:
            qo, ko = hsa.hsa_rope(rope, q, k, pd)
        out = hsa.hsa_prefill_attn(pool, layer, qo, ko, v.contiguous(), cu, _i32([0]), seq, P, SCALE, dev_err=err)
        near(out, attend(q64, k64, v64, window))
        if layer == 1:
            for i in range(B):
                hsa.hsa_kv_append(pool, 1, ko, v.contiguous(), cu, _i32([i]), zero, dev_err=err)
        else:  # the part of a page behind the shared ones is each sample's own
            for i in range(1, B):
                hsa.hsa_kv_append(pool, 0, ko[whole * PAGE:].contiguous(), v[whole * PAGE:].contiguous(),
                                  _i32([0, P - whole * PAGE]), _i32([i]), _i32([whole * PAGE]), dev_err=err)
        keys[layer] = [k64] * B
        vals[layer] = [v64] * B
    ws = hsa.decode_shared_workspace(pool, B, 1, 1)
    cu, sl = _i32([0, B]), _i32([P])
    for step in range(steps):
        cl = _i32([P + step] * B)
        at = torch.full((3, B), 60 + step)      # text goes on behind the image's largest position
        for layer in range(2):
            window = 10 ** 6 if layer == 0 else W
            q, k, v = bf(B, hq, D), bf(B, hkv, D), bf(B, hkv, D)
            qo, ko = hsa.hsa_rope(rope, q, k, at.int().cuda())
            out = hsa.hsa_decode_attn_shared(pool, layer, qo[:, None].contiguous(), ko[:, None].contiguous(),
                                             v[:, None].contiguous(), cl, cu, sl, SCALE, workspace=ws,
                                             dev_err=err, append=True)
            q64, k64 = turned(q, at), turned(k, at)
            for i in range(B):
                keys[layer][i] = torch.cat((keys[layer][i], k64[i:i + 1]))
                vals[layer][i] = torch.cat((vals[layer][i], v[i:i + 1].double()))
                near(out[i], attend(q64[i:i + 1], keys[layer][i], vals[layer][i], window))
    assert int(err) == 0


def test_shared_with_a_very_wide_block_table():
    """Room for 2^31 half pages (here 64 rows of 2^21 entries, 8 KV heads): the plain call's
    results, and with one entry less a row the shared kernels' own."""
    hsa = _hsa()
    g = _gen(14)
    B, hq, hkv, wide = 64, 16, 8, 2 ** 21
    q = torch.randn(B, 1, hq, D, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(B, 1, hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    cl = _i32([130 + b for b in range(B)])
    cu, sl = _i32([0, B]), _i32([128])
    outs = {}
    for width in (4, wide - 3, wide):
        table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        table[:, 1] = 1
        table[:, 2] = 2 + torch.arange(B, dtype=torch.int32, device="cuda")
        table[:, 3] = 66 + torch.arange(B, dtype=torch.int32, device="cuda")
        pool = hsa.DualPool.allocate([True], 130, B, table, torch.zeros(B, dtype=torch.int32, device="cuda"), hq, hkv)
        h = _gen(15)
        for t in (pool.k[0], pool.v[0]):
            t.copy_(torch.randn(t.shape, generator=h, device="cuda").bfloat16())
        plain = hsa.hsa_decode_attn(pool, 0, q, k, v, cl, SCALE)
        ws = hsa.decode_shared_workspace(pool, B, 1, 1)
        outs[width] = hsa.hsa_decode_attn_shared(pool, 0, q, k, v, cl, cu, sl, SCALE, workspace=ws)
        if width == wide:
            assert torch.equal(outs[width], plain)
        del table, pool
    assert torch.equal(outs[4], outs[wide - 3])
    assert float((outs[4].float() - outs[wide].float()).abs().max()) < 0.05
