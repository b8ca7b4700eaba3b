"""Decode attention that weighs its keys, on the GPU, against softmax in 64 bits.

Limits.  A score is 128 products of bf16 (FP8: fp16) values, exact, summed in fp32: off by at
most 128 2^-24 = 2^-17 of mag = scale sum |q k|, and by 2^-22 of itself for the scale's factor
and the exponential's argument.  A weight's relative error is its own score's and its lse's,
which is no more off than the worst score: at most 2^-16 (mag_max + 1) of it, mag_max over the
row's keys; sums over 32 rows and the decayed old weight add 2^-20 of what they sum.  Over a
sequence's weights the roundings are independent: sqrt(128) 2^-24 mag, under 2^-20 mag_max of the
weights' norm.  The output's limits are
those of the shared-prefix tests: P and the output round to bf16 once each."""
import pytest
import torch

import evict_ref as ref

pytestmark = pytest.mark.gpu

D, PAGE = 128, 64
SCALE = D ** -0.5


def _hsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import full_attention_kv_gb300 as hsa
    hsa.lib()
    return hsa


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _perm(n):
    l = torch.arange(n, device="cuda")
    return 16 * (l // 16) + 4 * ((l % 8) // 2) + l % 2 + 2 * (l % 16 // 8)


class Step:
    """Sequences of `cached` tokens in pages of random order, T new ones each."""

    def __init__(self, hsa, cached, T, hq, hkv, fmt=None, seed=1, prev=True, decay=0.75, garbage=float("nan"), extra=5,
                 vmag=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.hsa, self.cached, self.T, self.hq, self.hkv, self.fmt, self.decay = hsa, cached, T, hq, hkv, fmt, decay
        B = self.B = len(cached)
        pages = [(max(0, c) + T + PAGE - 1) // PAGE for c in cached]
        self.nb = sum(pages) + 1
        ids = torch.randperm(self.nb, generator=g, device="cuda").int().tolist()
        table = [[ids.pop() for _ in range(p)] + [-1] * (max(pages) + 1 - p) for p in pages]
        self.table = _i32(table)
        k = torch.randn(self.nb, hkv, PAGE, D, generator=g, device="cuda").bfloat16()
        v = torch.randn(self.nb, hkv, PAGE, D, generator=g, device="cuda").bfloat16()
        if vmag is not None:  # of position j, and of the new tokens
            for i, c in enumerate(cached):
                for j, block in enumerate(table[i][:pages[i]]):
                    v[block] *= vmag(torch.arange(j * PAGE, j * PAGE + PAGE, device="cuda"))[:, None]
        if fmt is None:
            self.bufs, self.values = (k, v), (k, v)
        else:
            self._quantise(k, v)
        # what lies behind a sequence's tokens, and in pages of no sequence, must not show
        for i, c in enumerate(cached):
            if garbage is not None:
                self._spoil(table[i][max(0, c) // PAGE] if max(0, c) // PAGE < pages[i] else -1, max(0, c) % PAGE, garbage)
        if garbage is not None:
            self._spoil(ids.pop(), 0, garbage)
        self.q = (torch.randn(B, T, hq, D, generator=g, device="cuda") * 2).bfloat16()
        self.k = torch.randn(B, T, hkv, D, generator=g, device="cuda").bfloat16()
        self.v = torch.randn(B, T, hkv, D, generator=g, device="cuda").bfloat16()
        if vmag is not None:
            for i, c in enumerate(cached):
                self.v[i] *= vmag(torch.arange(c, c + T, device="cuda"))[:, None, None]
        self.stride = (max(max(cached), 0) + T + extra + 3) // 4 * 4
        self.prev = torch.rand(B, hkv, self.stride, generator=g, device="cuda") if prev else None
        if prev:
            for i, c in enumerate(cached):
                self.prev[i, :, max(0, c):] = float("nan")  # new positions count nothing from it
        self.w = torch.full((B, hkv, self.stride), -7.0, device="cuda")
        self.err = _i32([0])
        self.cl = _i32(cached)
        self.pool = hsa.DualPool([True], [self.bufs[0]], [self.bufs[1]], self.table, _i32([0] * B), hq, kv_fp8=[fmt], Hkv=hkv, d=D,
                                 num_blocks=self.nb)
        self.ws = hsa.decode_weights_workspace(self.pool, B, T, self.stride).fill_(255)

    def _quantise(self, k, v):
        t, top = (torch.float8_e4m3fn, 448.0) if self.fmt == "e4m3" else (torch.float8_e5m2, 57344.0)
        cb = self.nb * self.hkv * PAGE * D
        bufs, values = [], []
        for x, is_v in ((k, False), (v, True)):
            scale = x.float().abs().amax(-1) / top
            code = (x.float() / scale[..., None]).nan_to_num(0.0).clamp(-top, top).to(t)
            buf = torch.empty(self.nb * self.hkv * PAGE * (D + 4), dtype=torch.uint8, device="cuda")
            if is_v:
                buf[:cb].view(self.nb, self.hkv, D, PAGE)[..., _perm(PAGE)] = code.view(torch.uint8).transpose(-1, -2)
            else:
                buf[:cb].view(self.nb, self.hkv, PAGE, D)[..., _perm(D)] = code.view(torch.uint8)
            buf[cb:].view(torch.float32).view(self.nb, self.hkv, PAGE)[:] = scale
            bufs.append(buf)
            values.append(code.double() * scale.double()[..., None])
        self.bufs, self.values = tuple(bufs), tuple(values)

    def _spoil(self, block, row, garbage):
        if block < 0:
            return
        if self.fmt is None:
            for b in self.bufs:
                b[block, :, row:] = garbage
            return
        cb = self.nb * self.hkv * PAGE * D
        self.bufs[0][:cb].view(self.nb, self.hkv, PAGE, D)[block, :, row:] = 127  # NaN in both formats
        self.bufs[1][:cb].view(self.nb, self.hkv, D, PAGE)[block][..., _perm(PAGE)[row:]] = 127
        for b in self.bufs:
            b[cb:].view(torch.float32).view(self.nb, self.hkv, PAGE)[block, :, row:] = garbage

    def run(self, **kw):
        a = dict(w_prev=self.prev, decay=self.decay, workspace=self.ws, dev_err=self.err)
        a.update(kw)
        return self.hsa.hsa_decode_attn_weights(self.pool, 0, self.q, self.k, self.v, self.cl, SCALE, a.pop("w", self.w), **a)

    def check(self, out, w=None, gone=(), prev="own"):
        """gone: (sequence, page) pairs whose keys are absent."""
        w = self.w if w is None else w
        prev = self.prev if isinstance(prev, str) else prev
        per = self.hq // self.hkv
        for i in range(self.B):
            c = max(0, self.cached[i])
            there = torch.tensor([(i, j // PAGE) not in gone for j in range(c)] + [True] * self.T, device="cuda")
            for h in range(self.hkv):
                safe = self.table[i].clamp(min=0, max=self.nb - 1)
                k = torch.cat((ref.rows(self.values[0], safe, c, h).double(), self.k[i, :, h].double()))[there]
                v = torch.cat((ref.rows(self.values[1], safe, c, h).double(), self.v[i, :, h].double()))[there]
                q = self.q[i, :, h * per:(h + 1) * per].reshape(-1, D)
                seen = [k.shape[0] - self.T + t for t in range(self.T) for _ in range(per)]
                o, p, mag = ref.attend(q, k, v, seen, SCALE)
                got = out[i, :, h * per:(h + 1) * per].reshape(-1, D).double()
                err, lim = (got - o).abs(), 2.0 ** -8 * (2 * o.abs() + mag) + 2.0 ** -10 * mag
                assert bool((err <= lim).all()), "out %d %d: %g over" % (i, h, float((err - lim).max()))
                big = (q.double().abs() @ k.abs().T * SCALE).amax(-1, keepdim=True)
                new = torch.zeros(c + self.T, dtype=torch.float64, device="cuda")
                rel = torch.zeros_like(new)
                new[there], rel[there] = p.sum(0), (p * (big + 1) * 2.0 ** -16).sum(0)
                old = torch.zeros_like(new)
                if prev is not None:
                    old[:c] = self.decay * prev[i, h, :c].double()
                got = w[i, h, :c + self.T].double()
                err, lim = (got - new - old).abs(), rel + 2.0 ** -20 * (new + old.abs()) + 1e-37
                assert bool((err <= lim).all()), "w %d %d: %g over at %d" % (i, h, float((err - lim).max()), int((err - lim).argmax()))
                assert float(err.norm()) <= 2.0 ** -20 * float(big.max() + 1) * float((new + old.abs()).norm())
                assert bool((w[i, h, c + self.T:] == -7.0).all())


CASES = {
    # cached lengths, T, Hq, Hkv
    "one token": ([1], 1, 32, 4),
    "nothing cached": ([0, 0, 0], 1, 16, 2),
    "nothing cached, verify": ([0, 5], 4, 16, 2),
    "page borders": ([63, 64, 65, 127, 128, 129], 1, 32, 4),
    "page borders, verify": ([61, 62, 63, 64, 125, 0], 4, 32, 4),
    "two": ([300, 64, 1], 2, 32, 4),
    "three": ([300, 64, 1, 2000], 3, 32, 4),
    "one head each": ([700, 3, 64], 1, 8, 8),
    "one head each, three": ([700, 3, 64], 3, 4, 4),
    "pairs": ([129, 1500], 3, 8, 4),
    "fours": ([129, 1500, 0], 4, 16, 4),
    "fours, one": ([5000, 10, 10], 1, 16, 4),
    "uneven": ([20000, 1, 0, 640, 33, 7001, 64, 2], 1, 16, 2),
    "one long": ([70001], 1, 32, 4),
    "one long, verify": ([40003], 4, 32, 4),
    "many": ([(37 * i) % 200 for i in range(150)], 1, 16, 2),
}


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("case", sorted(CASES))
def test_weights_and_output(case, fmt):
    cached, T, hq, hkv = CASES[case]
    s = Step(_hsa(), cached, T, hq, hkv, fmt)
    out = s.run()
    assert int(s.err) == 0
    s.check(out)


VALUES = {
    "tiny": lambda at: torch.full_like(at, 2.0 ** -30, dtype=torch.bfloat16),
    "large": lambda at: torch.full_like(at, 2.0 ** 30, dtype=torch.bfloat16),
    "unlike": lambda at: torch.exp2((at * 7919 % 25 - 12).float()).bfloat16(),
    "rising": lambda at: torch.exp2((at // PAGE).float() * 3 - 60).bfloat16(),
    "falling": lambda at: torch.exp2(60 - (at // PAGE).float() * 3).bfloat16(),
    "zero at first": lambda at: (at >= 100).bfloat16(),
}


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("values", sorted(VALUES))
def test_values_of_any_size(values, fmt):
    # an FP8 layer's P, times V's scale, is fp16: its precision follows the values' size
    s = Step(_hsa(), [2500, 64, 127], 2, 16, 2, fmt, garbage=None, vmag=VALUES[values])
    out = s.run(max_ctas=5)
    assert int(s.err) == 0
    s.check(out)


@pytest.mark.parametrize("max_ctas", [1, 3, 40, 1000])
def test_any_grid(max_ctas):
    s = Step(_hsa(), [900, 0, 64, 3000], 2, 16, 2, prev=False)
    s.check(s.run(max_ctas=max_ctas), prev=None)


def test_in_place_and_from_nothing():
    s = Step(_hsa(), [900, 130], 1, 32, 4)
    prev = s.prev.clone()
    w = torch.where(torch.arange(s.stride, device="cuda") < s.cl[:, None, None], prev, torch.tensor(-7.0, device="cuda"))
    s.check(s.run(w=w, w_prev=w), w=w, prev=prev)
    s.w.fill_(-7.0)
    s.check(s.run(w_prev=None), prev=None)


def test_more_sequences_than_fit_on_chip():
    hsa = _hsa()
    s = Step(hsa, [(i * 13) % 90 for i in range(1100)], 1, 8, 1, garbage=None)
    out = s.run()
    ids = [0, 1, 511, 1023, 1024, 1025, 1099]
    s.B, s.cached, s.table = len(ids), [s.cached[i] for i in ids], s.table[ids]
    s.q, s.k, s.v = s.q[ids], s.k[ids], s.v[ids]
    s.check(out[ids], w=s.w[ids], prev=s.prev[ids])


def test_left_out_and_absent():
    hsa = _hsa()
    for fmt in (None, "e4m3"):
        s = Step(hsa, [300, 700, 64, 129], 2, 16, 2, fmt)
        s.cl[1] = s.stride - 1  # does not fit: left out
        out = torch.full_like(s.q, 5.0)
        s.run(out=out, append=False)
        assert int(s.err) == hsa.HSA_DEVERR_BAD_LEN
        assert bool((out[1] == 5.0).all()) and bool((s.w[1] == -7.0).all())
        rest = [0, 2, 3]
        keep = s.B, s.cached, s.table, s.q, s.k, s.v
        s.B, s.cached, s.table, s.q, s.k, s.v = 3, [s.cached[i] for i in rest], s.table[rest], s.q[rest], s.k[rest], s.v[rest]
        s.check(out[rest], w=s.w[rest], prev=s.prev[rest])
        s.B, s.cached, s.table, s.q, s.k, s.v = keep
        # pages outside the pool, and a block table that is too narrow
        s.cl.copy_(_i32(s.cached))
        s.err.zero_()
        s.w.fill_(-7.0)
        full = s.table.clone()
        s.table[0, 2], s.table[1, 0], s.table[3, 1] = s.nb, -1, -5
        out = s.run()
        assert int(s.err) == hsa.HSA_DEVERR_BAD_BLOCK
        s.check(out, gone={(0, 2), (1, 0), (3, 1)})
        s.table.copy_(full)
        s.err.zero_()
        s.w.fill_(-7.0)
        narrow = s.table[:, :3].contiguous()
        pool = hsa.DualPool([True], [s.bufs[0]], [s.bufs[1]], narrow, _i32([0] * s.B), s.hq, kv_fp8=[fmt], Hkv=s.hkv, d=D,
                            num_blocks=s.nb)
        s.pool = pool
        out = s.run()
        assert int(s.err) == hsa.HSA_DEVERR_BAD_PAGE
        s.check(out, gone={(i, j) for i in range(4) for j in range(3, 20)})


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("T", [1, 4])
def test_append(fmt, T):
    """The same pool as hsa_kv_append afterwards, bit for bit, and a negative length as 0."""
    hsa = _hsa()
    cached = [62, 0, 640, -3, 700]
    a, b = Step(hsa, cached, T, 16, 2, fmt), Step(hsa, cached, T, 16, 2, fmt)
    a.check(a.run(append=True))
    n = torch.arange(a.B + 1, device="cuda", dtype=torch.int32) * T
    hsa.hsa_kv_append(b.pool, 0, b.k.view(-1, 2, D), b.v.view(-1, 2, D), n, torch.arange(a.B, device="cuda", dtype=torch.int32),
                      b.cl.clamp(min=0))
    assert int(a.err) == 0
    for x, y in zip(a.bufs, b.bufs):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_same_results_every_time_and_on_any_workspace():
    s = Step(_hsa(), [5000, 130, 9000], 1, 32, 4)
    out, w = s.run().clone(), s.w.clone()
    for fill in (0, 255, 127):
        s.ws.fill_(fill)
        s.w.fill_(-7.0)
        assert torch.equal(s.run(), out) and torch.equal(s.w, w)


def test_agrees_with_the_plain_decode():
    """Both round P once: twice the limit of one."""
    hsa = _hsa()
    s = Step(hsa, [5000, 130, 64], 2, 32, 4, garbage=0.0)
    a = s.run().float()
    b = hsa.hsa_decode_attn(s.pool, 0, s.q, s.k, s.v, s.cl, SCALE).float()
    assert float((a - b).abs().max()) <= 2.0 ** -6 * float(s.v.float().abs().max())


def test_captured_and_on_another_stream():
    s = Step(_hsa(), [900, 64, 2000], 1, 16, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = s.run(stream=side)
    side.synchronize()
    s.check(out)
    out = torch.empty_like(s.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(out=out)
    for seed in range(2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        s.q.copy_(torch.randn(s.q.shape, generator=g, device="cuda"))
        s.cached = [[700, 1, 1999], [900, 0, 1]][seed]
        s.cl.copy_(_i32(s.cached))
        s.prev.uniform_(generator=g)
        s.w.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        s.check(out)


def test_values_out_of_reach():
    """Scores that overflow no exponent: keys a thousand times the usual, weights at 0 and 1."""
    s = Step(_hsa(), [300, 200], 1, 16, 2, prev=False)
    s.q.mul_(8)
    s.k.mul_(4)
    s.check(s.run(), prev=None)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_nan_query_stays_in_its_head(fmt):
    """A row of NaN: its output and its KV head's weights, and nothing else."""
    s = Step(_hsa(), [300, 5000], 2, 16, 2, fmt)
    ok, w = s.run().clone(), s.w.clone()
    s.q[1, 0, 3, 7] = float("nan")
    out = s.run()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, 0, 3] = True
    assert bool(out[bad].isnan().all()) and torch.equal(out[~bad], ok[~bad])
    assert bool(s.w[1, 0, :5001].isnan().all())
    s.w[1, 0], w[1, 0] = 0.0, 0.0
    assert torch.equal(s.w, w)


def test_refusals():
    hsa = _hsa()
    s = Step(hsa, [100, 20], 1, 16, 2)
    for kw in (dict(workspace=s.ws[:-16]), dict(decay=float("inf")), dict(max_ctas=-1), dict(w_prev=s.w.flatten()[4:-s.w.numel() // 2])):
        with pytest.raises((hsa.HsaError, ValueError)):
            s.run(**kw)
    big = torch.empty(s.w.numel() + 4, device="cuda")
    a, b = big[:-4].view(s.w.shape), big[4:].view(s.w.shape)
    with pytest.raises(hsa.HsaError):
        s.run(w=a, w_prev=b)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(hsa.HsaError):
            hsa.hsa_decode_attn_weights(s.pool, 0, s.q, s.k, s.v, s.cl, scale, s.w)
    ring = hsa.DualPool.allocate([False], 1, 2, s.table, _i32([0, 1]), 16, 2)
    with pytest.raises(hsa.HsaError) as e:
        hsa.hsa_decode_attn_weights(ring, 0, s.q, s.k, s.v, s.cl, SCALE, s.w)
    assert e.value.status == hsa.HSA_UNSUPPORTED_SHAPE
    assert int(s.err) == 0
