"""Choice and move of the positions that stay, on the GPU: both are exact, so every value is
compared for equality with a plain form that sorts and copies one position at a time."""
import random

import pytest
import torch

import evict_ref as ref

pytestmark = pytest.mark.gpu

D, PAGE = 128, 64


def _hsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import full_attention_kv_gb300 as hsa
    hsa.lib()
    return hsa


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _spread(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").mul_(2.5).exp_()


VALUES = {
    "spread": lambda g, *s: _spread(g, *s),
    "ties": lambda g, *s: torch.randint(0, 4, s, generator=g, device="cuda").float(),
    "equal": lambda g, *s: torch.full(s, 0.125, device="cuda"),
    "zeros": lambda g, *s: torch.zeros(s, device="cuda") * torch.randint(-1, 2, s, generator=g, device="cuda"),
    "signs": lambda g, *s: torch.randn(s, generator=g, device="cuda"),
    "close": lambda g, *s: 1.0 + torch.randint(0, 9, s, generator=g, device="cuda") * 2.0 ** -23,
    "tiny": lambda g, *s: torch.randint(0, 9, s, generator=g, device="cuda") * 2.0 ** -149,
    "holes": lambda g, *s: torch.where(torch.rand(s, generator=g, device="cuda") < 0.3,
                                       torch.tensor(float("nan"), device="cuda"), _spread(g, *s)),
    "nothing": lambda g, *s: torch.full(s, float("nan"), device="cuda"),
    "infinities": lambda g, *s: torch.where(torch.rand(s, generator=g, device="cuda") < 0.3,
                                            torch.tensor(float("inf"), device="cuda"), -torch.rand(s, generator=g, device="cuda") / 0),
}

SIZES = [
    # lengths, row length, heads, budget, sinks, recent, reach
    ([0, 1, 2, 3, 5], 8, 1, 2, 0, 1, 0),
    ([1, 7, 64, 65, 127], 128, 2, 7, 1, 2, 1),
    ([40, 39, 41, 40], 44, 3, 40, 4, 30, 7),         # at the budget, below and above it
    ([100, 33, 97], 100, 2, 32, 16, 16, 2),          # the middle keeps nothing
    ([2049, 1, 600, 2048, 513], 2052, 2, 512, 4, 128, 3),
    ([5000, 4097, 9001], 9004, 1, 1, 0, 0, 0),
    ([20000, 333, 16384], 20000, 4, 4096, 3, 100, 7),
    ([20001], 40000, 1, 20000, 0, 0, 5),             # all but one
    ([20000, 18006, 18005, 18004], 20000, 2, 18005, 9000, 9000, 3),  # few of few
]


@pytest.mark.parametrize("kind", sorted(VALUES))
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_select(kind, case):
    hsa = _hsa()
    n, stride, heads, budget, sinks, recent, reach = SIZES[case]
    R = len(n)
    w = VALUES[kind](_gen(case), R + 1, heads, stride)
    for h in range(heads):  # nothing behind a row's end may compete
        for i in range(R):
            w[i, h, n[i]:] = float("inf") if i % 2 else float("nan")
    seq = random.Random(case).sample(range(R), R)
    length = [n[s] for s in seq]
    err = _i32([0])
    keep, new = hsa.hsa_kv_select(w, _i32(length), _i32(seq), budget, sinks=sinks, recent=recent, reach=reach, dev_err=err)
    host = w.cpu().tolist()
    assert int(err) == 0
    assert new.tolist() == [min(x, budget) for x in length]
    got = keep.tolist()
    for r in range(R):
        for h in range(heads):
            want = ref.choose(host[seq[r]][h], length[r], budget, sinks, recent, reach)
            assert got[r][h] == want + [-1] * (budget - len(want)), (r, h)


@pytest.mark.parametrize("reach", [0, 3])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
def test_select_long_rows(kind, reach):
    """Rows whose keys do not fit shared memory beside one another, split over clusters."""
    hsa = _hsa()
    n, stride, heads, budget = [1000003, 262144, 999999], 1000004, 2, 30001
    w = VALUES[kind](_gen(1), 3, heads, stride)
    keep, new = hsa.hsa_kv_select(w, _i32(n), _i32([0, 1, 2]), budget, sinks=5, recent=77, reach=reach)
    for r in range(3):
        x = w[r, :, :n[r]]
        score = x.clone()
        for d in range(1, reach + 1):
            score[:, d:] = torch.maximum(score[:, d:], x[:, :-d])
            score[:, :-d] = torch.maximum(score[:, :-d], x[:, d:])
        mid = score[:, 5:n[r] - 77].sort(dim=-1, descending=True, stable=True).indices[:, :budget - 82] + 5
        want = mid.sort(-1).values
        assert torch.equal(keep[r, :, 5:-77].long(), want)
        assert keep[r, :, :5].tolist() == [[0, 1, 2, 3, 4]] * heads
        assert torch.equal(keep[r, :, -77:].long(), (n[r] - 77 + torch.arange(77, device="cuda")).expand(heads, 77))
    assert new.tolist() == [budget] * 3


@pytest.mark.parametrize("n,budget,reach", [(16384, 100, 0), (40000, 3000, 0), (40000, 3000, 1), (300000, 20000, 0), (300000, 299000, 0)])
@pytest.mark.parametrize("kind", ["spread", "one in eight", "steps", "sorted", "few large"])
def test_select_where_a_sample_misleads(kind, n, budget, reach):
    """Rows that a sample of positions, evenly spaced, tells little or wrong things about."""
    hsa = _hsa()
    g = _gen(n)
    w = _spread(g, 2, 1, n)
    at = torch.arange(n, device="cuda")
    if kind == "one in eight":
        w = torch.where(at % 8 == 1, w * 1e6, w)
    elif kind == "steps":
        w = torch.where(at < n // 3, 1.0, torch.where(at < n // 2, 1.0 + 2.0 ** -23, 0.5)).expand(2, 1, n).contiguous()
    elif kind == "sorted":
        w = w.sort(dim=-1, descending=True).values
    elif kind == "few large":
        w = torch.where(at % 3001 == 7, w + 1e9, torch.zeros_like(w))
    keep, new = hsa.hsa_kv_select(w, _i32([n, n - 1]), _i32([0, 1]), budget, sinks=1, recent=2, reach=reach)
    for r in range(2):
        m = n - r
        x = w[r, 0, :m]
        score = x.clone()
        for d in range(1, reach + 1):
            score[d:] = torch.maximum(score[d:], x[:-d])
            score[:-d] = torch.maximum(score[:-d], x[d:])
        mid = score[1:m - 2].sort(descending=True, stable=True).indices[:budget - 3] + 1
        assert torch.equal(keep[r, 0, 1:-2].long(), mid.sort().values)
    assert new.tolist() == [budget] * 2


@pytest.mark.parametrize("kind", ["equal", "close"])
def test_select_longest_rows(kind):
    """As many positions a CTA as its counters hold, all with one exponent."""
    hsa = _hsa()
    n, budget = 1 << 22, 70000
    w = VALUES[kind](_gen(2), 1, 1, n)
    keep, new = hsa.hsa_kv_select(w, _i32([n]), _i32([0]), budget)
    want = w[0, 0].sort(descending=True, stable=True).indices[:budget].sort().values
    assert torch.equal(keep[0, 0].long(), want) and new.tolist() == [budget]


@pytest.mark.parametrize("R", [1, 20, 200])
def test_select_many_rows(R):
    """Fewer and more rows than SMs: another number of CTAs a row."""
    hsa = _hsa()
    g = _gen(R)
    n = torch.randint(0, 30000, (R,), generator=g, device="cuda", dtype=torch.int32)
    w = _spread(g, R, 4, 30000)
    keep, new = hsa.hsa_kv_select(w, n, torch.arange(R, device="cuda", dtype=torch.int32), 1000, sinks=4, recent=32)
    x = w.clone()
    at = torch.arange(30000, device="cuda")
    x.masked_fill_((at >= n[:, None])[:, None], -1)
    x.masked_fill_(((at < 4) | (at >= n[:, None] - 32) & (at < n[:, None]))[:, None], float("inf"))
    want = x.sort(dim=-1, descending=True, stable=True).indices[..., :1000].sort(-1).values.int()
    want = torch.where((n > 1000)[:, None, None], want,
                       torch.where(torch.arange(1000, device="cuda") < n[:, None], torch.arange(1000, device="cuda"), -1).int()[:, None])
    assert torch.equal(keep, want) and torch.equal(new, n.clamp(max=1000))


def test_select_on_another_stream_and_captured_over_clusters():
    hsa = _hsa()
    g = _gen(7)
    n, R = 30000, 5
    w, length, seq = _spread(g, R, 2, n), _i32([n, 20000, 3, 29999, 4097]), _i32([4, 2, 0, 1, 3])
    first = hsa.hsa_kv_select(w, length, seq, 2000, sinks=4, recent=100, reach=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = hsa.hsa_kv_select(w, length, seq, 2000, sinks=4, recent=100, reach=2, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    keep, new = torch.empty_like(first[0]), torch.empty_like(first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hsa.hsa_kv_select(w, length, seq, 2000, sinks=4, recent=100, reach=2, keep=keep, new_len=new)
    for _ in range(3):
        w.copy_(_spread(g, R, 2, n))
        want = hsa.hsa_kv_select(w, length, seq, 2000, sinks=4, recent=100, reach=2)
        keep.zero_()
        graph.replay()
        assert torch.equal(keep, want[0]) and torch.equal(new, want[1])


def test_select_in_place_is_refused():
    hsa = _hsa()
    length = _i32([5, 9])
    with pytest.raises(hsa.HsaError) as e:
        hsa.hsa_kv_select(torch.zeros(2, 1, 16, device="cuda"), length, _i32([0, 1]), 4, new_len=length)
    assert e.value.status == hsa.HSA_INVALID_ARG


def test_select_flags():
    hsa = _hsa()
    w = _spread(_gen(3), 2, 1, 16)
    for n, seq, bits in (([5, 17], [0, 1], hsa.HSA_DEVERR_BAD_LEN), ([5, -1], [0, 1], hsa.HSA_DEVERR_BAD_LEN),
                         ([5, 9], [0, 2], hsa.HSA_DEVERR_BAD_SEQ), ([5, 9], [0, -1], hsa.HSA_DEVERR_BAD_SEQ)):
        err = _i32([0])
        keep, new = hsa.hsa_kv_select(w, _i32(n), _i32(seq), 4, dev_err=err)
        assert int(err) == bits and new.tolist() == [4, 0] and keep[1].tolist() == [[-1] * 4]
        assert keep[0, 0].tolist() == ref.choose(w[0, 0].tolist(), 5, 4, 0, 0, 0)
    keep, new = hsa.hsa_kv_select(w, _i32([5, 0]), _i32([1, 0]), 0)
    assert new.tolist() == [0, 0] and keep.shape == (2, 1, 0)


class Moves:
    """A layer of pages, sequences of n[i] tokens in them, and free pages."""

    def __init__(self, hsa, n, budget, fmt, hkv, heads, seed):
        g, rng = _gen(seed), random.Random(seed)
        self.hsa, self.fmt, self.hkv, self.heads, self.budget = hsa, fmt, hkv, heads, budget
        R = len(n)
        self.seq = rng.sample(range(R), R)
        pages = [(x + PAGE - 1) // PAGE for x in n]
        self.kept = [min(x, budget) for x in n]
        dst = [(k + PAGE - 1) // PAGE for k in self.kept]
        self.nb = sum(pages) + sum(dst) + 1
        ids = list(range(self.nb))
        rng.shuffle(ids)
        self.width = max(pages) + 1
        self.table = [[-1] * self.width for _ in range(R)]
        for i in range(R):
            for j in range(pages[i]):
                self.table[self.seq[i]][j] = ids.pop()
        self.dst = [[ids.pop() for _ in range(d)] + [-1] * (max(dst) - d) for d in dst]
        if fmt is None:
            self.bufs = [torch.randn(self.nb, hkv, PAGE, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
        else:
            self.bufs = [torch.randint(0, 256, (self.nb * hkv * PAGE * (D + 4),), generator=g, device="cuda", dtype=torch.uint8)
                         for _ in range(2)]
        self.keep = [[sorted(rng.sample(range(x), k)) + [-1] * (budget - k) for _ in range(heads)] for x, k in zip(n, self.kept)]
        self.stride = (max(n + [budget]) + 3) // 4 * 4
        self.w = torch.randn(R, hkv, self.stride, generator=g, device="cuda")
        self.w_dst = torch.randn(R, hkv, self.stride, generator=g, device="cuda")
        self.err = _i32([0])
        self.pool = hsa.DualPool([True], self.bufs[:1], self.bufs[1:], _i32(self.table), _i32([0] * R), hkv * 2, kv_fp8=[fmt],
                                 Hkv=hkv, d=D, num_blocks=self.nb)

    def run(self, **kw):
        a = dict(keep=_i32(self.keep), new_len=_i32(self.kept), seq_idx=_i32(self.seq), dst_tables=_i32(self.dst), w=self.w,
                 w_dst=self.w_dst, dev_err=self.err)
        a.update(kw)
        self.hsa.hsa_kv_compact(self.pool, 0, **a)

    def views(self, bufs):
        if self.fmt is None:
            return [b.clone() for b in bufs]
        out = []
        cb = self.nb * self.hkv * PAGE * D
        for b, v in zip(bufs, (0, 1)):
            out.append(b[:cb].clone().view(self.nb, self.hkv, D, PAGE) if v else b[:cb].clone().view(self.nb, self.hkv, PAGE, D))
            out.append(b[cb:].clone().view(torch.int32).view(self.nb, self.hkv, PAGE))
        return out

    def moved(self, skip=()):
        """The layer's buffers and w_dst after the move, position by position."""
        perm = lambda l: 16 * (l // 16) + 4 * ((l % 8) // 2) + l % 2 + 2 * (l % 16 // 8)  # noqa: E731
        views = [x.cpu() for x in self.views(self.bufs)]
        w, w_dst = self.w.cpu(), self.w_dst.cpu().clone()
        for r, s in enumerate(self.seq):
            for h in range(self.hkv):
                for i in range(self.kept[r]):
                    pos = self.keep[r][h if self.heads > 1 else 0][i]
                    if (r, h, i) in skip:
                        continue
                    w_dst[s, h, i] = w[s, h, pos]
                    a, b = (self.table[s][pos // PAGE], pos % PAGE), (self.dst[r][i // PAGE], i % PAGE)
                    if self.fmt is None:
                        for x in views:
                            x[b[0], h, b[1]] = x[a[0], h, a[1]]
                    else:
                        k, ks, v, vs = views
                        k[b[0], h, b[1]] = k[a[0], h, a[1]]
                        v[b[0], h, :, perm(b[1])] = v[a[0], h, :, perm(a[1])]
                        ks[b[0], h, b[1]] = ks[a[0], h, a[1]]
                        vs[b[0], h, b[1]] = vs[a[0], h, a[1]]
        return views, w_dst

    def check(self, want, err=0):
        views, w_dst = want
        assert int(self.err) == err
        for got, x in zip(self.views(self.bufs), views):
            same = got.cpu().view(torch.int16) == x.view(torch.int16) if got.dtype == torch.bfloat16 else got.cpu() == x
            assert bool(same.all())
        assert torch.equal(self.w_dst.cpu(), w_dst)


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("n,budget,hkv,heads", [
    ([1, 64, 65, 3], 2, 2, 2),
    ([100, 64, 700, 63], 64, 4, 4),
    ([129, 500, 128, 1], 129, 1, 1),
    ([900, 40, 450], 200, 8, 1),
    ([1300], 1, 2, 2),
    ([300, 299], 299, 4, 1),
])
def test_compact(fmt, n, budget, hkv, heads):
    m = Moves(_hsa(), n, budget, fmt, hkv, heads, seed=budget)
    want = m.moved()
    m.run()
    m.check(want)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_compact_any_order(fmt):
    """Lists that do not ascend, and the same position twice."""
    m = Moves(_hsa(), [300, 90], 150, fmt, 2, 2, seed=5)
    rng = random.Random(1)
    m.keep = [[[rng.randrange(n) for _ in range(k)] + [-1] * (150 - k) for _ in range(2)] for n, k in ((300, 150), (90, 90))]
    want = m.moved()
    m.run()
    m.check(want)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_the_same_sequence_twice(fmt):
    """Two cuts of one sequence (branches of a search), each to pages of its own."""
    hsa = _hsa()
    m = Moves(hsa, [700, 700], 150, fmt, 2, 2, seed=6)
    a = hsa.hsa_kv_select(m.w, _i32([700, 700]), _i32([m.seq[0]] * 2), 150, sinks=3, dev_err=m.err)
    assert torch.equal(a[0][0], a[0][1]) and a[1].tolist() == [150, 150]
    m.table[m.seq[1]] = m.table[m.seq[0]]
    want = m.moved()[0]
    hsa.hsa_kv_compact(m.pool, 0, _i32(m.keep), _i32(m.kept), _i32([m.seq[0]] * 2), _i32(m.dst), dev_err=m.err)
    m.check((want, m.w_dst.cpu()))


@pytest.mark.parametrize("fmt", [None, "e5m2"])
def test_compact_flags(fmt):
    """What cannot be reached is flagged and left; everything else is moved."""
    hsa = _hsa()
    m = Moves(hsa, [200, 300], 100, fmt, 2, 2, seed=9)
    skip = {(0, 1, 7), (0, 0, 99)}
    m.moved()
    good = m.keep[0][1][7], m.keep[0][0][99]
    want = m.moved(skip)
    m.keep[0][1][7], m.keep[0][0][99] = -1, m.width * PAGE
    assert m.width * PAGE >= m.stride  # its weight is out of reach too
    m.run()
    m.check(want, hsa.HSA_DEVERR_BAD_LEN | hsa.HSA_DEVERR_BAD_PAGE)
    m.keep[0][1][7], m.keep[0][0][99] = good
    state = m.views(m.bufs)
    for kw, bits in ((dict(seq_idx=_i32([2, -1])), hsa.HSA_DEVERR_BAD_SEQ), (dict(new_len=_i32([101, -1])), hsa.HSA_DEVERR_BAD_LEN),
                     (dict(dst_tables=_i32([[m.nb, -1]] * 2)), hsa.HSA_DEVERR_BAD_BLOCK)):
        m.err.zero_()
        m.run(w=None, w_dst=None, **kw)
        assert int(m.err) == bits
        for a, b in zip(state, m.views(m.bufs)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # one page too few: the first 64 rows move
    m.err.zero_()
    want = m.moved({(r, h, i) for r in range(2) for h in range(2) for i in range(64, 100)})
    m.run(dst_tables=_i32([x[:1] for x in m.dst]))
    m.check(want, hsa.HSA_DEVERR_BAD_PAGE)
    # a bad page of the block table
    m.err.zero_()
    m.table[m.seq[1]][0] = m.nb
    m.pool.block_tables.copy_(_i32(m.table))
    lost = {(1, h, i) for h in range(2) for i in range(100) if m.keep[1][h][i] < PAGE}
    m.table[m.seq[1]][0] = 0
    want = m.moved(lost)
    for r, h, i in lost:
        want[1][m.seq[r], h, i] = m.w.cpu()[m.seq[r], h, m.keep[r][h][i]]
    m.run()
    m.check(want, hsa.HSA_DEVERR_BAD_BLOCK)


def test_select_and_compact_captured():
    """Captured in a graph and replayed on new weights."""
    hsa = _hsa()
    m = Moves(hsa, [500, 260], 128, None, 2, 2, seed=11)
    length, seq, dst = _i32([500, 260]), _i32([0, 1]), _i32(m.dst)
    m.pool.block_tables.copy_(_i32([m.table[m.seq[0]], m.table[m.seq[1]]]))
    m.table = [m.table[m.seq[0]], m.table[m.seq[1]]]
    m.seq = [0, 1]
    keep, new = torch.empty((2, 2, 128), dtype=torch.int32, device="cuda"), _i32([0, 0])
    args = dict(sinks=2, recent=16, reach=1, keep=keep, new_len=new)

    def step():
        hsa.hsa_kv_select(m.w, length, seq, 128, **args)
        hsa.hsa_kv_compact(m.pool, 0, keep, new, seq, dst, w=m.w, w_dst=m.w_dst, dev_err=m.err)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        m.w.copy_(torch.randn(m.w.shape, generator=_gen(seed), device="cuda"))
        host = m.w.tolist()
        m.keep = [[ref.choose(host[r][h], [500, 260][r], 128, 2, 16, 1) for h in range(2)] for r in range(2)]
        want = m.moved()
        graph.replay()
        torch.cuda.synchronize()
        m.check(want)
