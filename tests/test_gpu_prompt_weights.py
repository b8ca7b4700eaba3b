"""The weight of a prompt's last queries on every cached key, on the GPU, against softmax in 64
bits.  Limits as in the weighing decode's tests: a score is off by at most 2^-17 of scale sum |q k|,
a weight relatively by its score's error and its lse's, 2^-16 (mag_max + 1); sums over at most 512
rows and the decayed old weight add 2^-20 of what they sum; over a sequence the roundings are
independent, 2^-20 (mag_max + 1) of the weights' norm."""
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


class Prompts:
    """Requests of n[i] tokens in the pool, the newest m[i] of them with queries."""

    def __init__(self, hsa, n, m, window, hq, hkv, seed=1, prev=True, decay=0.75, garbage=float("nan"), batch=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.hsa, self.n, self.m, self.window, self.hq, self.hkv, self.decay = hsa, n, m, window, hq, hkv, decay
        R = len(n)
        batch = batch or R + 1
        self.seq = torch.randperm(batch, generator=g, device="cuda")[:R].tolist()
        pages = [(x + PAGE - 1) // PAGE for x in n]
        self.nb = sum(pages) + 1
        ids = torch.randperm(self.nb, generator=g, device="cuda").int().tolist()
        width = max(pages) + 1
        table = [[-1] * width for _ in range(batch)]
        for i in range(R):
            table[self.seq[i]] = [ids.pop() for _ in range(pages[i])] + [-1] * (width - pages[i])
        self.table = _i32(table)
        self.kp = torch.randn(self.nb, hkv, PAGE, D, generator=g, device="cuda").bfloat16()
        for i in range(R):
            if n[i] % PAGE:
                self.kp[table[self.seq[i]][n[i] // PAGE], :, n[i] % PAGE:] = garbage
        self.kp[ids.pop()] = garbage
        rows = sum(m)
        self.q = (torch.randn(rows, hq, D, generator=g, device="cuda") * 2).bfloat16()
        self.cu = _i32([sum(m[:i]) for i in range(R + 1)])
        self.stride = (max(n) + 5 + 3) // 4 * 4
        self.prev = torch.rand(batch, hkv, self.stride, generator=g, device="cuda") if prev else None
        if prev:
            for i in range(R):
                self.prev[self.seq[i], :, n[i] - m[i]:] = float("nan")  # new positions count nothing from it
        self.w = torch.full((batch, hkv, self.stride), -7.0, device="cuda")
        self.err = _i32([0])
        self.len, self.at = _i32(n), _i32(self.seq)
        self.pool = hsa.DualPool([True], [self.kp], [torch.zeros_like(self.kp)], self.table, _i32([0] * batch), hq)
        self.ws = hsa.prefill_weights_workspace(self.pool, R, window).fill_(255)

    def run(self, **kw):
        a = dict(w_prev=self.prev, decay=self.decay, workspace=self.ws, dev_err=self.err)
        a.update(kw)
        return self.hsa.hsa_prefill_weights(self.pool, 0, self.q, self.cu, self.len, self.at, self.window, SCALE, a.pop("w", self.w), **a)

    def check(self, w=None, gone=(), prev="own", skip=()):
        w = self.w if w is None else w
        prev = self.prev if isinstance(prev, str) else prev
        per = self.hq // self.hkv
        cu = self.cu.tolist()
        named = set()
        for i, (n, m, s) in enumerate(zip(self.n, self.m, self.seq)):
            if i in skip or m == 0:
                continue
            named.add(s)
            T = min(self.window, m)
            there = torch.tensor([(i, j // PAGE) not in gone for j in range(n)], device="cuda")
            for h in range(self.hkv):
                k = ref.rows(self.kp, self.table[s].clamp(min=0, max=self.nb - 1), n, h)
                k = torch.where(there[:, None], k, torch.zeros((), device="cuda", dtype=k.dtype)).double()
                q = self.q[cu[i + 1] - T:cu[i + 1], h * per:(h + 1) * per].reshape(-1, D).double()
                x = q @ k.T * SCALE
                late = torch.arange(n, device="cuda") > n - T + torch.arange(T * per, device="cuda")[:, None] // per
                p = torch.softmax(x.masked_fill(late | ~there, float("-inf")), -1).nan_to_num(0.0)
                big = (q.abs() @ k.abs().T * SCALE).amax(-1, keepdim=True)
                new, rel = p.sum(0), (p * (big + 1) * 2.0 ** -16).sum(0)
                old = torch.zeros_like(new)
                if prev is not None:
                    old[:n - m] = self.decay * prev[s, h, :n - m].double()
                err, lim = (w[s, h, :n].double() - new - old).abs(), rel + 2.0 ** -20 * (new + old.abs()) + 1e-37
                assert bool((err <= lim).all()), "%d %d: %g over at %d" % (i, h, float((err - lim).max()), int((err - lim).argmax()))
                assert float(err.norm()) <= 2.0 ** -20 * float(big.max() + 1) * float((new + old.abs()).norm())
                assert bool((w[s, h, n:] == -7.0).all())
        for s in set(range(w.shape[0])) - named:
            assert bool((w[s] == -7.0).all())


CASES = {
    # tokens, new rows, window, Hq, Hkv
    "one token": ([1], [1], 1, 32, 4),
    "one query": ([1000, 64, 65], [1, 1, 1], 1, 32, 4),
    "fewer rows than the window": ([300, 129, 5], [3, 129, 5], 32, 32, 4),
    "page borders": ([63, 64, 65, 127, 128, 129], [20, 64, 1, 127, 128, 129], 16, 16, 2),
    "one row tile": ([1000, 640, 3], [100, 16, 3], 16, 32, 4),
    "two row tiles": ([1500, 31, 900], [300, 31, 33], 32, 32, 4),
    "three row tiles": ([1500, 40, 900], [300, 40, 33], 33, 32, 4),
    "four row tiles": ([2000, 63, 64, 1], [2000, 63, 64, 1], 64, 32, 4),
    "mixed row tiles": ([700, 800, 900, 1000], [1, 17, 40, 1000], 64, 16, 2),
    "one head each": ([900, 77], [90, 77], 64, 8, 8),
    "pairs": ([900, 77], [90, 77], 33, 8, 4),
    "fours": ([900, 77, 2], [90, 7, 2], 50, 16, 4),
    "no rows": ([500, 200, 300], [0, 30, 0], 16, 16, 2),
    "many": ([(37 * i) % 500 + 1 for i in range(100)], [(37 * i) % 500 % 20 + 1 for i in range(100)], 8, 16, 2),
    "uneven": ([30000, 1, 400, 8001], [500, 1, 400, 64], 32, 32, 4),
    "long": ([120001], [700], 64, 32, 4),
}


@pytest.mark.parametrize("case", sorted(CASES))
def test_weights(case):
    p = Prompts(_hsa(), *CASES[case])
    p.run()
    assert int(p.err) == 0
    p.check()


def test_in_place_from_nothing_and_again():
    p = Prompts(_hsa(), [900, 130], [200, 5], 32, 16, 2)
    prev = p.prev.clone()
    w = p.prev.clone()
    for i, s in enumerate(p.seq):
        w[s, :, p.n[i]:] = -7.0
    w[[s for s in range(3) if s not in p.seq]] = -7.0
    p.run(w=w, w_prev=w)
    p.check(w=w, prev=prev)
    p.run(w_prev=None)
    p.check(prev=None)
    first = p.w.clone()
    for fill in (0, 127):
        p.ws.fill_(fill)
        p.w.fill_(-7.0)
        p.run(w_prev=None)
        assert torch.equal(first, p.w)


def test_left_out_and_absent():
    hsa = _hsa()
    L, S = hsa.HSA_DEVERR_BAD_LEN, hsa.HSA_DEVERR_BAD_SEQ
    n, m = [300, 700, 129], [50, 60, 70]
    p = Prompts(hsa, n, m, 16, 16, 2)
    for field, i, value, bits, skip in (("len", 1, 59, L, {1}), ("len", 1, -1, L, {1}), ("len", 0, p.stride + 1, L, {0}),
                                        ("at", 2, 4, S, {2}), ("at", 2, -1, S, {2}), ("cu", 3, 181, L, {2}), ("cu", 0, -1, L, {0}),
                                        ("cu", 1, 111, L, {1})):
        t = getattr(p, field)
        was = int(t[i])
        t[i] = value
        p.err.zero_()
        p.w.fill_(-7.0)
        p.run()
        assert int(p.err) == bits, (field, value)
        t[i] = was
        if (field, value) == ("cu", 111):  # request 0 owns 111 rows of q now, request 1 none
            p.m, p.cu[1] = [111, -1, 70], 111
            p.check(skip={1})
            p.m, p.cu[1] = m, was
            continue
        p.check(skip=skip)
    p.err.zero_()
    p.w.fill_(-7.0)
    full = p.table.clone()
    p.table[p.seq[0], 2], p.table[p.seq[1], 0], p.table[p.seq[2], 1] = p.nb, -1, -5
    p.run()
    assert int(p.err) == hsa.HSA_DEVERR_BAD_BLOCK
    p.check(gone={(0, 2), (1, 0), (2, 1)})
    p.table.copy_(full)
    p.err.zero_()
    p.w.fill_(-7.0)
    p.pool = hsa.DualPool([True], [p.kp], [p.kp], p.table[:, :3].contiguous(), _i32([0] * 4), 16)
    p.run()
    assert int(p.err) == hsa.HSA_DEVERR_BAD_PAGE
    p.check(gone={(i, j) for i in range(3) for j in range(3, 20)})


def test_captured_and_on_another_stream():
    p = Prompts(_hsa(), [900, 640], [64, 640], 32, 16, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.run(stream=side)
    side.synchronize()
    p.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    p.q.copy_(torch.randn(p.q.shape, generator=g, device="cuda"))
    p.n = [800, 640]
    p.len.copy_(_i32(p.n))
    p.prev[p.seq[0], :, 736:] = float("nan")
    p.w.fill_(-7.0)
    graph.replay()
    torch.cuda.synchronize()
    p.check()


def test_refusals():
    hsa = _hsa()
    p = Prompts(hsa, [100], [20], 16, 16, 2)
    for kw in (dict(workspace=p.ws[:-16]), dict(decay=float("nan"))):
        with pytest.raises(hsa.HsaError):
            p.run(**kw)
    p.window = 65
    with pytest.raises(hsa.HsaError) as e:
        p.run(workspace=None)
    assert e.value.status == hsa.HSA_UNSUPPORTED_SHAPE
    fp8 = hsa.DualPool.allocate([True], 4, 1, p.table, _i32([0] * 2), 16, 2, kv_fp8=True)
    with pytest.raises(hsa.HsaError) as e:
        hsa.hsa_prefill_weights(fp8, 0, p.q, p.cu, p.len, p.at, 16, SCALE, p.w)
    assert e.value.status == hsa.HSA_UNSUPPORTED_SHAPE
    assert int(p.err) == 0 and bool((p.w == -7.0).all())
