"""Eviction in a model of both kinds of layer, on the GPU: the full layer is cut to a budget and goes on
from its shorter length, the sliding layer beside it goes on from the true one, past the ring's end
and through a second eviction.  Both layers' outputs against 64 bits, the ring bit for bit.  The
prompt comes in two chunks, the second weighed on the first one's weights; an FP8 layer's by the
append, weighed by its last token's decode.  And a verify step made again for the accepted tokens."""
import pytest
import torch

import evict_ref as ref
import test_gpu_evict_run as run
import test_gpu_weigh as weigh

pytestmark = pytest.mark.gpu

D, W, SCALE = 128, 128, 128 ** -0.5
HQ, HKV = 16, 2
PER = HQ // HKV


class Hybrid(run.Server):
    """Layer 0 full, layer 1 sliding; the sliding layer's rows of every token beside."""

    def __init__(self, hsa, fmt):
        super().__init__(hsa, fmt, HQ, HKV)
        self.pool = hsa.DualPool.allocate([True, False], 64, 2, self.tables, run._i32([1, 0]), HQ, HKV, kv_fp8=fmt or False)
        self.seen = [[torch.zeros(0, HKV, D, device="cuda", dtype=torch.bfloat16)] * 2 for _ in range(2)]

    def remember(self, i, k, v):
        self.seen[i] = [torch.cat((a, b)) for a, b in zip(self.seen[i], (k, v))]

    def check_ring(self):
        for i in range(2):
            n = self.seen[i][0].shape[0]
            for pos in range(max(0, n - W), n):
                for x, pool in zip(self.seen[i], (self.pool.k, self.pool.v)):
                    assert torch.equal(pool[1][1 - i, :, pos % W], x[pos])

    def check_sliding(self, i, pos, q, out):
        """A query [hq, D] at `pos` and its output."""
        for h in range(HKV):
            k, v = (x[max(0, pos + 1 - W):pos + 1, h].double() for x in self.seen[i])
            _near(out[h * PER:(h + 1) * PER], *ref.attend(q[h * PER:(h + 1) * PER], k, v, [k.shape[0] - 1] * PER, SCALE))


def _near(got, o, p, mag):
    err = (got.double() - o).abs()
    assert bool((err <= 2.0 ** -8 * (2 * o.abs() + mag) + 2.0 ** -10 * mag).all())


def _big(q, k):
    return float((q.double().abs() @ k.double().abs().T).max()) * SCALE


def _chunk(s, m, first, cu):
    """A chunk of each sequence through both layers (full layer bf16), weighed on what came before."""
    hsa, i32 = s.hsa, run._i32
    rows, start, seq = cu[-1], i32(s.n), i32([0, 1])
    was = list(s.n)
    pos = torch.cat([torch.arange(was[i], was[i] + m[i], device="cuda", dtype=torch.int32) for i in range(2)])
    for i in range(2):
        s.grow(i, was[i] + m[i])
    # the full layer: rotated and appended, then the attention of the new rows
    q, k, v = s.randn(rows, HQ, D) * 2, s.randn(rows, HKV, D), s.randn(rows, HKV, D)
    q, k = hsa.hsa_rope_kv_append(s.pool, 0, s.rope, q, k, v, i32(cu), seq, start, positions=pos, dev_err=s.err)
    hsa.hsa_prefill_attn(s.pool, 0, q, k, v, i32(cu), start, seq, max(m), SCALE, dev_err=s.err)
    s.n = [was[i] + m[i] for i in range(2)]
    old = s.w[0].clone()
    hsa.hsa_prefill_weights(s.pool, 0, q, i32(cu), i32(s.n), seq, 32, SCALE, s.w[0], w_prev=None if first else s.w[0],
                            decay=0.5, dev_err=s.err)
    for i in range(2):
        for h in range(HKV):
            keys, vals = s.rows(i, h)
            x = q[cu[i + 1] - 32:cu[i + 1], h * PER:(h + 1) * PER].reshape(-1, D)
            want = ref.attend(x, keys, vals, [s.n[i] - 32 + t for t in range(32) for _ in range(PER)], SCALE)[1].sum(0)
            want[:was[i]] += 0.5 * old[i, h, :was[i]].double()
            run._close(s.w[0][i, h, :s.n[i]], want, _big(x, keys))
    # the sliding layer: attention first, then the append
    q, k, v = s.randn(rows, HQ, D), s.randn(rows, HKV, D), s.randn(rows, HKV, D)
    q, k = hsa.hsa_rope(s.rope, q, k, pos)
    out = hsa.hsa_prefill_attn(s.pool, 1, q, k, v, i32(cu), start, seq, max(m), SCALE, dev_err=s.err)
    hsa.hsa_kv_append(s.pool, 1, k, v, i32(cu), seq, start, dev_err=s.err)
    for i in range(2):
        s.remember(i, k[cu[i]:cu[i + 1]], v[cu[i]:cu[i + 1]])
        for row in (cu[i], cu[i + 1] - 1):
            s.check_sliding(i, was[i] + row - cu[i], q[row], out[row])


def _step(s, length, check, prev=True):
    """A decode step: the full layer from s.n cached tokens, the sliding one from `length`; both append."""
    hsa, i32 = s.hsa, run._i32
    for i in range(2):
        s.grow(i, s.n[i] + 1)
    qkv = s.randn(2, 2, HQ + 2 * HKV, D)  # of each layer
    turned = [hsa.hsa_rope(s.rope, x[:, :HQ], x[:, HQ:HQ + HKV], i32(length)) + (x[:, HQ + HKV:].contiguous(),) for x in qkv]
    (q, k, v), (q1, k1, v1) = [(a.view(2, 1, HQ, D), b.view(2, 1, HKV, D), c.view(2, 1, HKV, D)) for a, b, c in turned]
    before = {(i, h): s.rows(i, h) for i in range(2) for h in range(HKV)} if check else {}
    old = s.w[0].clone()
    out = hsa.hsa_decode_attn_weights(s.pool, 0, q, k, v, i32(s.n), SCALE, s.w[0], w_prev=s.w[0] if prev else None, decay=0.9,
                                      dev_err=s.err, append=True)
    out1 = hsa.hsa_decode_attn_append(s.pool, 1, q1, k1, v1, i32(length), SCALE, dev_err=s.err)
    for (i, h), (keys, vals) in before.items():
        keys, vals = torch.cat((keys, k[i, 0, h][None].double())), torch.cat((vals, v[i, 0, h][None].double()))
        x = q[i, 0, h * PER:(h + 1) * PER]
        o, p, mag = ref.attend(x, keys, vals, [s.n[i]] * PER, SCALE)
        _near(out[i, 0, h * PER:(h + 1) * PER], o, p, mag)
        want = p.sum(0)
        if prev:
            want[:-1] += 0.9 * old[i, h, :s.n[i]].double()
        run._close(s.w[0][i, h, :s.n[i] + 1], want, _big(x, keys))
    for i in range(2):
        s.remember(i, k1[i], v1[i])
        if check:
            s.check_sliding(i, length[i], q1[i, 0], out1[i, 0])
    s.n = [n + 1 for n in s.n]
    return [n + 1 for n in length]


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
def test_full_layer_evicted_beside_a_ring(fmt):
    hsa = run._hsa()
    s = Hybrid(hsa, fmt)
    if fmt is None:
        _chunk(s, [400, 233], True, [0, 400, 633])
        _chunk(s, [300, 100], False, [0, 300, 400])
        length = [700, 333]
    else:
        m = [699, 332]
        cu, start = run._i32([0, m[0], sum(m)]), run._i32([0, 0])
        for i in range(2):
            s.grow(i, m[i])
        for layer in (0, 1):
            k, v = s.randn(sum(m), HKV, D), s.randn(sum(m), HKV, D)
            pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in m])
            _, k = hsa.hsa_rope(s.rope, None, k, pos)
            hsa.hsa_kv_append(s.pool, layer, k, v, cu, run._i32([0, 1]), start, dev_err=s.err)
        for i in range(2):
            s.remember(i, *(x[int(cu[i]):int(cu[i + 1])] for x in (k, v)))
        s.n = list(m)
        length = _step(s, m, True, prev=False)  # the prompt's last token weighs it
    s.evict(256, sinks=4, recent=32, reach=2)
    for step in range(140):
        length = _step(s, length, step % 23 == 0)
        if step == 70:
            s.evict(192, sinks=1, recent=64, reach=0)
    s.check_ring()
    assert int(s.err) == 0 and s.n == [192 + 69] * 2 and length == [840, 473]


@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("accepted", [1, 2, 3])
def test_verify_step_again_for_the_accepted_tokens(fmt, accepted):
    """w_prev kept: the accepted tokens' weights without the rejected ones'."""
    s = weigh.Step(weigh._hsa(), [300, 64, 1000], 4, HQ, HKV, fmt)
    s.check(s.run())
    s.T = accepted
    s.q, s.k, s.v = (x[:, :accepted].contiguous() for x in (s.q, s.k, s.v))
    s.w.fill_(-7.0)
    s.check(s.run(append=True))
    assert int(s.err) == 0
