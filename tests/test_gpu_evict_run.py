"""A bounded cache from prompt to decode on the GPU, the operators together as a server would call
them: chunked prefill and rotating append, the weight of the last queries, the choice, the move to
pages of their own, then decode steps that weigh and append, another eviction among them.  Checked
against a cache kept as lists of rows in 64 bits: the rows that stay bit for bit, weights and
outputs to the limits of their own tests."""
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


class Server:
    """Two sequences on one full layer; free pages handed out from a list."""

    def __init__(self, hsa, fmt, hq, hkv):
        self.hsa, self.fmt, self.hq, self.hkv = hsa, fmt, hq, hkv
        self.free = list(range(64))[::-1]
        self.table = [[-1] * 24 for _ in range(2)]
        self.tables = _i32(self.table)
        self.pool = hsa.DualPool.allocate([True], 64, 1, self.tables, _i32([0, 0]), hq, hkv, kv_fp8=fmt or False)
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(5)
        self.err = _i32([0])
        self.n = [0, 0]
        self.rope = hsa.Rope(D)
        self.w = [torch.zeros(2, hkv, 24 * PAGE, device="cuda") for _ in range(2)]

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").bfloat16()

    def grow(self, seq, n):
        while len([b for b in self.table[seq] if b >= 0]) * PAGE < n:
            self.table[seq][[b >= 0 for b in self.table[seq]].index(False)] = self.free.pop()
        self.tables.copy_(_i32(self.table))

    def rows(self, seq, h):
        """The sequence's K and V values in the pool, float64."""
        n = self.n[seq]
        t = self.tables[seq].clamp(min=0)
        if self.fmt is None:
            return [ref.rows(x[0], t, n, h).double() for x in (self.pool.k, self.pool.v)]
        kc, ks, vc, vs = self.pool.fp8_views(0)
        f = torch.float8_e4m3fn if self.fmt == "e4m3" else torch.float8_e5m2
        perm = lambda m: 16 * (torch.arange(m, device="cuda") // 16) + torch.tensor(  # noqa: E731
            [4 * ((l % 8) // 2) + l % 2 + 2 * (l // 8) for l in range(16)], device="cuda").repeat(m // 16)
        k = kc[..., perm(D)].view(f).double() * ks.double()[..., None]
        v = vc[..., perm(PAGE)].transpose(-1, -2).contiguous().view(f).double() * vs.double()[..., None]
        return [ref.rows(x, t, n, h) for x in (k, v)]

    def evict(self, budget, **choice):
        """Every sequence cut to the budget; the model of what stays comes from the rows before."""
        hsa, w = self.hsa, self.w[0]
        before = {(s, h): self.rows(s, h) for s in range(2) for h in range(self.hkv)}
        keep, new = hsa.hsa_kv_select(w, _i32(self.n), _i32([0, 1]), budget, dev_err=self.err, **choice)
        pages = [(min(n, budget) + PAGE - 1) // PAGE for n in self.n]
        dst = [[self.free.pop() for _ in range(p)] + [-1] * (max(pages) - p) for p in pages]
        hsa.hsa_kv_compact(self.pool, 0, keep, new, _i32([0, 1]), _i32(dst), w=w, w_dst=self.w[1], dev_err=self.err)
        old = [list(t) for t in self.table]
        picked, weights = keep.tolist(), w.tolist()
        for s in range(2):
            self.free += [b for b in old[s] if b >= 0]
            self.table[s] = [b for b in dst[s] if b >= 0]
            self.table[s] += [-1] * (24 - len(self.table[s]))
        self.tables.copy_(_i32(self.table))
        was, self.n = self.n, new.tolist()
        self.w.reverse()
        for s in range(2):
            assert self.n[s] == min(was[s], budget)
            for h in range(self.hkv):
                want = ref.choose(weights[s][h], was[s], budget, choice["sinks"], choice["recent"], choice["reach"])
                assert picked[s][h][:len(want)] == want
                for x, y in zip(self.rows(s, h), before[s, h]):
                    assert torch.equal(x, y[want])
                assert self.w[0][s, h, :len(want)].tolist() == [weights[s][h][i] for i in want]


def _close(got, want, big):
    assert bool(((got.double() - want).abs() <= want * (2.0 ** -16 * (big + 1) + 2.0 ** -20) + 1e-30).all())


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("hq,hkv", [(16, 2), (8, 8)])
def test_prompt_eviction_decode(fmt, hq, hkv):
    hsa = _hsa()
    s = Server(hsa, fmt, hq, hkv)
    per = hq // hkv
    # ---- the prompt, in one chunk: rotated, attended (bf16), appended ---------------------------
    m = [700, 333]
    cu = _i32([0, m[0], sum(m)])
    q, k, v = s.randn(sum(m), hq, D) * 2, s.randn(sum(m), hkv, D), s.randn(sum(m), hkv, D)
    for i in range(2):
        s.grow(i, m[i])
    q, k = hsa.hsa_rope_kv_append(s.pool, 0, s.rope, q, k, v, cu, _i32([0, 1]), _i32([0, 0]), dev_err=s.err)
    s.n = list(m)
    if fmt is None:
        hsa.hsa_prefill_attn(s.pool, 0, q, k, v, cu, _i32([0, 0]), _i32([0, 1]), max(m), SCALE, dev_err=s.err)
        hsa.hsa_prefill_weights(s.pool, 0, q, cu, _i32(m), _i32([0, 1]), 32, SCALE, s.w[0], dev_err=s.err)
        for i in range(2):
            last = int(cu[i + 1])
            for h in range(hkv):
                keys, vals = s.rows(i, h)
                x = q[last - 32:last, h * per:(h + 1) * per].reshape(-1, D)
                _, p, _ = ref.attend(x, keys, vals, [m[i] - 32 + t for t in range(32) for _ in range(per)], SCALE)
                big = float((x.double().abs() @ keys.abs().T).max()) * SCALE
                _close(s.w[0][i, h, :m[i]], p.sum(0), big)
    else:  # an FP8 layer's prompt is weighed by its last token's decode
        s.w[0].copy_(torch.rand(s.w[0].shape, generator=s.gen, device="cuda"))
    s.evict(256, sinks=4, recent=32, reach=2)
    # ---- decode: attend, weigh, append; positions go on from the prompt's -----------------------
    ws = hsa.decode_weights_workspace(s.pool, 2, 1, s.w[0].shape[2])
    for step in range(70):
        for i in range(2):
            s.grow(i, s.n[i] + 1)
        qkv = s.randn(2, hq + 2 * hkv, D)
        q, k = hsa.hsa_rope(s.rope, qkv[:, :hq], qkv[:, hq:hq + hkv], _i32([m[0] + step, m[1] + step]))
        v = qkv[:, hq + hkv:].contiguous()
        before = {(i, h): s.rows(i, h) for i in range(2) for h in range(hkv)} if step % 23 == 0 else None
        old = s.w[0].clone()
        out = hsa.hsa_decode_attn_weights(s.pool, 0, q.view(2, 1, hq, D), k.view(2, 1, hkv, D), v.view(2, 1, hkv, D), _i32(s.n), SCALE,
                                          s.w[0], w_prev=s.w[0], decay=0.9, workspace=ws, dev_err=s.err, append=True)
        if before:
            for (i, h), (keys, vals) in before.items():
                keys, vals = torch.cat((keys, k[i, h][None].double())), torch.cat((vals, v[i, h][None].double()))
                x = q[i, h * per:(h + 1) * per]
                o, p, mag = ref.attend(x, keys, vals, [s.n[i]] * per, SCALE)
                err = (out[i, 0, h * per:(h + 1) * per].double() - o).abs()
                assert bool((err <= 2.0 ** -8 * (2 * o.abs() + mag) + 2.0 ** -10 * mag).all())
                want = p.sum(0)
                want[:-1] += 0.9 * old[i, h, :s.n[i]].double()
                big = float((x.double().abs() @ keys.abs().T).max()) * SCALE
                _close(s.w[0][i, h, :s.n[i] + 1], want, big)
        s.n = [n + 1 for n in s.n]
        if step == 40:
            s.evict(192, sinks=1, recent=64, reach=0)
    assert int(s.err) == 0 and s.n == [192 + 29] * 2
