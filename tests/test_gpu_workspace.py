"""One decode workspace, sized for the pools' whole batch, under calls of different batch
sizes: what a smaller call leaves in it must not reach a larger one's arrival counters.
Each result is compared bit for bit with the same call on a workspace of its own."""
import pytest
import torch

import test_gpu_shared as base

pytestmark = pytest.mark.gpu

D, PAGE, W, SCALE = base.D, base.PAGE, base.W, base.SCALE
BATCH, HQ, HKV, WIDTH = 32, 32, 4, 12


class Layers:
    """A full bf16 and a sliding layer, and an FP8 full layer, of pools with the same batch."""

    def __init__(self, hsa, T, seed=1):
        g = base._gen(seed)
        self.hsa, self.T = hsa, T
        shared = 4  # pages, in groups of eight rows
        nb = BATCH // 8 * shared + BATCH * (WIDTH - shared)
        ids = torch.randperm(nb, generator=g, device="cuda").int()
        heads = ids[:BATCH // 8 * shared].view(-1, 1, shared).expand(-1, 8, -1).reshape(BATCH, shared)
        self.table = torch.cat((heads, ids[BATCH // 8 * shared:].view(BATCH, -1)), 1).contiguous()
        rows = torch.randperm(BATCH, generator=g, device="cuda").int()
        self.cl = torch.randint(4 * PAGE, WIDTH * PAGE - T, (BATCH,), generator=g, device="cuda").int()
        bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.q, self.k, self.v = bf(BATCH, T, HQ, D), bf(BATCH, T, HKV, D), bf(BATCH, T, HKV, D)
        self.pool = hsa.DualPool([True, False], [bf(nb, HKV, PAGE, D), bf(BATCH, HKV, W, D)],
                                 [bf(nb, HKV, PAGE, D), bf(BATCH, HKV, W, D)], self.table, rows, HQ)
        self.fp8 = hsa.DualPool.allocate([True], nb, BATCH, self.table, rows, HQ, HKV, kv_fp8="e4m3")
        n = WIDTH * PAGE
        for b in range(BATCH):  # (shared pages are written by every one of their sequences)
            hsa.hsa_kv_append(self.fp8, 0, bf(n, HKV, D), bf(n, HKV, D), base._i32([0, n]), base._i32([b]),
                              base._i32([0]))
        self.cu = base._i32(list(range(0, BATCH + 1, 8)))
        self.sl = base._i32([shared * PAGE] * (BATCH // 8))

    def run(self, what, B, ws):
        """The output, in a buffer that holds NaN before the call."""
        out = torch.full_like(self.q[:B], float("nan"))
        a = (self.q[:B], self.k[:B], self.v[:B], self.cl[:B])
        if what == "shared":
            return self.hsa.hsa_decode_attn_shared(self.pool, 0, *a, self.cu[:B // 8 + 1], self.sl[:B // 8], SCALE,
                                                   out=out, workspace=ws)
        pool, layer = {"full": (self.pool, 0), "ring": (self.pool, 1), "fp8": (self.fp8, 0)}[what]
        return self.hsa.hsa_decode_attn(pool, layer, *a, SCALE, out=out, workspace=ws)


@pytest.mark.parametrize("T", [1, 3])
def test_workspace_of_the_largest_batch_serves_smaller_ones(T):
    hsa = base._hsa()
    c = Layers(hsa, T)
    ws = hsa.decode_shared_workspace(c.pool, BATCH, T, BATCH // 8)
    assert ws.numel() >= hsa.hsa_decode_workspace_bytes(c.pool, BATCH, T)

    def fresh():
        return torch.zeros_like(ws)

    plan = []
    for first in ("shared", "full", "fp8", "ring"):
        for then in ("full", "fp8", "ring", "shared"):
            # 17 sequences x 4 heads leave a ring's two halves to two CTAs
            plan += [(first, 8), (then, 17 if then == "ring" else BATCH), (first, 16), (then, 24)]
    want = {p: c.run(*p, fresh()) for p in set(plan)}
    for p, w in want.items():
        assert not bool(w.isnan().any()), p
    for i, p in enumerate(plan):
        got = c.run(*p, ws)
        assert torch.equal(got, want[p]), "call %d, %s of %d sequences after %s of %d" % ((i,) + p + plan[i - 1])


def test_workspace_between_pools_of_the_plain_sizes():
    """The plain call's own workspace, small batches and large ones in turn."""
    hsa = base._hsa()
    c = Layers(hsa, 1, seed=2)
    ws = hsa.decode_workspace(c.pool, BATCH, 1)
    want = {B: c.run("full", B, torch.zeros_like(ws)) for B in (1, 5, 16, 31, BATCH)}
    for B in (1, BATCH, 5, 31, 16, BATCH, 1, 31):
        assert torch.equal(c.run("full", B, ws), want[B]), B
