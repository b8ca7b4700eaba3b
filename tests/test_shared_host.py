"""Host side of the shared-prefix decode, without a GPU: refusals, workspace size, and the
arithmetic of its segments and slots."""
import ctypes
import random

import pytest
import torch

import test_binding_host as host
import test_cabi as cabi
from full_attention_kv_gb300 import binding

fake = host.fake


def test_shared_arguments_refused():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    INV, UNS, OK = hsa.HSA_INVALID_ARG, hsa.HSA_UNSUPPORTED_SHAPE, hsa.HSA_OK
    base = dict(p=ctypes.byref(cabi._pools(hsa)), layer=1, q=256, k=256, v=256, cl=256, cu=256, sl=256, n=1,
                B=2, T=1, scale=0.1, out=256, ws=256, bytes=0, ctas=0, opts=0)

    def call(**kw):
        a = dict(base, **kw)
        return L.hsa_decode_attn_shared(a["p"], a["layer"], a["q"], a["k"], a["v"], a["cl"], a["cu"], a["sl"], a["n"],
                                        a["B"], a["T"], a["scale"], a["out"], a["ws"], a["bytes"], a["ctas"], a["opts"],
                                        None, None)
    assert call(p=None) == INV and call(layer=2) == INV and call(opts=4) == INV
    assert call(n=-1) == INV and call(cu=None) == INV and call(sl=None) == INV
    assert call(scale=0.0) == INV and call(scale=-1.0) == INV and call(scale=float("nan")) == INV
    assert call(scale=float("inf")) == INV
    assert call(B=3) == INV and call(B=-1) == INV and call(T=0) == INV and call(ctas=-1) == INV
    assert call(T=5) == UNS and call(q=264) == INV and call(cl=None) == INV and call(out=None) == INV
    assert call(B=0, n=0, q=None, k=None, v=None, cl=None, cu=None, sl=None, out=None, ws=None) == OK
    assert call(p=ctypes.byref(cabi._pools(hsa, d=64))) == UNS


def test_shared_workspace_covers_the_plain_one():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    p = ctypes.byref(cabi._pools(hsa, batch=64))
    f = L.hsa_decode_shared_workspace_bytes
    assert f(None, 1, 1, 1) == 0 and f(p, -1, 1, 1) == 0 and f(p, 1, 1, -1) == 0 and f(p, 1, 0, 1) == 0
    last = 0
    for B, T, n in ((1, 1, 0), (1, 1, 1), (8, 1, 1), (8, 4, 8), (64, 4, 64)):
        size = f(p, B, T, n)
        assert size >= L.hsa_decode_workspace_bytes(p, B, T) and size > last
        last = size


def test_shared_binding_checks(fake):
    bf, i32 = host._bf, host._i32
    pool = host._pool()
    B, T = 3, 2
    q, k, v, cl = bf(B, T, host.Hq, 128), bf(B, T, host.Hkv, 128), bf(B, T, host.Hkv, 128), i32(B)
    ws = torch.zeros(64, dtype=torch.uint8)
    binding.hsa_decode_attn_shared(pool, 1, q, k, v, cl, i32(3), i32(2), 0.1, workspace=ws, stream=0, append=True)
    name, a = fake.calls[-1]
    assert name == "hsa_decode_attn_shared" and a[8:11] == (2, B, T) and a[16] == binding.HSA_DECODE_APPEND
    done = len(fake.calls)
    for bad in [(q, k, v, cl, i32(2), i32(2)), (q, k, v, cl, i32(4), i32(2)), (q, k, v, i32(B - 1), i32(3), i32(2)),
                (q[:, :1].contiguous(), k, v, cl, i32(3), i32(2)), (q, k[:, :, :1].contiguous(), v, cl, i32(3), i32(2)),
                (q, k, v, cl, i32(3, 1), i32(2))]:
        with pytest.raises(ValueError):
            binding.hsa_decode_attn_shared(pool, 1, *bad, 0.1, workspace=ws, stream=0)
    with pytest.raises(TypeError):
        binding.hsa_decode_attn_shared(pool, 1, q, k, v, cl, i32(3).long(), i32(2), 0.1, workspace=ws, stream=0)
    assert len(fake.calls) == done


@pytest.mark.parametrize("seed", range(60))
def test_segments_cover_the_items_and_slots_are_their_own(seed):
    """Part 1's split: every (unit, page) in exactly one segment; a segment's slot, CTA + unit,
    is its own and inside the workspace's count; and the range of CTAs that the merge computes
    for a unit is the one that wrote it."""
    rng = random.Random(seed)
    G, T, Hkv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4]), rng.choice([1, 2, 4, 8])
    members = [rng.choice([0, 1, 2, 5, 40, 300]) for _ in range(rng.randint(1, 40))]
    pages = [rng.choice([0, 0, 1, 2, 3, 17, 200]) for _ in members]
    ctas = rng.choice([1, 2, 13, 152])
    B = sum(members)
    weight = lambda rows: 1 if rows <= 128 else 2  # noqa: E731
    groups, item0, unit0 = [], 0, 0
    for m, pg in zip(members, pages):
        rows = m * T * G
        pairs = (rows + 255) // 256 if pg else 0
        head = pg * (2 * (pairs - 1) + weight(rows - (pairs - 1) * 256)) if pairs else 0
        groups.append((item0, unit0, pairs, pg, rows, head))
        item0 += head * Hkv
        unit0 += pairs * Hkv
    N, slots = item0, ctas + (B * T * G // 256 + min(len(members), B)) * Hkv
    if N == 0:
        return
    C = (N + 1) // 2 if N < 2 * ctas else ctas
    wrote, used = {}, set()
    for c in range(C):
        it, i1 = c * N // C, (c + 1) * N // C
        while it < i1:
            g = next(k for k, x in enumerate(groups) if x[0] <= it < x[0] + x[5] * Hkv)
            s, u0, pr, pg, rows, head = groups[g]
            h, in_head = divmod(it - s, head)
            pair = min(in_head // (2 * pg), pr - 1)
            wt = weight(rows - pair * 256)
            o0 = in_head - pair * 2 * pg
            o1 = min(pg * wt, o0 + i1 - it)
            it += o1 - o0
            n0, n1 = -(-o0 // wt), -(-o1 // wt)
            if n0 == n1:
                continue
            u = h * pr + pair
            slot = c + u0 + u
            assert slot not in used and slot < slots
            used.add(slot)
            wrote.setdefault((g, u), []).append((c, n0, n1, slot))
    for g, (s, u0, pr, pg, rows, head) in enumerate(groups):
        for u in range(pr * Hkv):
            segs = wrote[(g, u)]
            assert segs[0][1] == 0 and segs[-1][2] == pg
            assert all(a[2] == b[1] for a, b in zip(segs, segs[1:]))
            h, pair = divmod(u, pr)
            a = s + h * head + pair * 2 * pg
            b = a + (pg - 1) * weight(rows - pair * 256)
            lo, hi = ((a + 1) * C - 1) // N, ((b + 1) * C - 1) // N
            assert [x[0] for x in segs] == list(range(lo, hi + 1))
            assert [x[3] for x in segs] == [c + u0 + u for c in range(lo, hi + 1)]
