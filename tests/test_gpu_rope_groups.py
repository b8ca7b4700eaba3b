"""The two ways in which a rotating append writes an FP8 layer's values -- by groups of keys,
and beside a token's keys -- around the sizes where the call changes from one to the other:
one call's pool is that of many short ones, byte for byte."""
import pytest
import torch

import test_gpu_shared as base

pytestmark = pytest.mark.gpu

D, PAGE = 128, 64
# by groups from n (Hkv + 4) = 12000 on where requests have 300 tokens and more, from 18000
# where they are shorter, and from 32 tokens a request
CASES = [(hq, hkv, [c]) for hq, hkv, at in ((16, 2, 2000), (32, 4, 1500), (8, 8, 1000)) for c in (at - 1, at, at + 17)]
CASES += [(32, 4, [140] * 16), (32, 4, [141] * 16), (8, 8, [93, 94] * 8), (8, 8, [95, 94] * 8), (4, 1, [2405]),
          (16, 2, [31] * 99), (16, 2, [33] * 99), (32, 4, [299, 301, 1, 1000]), (32, 4, [1201, 300, 2])]


@pytest.mark.parametrize("layer", ["e4m3", "e5m2"])
@pytest.mark.parametrize("hq,hkv,counts", CASES)
def test_values_by_groups_equal_values_beside_the_keys(layer, hq, hkv, counts):
    hsa = base._hsa()
    g = base._gen(sum(counts) + hkv)
    R, n = len(counts), sum(counts)
    starts = torch.randint(0, 100, (R,), generator=torch.Generator().manual_seed(n)).tolist()
    wide = max(c + s for c, s in zip(counts, starts)) // PAGE + 1
    table = torch.randperm(R * wide, generator=g, device="cuda").int().view(R, wide)
    pools = [hsa.DualPool.allocate([True], R * wide, R, table, torch.zeros(R, dtype=torch.int32, device="cuda"),
                                   hq, hkv, kv_fp8=layer) for _ in range(2)]
    rope = hsa.Rope(D)
    qkv = torch.randn(n, hq + 2 * hkv, D, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    cu = [sum(counts[:i]) for i in range(R + 1)]
    err = base._i32([0])
    one = hsa.hsa_rope_kv_append(pools[0], 0, rope, q, k, v, base._i32(cu), base._i32(list(range(R))),
                                 base._i32(starts), dev_err=err)
    for r in range(R):
        for at in range(0, counts[r], 150):
            m = min(150, counts[r] - at)
            part = slice(cu[r] + at, cu[r] + at + m)
            few = hsa.hsa_rope_kv_append(pools[1], 0, rope, q[part], k[part], v[part], base._i32([0, m]), base._i32([r]),
                                         base._i32([starts[r] + at]), dev_err=err)
            assert torch.equal(few[0], one[0][part]) and torch.equal(few[1], one[1][part])
    for a, b in ((pools[0].k[0], pools[1].k[0]), (pools[0].v[0], pools[1].v[0])):
        assert torch.equal(a, b)
    assert int(err) == 0


def _call(hsa, pool, rope, qkv, hq, hkv, cu, seq, starts, part=slice(None), err=None):
    q, k, v = qkv[part, :hq], qkv[part, hq:hq + hkv], qkv[part, hq + hkv:]
    return hsa.hsa_rope_kv_append(pool, 0, rope, None, k, v, base._i32(cu), base._i32(seq), base._i32(starts),
                                  k_out=False, dev_err=err)


@pytest.mark.parametrize("layer", ["e4m3", "e5m2"])
def test_a_sequence_in_many_requests_by_groups(layer):
    """One call that names a sequence many times, its ranges end to end: they meet inside groups
    of 16 positions, whose bytes are then written by several warps."""
    hsa = base._hsa()
    hq = hkv = 8
    counts = [17, 5, 70, 1, 30, 64, 41] * 9 + [50]
    n = sum(counts)
    assert n * (hkv + 4) >= 18000 and n >= 32 * len(counts)
    table = torch.randperm(40, generator=base._gen(50), device="cuda").int().view(1, 40).contiguous()
    pools = [hsa.DualPool.allocate([True], 40, 1, table, base._i32([0]), hq, hkv, kv_fp8=layer) for _ in range(3)]
    qkv = torch.randn(n, hq + 2 * hkv, D, generator=base._gen(51), device="cuda").bfloat16()
    rope = hsa.Rope(D)
    cu = [sum(counts[:i]) for i in range(len(counts) + 1)]
    _call(hsa, pools[0], rope, qkv, hq, hkv, cu, [0] * len(counts), [7 + c for c in cu[:-1]])
    _call(hsa, pools[1], rope, qkv, hq, hkv, [0, n], [0], [7])
    for at in range(0, n, 100):
        m = min(100, n - at)
        _call(hsa, pools[2], rope, qkv, hq, hkv, [0, m], [0], [7 + at], slice(at, at + m))
    for p in pools[1:]:
        assert torch.equal(pools[0].k[0], p.k[0]) and torch.equal(pools[0].v[0], p.v[0])


def test_rows_that_cannot_be_reached_by_groups():
    """Entries and sequences that are not there, starts below 0, tokens of no request, pages past
    the block table: flagged, nothing of them written, the rest as by short calls."""
    hsa = base._hsa()
    hq, hkv = 32, 4
    counts, starts = [700, 400, 300, 500, 350], [5, -20, 3, 60, 9]
    seq, first = [0, 1, 9, 2, 3], 100
    n = first + sum(counts) + 40  # tokens before and behind every request
    assert n * (hkv + 4) >= 12000 and n >= 300 * len(counts)
    table = torch.arange(4 * 12, dtype=torch.int32, device="cuda").view(4, 12)[:, :9].contiguous()
    table[0, 2], table[2, 4], table[3, 0] = -1, 48, 2 ** 31 - 1
    pools = [hsa.DualPool.allocate([True], 48, 4, table, base._i32([0] * 4), hq, hkv, kv_fp8="e4m3") for _ in range(2)]
    for p in pools:
        for t in (p.k[0], p.v[0]):
            t.copy_(torch.randint(0, 60, t.shape, generator=base._gen(60), device="cuda", dtype=torch.uint8))
    qkv = torch.randn(n, hq + 2 * hkv, D, generator=base._gen(61), device="cuda").bfloat16()
    rope = hsa.Rope(D)
    cu = [first + sum(counts[:i]) for i in range(len(counts) + 1)]
    errs = [base._i32([0]) for _ in pools]
    _call(hsa, pools[0], rope, qkv, hq, hkv, cu, seq, starts, err=errs[0])
    for r, c in enumerate(counts):
        for at in range(0, c, 150):
            m = min(150, c - at)
            _call(hsa, pools[1], rope, qkv, hq, hkv, [0, m], seq[r:r + 1], [starts[r] + at],
                  slice(cu[r] + at, cu[r] + at + m), err=errs[1])
    assert torch.equal(pools[0].k[0], pools[1].k[0]) and torch.equal(pools[0].v[0], pools[1].v[0])
    want = hsa.HSA_DEVERR_BAD_LEN | hsa.HSA_DEVERR_BAD_SEQ | hsa.HSA_DEVERR_BAD_BLOCK | hsa.HSA_DEVERR_BAD_PAGE
    assert int(errs[0]) == want and int(errs[1]) == want
