"""Rotary positions and the rotating KV append on the GPU, against the formula in 64
bits (tests/rope_ref.py holds it and the derivation of the limits)."""
import pytest
import torch

import rope_ref

pytestmark = pytest.mark.gpu

BASE = 1.0e6
D, PAGE, W = 128, 64, 128


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


def _bf(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _axes(rot, n_axes):
    return [i % n_axes for i in range(rot // 2)]


def _heads(g, n, hq, hkv, fused):
    if fused:
        qkv = _bf(g, n, hq + 2 * hkv, D)
        return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    return _bf(g, n, hq, D), _bf(g, n, hkv, D), _bf(g, n, hkv, D)


def _rope(hsa, rot, n_axes, inter, scale=1.0, inv=None):
    inv = [BASE ** (-2.0 * i / rot) for i in range(rot // 2)] if inv is None else inv
    ax = _axes(rot, n_axes)
    return hsa.Rope(rot, inv_freq=inv, axis_of_pair=ax, interleaved=inter, scale=scale), inv, ax


def _close(got, ref, mag, what):
    err = (got.double().cpu() - ref).abs()
    lim = rope_ref.bf16_limit(ref, mag)
    assert bool((err <= lim).all()), "%s: %g over its limit" % (what, float((err - lim).max()))


CASES = [
    # n, Hq, Hkv, rot, axes, interleaved, fused, scale
    (1, 32, 4, 128, 1, False, True, 1.0),
    (7, 32, 4, 128, 3, False, True, 1.0),
    (33, 16, 2, 64, 1, True, False, 1.0),
    (130, 16, 4, 96, 2, False, True, 1.25),
    (64, 8, 8, 32, 4, True, True, 1.0),
    (257, 5, 3, 16, 1, False, False, -0.5),
    (19, 1, 1, 112, 3, True, False, 1.0),
    (600, 6, 1, 48, 2, False, True, 1.0),
]


@pytest.mark.parametrize("n,hq,hkv,rot,axes,inter,fused,scale", CASES)
def test_rope_matches_the_formula(n, hq, hkv, rot, axes, inter, fused, scale):
    hsa = _hsa()
    g = _gen(n + rot)
    rope, inv, ax = _rope(hsa, rot, axes, inter, scale)
    q, k, _ = _heads(g, n, hq, hkv, fused)
    pos = torch.randint(-1000, 1 << 20, (axes, n), generator=g, device="cuda", dtype=torch.int32)
    before = q.clone(), k.clone()
    qo, ko = hsa.hsa_rope(rope, q, k, pos)
    cos, sin = rope_ref.angles(pos.tolist(), inv, ax)
    for got, x, nm in ((qo, q, "q"), (ko, k, "k")):
        _close(got, *rope_ref.turn(x, cos, sin, rot, inter, scale), nm)
        assert torch.equal(got[..., rot:], x[..., rot:])
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])


@pytest.mark.parametrize("inv", [[1.0, 0.3, 1e-6, -0.7, 6.5, 1e5, -1e-12, 0.0]])
def test_rope_holds_at_every_position(inv):
    """The largest, smallest and negative positions, frequencies above a turn a token,
    negative, tiny and zero."""
    hsa = _hsa()
    g = _gen(5)
    at = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 1048575, -77777, 2 ** 30 + 1]
    rope, inv, ax = _rope(hsa, 16, 1, False, inv=inv)
    x = _bf(g, len(at), 2, D)
    pos = torch.tensor([at], dtype=torch.int32, device="cuda")
    qo, _ = hsa.hsa_rope(rope, x, None, pos)
    cos, sin = rope_ref.angles([at], inv, ax)
    _close(qo, *rope_ref.turn(x, cos, sin, 16, False), "far positions")


def test_rope_in_place_one_side_and_untouched_values():
    hsa = _hsa()
    g = _gen(6)
    rope, inv, ax = _rope(hsa, 64, 1, False)
    x, k = _bf(g, 50, 4, D), _bf(g, 50, 2, D)
    x[3, 1, 64] = float("inf")     # past rot_dim: passes as it is
    x[4, 1, 127] = float("nan")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    a, b = hsa.hsa_rope(rope, x, k, pos)
    assert a[3, 1, 64] == float("inf") and torch.isnan(a[4, 1, 127])
    assert torch.isfinite(a[3, 1, :64].float()).all()
    only_q, none = hsa.hsa_rope(rope, x, None, pos)
    assert none is None and torch.equal(only_q.view(torch.int16), a.view(torch.int16))
    none, only_k = hsa.hsa_rope(rope, None, k, pos)
    assert none is None and torch.equal(only_k, b)
    y, z = x.clone(), k.clone()
    qo, ko = hsa.hsa_rope(rope, y, z, pos, q_out=y, k_out=z)
    assert qo.data_ptr() == y.data_ptr() and torch.equal(y.view(torch.int16), a.view(torch.int16))
    assert torch.equal(z, b)
    # turning by negated positions undoes it, within two roundings
    back, _ = hsa.hsa_rope(rope, b, None, -pos)
    assert float((back.float() - k.float()).abs().max()) <= 2 * 2.0 ** -8 * 2 * float(k.abs().max())
    empty = x[:0]
    qo, _ = hsa.hsa_rope(rope, empty, None, pos[:0])
    assert qo.shape == (0, 4, D)


def _requests(seed, counts, starts):
    """Sequences in another order than the requests, pages scattered, ring rows permuted."""
    g = _gen(seed)
    r = len(counts)
    cu = [sum(counts[:i]) for i in range(r + 1)]
    width = max((s + c + PAGE - 1) // PAGE for s, c in zip(starts, counts)) + 1
    nb = r * width
    tables = torch.randperm(nb, generator=g, device="cuda").int().view(r, width).contiguous()
    rows = torch.randperm(r + 2, generator=g, device="cuda").int()[:r].contiguous()
    seq = torch.randperm(r, generator=g, device="cuda").int()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(cu), seq, i32(starts), tables, rows, nb


LAYERS = ["full", "ring", "e4m3", "e5m2"]
REQUESTS = [
    ([1], [0]),
    ([1, 1, 1, 1, 1], [0, 63, 64, 127, 5000]),
    ([3, 0, 130, 64, 1, 300, 0], [62, 9, 0, 64, 128, 1000, 3]),
    ([1] * 70 + [2] * 3, list(range(0, 730, 10))),
]


def _pool(hsa, layer, tables, rows, nb, hq, hkv, seed):
    g = _gen(seed)
    full = layer != "ring"
    fp8 = layer if layer in ("e4m3", "e5m2") else False
    pool = hsa.DualPool.allocate([full], nb, rows.numel() + 2, tables, rows, hq, hkv, kv_fp8=fp8)
    for t in (pool.k[0], pool.v[0]):
        if fp8:  # finite scales: code bytes and fp32 scales of their own
            t.copy_(torch.randint(0, 60, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        else:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").bfloat16())
    return pool


@pytest.mark.parametrize("layer", ["full", "ring"])
@pytest.mark.parametrize("counts,starts", REQUESTS)
@pytest.mark.parametrize("hq,hkv,fused,inter", [(32, 4, True, False), (16, 2, False, True), (8, 8, True, False)])
def test_append_equals_rope_then_append(layer, counts, starts, hq, hkv, fused, inter):
    """bf16 pools: every bit of the pool (stale rows among it), q_out and k_out."""
    hsa = _hsa()
    cu, seq, start, tables, rows, nb = _requests(1, counts, starts)
    n = sum(counts)
    q, k, v = _heads(_gen(2), n, hq, hkv, fused)
    rope, inv, ax = _rope(hsa, 64, 2, inter)
    pos = torch.randint(0, 9000, (2, n), generator=_gen(3), device="cuda", dtype=torch.int32)
    a, b = (_pool(hsa, layer, tables, rows, nb, hq, hkv, 4) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = hsa.hsa_rope_kv_append(a, 0, rope, q, k, v, cu, seq, start, positions=pos, dev_err=err)
    q1, k1 = hsa.hsa_rope(rope, q, k, pos)
    hsa.hsa_kv_append(b, 0, k1, v.contiguous(), cu, seq, start, dev_err=err)
    assert int(err) == 0
    assert torch.equal(qo, q1) and torch.equal(ko, k1)
    assert torch.equal(a.k[0], b.k[0]) and torch.equal(a.v[0], b.v[0])
    # keys alone, and no turned keys wanted: the pool is the same
    d = _pool(hsa, layer, tables, rows, nb, hq, hkv, 4)
    assert hsa.hsa_rope_kv_append(d, 0, rope, None, k, v, cu, seq, start, positions=pos,
                                  k_out=False, dev_err=err) == (None, None)
    assert torch.equal(a.k[0], d.k[0]) and torch.equal(a.v[0], d.v[0])


@pytest.mark.parametrize("layer", LAYERS)
def test_append_takes_the_cache_position(layer):
    """positions=None: start_pos + i on every axis."""
    hsa = _hsa()
    counts, starts = REQUESTS[2]
    cu, seq, start, tables, rows, nb = _requests(7, counts, starts)
    n = sum(counts)
    q, k, v = _heads(_gen(8), n, 16, 2, True)
    rope, inv, ax = _rope(hsa, 128, 3, False)
    at = torch.tensor([s + i for s, c in zip(starts, counts) for i in range(c)], dtype=torch.int32, device="cuda")
    a, b = (_pool(hsa, layer, tables, rows, nb, 16, 2, 9) for _ in range(2))
    one = hsa.hsa_rope_kv_append(a, 0, rope, q, k, v, cu, seq, start)
    two = hsa.hsa_rope_kv_append(b, 0, rope, q, k, v, cu, seq, start, positions=at.repeat(3, 1).contiguous())
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert torch.equal(a.k[0], b.k[0]) and torch.equal(a.v[0], b.v[0])


PERM16 = torch.tensor([4 * ((l % 8) // 2) + l % 2 + 2 * (l // 8) for l in range(16)])


@pytest.mark.parametrize("layer", ["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,starts", REQUESTS)
@pytest.mark.parametrize("rot,inter,hq,hkv", [(128, False, 32, 4), (96, True, 16, 2), (16, False, 8, 8), (48, False, 4, 1)])
def test_append_fp8_rows(layer, counts, starts, rot, inter, hq, hkv):
    """Scales within the fp32 part; codes the nearest of their grid; other rows as they were."""
    hsa = _hsa()
    top, half_rel, half_sub = (448.0, 2.0 ** -4, 2.0 ** -10) if layer == "e4m3" else (57344.0, 2.0 ** -3, 2.0 ** -17)
    cu, seq, start, tables, rows, nb = _requests(11, counts, starts)
    n = sum(counts)
    q, k, v = _heads(_gen(12), n, hq, hkv, True)
    k[n // 2, 0] = 0               # an all-zero row stores scale 0
    v[0, hkv - 1] = 0
    rope, inv, ax = _rope(hsa, rot, 2, inter)
    pos = torch.randint(0, 90000, (2, n), generator=_gen(13), device="cuda", dtype=torch.int32)
    pool = _pool(hsa, layer, tables, rows, nb, hq, hkv, 14)
    was = [t.clone() for t in pool.fp8_views(0)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = hsa.hsa_rope_kv_append(pool, 0, rope, q, k, v, cu, seq, start, positions=pos, dev_err=err)
    assert int(err) == 0
    kc, ks, vc, vs = pool.fp8_views(0)
    cos, sin = rope_ref.angles(pos.tolist(), inv, ax)
    k64, kmag = rope_ref.turn(k, cos, sin, rot, inter)
    _close(qo, *rope_ref.turn(q, cos, sin, rot, inter), "q")
    _close(ko, k64, kmag, "k")
    v64 = v.double().cpu()
    vmag = v64.abs()
    r = [i for i, c in enumerate(counts) for _ in range(c)]
    at = torch.tensor([s + i for s, c in zip(starts, counts) for i in range(c)])
    sq = seq.cpu().long()[torch.tensor(r)]
    blk, off = tables.cpu()[sq, at // PAGE].long(), at % PAGE
    dt = torch.float8_e4m3fn if layer == "e4m3" else torch.float8_e5m2
    place = 16 * (torch.arange(D) // 16) + PERM16.repeat(D // 16)
    byte = 16 * (off // 16) + PERM16[off % 16]
    got_k = kc.cpu().view(dt).float()[blk, :, off][..., place].double()
    got_v = vc.cpu().view(dt).float()[blk, :, :, byte].double()
    for got, sc, ref, mag, nm in ((got_k, ks, k64, kmag, "k"), (got_v, vs, v64, vmag, "v")):
        s = sc.cpu()[blk, :, off].double()
        want = ref.abs().amax(-1) / top
        slack = (rope_ref.FP32_PART * mag).amax(-1) / top + want * 2.0 ** -23
        assert bool(((s - want).abs() <= slack).all()), nm
        val = got * s[..., None]
        # half a step of the code, the scale's and the value's own fp32 part
        lim = torch.maximum(ref.abs() * half_rel, half_sub * s[..., None]) * (1 + 2.0 ** -6) + \
            mag * rope_ref.FP32_PART * 4
        assert bool(((val - ref).abs() <= lim).all()), nm
        zero = want == 0
        assert bool((s[zero] == 0).all()) and bool((got[zero] == 0).all())
    # what no token was written to is as it was
    keep = torch.ones(nb, PAGE, dtype=torch.bool)
    keep[blk, off] = False
    for now, old, rowdim in ((kc, was[0], 2), (ks, was[1], 2)):
        m = keep[:, None, :].expand(nb, hkv, PAGE).cuda()
        assert torch.equal(now[m], old[m])
    m = torch.ones(nb, hkv, D, PAGE, dtype=torch.bool)
    m[blk, :, :, byte] = False
    assert torch.equal(vc[m.cuda()], was[2][m.cuda()])


@pytest.mark.parametrize("layer", LAYERS)
def test_append_flags_and_skips(layer):
    """Tokens of no request, a negative start, bad sequences and unreachable rows."""
    hsa = _hsa()
    hq, hkv = 16, 2
    tables = torch.tensor([[0, 1], [2, -1], [9, 3], [1, 0]], dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 1, 99, 2], dtype=torch.int32, device="cuda")
    pool = _pool(hsa, layer, tables, rows, 4, hq, hkv, 20)
    k0, v0 = pool.k[0].clone(), pool.v[0].clone()
    n = 8
    q, k, v = _heads(_gen(21), n, hq, hkv, False)
    rope, inv, ax = _rope(hsa, 128, 1, False)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    call = lambda cu, seq, start: hsa.hsa_rope_kv_append(  # noqa: E731
        pool, 0, rope, q, k, v, i32(*cu), i32(*seq), i32(*start),
        positions=torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous(),
        q_out=qo, k_out=ko, dev_err=err)
    want_q, want_k = hsa.hsa_rope(rope, q, k, torch.arange(n, dtype=torch.int32, device="cuda"))

    def fresh():
        return (torch.full_like(q, 7.0), torch.full_like(k, 7.0), i32(0))

    def unchanged():
        return torch.equal(pool.k[0], k0) and torch.equal(pool.v[0], v0)

    # rows behind the last request and at negative cache positions: left as they were
    qo, ko, err = fresh()
    call((2, 2, 2), (0, 3), (0, 0))
    assert int(err) == hsa.HSA_DEVERR_BAD_LEN and unchanged()
    assert bool((qo == 7).all()) and bool((ko == 7).all())
    qo, ko, err = fresh()
    call((0, 8), (0,), (-8,))
    assert int(err) == hsa.HSA_DEVERR_BAD_LEN and unchanged() and bool((qo == 7).all())
    # no such sequence; turned all the same
    for seq in (-1, 4):
        qo, ko, err = fresh()
        call((0, 8), (seq,), (0,))
        assert int(err) == hsa.HSA_DEVERR_BAD_SEQ and unchanged()
        assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    qo, ko, err = fresh()
    if layer == "ring":
        call((0, 8), (2,), (0,))
        assert int(err) == hsa.HSA_DEVERR_BAD_RING and unchanged()
    else:
        call((0, 8), (1,), (64,))      # an unallocated page (-1)
        assert int(err) == hsa.HSA_DEVERR_BAD_BLOCK and unchanged()
        qo, ko, err = fresh()
        call((0, 8), (2,), (0,))       # a page past the pool
        assert int(err) == hsa.HSA_DEVERR_BAD_BLOCK and unchanged()
        qo, ko, err = fresh()
        call((0, 8), (0,), (128,))     # past the block table
        assert int(err) == hsa.HSA_DEVERR_BAD_PAGE and unchanged()
        qo, ko, err = fresh()
        call((0, 8), (0,), (2 ** 31 - 4,))
        assert int(err) == hsa.HSA_DEVERR_BAD_PAGE and unchanged()
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    # no dev_err: skipped as quietly
    hsa.hsa_rope_kv_append(pool, 0, rope, q, k, v, i32(0, 8), i32(7), i32(0))
    assert unchanged()


def test_rope_on_another_stream_and_in_a_graph():
    hsa = _hsa()
    g = _gen(30)
    rope, inv, ax = _rope(hsa, 128, 1, False)
    counts, starts = [1] * 6, [5, 64, 130, 0, 63, 700]
    cu, seq, start, tables, rows, nb = _requests(31, counts, starts)
    q, k, v = _heads(g, 6, 32, 4, True)
    want_pool = _pool(hsa, "full", tables, rows, nb, 32, 4, 32)
    want = hsa.hsa_rope_kv_append(want_pool, 0, rope, q, k, v, cu, seq, start)
    torch.cuda.synchronize()
    for captured in (False, True):
        pool = _pool(hsa, "full", tables, rows, nb, 32, 4, 32)
        qo, ko = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call = lambda: hsa.hsa_rope_kv_append(pool, 0, rope, q, k, v, cu, seq, start,  # noqa: E731
                                                  q_out=qo, k_out=ko)
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    call()
                graph.replay()
                qo.zero_()
                graph.replay()
            else:
                call()
        s.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
        assert torch.equal(pool.k[0], want_pool.k[0]) and torch.equal(pool.v[0], want_pool.v[0])


@pytest.mark.parametrize("layer", ["full", "e4m3", "e5m2"])
def test_append_with_offsets_past_the_tokens(layer):
    """cu_tokens that end past ntok: the tokens that are there are appended, and nothing is read
    behind them (a long FP8 append gathers the values of 16 positions at a time)."""
    hsa = _hsa()
    n = 2100
    tables = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
    rows = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = _heads(_gen(40), n, 16, 2, False)
    rope, inv, ax = _rope(hsa, 128, 1, False)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pools = [_pool(hsa, layer, tables, rows, 40, 16, 2, 41) for _ in range(2)]
    err = i32(0)
    for pool, end in zip(pools, (n, n + 300)):
        hsa.hsa_rope_kv_append(pool, 0, rope, None, k, v, i32(0, end), i32(0), i32(5), k_out=False, dev_err=err)
    assert int(err) == 0
    assert torch.equal(pools[0].k[0], pools[1].k[0]) and torch.equal(pools[0].v[0], pools[1].v[0])


@pytest.mark.parametrize("layer", ["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,starts", [([2048], [0]), ([700, 3, 1500, 40], [9, 62, 16, 1000]), ([2500], [4001])])
def test_long_fp8_append_equals_short_ones(layer, counts, starts):
    """The grouped way of long appends and the token by token way of short ones: every byte of
    the layer, stale rows among them."""
    hsa = _hsa()
    cu, seq, start, tables, rows, nb = _requests(42, counts, starts)
    n = sum(counts)
    q, k, v = _heads(_gen(43), n, 16, 2, True)
    v[5, 1] = 0
    v[n - 1, 0, 3] = 300.0
    rope, inv, ax = _rope(hsa, 64, 1, True)
    a, b = (_pool(hsa, layer, tables, rows, nb, 16, 2, 44) for _ in range(2))
    hsa.hsa_rope_kv_append(a, 0, rope, None, k, v, cu, seq, start, k_out=False)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for r, c in enumerate(counts):
        for lo in range(0, c, 999):
            hi = min(c, lo + 999)
            at = slice(int(cu[r]) + lo, int(cu[r]) + hi)
            hsa.hsa_rope_kv_append(b, 0, rope, None, k[at], v[at], i32([0, hi - lo]), seq[r:r + 1].contiguous(),
                                   i32([starts[r] + lo]), k_out=False)
    assert torch.equal(a.k[0], b.k[0]) and torch.equal(a.v[0], b.v[0])


@pytest.mark.parametrize("layer", LAYERS)
def test_a_sequence_in_many_requests_of_one_call(layer):
    """One call that names a sequence many times, its ranges end to end (they meet inside groups
    of 16 positions): every byte as from one request."""
    hsa = _hsa()
    counts = [17, 5, 70, 1, 30, 64, 41] * 9 + [50]
    n = sum(counts)
    assert n >= 2048 and n >= 32 * len(counts)
    cu, starts = [0], [7]
    for c in counts:
        cu.append(cu[-1] + c)
        starts.append(starts[-1] + c)
    tables = torch.randperm(40, generator=_gen(50), device="cuda").int().view(1, 40).contiguous()
    rows = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = _heads(_gen(51), n, 16, 2, True)
    rope, inv, ax = _rope(hsa, 128, 1, False)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    a, b = (_pool(hsa, layer, tables, rows, 40, 16, 2, 52) for _ in range(2))
    tail = slice(n - 100, n)           # a ring of 128 slots holds the last tokens alone
    if layer == "ring":
        cu, starts = [0, 17, 22, 92, 93, 100], [7, 24, 29, 99, 100, 107]
        q, k, v, n = q[tail], k[tail], v[tail], 100
    one = hsa.hsa_rope_kv_append(a, 0, rope, q, k, v, i32(cu), i32([0] * (len(cu) - 1)), i32(starts[:len(cu) - 1]))
    two = hsa.hsa_rope_kv_append(b, 0, rope, q, k, v, i32([0, n]), i32([0]), i32([7]))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert torch.equal(a.k[0], b.k[0]) and torch.equal(a.v[0], b.v[0])
