"""Host side of the rotary entry points, without a GPU: refusals of the C ABI and of the
binding, and the request search of the append kernel."""
import ctypes

import pytest
import torch

import test_binding_host as host
import test_cabi as cabi
from full_attention_kv_gb300 import binding

fake = host.fake


def _rope(n=64, rot=128, axes=1, inter=0, scale=1.0, inv=0.5, axis=None):
    import full_attention_kv_gb300 as hsa
    f = (ctypes.c_double * n)(*([inv] * n))
    a = (ctypes.c_uint8 * n)(*axis) if axis is not None else None
    p = hsa.HsaRopeParams(rot_dim=rot, n_axes=axes, interleaved=inter, scale=scale,
                          inv_freq=ctypes.cast(f, ctypes.POINTER(ctypes.c_double)),
                          axis_of_pair=ctypes.cast(a, ctypes.POINTER(ctypes.c_uint8)) if a else None)
    p._keep = (f, a)
    return p


BAD_ROPE = [
    (dict(rot=0), "HSA_UNSUPPORTED_SHAPE"),
    (dict(rot=24), "HSA_UNSUPPORTED_SHAPE"),
    (dict(rot=144, n=72), "HSA_UNSUPPORTED_SHAPE"),
    (dict(rot=-16), "HSA_UNSUPPORTED_SHAPE"),
    (dict(axes=0), "HSA_INVALID_ARG"),
    (dict(axes=5), "HSA_INVALID_ARG"),
    (dict(inter=2), "HSA_INVALID_ARG"),
    (dict(scale=float("nan")), "HSA_INVALID_ARG"),
    (dict(inv=float("inf")), "HSA_INVALID_ARG"),
    (dict(inv=float("nan")), "HSA_INVALID_ARG"),
    (dict(inv=1e15), "HSA_INVALID_ARG"),
    (dict(axes=2, axis=[0] * 63 + [2]), "HSA_INVALID_ARG"),
]


@pytest.mark.parametrize("change,status", BAD_ROPE)
def test_rope_descriptions_refused(change, status):
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    want = getattr(hsa, status)
    r = ctypes.byref(_rope(**change))
    assert L.hsa_rope(r, 4096, 0, 65536, 0, 256, 1, 1, 1, 128, 131072, 262144, None) == want
    p = ctypes.byref(cabi._pools(hsa))
    assert L.hsa_rope_kv_append(p, 1, r, 4096, 0, 65536, 0, 131072, 0, 256, 256, 256, 256, 1, 1,
                                262144, 524288, None, None) == want


def test_rope_arguments_refused():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    INV, OK = hsa.HSA_INVALID_ARG, hsa.HSA_OK
    r = ctypes.byref(_rope())
    q, k, qo, ko, pos = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 256
    call = lambda n=4, Hq=32, Hkv=4, d=128, q=q, qs=0, k=k, ks=0, pos=pos, qo=qo, ko=ko, r=r: \
        L.hsa_rope(r, q, qs, k, ks, pos, n, Hq, Hkv, d, qo, ko, None)  # noqa: E731
    assert call(r=None) == INV
    assert call(n=-1) == INV and call(Hq=-1) == INV and call(Hkv=-1) == INV
    assert call(d=64) == hsa.HSA_UNSUPPORTED_SHAPE
    assert call(q=None) == INV and call(k=None) == INV and call(pos=None) == INV
    assert call(qo=None) == INV and call(ko=None) == INV
    assert call(q=q + 8) == INV and call(ko=ko + 2) == INV
    assert call(qs=32 * 128 - 8) == INV      # a token's heads do not fit its stride
    assert call(qs=32 * 128 + 4) == INV      # 16-byte steps
    assert call(ks=-8) == INV
    # outputs over inputs or over each other; in place only where the rows are the same
    assert call(qo=k) == INV and call(ko=q) == INV and call(ko=qo) == INV
    assert call(qo=q + 4096) == INV
    assert call(qo=q, qs=40 * 128) == INV
    assert call(n=0, q=None, k=None, pos=None, qo=None, ko=None) == OK
    assert call(Hq=0, Hkv=0, q=None, k=None, qo=None, ko=None) == OK


def test_rope_append_arguments_refused():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    INV, OK = hsa.HSA_INVALID_ARG, hsa.HSA_OK
    r, p = ctypes.byref(_rope()), ctypes.byref(cabi._pools(hsa))
    M = 1 << 20
    base = dict(p=p, layer=1, r=r, q=M, qs=0, k=2 * M, ks=0, v=3 * M, vs=0, pos=256, cu=256, seq=256,
                start=256, R=1, n=4, qo=4 * M, ko=5 * M)

    def call(**kw):
        a = dict(base, **kw)
        return L.hsa_rope_kv_append(a["p"], a["layer"], a["r"], a["q"], a["qs"], a["k"], a["ks"],
                                    a["v"], a["vs"], a["pos"], a["cu"], a["seq"], a["start"],
                                    a["R"], a["n"], a["qo"], a["ko"], None, None)
    assert call(p=None) == INV and call(layer=2) == INV and call(r=None) == INV
    assert call(R=-1) == INV and call(n=-1) == INV
    assert call(cu=None) == INV and call(seq=None) == INV and call(start=None) == INV
    assert call(k=None) == INV and call(v=None) == INV and call(v=3 * M + 8) == INV
    assert call(q=None) == INV and call(qo=None) == INV   # both or neither
    assert call(vs=4 * 128 - 8) == INV and call(ks=12) == INV
    assert call(qo=3 * M) == INV and call(ko=M) == INV and call(ko=4 * M) == INV
    assert call(ko=2 * M, ks=48 * 128) == INV
    assert call(n=0, q=None, k=None, v=None, qo=None, ko=None) == OK
    assert call(R=0) == OK
    assert call(p=ctypes.byref(cabi._pools(hsa, d=64))) == hsa.HSA_UNSUPPORTED_SHAPE


def test_rope_builder():
    r = binding.Rope(128, base=10000.0, sections=(16, 24, 24))
    assert r.n_axes == 3 and list(r._axis) == [0] * 16 + [1] * 24 + [2] * 24
    assert r._inv[0] == 1.0 and abs(r._inv[32] - 0.01) < 1e-12
    assert binding.Rope(64, inv_freq=torch.ones(32)).c.rot_dim == 64
    assert binding.Rope(32, axis_of_pair=[0, 1] * 8).n_axes == 2
    for kw in (dict(sections=(16, 24)), dict(sections=(-1, 65)), dict(inv_freq=[1.0] * 63),
               dict(axis_of_pair=[0] * 63), dict(axis_of_pair=[4] * 64), dict(axis_of_pair=[-1] * 64),
               dict(sections=(64,), axis_of_pair=[0] * 64), dict(sections=(60, 1, 1, 1, 1))):
        with pytest.raises(ValueError):
            binding.Rope(128, **kw)


def test_rope_binding_checks(fake):
    bf, i32 = host._bf, host._i32
    r = binding.Rope(128, sections=(16, 24, 24))
    n = 6
    qkv = bf(n, host.Hq + 2 * host.Hkv, 128)
    q, k, v = qkv[:, :host.Hq], qkv[:, host.Hq:host.Hq + host.Hkv], qkv[:, host.Hq + host.Hkv:]
    binding.hsa_rope(r, q, k, i32(3, n), stream=0)
    name, a = fake.calls[-1]
    row = (host.Hq + 2 * host.Hkv) * 128
    assert name == "hsa_rope" and (a[2], a[4]) == (row, row) and a[6:10] == (n, host.Hq, host.Hkv, 128)
    pool = host._pool()
    cu, seq, start = i32(3), i32(2), i32(2)
    binding.hsa_rope_kv_append(pool, 0, r, q, k, v, cu, seq, start, positions=i32(3, n), stream=0)
    name, a = fake.calls[-1]
    assert name == "hsa_rope_kv_append" and (a[4], a[6], a[8]) == (row,) * 3 and a[13:15] == (2, n)
    binding.hsa_rope_kv_append(pool, 1, r, None, k, v, cu, seq, start, k_out=False, stream=0)
    a = fake.calls[-1][1]
    assert a[3] is None and a[9] is None and a[15] is None and a[16] is None
    done = len(fake.calls)
    for args in [(q, k, i32(2, n)), (q, k, i32(3, n + 1)), (q, k[:-1], i32(3, n)), (q[..., :64], k, i32(3, n)),
                 (q.transpose(0, 1), k, i32(3, n)), (q[:, :, ::2], k, i32(3, n)), (q[:1].expand(n, -1, -1), k, i32(3, n)),
                 (None, None, i32(3, n)), (qkv[0], k, i32(3, n)), (qkv[:, ::2], k, i32(3, n))]:
        with pytest.raises(ValueError):
            binding.hsa_rope(r, *args, stream=0)
    with pytest.raises(TypeError):
        binding.hsa_rope(r, q.float(), k, i32(3, n), stream=0)
    with pytest.raises(ValueError):
        binding.hsa_rope(r, q, k, i32(3, n), q_out=bf(n, host.Hq - 1, 128), stream=0)
    for kw in (dict(q=q[:, :-1]), dict(k=k[:, :1]), dict(v=v[:-1]), dict(cu=i32(2)), dict(start=i32(3)),
               dict(pos=i32(3, n - 1)), dict(qo=bf(n + 1, host.Hq, 128)), dict(ko=bf(n, host.Hq, 128))):
        with pytest.raises(ValueError):
            binding.hsa_rope_kv_append(pool, 1, r, kw.get("q", q), kw.get("k", k), kw.get("v", v), kw.get("cu", cu), seq,
                                       kw.get("start", start), positions=kw.get("pos", i32(3, n)), q_out=kw.get("qo"),
                                       k_out=kw.get("ko"), stream=0)
    assert len(fake.calls) == done


def _search(cu, R, tok):
    """The kernel's 32-way search, lane by lane; every read inside cu."""
    lo, hi = 0, R
    while hi - lo > 1:
        step = (hi - lo + 31) // 32
        k = 0
        for lane in range(32):
            at = lo + (lane + 1) * step
            if at < hi:
                assert 0 < at < len(cu) - 1 + 1
                k += cu[at] <= tok
        nlo = lo + k * step
        hi, lo = min(hi, nlo + step), nlo
        assert 0 <= lo < hi <= R
    return lo


@pytest.mark.parametrize("R", [1, 2, 31, 32, 33, 64, 65, 1000, 1025])
def test_request_search(R):
    g = torch.Generator().manual_seed(R)
    counts = torch.randint(0, 4, (R,), generator=g).tolist()
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    owner = [r for r, c in enumerate(counts) for _ in range(c)]
    for tok, r in enumerate(owner):
        assert _search(cu, R, tok) == r
    _search(cu, R, cu[-1] + 5)
    _search([0] + torch.randint(-50, 50, (R,), generator=g).tolist(), R, 3)  # out of order: ends, in bounds
