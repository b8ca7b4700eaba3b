"""Host side of the eviction entry points, without a GPU: refusals of the C ABI and of the
binding, and the order of the selection kernel's keys."""
import ctypes
import math
import struct

import pytest
import torch

import test_binding_host as host
import test_cabi as cabi
from full_attention_kv_gb300 import binding

fake = host.fake
M = 1 << 20


def _f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def test_select_arguments_refused():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    INV, OK = hsa.HSA_INVALID_ARG, hsa.HSA_OK
    base = dict(w=M, stride=64, batch=4, heads=2, n=256, seq=256, R=2, budget=16, sinks=4, recent=8, reach=1,
                keep=2 * M, new=512)

    def call(**kw):
        a = dict(base, **kw)
        return L.hsa_kv_select(a["w"], a["stride"], a["batch"], a["heads"], a["n"], a["seq"], a["R"], a["budget"],
                               a["sinks"], a["recent"], a["reach"], a["keep"], a["new"], None, None)
    for kw in (dict(w=None), dict(w=M + 4), dict(stride=62), dict(stride=-4), dict(batch=-1), dict(heads=0),
               dict(n=None), dict(seq=None), dict(R=-1), dict(budget=-1), dict(sinks=-1), dict(recent=-1),
               dict(reach=-1), dict(sinks=9), dict(keep=None), dict(new=None), dict(R=1 << 27),
               dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(new=256), dict(new=260), dict(new=252)):
        assert call(**kw) == INV, kw
    assert call(reach=8) == hsa.HSA_UNSUPPORTED_SHAPE and call(stride=(1 << 22) + 4) == hsa.HSA_UNSUPPORTED_SHAPE
    assert call(R=0, w=None, n=None, seq=None, keep=None, new=None) == OK


def test_compact_arguments_refused():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    INV, SHAPE, OK = hsa.HSA_INVALID_ARG, hsa.HSA_UNSUPPORTED_SHAPE, hsa.HSA_OK
    base = dict(p=ctypes.byref(cabi._pools(hsa)), layer=1, keep=M, heads=4, budget=64, new=256, seq=256, R=2, dst=512,
                blocks=1, w=2 * M, wd=3 * M, stride=64)

    def call(**kw):
        a = dict(base, **kw)
        return L.hsa_kv_compact(a["p"], a["layer"], a["keep"], a["heads"], a["budget"], a["new"], a["seq"], a["R"], a["dst"],
                                a["blocks"], a["w"], a["wd"], a["stride"], None, None)
    assert call(layer=0) == SHAPE  # a ring evicts by position
    assert call(heads=2) == SHAPE and call(heads=0) == SHAPE
    for kw in (dict(p=None), dict(layer=2), dict(keep=None), dict(budget=-1), dict(new=None), dict(seq=None), dict(R=-1),
               dict(dst=None), dict(blocks=-1), dict(w=None), dict(wd=None), dict(w=2 * M + 4), dict(wd=3 * M + 8),
               dict(stride=63), dict(stride=-4), dict(wd=2 * M), dict(wd=2 * M + 16), dict(wd=2 * M - 16),
               dict(R=1 << 30)):
        assert call(**kw) == INV, kw
    assert call(R=0, keep=None, dst=None) == OK and call(budget=0) == OK
    for change, layer, status in cabi._BAD_POOLS:
        p = ctypes.byref(cabi._pools(hsa, **dict(change)))
        assert call(p=p, layer=layer) in (getattr(hsa, status), SHAPE), (change, layer)


def test_select_and_compact_binding_checks(fake):
    i32 = host._i32
    w = _f32(4, 2, 64)
    keep, new = binding.hsa_kv_select(w, i32(3), i32(3), 16, sinks=1, recent=2, reach=3, stream=0)
    name, a = fake.calls[-1]
    assert name == "hsa_kv_select" and a[1:4] == (64, 4, 2) and a[6:11] == (3, 16, 1, 2, 3)
    assert keep.shape == (3, 2, 16) and new.shape == (3,)
    pool = host._pool()
    binding.hsa_kv_compact(pool, 1, keep, new, i32(3), i32(3, 5), w=w, w_dst=w.clone(), stream=0)
    name, a = fake.calls[-1]
    assert name == "hsa_kv_compact" and a[3:5] == (2, 16) and a[7] == 3 and a[9] == 5 and a[12] == 64
    binding.hsa_kv_compact(pool, 1, keep[:, :1].contiguous(), new, i32(3), i32(3, 5), stream=0)
    assert fake.calls[-1][1][3] == 1 and fake.calls[-1][1][10] is None
    done = len(fake.calls)
    for args, kw in [((w, i32(2), i32(3), 16), {}), ((_f32(4, 2, 62), i32(3), i32(3), 16), {}), ((w[0], i32(3), i32(3), 16), {}),
                     ((w, i32(3), i32(3), -1), {}), ((w, i32(3), i32(3), 16), dict(keep=i32(3, 2, 15))),
                     ((w, i32(3), i32(3), 16), dict(new_len=i32(4))), ((w[:, :, ::2], i32(3), i32(3), 16), {})]:
        with pytest.raises(ValueError):
            binding.hsa_kv_select(*args, stream=0, **kw)
    with pytest.raises(TypeError):
        binding.hsa_kv_select(w.double(), i32(3), i32(3), 16, stream=0)
    for kw in (dict(keep=i32(3, 3, 16)), dict(new=i32(2)), dict(seq=i32(4)), dict(dst=i32(2, 5)), dict(w=w), dict(wd=w),
               dict(w=_f32(3, 2, 64), wd=_f32(3, 2, 64)), dict(w=w, wd=_f32(4, 2, 60)), dict(w=_f32(4, 1, 64), wd=_f32(4, 1, 64))):
        with pytest.raises(ValueError):
            binding.hsa_kv_compact(pool, 1, kw.get("keep", keep), kw.get("new", new), kw.get("seq", i32(3)),
                                   kw.get("dst", i32(3, 5)), w=kw.get("w"), w_dst=kw.get("wd"), stream=0)
    assert len(fake.calls) == done


def test_decode_weights_arguments_refused():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    INV, SHAPE, OK = hsa.HSA_INVALID_ARG, hsa.HSA_UNSUPPORTED_SHAPE, hsa.HSA_OK
    base = dict(p=ctypes.byref(cabi._pools(hsa)), layer=1, q=M, k=2 * M, v=3 * M, c=256, B=2, T=1, scale=0.1, out=4 * M,
                prev=5 * M, decay=1.0, w=6 * M, stride=256, ws=7 * M, bytes=1 << 40, ctas=0, opt=0)

    def call(**kw):
        a = dict(base, **kw)
        return L.hsa_decode_attn_weights(a["p"], a["layer"], a["q"], a["k"], a["v"], a["c"], a["B"], a["T"], a["scale"], a["out"],
                                         a["prev"], a["decay"], a["w"], a["stride"], a["ws"], a["bytes"], a["ctas"], a["opt"],
                                         None, None)
    for kw in (dict(p=None), dict(layer=2), dict(q=None), dict(k=None), dict(v=None), dict(c=None), dict(out=None), dict(w=None),
               dict(q=M + 8), dict(out=4 * M + 2), dict(w=6 * M + 4), dict(prev=5 * M + 4), dict(B=-1), dict(B=3), dict(T=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(decay=math.nan),
               dict(decay=-math.inf), dict(stride=255), dict(stride=-4), dict(stride=(1 << 30) + 4), dict(ctas=-1),
               dict(opt=2), dict(opt=4), dict(prev=6 * M + 16), dict(prev=6 * M - 16)):
        assert call(**kw) == INV, kw
    assert call(layer=0) == SHAPE and call(T=5) == SHAPE
    assert call(B=0) == OK
    p = cabi._pools(hsa)
    size = lambda B, T, n: L.hsa_decode_weights_workspace_bytes(ctypes.byref(p), B, T, n)  # noqa: E731
    assert size(2, 1, 1024) >= 4 * 2 * 32 * 1024 and size(2, 4, 1024) >= 4 * size(2, 1, 1024) // 2
    assert size(-1, 1, 4) == 0 and size(1, 0, 4) == 0 and size(1, 1, -4) == 0
    assert L.hsa_decode_weights_workspace_bytes(None, 1, 1, 4) == 0


def test_decode_weights_binding_checks(fake, monkeypatch):
    monkeypatch.setattr(binding, "decode_weights_workspace", lambda *a, **k: torch.zeros(64, dtype=torch.uint8))
    pool, i32, bf = host._pool(), host._i32, host._bf
    B, T = 3, 2
    q, k, v, cl, w = bf(B, T, host.Hq, 128), bf(B, T, host.Hkv, 128), bf(B, T, host.Hkv, 128), i32(B), _f32(B, host.Hkv, 64)
    binding.hsa_decode_attn_weights(pool, 1, q, k, v, cl, 0.1, w, w_prev=w, append=True, stream=0)
    name, a = fake.calls[-1]
    assert name == "hsa_decode_attn_weights" and a[6:8] == (B, T) and a[13] == 64 and a[17] == binding.HSA_DECODE_APPEND
    binding.hsa_decode_attn_weights(pool, 1, q, k, v, cl, 0.1, w, stream=0)
    assert fake.calls[-1][1][10] is None and fake.calls[-1][1][17] == 0
    done = len(fake.calls)
    for kw in (dict(q=q[:, :, :-1]), dict(k=k[:-1]), dict(v=v[:, :1]), dict(cl=i32(2)), dict(w=_f32(B, host.Hkv, 62)),
               dict(w=_f32(2, host.Hkv, 64)), dict(w=w[0]), dict(prev=_f32(B, host.Hkv, 60)), dict(out=bf(B, T, host.Hq, 64))):
        with pytest.raises(ValueError):
            binding.hsa_decode_attn_weights(pool, 1, kw.get("q", q), kw.get("k", k), kw.get("v", v), kw.get("cl", cl), 0.1,
                                            kw.get("w", w), w_prev=kw.get("prev"), out=kw.get("out"), stream=0)
    with pytest.raises(TypeError):
        binding.hsa_decode_attn_weights(pool, 1, q, k, v, cl, 0.1, w.double(), stream=0)
    assert len(fake.calls) == done


def test_prefill_weights_arguments_refused():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    INV, SHAPE, OK = hsa.HSA_INVALID_ARG, hsa.HSA_UNSUPPORTED_SHAPE, hsa.HSA_OK
    base = dict(p=ctypes.byref(cabi._pools(hsa)), layer=1, q=M, cu=256, n=256, seq=256, R=2, rows=40, window=16, scale=0.1,
                prev=5 * M, decay=1.0, w=6 * M, stride=256, ws=7 * M, bytes=1 << 40)

    def call(**kw):
        a = dict(base, **kw)
        return L.hsa_prefill_weights(a["p"], a["layer"], a["q"], a["cu"], a["n"], a["seq"], a["R"], a["rows"], a["window"],
                                     a["scale"], a["prev"], a["decay"], a["w"], a["stride"], a["ws"], a["bytes"], None, None)
    for kw in (dict(p=None), dict(layer=2), dict(q=None), dict(q=M + 8), dict(cu=None), dict(n=None), dict(seq=None), dict(R=-1),
               dict(rows=-1), dict(window=0), dict(window=-1), dict(scale=0.0), dict(scale=math.nan), dict(decay=math.nan),
               dict(w=None), dict(w=6 * M + 4), dict(prev=5 * M + 4), dict(stride=255), dict(stride=-4), dict(prev=6 * M + 16),
               dict(stride=(1 << 30) + 4)):
        assert call(**kw) == INV, kw
    assert call(layer=0) == SHAPE and call(window=65) == SHAPE
    assert call(p=ctypes.byref(cabi._pools(hsa, fp8=[0, 1]))) == SHAPE
    assert call(R=0, q=None, w=None) == OK and call(rows=0, q=None) == OK
    size = lambda R, n: L.hsa_prefill_weights_workspace_bytes(base["p"], R, n)  # noqa: E731
    assert size(2, 64) >= size(2, 16) > size(1, 16) > 0 and size(-1, 4) == 0 and size(1, 0) == 0


def test_prefill_weights_binding_checks(fake, monkeypatch):
    monkeypatch.setattr(binding, "prefill_weights_workspace", lambda *a, **k: torch.zeros(64, dtype=torch.uint8))
    pool, i32, bf = host._pool(), host._i32, host._bf
    q, w = bf(40, host.Hq, 128), _f32(4, host.Hkv, 64)
    binding.hsa_prefill_weights(pool, 1, q, i32(3), i32(2), i32(2), 16, 0.1, w, w_prev=w, decay=0.5, stream=0)
    name, a = fake.calls[-1]
    assert name == "hsa_prefill_weights" and a[6:9] == (2, 40, 16) and a[13] == 64 and a[10] == w.data_ptr()
    done = len(fake.calls)
    for kw in (dict(q=q[:, :-1].contiguous()), dict(q=q[0]), dict(cu=i32(2)), dict(n=i32(3)), dict(seq=i32(3)),
               dict(w=_f32(3, host.Hkv, 64)), dict(w=_f32(4, host.Hkv, 63)), dict(prev=_f32(4, host.Hkv, 60))):
        with pytest.raises(ValueError):
            binding.hsa_prefill_weights(pool, 1, kw.get("q", q), kw.get("cu", i32(3)), kw.get("n", i32(2)), kw.get("seq", i32(2)),
                                        16, 0.1, kw.get("w", w), w_prev=kw.get("prev"), stream=0)
    assert len(fake.calls) == done


def _key(x):
    """The kernel's integer of an fp32 value."""
    x = -math.inf if math.isnan(x) else x + 0.0
    u = struct.unpack("<I", struct.pack("<f", x))[0]
    return u ^ (0xffffffff if u >> 31 else 0x80000000)


def test_key_order():
    tiny = 2.0 ** -149
    v = [-math.inf, -3.4e38, -1.0, -2.0 ** -126, -tiny, 0.0, tiny, 2.0 ** -126, 1e-4, 1.0, 1.0 + 2.0 ** -23, 3.4e38, math.inf]
    keys = [_key(x) for x in v]
    assert keys == sorted(set(keys)) and keys[0] > 0
    assert _key(-0.0) == _key(0.0) and _key(math.nan) == _key(-math.inf)
