"""Calls on a stream other than the current one, with outputs and workspaces made by the
call: their memory must not be taken from under the kernels, nor from under work that the
current stream has yet to do."""
import pytest
import torch

import test_gpu_shared as base

pytestmark = pytest.mark.gpu

D, SCALE = base.D, base.SCALE
PAUSE = 40_000_000  # clocks: about 20 ms


def _calls(hsa):
    """name -> a function of the stream that makes its own outputs and workspace."""
    c = base.Case(hsa, *base.CASES["verify"], seed=2)
    n = 37
    g = base._gen(3)
    q = torch.randn(n, c.hq, D, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(n, c.hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    rope = hsa.Rope(D)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    spare = hsa.DualPool.allocate([True], 2, 1, base._i32([[0, 1]]), base._i32([0]), c.hq, c.hkv)
    cu, zero = base._i32([0, n]), base._i32([0])
    lens = base._i32([40] * 500)
    slots = torch.arange(128, dtype=torch.int32, device="cuda").repeat(500, 1)
    return {
        "shared": lambda s: hsa.hsa_decode_attn_shared(c.pool, 0, c.q, c.k, c.v, c.cl, c.cu, c.sl, SCALE, stream=s),
        "decode": lambda s: hsa.hsa_decode_attn(c.pool, 0, c.q, c.k, c.v, c.cl, SCALE, stream=s),
        "rope": lambda s: hsa.hsa_rope(rope, q, k, pos, stream=s),
        "append": lambda s: hsa.hsa_rope_kv_append(spare, 0, rope, q, k, v, cu, zero, zero, stream=s),
        "prefill": lambda s: hsa.hsa_prefill_attn(spare, 0, q, k, v, cu, zero, zero, n, SCALE, stream=s),
        "window": lambda s: hsa.hsa_window_safe_len(lens, slots, 128, stream=s),
    }


def _flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,))]


@pytest.mark.parametrize("kind", ["stream", "number", "default"])
@pytest.mark.parametrize("name", ["shared", "decode", "rope", "append", "prefill", "window"])
def test_memory_made_for_a_call_on_another_stream(name, kind):
    hsa = base._hsa()
    call = _calls(hsa)[name]
    want = _flat(call(None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    here = torch.cuda.Stream() if kind == "default" else torch.cuda.current_stream()
    on, given = {"stream": (side, side), "number": (side, side.cuda_stream),
                 "default": (torch.cuda.default_stream(), 0)}[kind]
    sizes = sorted({t.numel() * t.element_size() for t in want} | {1 << 20, 4 << 20, 16 << 20})
    with torch.cuda.stream(here):
        for _ in range(2):
            # the stream is busy when the call comes: what the current stream takes and fills
            # meanwhile must be other memory than the call's
            with torch.cuda.stream(on):
                torch.cuda._sleep(PAUSE)
            got = _flat(call(given))
            for size in sizes * 4:
                torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            del got
            # the current stream is busy, and reads memory that it has given back since
            old = [torch.full_like(t, 3) for t in want]
            torch.cuda.synchronize()
            torch.cuda._sleep(PAUSE)
            kept = [t.clone() for t in old]
            del old
            got = _flat(call(given))
            torch.cuda.synchronize()
            for t in kept:
                assert bool((t == 3).all())
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            # a result that the current stream still reads when it is given back, and the next
            # call on the same stream
            torch.cuda._sleep(PAUSE)
            kept = [t.clone() for t in got]
            del got
            with torch.cuda.stream(on):
                for size in sizes * 4:
                    torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
            torch.cuda.synchronize()
            for a, b in zip(kept, want):
                assert torch.equal(a, b)


def test_two_host_threads_at_once():
    """Every call from two threads, each on a stream and a workspace of its own."""
    import threading
    hsa = base._hsa()
    cases = [base.Case(hsa, *base.CASES[n], seed=4) for n in ("three tokens", "odd pages")]
    want = [c.run() for c in cases]
    plain = [hsa.hsa_decode_attn(c.pool, 0, c.q, c.k, c.v, c.cl, SCALE) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(c, w, p):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(50):
                    a = c.run()
                    b = hsa.hsa_decode_attn(c.pool, 0, c.q, c.k, c.v, c.cl, SCALE)
                s.synchronize()
                if not torch.equal(a, w) or not torch.equal(b, p):
                    bad.append("values")
        except Exception as e:  # noqa: BLE001 - told by the test's thread
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=x) for x in zip(cases, want, plain)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
