"""Calls from host threads: one that has called nothing of CUDA's before (the tensor maps are encoded
by the driver, which wants the thread to have a current context), and two at once."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _hsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import full_attention_kv_gb300 as hsa
    hsa.lib()
    return hsa


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("name", ["decode", "decode fp8", "shared", "prefill", "weights", "weights fp8", "prompt weights"])
def test_first_call_of_a_thread(name):
    hsa = _hsa()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    n, hq, hkv, d = 100, 16, 2, 128
    pool = hsa.DualPool.allocate([True], 4, 1, _i32([[0, 1], [2, 3]]), _i32([0, 0]), hq, hkv,
                                 kv_fp8="e4m3" if "fp8" in name else False)
    hsa.hsa_kv_append(pool, 0, bf(2 * n, hkv, d), bf(2 * n, hkv, d), _i32([0, n, 2 * n]), _i32([0, 1]), _i32([0, 0]))
    q, k, v = bf(2, 1, hq, d), bf(2, 1, hkv, d), bf(2, 1, hkv, d)
    cl, seq, cu = _i32([n, n]), _i32([0, 1]), _i32([0, 1, 2])
    group, zero = _i32([0, 2]), _i32([0])
    out, w = torch.empty_like(q), torch.zeros(2, hkv, 128, device="cuda")
    flat = out.view(2, hq, d)
    stream = torch.cuda.current_stream()
    if name.startswith("decode"):
        ws = hsa.decode_workspace(pool, 2, 1)
        call = lambda: hsa.hsa_decode_attn(pool, 0, q, k, v, cl, 0.1, out=out, workspace=ws, stream=stream)  # noqa: E731
    elif name == "shared":
        ws = hsa.decode_shared_workspace(pool, 2, 1, 1)
        call = lambda: hsa.hsa_decode_attn_shared(pool, 0, q, k, v, cl, group, zero, 0.1, out=out, workspace=ws,  # noqa: E731
                                                  stream=stream)
    elif name == "prefill":
        call = lambda: hsa.hsa_prefill_attn(pool, 0, q.view(2, hq, d), k.view(2, hkv, d), v.view(2, hkv, d), cu, cl, seq,  # noqa: E731
                                            1, 0.1, out=flat, stream=stream)
    elif name.startswith("weights"):
        ws = hsa.decode_weights_workspace(pool, 2, 1, 128)
        call = lambda: hsa.hsa_decode_attn_weights(pool, 0, q, k, v, cl, 0.1, w, out=out, workspace=ws, stream=stream)  # noqa: E731
    else:
        ws = hsa.prefill_weights_workspace(pool, 2, 16)
        call = lambda: hsa.hsa_prefill_weights(pool, 0, q.view(2, hq, d), cu, cl, seq, 16, 0.1, w, workspace=ws,  # noqa: E731
                                               stream=stream)
    call()
    torch.cuda.synchronize()
    want = out.clone(), w.clone()
    out.zero_()
    w.zero_()
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001 - told by the test's thread
            bad.append(repr(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not bad
    if name != "prompt weights":
        assert torch.equal(out, want[0])
    assert torch.equal(w, want[1])


class Cut:
    """A sequence cut to a budget, then a step: the four calls of an eviction, on pages of its own."""

    def __init__(self, hsa, n, hq, hkv, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.hsa, self.n, self.budget, d = hsa, n, n // 3, 128
        pages, kept = (n + 63) // 64, (self.budget + 64) // 64
        self.dst = _i32([list(range(pages, pages + kept))])
        self.old = _i32([list(range(pages))])
        self.new = _i32([list(range(pages, pages + kept)) + [0] * (pages - kept)])
        self.pool = hsa.DualPool.allocate([True], pages + kept, 1, self.old.clone(), _i32([0]), hq, hkv)
        self.q, self.k, self.v = bf(n, hq, d), bf(n, hkv, d), bf(n, hkv, d)
        self.step = bf(1, 1, hq, d), bf(1, 1, hkv, d), bf(1, 1, hkv, d)
        self.cu, self.len, self.zero, self.err = _i32([0, n]), _i32([n]), _i32([0]), _i32([0])
        self.w = torch.zeros(2, 1, hkv, pages * 64, device="cuda")
        self.ws = hsa.prefill_weights_workspace(self.pool, 1, 64), hsa.decode_weights_workspace(self.pool, 1, 1, pages * 64)

    def run(self):
        hsa, w, kept = self.hsa, self.w[0], self.w[1]
        self.pool.block_tables.copy_(self.old)
        hsa.hsa_kv_append(self.pool, 0, self.k, self.v, self.cu, self.zero, self.zero, dev_err=self.err)
        hsa.hsa_prefill_weights(self.pool, 0, self.q, self.cu, self.len, self.zero, 64, 0.1, w, workspace=self.ws[0],
                                dev_err=self.err)
        keep, left = hsa.hsa_kv_select(w, self.len, self.zero, self.budget, sinks=4, recent=16, reach=1, dev_err=self.err)
        hsa.hsa_kv_compact(self.pool, 0, keep, left, self.zero, self.dst, w=w, w_dst=kept, dev_err=self.err)
        self.pool.block_tables.copy_(self.new)
        out = hsa.hsa_decode_attn_weights(self.pool, 0, *self.step, left, 0.1, kept, w_prev=kept, workspace=self.ws[1],
                                          append=True, dev_err=self.err)
        return keep, out, kept[..., :self.budget + 1].clone()


def test_evictions_from_two_host_threads_at_once():
    hsa = _hsa()
    cases = [Cut(hsa, 50000, 32, 4, 1), Cut(hsa, 3001, 16, 2, 2)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(c, w):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got = c.run()
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, w)):
                        bad.append("values")
        except Exception as e:  # noqa: BLE001 - told by the test's thread
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=x) for x in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and all(int(c.err) == 0 for c in cases)
