"""Calls from a host thread that has called nothing of CUDA's before: the tensor maps are encoded by
the driver, which wants the thread to have a current context."""
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
