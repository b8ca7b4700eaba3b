"""The bounded waits of the eviction kernels, on the GPU and without a hang: in a test-only variant of the
library, built into a temporary directory with a 2 ms limit, the weighing decode's, the prompt
weights' and the FP8 move's producers issue no load at all (so nothing is in flight when a CTA
exits).  Each call must return and flag the timeout, with no garbage behind it, and
leave the context usable: the product library's same call is right afterwards."""
import pytest
import torch

import test_gpu_evict as evict
import test_gpu_prompt_weights as prompt
import test_gpu_weigh as weigh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def variant(tmp_path_factory):
    weigh._hsa()
    from full_attention_kv_gb300 import build as libbuild
    return libbuild.build(out_dir=str(tmp_path_factory.mktemp("withheld")),
                          defines=("HSA_WAIT_NS=2000000ull", "HSA_TEST_WITHHOLD_LOADS"))


@pytest.fixture
def withheld(variant, monkeypatch):
    """Runs a call against the variant."""
    from full_attention_kv_gb300 import binding

    def run(call):
        with monkeypatch.context() as m:
            m.setattr(binding, "LIB_PATH", variant)
            m.setattr(binding, "_lib", None)
            call()
            torch.cuda.synchronize()  # returns: each wait gave up after 2 ms
        assert binding.lib()._name == binding.LIB_PATH != variant
    return run


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("T", [1, 4])
def test_weighing_decode(withheld, T, fmt):
    hsa = weigh._hsa()
    s = weigh.Step(hsa, [300, 64, 5000], T, 16, 2, fmt)
    out = torch.full_like(s.q, 5.0)
    withheld(lambda: s.run(out=out))
    assert int(s.err) == hsa.HSA_DEVERR_TIMEOUT
    assert torch.isfinite(out.float()).all()  # of the new tokens alone
    s.err.zero_()
    s.w.fill_(-7.0)
    s.check(s.run())
    assert int(s.err) == 0


@pytest.mark.parametrize("window", [1, 16, 33, 64])  # one to four row tiles
def test_prompt_weights(withheld, window):
    hsa = weigh._hsa()
    s = prompt.Prompts(hsa, [3000, 70], [64, 64], window, 32, 4)
    withheld(s.run)
    assert int(s.err) == hsa.HSA_DEVERR_TIMEOUT
    assert bool((s.w == -7.0).all())
    s.err.zero_()
    s.run()
    s.check()
    assert int(s.err) == 0


def test_move_of_an_fp8_layer(withheld):
    hsa = weigh._hsa()
    m = evict.Moves(hsa, [700, 90], 150, "e4m3", 2, 2, seed=5)
    want, before = m.moved(), m.views(m.bufs)
    withheld(m.run)
    assert int(m.err) == hsa.HSA_DEVERR_TIMEOUT
    assert torch.equal(m.views(m.bufs)[2], before[2])  # V's codes
    m.err.zero_()
    m.run()
    m.check(want)
