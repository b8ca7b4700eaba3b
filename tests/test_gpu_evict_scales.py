"""Softmax scales far from the usual, on the GPU against 64 bits: weights all alike at one end, a single key's
at the other.  Limits as in the calls' own tests."""
import pytest
import torch

import test_gpu_prompt_weights as prompt
import test_gpu_weigh as weigh

pytestmark = pytest.mark.gpu

SCALES = [2.0 ** -96, 2.0 ** -40, 1e-4, 4.0, 2.0 ** 18]


@pytest.mark.parametrize("scale", SCALES)
def test_prompt_weights(scale, monkeypatch):
    monkeypatch.setattr(prompt, "SCALE", scale)
    s = prompt.Prompts(prompt._hsa(), [900, 70, 3000], [64, 70, 5], 32, 32, 4)
    s.run()
    s.check()
    assert int(s.err) == 0


@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("scale", SCALES)
def test_weighing_decode(scale, fmt, monkeypatch):
    monkeypatch.setattr(weigh, "SCALE", scale)
    s = weigh.Step(weigh._hsa(), [900, 70, 3000], 2, 16, 2, fmt)
    s.check(s.run())
    assert int(s.err) == 0
