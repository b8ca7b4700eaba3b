"""Weighing decode where one key says nothing about the others, on the GPU against 64 bits: a row of
V a million times the rest that no query looks at, and a key that takes nearly all of the weight
and has no V (an attention sink).  The output is then the other keys', and so are its limits.

Limits as in test_gpu_weigh: P rounds once before the product with V, to bf16 (2^-9 of itself) or,
on an FP8 layer, to fp16 (2^-11), the bf16 sum of weights with it; the output rounds to bf16 (2^-9).
mag = sum p |v| holds the keys that carry the output, not the one beside them: with no weight, or
no V, it adds nothing to the sum."""
import pytest
import torch

import test_gpu_weigh as weigh

pytestmark = pytest.mark.gpu

# The first key's place on an axis of its own, in nats / 1.41 over the others, its V and, where only
# one dimension of it has a value, which.
FIRST = {
    "large V without weight": (-32.0, 2.0 ** 18, None),
    "larger V without weight": (-32.0, 2.0 ** 24, None),
    "sink without V": (14.0, 0.0, None),
    "sink with little V": (14.0, 2.0 ** -34, None),
    "sink far above, without V": (28.0, 0.0, None),
    "sink with V in one dimension": (10.0, 1.0, 5),
}


class First(weigh.Step):
    def __init__(self, first, *args, **kw):
        self.first = first
        super().__init__(*args, garbage=None, **kw)
        if self.fmt is None:
            self._shape(*self.bufs)
        self.q[..., 0] = 16.0
        self.k[..., 0] = 0.0
        self.v.zero_()

    def _shape(self, k, v):
        far, size, dim = FIRST[self.first]
        k[..., 0] = 0.0
        for block in self.table[:, 0].tolist():
            k[block, :, 0, 0] = far
            v[block, :, 0] *= size
            if dim is not None:
                v[block, :, 0] = 0.0
                v[block, :, 0, dim] = size

    def _quantise(self, k, v):
        self._shape(k, v)
        super()._quantise(k, v)


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("T", [1, 2, 4])
@pytest.mark.parametrize("first", sorted(FIRST))
def test_one_key_apart(first, T, fmt):
    s = First(first, weigh._hsa(), [60, 64, 500], T, 16, 2, fmt)
    for max_ctas in (0, 1):  # a state for each page, and pages that share a few
        s.w.fill_(-7.0)
        out = s.run(max_ctas=max_ctas)
        assert int(s.err) == 0
        s.check(out)
