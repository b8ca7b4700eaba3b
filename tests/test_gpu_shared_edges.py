"""Shared-prefix decode at the edges of its contract: members of unlike lengths, pages that
nobody has written, entries that are not there, values near the top of bf16's range.  Limits
as in test_gpu_shared."""
import pytest
import torch

import test_gpu_shared as base

pytestmark = pytest.mark.gpu

D, PAGE, SCALE = base.D, base.PAGE, base.SCALE


@pytest.mark.parametrize("max_ctas", [0, 2])
@pytest.mark.parametrize("past", ["absent", "stale"])
def test_a_first_member_that_holds_less(past, max_ctas):
    """Rows agree as far as a member's cached tokens go; behind its own, a short member's row
    holds -1 or another sequence's block.  The first member is one of the short ones."""
    hsa = base._hsa()
    for own in ([-640, 5, -100, 130], [-300, 0, 64, -640], [-1, 70, 1, 2], [-64, -128, -63, 9]):
        for T in (1, 3):
            c = base.Case(hsa, [4, 2], [640, 200], own, T, 16, 2, seed=len(own) + T)
            for i, n in enumerate(c.cached):
                # a block of other values, and where there is no such block, none
                c.table[i, (n + T + PAGE - 1) // PAGE:] = -1 if past == "absent" else c.spare
            out = c.run(max_ctas=max_ctas)
            assert int(c.err) == 0
            c.check(out)


@pytest.mark.parametrize("T", [1, 4])
def test_members_that_all_hold_less_see_no_unwritten_page(T):
    """Nobody holds the last shared pages: they may hold anything, NaN and infinities too."""
    hsa = base._hsa()
    c = base.Case(hsa, [3, 2], [640, 256], [-100, -300, -193, -70, -256], T, 32, 4, seed=4)
    written = torch.zeros(c.kp.shape[0], PAGE, dtype=torch.bool, device="cuda")
    for i, n in enumerate(c.cached):
        for at in range(0, n, PAGE):
            written[int(c.table[i, at // PAGE]), :n - at] = True
    hole = ~written[:, None, :, None]
    c.kp.masked_fill_(hole, float("nan"))
    c.vp.masked_fill_(hole, float("inf"))
    c.vp[..., 1::2].masked_fill_(hole, float("nan"))
    c.check(c.run())
    assert int(c.err) == 0


def test_bad_entries_read_no_block():
    """The keys of an entry outside the pool are absent: no block stands in for them, whatever
    block 0 holds."""
    hsa = base._hsa()
    c = base.Case(hsa, [3, 40], [640, 450], [5, 130], 1, 16, 2, seed=10)
    # block 0 takes the place of the spare one
    c.kp[c.spare], c.vp[c.spare] = c.kp[0].clone(), c.vp[0].clone()
    c.table[c.table == 0] = c.spare
    c.kp[0], c.vp[0] = float("nan"), float("nan")
    c.table[:3, 4] = -1
    c.table[:3, 9] = c.kp.shape[0]
    c.table[3:, 6] = 10 ** 9
    c.table[3:, 0] = 2 ** 31 - 1
    out = c.run()
    assert int(c.err) == hsa.HSA_DEVERR_BAD_BLOCK
    c.check(out)


@pytest.mark.parametrize("max_ctas", [0, 1])
def test_large_values_behind_a_leap_of_the_scores(max_ctas):
    """Scores 2^12 to 2^56 above those of the pages before, on values of 1e30: a weight that
    is held above 1 for a page must leave fp32 room for them."""
    hsa = base._hsa()
    for leap in (12, 20, 56):
        for members in (3, 40):  # one tile of rows, two
            c = base.Case(hsa, [members], [64 * 30], [20, 3], 1, 16, 2, seed=31, sharp=0.0)
            c.q[:] = 1
            c.kp.mul_(0.02)
            # a key of all u scores 128 u D^-1/2, log2 e times that in powers of two
            u = leap / (D * SCALE * 1.4427)
            for i in range(7, 30):
                c.kp[int(c.table[0, i])] += u
            for x in (c.vp, c.v):
                x.mul_(1e30)
            out = c.run(max_ctas=max_ctas)
            assert bool(out.isfinite().all())
            c.check(out)
