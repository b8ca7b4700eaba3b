"""Host side of the eviction entry points' size queries, without a GPU: nothing for a shape that the
call refuses, however far out of range, and at once."""
import ctypes

import pytest

import test_cabi as cabi


@pytest.mark.parametrize("T", [5, 8, 1 << 20, (1 << 28) + 1, (1 << 31) - 1])
def test_no_workspace_for_more_tokens_than_a_step_takes(T):
    import full_attention_kv_gb300 as hsa
    p = ctypes.byref(cabi._pools(hsa))
    assert hsa.lib().hsa_decode_weights_workspace_bytes(p, 2, 4, 1024) > 0
    assert hsa.lib().hsa_decode_weights_workspace_bytes(p, 2, T, 1024) == 0


def test_no_workspace_for_heads_or_rows_that_are_refused():
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    for hq in (48, 64, 1 << 30, 31):  # 12, 16 and more queries a head, and no whole number
        p = ctypes.byref(cabi._pools(hsa, Hq=hq))
        assert L.hsa_decode_weights_workspace_bytes(p, 2, 1, 1024) == 0
        assert L.hsa_prefill_weights_workspace_bytes(p, 2, 16) == 0
    p = ctypes.byref(cabi._pools(hsa))
    for stride in (1022, (1 << 30) + 4):
        assert L.hsa_decode_weights_workspace_bytes(p, 2, 1, stride) == 0
    for window in (65, (1 << 31) - 1):
        assert L.hsa_prefill_weights_workspace_bytes(p, 2, window) == 0
    assert L.hsa_prefill_weights_workspace_bytes(p, 2, 64) > 0
