"""Sizes of the decode workspaces, without a GPU: the arrival counters at the start have room
for the pools' whole batch, whatever the call's."""
import ctypes

import pytest

import test_cabi as cabi


@pytest.mark.parametrize("Hkv", [1, 2, 8])
def test_counters_have_room_for_the_whole_batch(Hkv):
    import full_attention_kv_gb300 as hsa
    L = hsa.lib()
    plain, shared = L.hsa_decode_workspace_bytes, L.hsa_decode_shared_workspace_bytes

    def pools(batch):
        return ctypes.byref(cabi._pools(hsa, batch=batch, Hkv=Hkv, Hq=8 * Hkv))

    for B in (1, 7, 64):
        # pools of 64 rows and of 1 << 20: the counters' bytes, and nothing else, between them
        more = ((1 << 20) - 64) * Hkv * 4
        assert abs(plain(pools(1 << 20), B, 1) - plain(pools(64), B, 1) - more) < 256
        a, b = shared(pools(1 << 20), B, 1, 1), shared(pools(64), B, 1, 1)
        assert abs(a - b - more) < 512
        # a workspace of the largest call is one for every smaller call
        p = pools(64)
        assert plain(p, 64, 4) >= plain(p, B, 1) and shared(p, 64, 4, 64) >= shared(p, B, 1, 1)
        assert shared(p, B, 1, 0) >= plain(p, B, 1)
