"""Host side of the eviction entry points, without a GPU: refusals beside those of test_evict_host."""
import ctypes

import pytest

import test_cabi as cabi

M = 1 << 20


@pytest.mark.parametrize("new", [768, 772, 764])
def test_select_new_len_over_the_sequences(new):
    """Every CTA of a request reads its sequence; the first one writes the new length."""
    import full_attention_kv_gb300 as hsa
    s = hsa.lib().hsa_kv_select(M, 64, 4, 2, 256, 768, 2, 16, 4, 8, 1, 2 * M, new, None, None)
    assert s == hsa.HSA_INVALID_ARG


@pytest.mark.parametrize("scale", [2.0 ** -97, 1e-38, 1e-45, 2.0 ** 97, 3e38])
def test_scales_whose_log_sum_leaves_fp32(scale):
    import full_attention_kv_gb300 as hsa
    p = ctypes.byref(cabi._pools(hsa))
    s = hsa.lib().hsa_prefill_weights(p, 1, M, 256, 256, 256, 2, 40, 16, scale, None, 1.0, 6 * M, 256, 7 * M, 1 << 40, None, None)
    assert s == hsa.HSA_INVALID_ARG
    s = hsa.lib().hsa_decode_attn_weights(p, 1, M, 2 * M, 3 * M, 256, 2, 1, scale, 4 * M, None, 1.0, 6 * M, 256, 7 * M, 1 << 40, 0, 0,
                                          None, None)
    assert s == hsa.HSA_INVALID_ARG
