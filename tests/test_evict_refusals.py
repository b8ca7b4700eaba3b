"""Host side of the eviction entry points, without a GPU: refusals beside those of test_evict_host."""
import pytest

M = 1 << 20


@pytest.mark.parametrize("new", [768, 772, 764])
def test_select_new_len_over_the_sequences(new):
    """Every CTA of a request reads its sequence; the first one writes the new length."""
    import full_attention_kv_gb300 as hsa
    s = hsa.lib().hsa_kv_select(M, 64, 4, 2, 256, 768, 2, 16, 4, 8, 1, 2 * M, new, None, None)
    assert s == hsa.HSA_INVALID_ARG
