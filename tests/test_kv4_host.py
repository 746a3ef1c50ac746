"""Host side of the 4-bit cache's binding (no GPU needed)."""
import pytest

from w8a8_online_quantized_amd import cider

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D,gs", [(128, 48), (128, 256), (128, -32), (128, 16), (128, 24), (256, 32), (64, 16), (64, 40), (128, 1)])
def test_cache_refuses_groups_that_no_call_takes(D, gs):
    """(48 gave two groups of 64, 256 an array of no scales.)"""
    with pytest.raises(ValueError, match="group_size"):
        cider.kv4_cache(2, 2, 16, D, gs, device="cpu")


@pytest.mark.parametrize("D,gs,G", [(64, 0, 1), (64, 64, 1), (64, 32, 2), (128, 32, 4), (128, 128, 1), (256, 64, 4), (256, 256, 1)])
def test_cache_groups(D, gs, G):
    cache = cider.kv4_cache(3, 2, 16, D, gs, device="cpu")
    assert cache.k_codes.shape == cache.v_codes.shape == (3, 2, 16, D // 2)
    assert cache.k_scale.shape == cache.v_scale.shape == (3, 2, G, 16)


def test_refusals_name_what_is_not_aligned():
    ids = torch.arange(8, dtype=torch.int32)
    cache = cider.kv4_cache(1, 1, 16, 64, device="cpu")
    with pytest.raises(cider.CiderError, match=r"slots, q must start at a multiple of 16 bytes") as e:
        cider._refused("cider_kv4_append", cider.CIDER_ERROR_INVALID_VALUE, cache, slots=ids[1:], positions=ids, q=ids[2:], q_norm=None)
    assert e.value.status == cider.CIDER_ERROR_INVALID_VALUE
    shifted = cache._replace(v_scale=torch.zeros(20)[1:17].view(1, 1, 1, 16))
    for arrays in (shifted, tuple(shifted)):
        with pytest.raises(cider.CiderError, match=r": v_scale must start"):
            cider._refused("cider_kv4_read", cider.CIDER_ERROR_INVALID_VALUE, arrays, slots=ids)
    for status, tensors in ((cider.CIDER_ERROR_INVALID_VALUE, ids[4:]), (cider.CIDER_ERROR_LAUNCH, ids[1:])):
        with pytest.raises(cider.CiderError) as e:
            cider._refused("cider_rope", status, x=tensors)
        assert "16 bytes" not in str(e.value)
