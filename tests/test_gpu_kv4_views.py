"""Slices that start between two multiples of 16 bytes: the attention block's calls refuse them by name."""
import pytest

from tests.test_gpu_parity import cider

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests.test_gpu_kv4 import i32  # noqa: E402


def test_slices_are_named():
    c = cider()
    cache, freq = c.kv4_cache(4, 2, 16, 64), c.rope_frequencies(64)[0]
    q, k = torch.ones(3, 4, 64, device="cuda").half(), torch.ones(3, 2, 64, device="cuda").half()
    ids, table = i32([0, 1, 2, 3]), i32([[0], [1], [2]])
    odd = torch.ones(8 + q.numel(), device="cuda").half()[1:1 + q.numel()].view(q.shape)
    cut = ids[1:]
    for name, call in (
        ("positions", lambda: c.cider_rope(q, cut, freq)), ("x", lambda: c.cider_rope(odd, ids[:3], freq)),
        ("slots", lambda: c.cider_kv4_append(cache, k, k, cut)), ("q", lambda: c.cider_kv4_append(cache, k, k, ids[:3], q=odd)),
        ("slots", lambda: c.cider_kv4_read(cache, cut)), ("lengths", lambda: c.cider_kv4_attention(q, cache, table, cut)),
        ("q", lambda: c.cider_kv4_attention(odd, cache, table, ids[:3])),
    ):
        with pytest.raises(c.CiderError, match=rf": {name} must start at a multiple of 16 bytes"):
            call()
    # their copies are taken
    c.cider_kv4_append(cache, k, k, cut.clone())
    assert c.cider_kv4_attention(q, cache, table, cut.clone()).shape == q.shape
