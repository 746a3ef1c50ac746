"""Head norms of the cache's writer where fp32 ends."""
import pytest

from tests.test_gpu_parity import cider

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests.test_gpu_kv4 import gen, rnd  # noqa: E402


@pytest.mark.parametrize("D", [64, 128, 256])
def test_heads_whose_squares_overflow_are_nan(D):
    """NaN in q_out, and for k a scale of NaN with codes 0; other heads, and sums that just fit, are as they were."""
    c, g = cider(), gen(D)
    t = torch.bfloat16
    q, k, v = rnd(g, 5, 4, D, t=t), rnd(g, 5, 2, D, t=t), rnd(g, 5, 2, D, t=t)
    w = torch.ones(D, dtype=t, device="cuda")
    slots = torch.arange(5, device="cuda").to(torch.int32)
    plain, cache = c.kv4_cache(1, 2, 16, D, 32 if D < 256 else 64), c.kv4_cache(1, 2, 16, D, 32 if D < 256 else 64)
    want = c.cider_kv4_append(plain, k, v, slots, q=q, q_norm=w, k_norm=w)
    q[1, 2, 3], k[2, 1, 7], q[3, 0] = 1e20, -3e19, 1e18       # squares of 1e40 and 9e38 overflow, D of 1e36 do not
    out = c.cider_kv4_append(cache, k, v, slots, q=q, q_norm=w, k_norm=w)
    hit = torch.zeros(5, 4, dtype=torch.bool, device="cuda")
    hit[1, 2] = True
    assert bool(out[hit].isnan().all()) and bool((out[3, 0] == 1).all())
    hit[3, 0] = True
    assert torch.equal(out[~hit], want[~hit])
    assert bool(cache.k_scale[0, 1, :, 2].isnan().all()) and bool((cache.k_codes[0, 1, 2] == 0x88).all())
    for a, b in zip(cache[:2], plain[:2]):
        a, b = (a, b) if a.dtype == torch.uint8 else (a.transpose(2, 3), b.transpose(2, 3))
        keep = torch.ones(2, 16, dtype=torch.bool, device="cuda")
        keep[1, 2] = False
        assert torch.equal(a[0][keep], b[0][keep])
    assert torch.equal(cache.v_codes, plain.v_codes) and torch.equal(cache.v_scale, plain.v_scale)
