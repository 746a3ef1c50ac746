"""Query offsets of attention: what may come in them, and what a batch may mix."""
import pytest

from tests.test_gpu_parity import cider

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests.test_gpu_kv4 import DT, check, gen, i32, setup  # noqa: E402


@pytest.mark.parametrize("n,Hq,L,offsets", [
    (1024, 4, 300, lambda T: [0, T // 2, 0, T]),                   # more tiles than the launch has places for
    (300, 2, 3000, lambda T: [T // 3, T, -T, T]),                  # the same in parts
    (5, 4, 700, lambda T: [0, T, 2, T]),                           # few rows
    (5, 4, 700, lambda T: [T, 0, -1, 1 << 30]),
])
def test_offsets_that_do_not_ascend_stay_in_bounds(n, Hq, L, offsets):
    """Rows behind T, and bytes behind the workspace, are left as they were; sequences of another call are not touched."""
    c, g = cider(), gen(n)
    q, cache, table, ends = setup(c, g, [L] * 3, [n] * 3, Hq, 2, 128, 64, 16, torch.float16)
    T = ends[-1]
    before = [a.clone() for a in cache]
    size = c.cider_kv4_attention_workspace_size(T, 3, Hq, 2, 128, table.shape[1] * 16)
    space = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 64, Hq, 128), 5.0, dtype=torch.float16, device="cuda")
    c.cider_kv4_attention(q, cache, table, i32([L] * 3), query_offsets=i32(offsets(T)), y=out[:T], workspace=space[:size])
    torch.cuda.synchronize()
    assert bool((out[T:] == 5).all()) and bool((space[size:] == 77).all())
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    y = c.cider_kv4_attention(q, cache, table, i32([L] * 3), query_offsets=i32(ends))
    check(y, q, cache, table, [L] * 3, ends)


# queries of each sequence, query heads, key/value heads: prompts and chunks between single tokens, on both sides of the
# rule that chooses a kernel by the average
MIXED = [([1] * 40 + [300] + [1] * 23, 4, 2), ([1, 700, 1, 1, 0, 33], 4, 2), ([1] * 30 + [90, 0, 5], 16, 2), ([1, 1, 2000], 2, 1)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,gs", [(64, 32), (128, 0), (256, 64)])
@pytest.mark.parametrize("counts,Hq,Hkv", MIXED)
def test_prompts_and_single_tokens_in_one_call(counts, Hq, Hkv, D, gs, dtype):
    """A page table as wide as the largest context that a captured call is to serve, most of it unused."""
    c, g = cider(), gen(sum(counts) + D)
    lens = [n + (b * 977) % 1500 if n else 40 for b, n in enumerate(counts)]
    q, cache, table, ends = setup(c, g, lens, counts, Hq, Hkv, D, gs, 32, DT[dtype], extra_pages=300)
    y = c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=i32(ends))
    check(y, q, cache, table, lens, ends)
