"""Sums of attention over long caches, to a tolerance that does not grow with the
length: a row's error is that of the weights' fp16 rounding and of its result."""
import pytest

from tests.test_gpu_parity import cider

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests import kv4_reference as ref  # noqa: E402
from tests.test_gpu_kv4 import DT, gen, rnd  # noqa: E402

U = 2.0 ** -24


def long_cache(g, c, L, Hkv, D, G, v_mean, page=128):
    pages = -(-L // page)
    code = lambda mean: rnd(g, pages, Hkv, page, D, scale=2.6, mean=mean).round_().clamp_(-7, 7)  # noqa: E731
    scale = lambda: 0.3 + 0.3 * torch.rand(pages, Hkv, G, page, generator=g, device="cuda")      # noqa: E731
    return c.KV4Cache(ref.pack(code(0.0)), scale(), ref.pack(code(v_mean)), scale())


def row(q, k, v, scale, sk):
    """A row in 64 bits, the norm of independent relative errors of its weights,
    and the size of an error of its scores."""
    s = scale * (k @ q)
    p = torch.softmax(s, 0)
    # a score: D products of up to 2 * 279 |q| s_k before the offset is off, each fp32
    # step cut (2 U), as independent errors three times the root of their number; then
    # its scaling, the difference to the maximum and the exponential
    score = 3 * scale * float(q.abs().sum()) * 2 * 279 * sk * U / len(q) ** 0.5 + (float(s.abs().max()) + 16) * 4 * U
    return p @ v, (p.square() @ v.square()).sqrt(), score


def check_rows(y, picks, q, k, v, per, scale, sk, extra=0.0):
    """Joint error over the picked rows. Weights: half a step of fp16 each, 2^-11,
    as independent errors (and `extra`). fp32 sums: up to 2^14 steps of a wave, each
    cut by 2^-23, and 2^17 terms of the sum of weights, each rounded by 2^-24, as
    independent ones 2^-16 and 2^-15.5: 2^-14. The result: half a step of its type."""
    err = 0.0
    weights = size = 0.0
    for t, h in picks:
        want, spread, score = row(q[t, h].double(), k[:, h // per], v[:, h // per], scale, sk)
        err += float((y[t, h].double() - want).square().sum())
        weights += float((spread * (2.0 ** -11 + extra + 2 * score)).square().sum())
        size += float(want.square().sum())
    allowed = weights ** 0.5 + size ** 0.5 * (torch.finfo(y.dtype).eps / 2 + 2.0 ** -14)
    assert err ** 0.5 <= allowed, (err ** 0.5 / size ** 0.5, allowed / size ** 0.5)


# standard deviation of q (0: every token weighs the same; 8: a few tokens have nearly all weight), mean of V's codes
KINDS = [(0.0, 0.0), (1.0, 0.0), (8.0, 0.0), (0.0, 2.0)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 1), (64, 2), (128, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("B,n,Hq,Hkv,L", [(1, 2048, 32, 4, 131072), (64, 1, 8, 8, 131072), (1, 70, 4, 1, 131072),
                                          (1, 1, 16, 8, 500000)])
def test_long_sums(B, n, Hq, Hkv, L, D, G, dtype):
    """Long ranges of one wave (many rows, and many sequences over the same pages), and parts that are joined."""
    c, t, g = cider(), DT[dtype], gen(L + D + G + n)
    for q_std, v_mean in KINDS:
        cache = long_cache(g, c, L, Hkv, D, G, v_mean)
        table = torch.arange(cache.k_codes.shape[0], device="cuda", dtype=torch.int32).repeat(B, 1)
        q = rnd(g, B * n, Hq, D, t=t, scale=q_std)
        y = c.cider_kv4_attention(q, cache, table, torch.full((B,), L, dtype=torch.int32, device="cuda"), causal=False)
        k, v = ref.stored_rows(cache, torch.arange(L, device="cuda"))
        at = torch.randint(0, B * n, (3,), generator=g, device="cuda").tolist()
        picks = {(i, h) for i in at for h in range(0, Hq, max(1, Hq // 4))}
        check_rows(y, picks, q, k, v, Hq // Hkv, D ** -0.5, float(cache.k_scale.max()))
        del k, v


# lengths, queries of each, query heads, key/value heads
SPREAD = [([300, 90], [1, 1], 4, 2), ([500, 400], [3, 3], 4, 2), ([300], [300], 4, 2), ([700, 500], [90, 200], 4, 2),
          ([4000], [1100], 2, 2), ([9000], [8800], 1, 1)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,gs", [(64, 0), (128, 32), (256, 128)])
@pytest.mark.parametrize("lens,counts,Hq,Hkv", SPREAD)
def test_a_large_scale_of_no_weight(lens, counts, Hq, Hkv, D, gs, dtype):
    """A token in the middle of each sequence with keys opposed to every query, and a scale of V far above the others':
    it has no weight, rows before it do not see it, and what is left of the others' weights is in units of its scale."""
    from tests.test_gpu_kv4 import i32, setup
    c, t, g = cider(), DT[dtype], gen(sum(lens) + D + gs)
    page, G = 32, D // gs if gs else 1
    for factor in (1e4, 1e5, 1e6):
        q, cache, table, ends = setup(c, g, lens, counts, Hq, Hkv, D, gs, page, t)
        q = (q.abs() + 0.25).to(t)
        for b, L in enumerate(lens):
            at = L - counts[b] // 2 - 2
            p, o = int(table[b, at // page]), at % page
            cache.k_codes[p, :, o] = 0x11                    # -7, of scores below -200
            cache.k_scale[p, :, :, o] = 10.0
            cache.v_scale[p, :, :, o] *= factor
        y = c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=i32(ends))
        err = weights = size = 0.0
        for b, (L, n) in enumerate(zip(lens, counts)):
            at = torch.arange(L, device="cuda")
            at = at[at != L - n // 2 - 2]                    # the token itself adds nothing: 2^-200
            k, v = ref.stored_rows(cache, table[b].long()[at // page] * page + at % page)
            sv = cache.v_scale[table[b].long()[at // page], :, :, at % page].double().repeat_interleave(D // G, -1)
            for i in {0, n // 3, n - 1}:
                seen = at <= L - n + i
                for h in range(Hq):
                    u, q64 = h // (Hq // Hkv), q[ends[b] + i, h].double()
                    want, spread, score = row(q64, k[seen, u], v[seen, u], D ** -0.5, 0.6)
                    p = torch.softmax(D ** -0.5 * (k[seen, u] @ q64), 0)
                    # half of the smallest step of fp16, 2^-25, in units of at most 1/64 of the largest scale; the
                    # largest weight of a row is one at least
                    lost = 2.0 ** -25 / 64 * 0.6 * factor * float(p.max()) * (v[seen, u] / sv[seen, u]).square().sum(0).sqrt()
                    err += float((y[ends[b] + i, h].double() - want).square().sum())
                    weights += float((spread * (2.0 ** -11 + 2 * score) + lost).square().sum())
                    size += float(want.square().sum())
        allowed = weights ** 0.5 + size ** 0.5 * (torch.finfo(t).eps / 2 + 2.0 ** -14)
        assert err ** 0.5 <= allowed, (factor, err ** 0.5 / size ** 0.5, allowed / size ** 0.5)


@pytest.mark.parametrize("power", [-127, -119, -118, 118, 124])
@pytest.mark.parametrize("n,L", [(1, 400), (90, 400), (40, 4000)])      # two joins of a few parts, one of many
def test_scales_at_the_ends_of_the_type(n, L, power):
    """Scales of V up to where bf16 results end, and down to where fp32 scales lose bits. (Sums of averages times their
    weights would pass fp32's largest number before the results do.)"""
    from tests.test_gpu_kv4 import i32, setup
    c, g = cider(), gen(n)
    q, cache, table, ends = setup(c, g, [L], [n], 4, 2, 128, 64, 16, torch.bfloat16)
    cache.v_scale.mul_(2.0 ** power)
    y = c.cider_kv4_attention(q, cache, table, i32([L]))
    at = torch.arange(L, device="cuda")
    k, v = ref.stored_rows(cache, table[0].long()[at // 16] * 16 + at % 16)
    fin = torch.finfo(torch.bfloat16)
    for i in {0, n // 2, n - 1}:
        seen = L - n + i + 1
        for h in range(4):
            want, spread, score = row(q[i, h].double(), k[:seen, h // 2], v[:seen, h // 2], 128 ** -0.5, 0.6)
            # (results and their roundings below the normal range: half a smallest step each, the fp32 ones' too)
            allowed = spread.norm() * (2.0 ** -11 + 2 * score) + want.norm() * (fin.eps / 2 + 2.0 ** -14) + \
                (fin.tiny * fin.eps + 2.0 ** -149) / 2 * 128 ** 0.5
            assert float((y[i, h].double() - want).norm()) <= float(allowed), (i, h)
            assert bool(y[i, h].isfinite().all())


@pytest.mark.parametrize("D,G", [(64, 2), (128, 1), (256, 2)])
@pytest.mark.parametrize("B,n,Hq,Hkv,L", [(1, 2048, 32, 4, 131001), (64, 1, 8, 8, 131001), (1, 70, 4, 1, 131001),
                                          (1, 1, 16, 8, 131001), (1, 1000, 2, 1, 131001)])
def test_no_part_of_a_long_range_is_lost(B, n, Hq, Hkv, L, D, G):
    """Equal weights over codes of V that rise from 0 to 6: without the first or the last page of 1024 the average would be
    off by 2^-10 of itself, without a part of a join by far more, and the bound is 2^-10.8."""
    c, g = cider(), gen(L + D + n)
    cache = long_cache(g, c, L, Hkv, D, G, 0.0)
    pages = cache.k_codes.shape[0]
    rise = torch.linspace(0.0, 6.0, pages, device="cuda").view(-1, 1, 1, 1) + 1.5 * torch.rand(pages, Hkv, 128, D, generator=g, device="cuda") - 0.75
    cache.v_codes.copy_(ref.pack(rise.round_().clamp_(-7, 7)))
    cache.v_scale.fill_(0.4)
    table = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(B, 1)
    q = torch.zeros(B * n, Hq, D, dtype=torch.float16, device="cuda")
    y = c.cider_kv4_attention(q, cache, table, torch.full((B,), L, dtype=torch.int32, device="cuda"), causal=False)
    _, v = ref.stored_rows(cache, torch.arange(L, device="cuda"))
    want = v.mean(0).repeat_interleave(Hq // Hkv, 0)
    off = (y.double() - want).flatten(1).norm(dim=1) / want.norm()
    assert float(off.max()) <= 2.0 ** -11 + 2.0 ** -14, float(off.max())
