"""Rotary positions, the 4-bit cache and attention over it, against plain forms
in 64 bits (tests/kv4_reference.py)."""
import math

import pytest

from tests.test_gpu_parity import cider

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests import kv4_reference as ref  # noqa: E402

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
GROUPS = [(64, 0), (64, 32), (128, 0), (128, 64), (128, 32), (256, 0), (256, 128), (256, 64)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, t=torch.float32, scale=1.0, mean=0.0):
    return (mean + scale * torch.randn(*shape, generator=g, device="cuda")).to(t)


def within(got, want, bound):
    """|got - want| <= bound, and both NaN in the same places."""
    assert torch.equal(got.isnan(), want.isnan())
    off = torch.where(want.isnan(), 0.0, (got.double() - want).abs() - bound)
    assert float(off.max()) <= 0.0, (float(off.max()), int(off.argmax()))


def rounding(y, t):
    return y.abs() * (torch.finfo(t).eps / 2) + torch.finfo(t).tiny * torch.finfo(t).eps / 2


# ---- rotary positions -------------------------------------------------------

ROPE = [(1, 1, 2, 2), (3, 2, 10, 4), (5, 3, 64, 64), (2, 9, 96, 24), (7, 5, 80, 48), (16, 16, 128, 128), (9, 24, 128, 64),
        (130, 3, 256, 256), (33, 40, 64, 16), (4, 2, 1024, 512), (2, 1, 36, 32), (3, 7, 128, 100), (1030, 6, 128, 96)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rd", ROPE)
def test_rope(T, H, D, rd, interleaved, dtype):
    c, t, g = cider(), DT[dtype], gen(T + D)
    x = rnd(g, T, H, D, t=t)
    pos = torch.randint(-1000, 1 << 20, (T,), generator=g, device="cuda").to(torch.int32)
    pos[0] = (1 << 31) - 1 if T > 1 else 0
    freq, scale = c.rope_frequencies(rd, scaling="parts", factor=8.0, trained=4096)
    want = ref.rotate(x, pos, freq, interleaved, scale)
    # positions near 2^31: the fp64 angle itself is off by 2^31 * 2^-53 * a few
    bound = (ref.rotation_error(x.double(), freq, interleaved, scale) + 2e-6 * x.double().abs().amax()) * 1.01
    y = c.cider_rope(x, pos, freq, interleaved=interleaved, scale=scale)
    within(y, want, bound + rounding(want, t) * 1.01)
    assert torch.equal(y[..., rd:], x[..., rd:])
    # strided rows in, rows with guards out, and in place: the same bits
    wide = torch.full((T, H + 2, D + 8), float("nan"), dtype=t, device="cuda")
    wide[:, 1:-1, :D] = x
    out = torch.full((T, H + 1, D + 16), 7.0, dtype=t, device="cuda")
    if (D + 8) * 2 % 16 == 0 and D * 2 % 16 == 0:      # 16-byte aligned starts
        view = wide[:, 1:-1, :D]
        c.cider_rope(view, pos, freq, interleaved=interleaved, scale=scale, y=out[:, :H, :D])
        assert torch.equal(out[:, :H, :D], y)
        assert bool((out[:, H:] == 7).all()) and bool((out[..., D:] == 7).all())
        c.cider_rope(view, pos, freq, interleaved=interleaved, scale=scale, y=view)
        assert torch.equal(view, y) and bool(wide[:, 0].isnan().all()) and bool(wide[..., D:].isnan().all())
    # heads before tokens
    flip = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(c.cider_rope(flip, pos, freq, interleaved=interleaved, scale=scale), y)


def test_rope_paths_agree():
    """The chunked kernels and the element one give the same bits (an odd head stride takes the latter)."""
    c, g = cider(), gen(3)
    for t in DT.values():
        for interleaved in (False, True):
            x = rnd(g, 37, 6, 128, t=t)
            pos = torch.arange(37, device="cuda").to(torch.int32) * 999
            freq, _ = c.rope_frequencies(64)
            odd = torch.empty(37, 6, 129, dtype=t, device="cuda")[..., :128]
            odd.copy_(x)
            assert torch.equal(c.cider_rope(odd, pos, freq, interleaved=interleaved),
                               c.cider_rope(x, pos, freq, interleaved=interleaved))


def test_rope_turns_back():
    """Positions p and -p undo each other, scores depend on differences of positions only, lengths are kept."""
    c, g = cider(), gen(4)
    x = rnd(g, 64, 4, 128, t=torch.float16)
    freq, _ = c.rope_frequencies(128)
    pos = torch.randint(0, 1 << 17, (64,), generator=g, device="cuda").to(torch.int32)
    y = c.cider_rope(x, pos, freq)
    back = c.cider_rope(y, -pos, freq)
    # two roundings of 2^-11 of values up to the pair's length, and the fp32 steps
    pair = torch.hypot(x[..., :64].double(), x[..., 64:].double()).repeat(1, 1, 2)
    assert bool(((back.double() - x.double()).abs() <= pair * (2 * 1.5 * 2.0 ** -11 + 1e-5)).all())
    a, b = rnd(g, 1, 1, 128, t=torch.float16).expand(64, 1, 128), rnd(g, 1, 1, 128, t=torch.float16).expand(64, 1, 128)
    s = (c.cider_rope(a, pos, freq).double() * c.cider_rope(b, pos - 77, freq).double()).sum(-1)
    assert float((s - s[0]).abs().max()) <= float((a[0].double().norm() * b[0].double().norm()) * (2 * 2.0 ** -11 + 1e-4))


# ---- the cache --------------------------------------------------------------

APPEND = [(1, 1, 1), (3, 4, 2), (17, 9, 3), (64, 0, 8), (5, 40, 1), (130, 16, 8), (1031, 6, 2)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,gs", GROUPS)
@pytest.mark.parametrize("T,Hq,Hkv", APPEND)
def test_append(T, Hq, Hkv, D, gs, dtype):
    c, t, g = cider(), DT[dtype], gen(T * 7 + D + gs)
    page, G = (16, 32, 128)[T % 3], D // gs if gs else 1
    pages = -(-T // page) + 2
    cache = c.kv4_cache(pages, Hkv, page, D, gs)
    for a in cache:                                   # what is not written stays
        a.copy_(torch.randint(0, 255, a.shape, generator=g, device="cuda").to(a.dtype))
    before = [a.clone() for a in cache]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 4:
        slots[1], slots[3] = -1, pages * page
    kept = (slots >= 0) & (slots < pages * page)
    k, v = rnd(g, T, Hkv, D, t=t) * 3, rnd(g, T, Hkv, D, t=t)
    q = rnd(g, T, Hq, D, t=t) if Hq else None
    rd, interleaved, normed = (D, D // 2, D // 4)[(T + Hq) % 3], bool(T % 2), bool((T + Hkv) % 2)
    freq, scale = c.rope_frequencies(rd, scaling="parts", factor=4.0)
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda").to(torch.int32)
    nq, nk = (rnd(g, D, t=t, mean=1.0, scale=0.2), rnd(g, D, t=t, mean=1.0, scale=0.2)) if normed else (None, None)
    kw = dict(positions=pos, inv_freq=freq, interleaved=interleaved, rope_scale=scale, eps=1e-5)
    out = c.cider_kv4_append(cache, k, v, slots, q=q, q_norm=nq if Hq else None, k_norm=nk, **kw)
    if not Hq:
        assert out is None
    # k's 16-bit values: the same rows given as q
    seen = c.cider_kv4_append(c.kv4_cache(pages, Hkv, page, D, gs), k, v, slots, q=k, q_norm=nk, k_norm=nk, **kw)
    for x, w, y in ((q, nq, out), (k, nk, seen)):
        if x is None:
            continue
        n = x.double()
        # a sum of D squares over lanes, its root and quotient, two products
        rel = 0.0
        if w is not None:
            n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + 1e-5) * w.double()
            rel = ((8 + 6) / 2 + 4 + 2) * ref.U
        err = ref.rotation_error(n, freq, interleaved, scale)
        pair = ref.rotation_error(n, freq, interleaved, scale) / ((math.pi + 12) * ref.U) * rel
        want = ref.rotate(n, pos, freq, interleaved, scale)
        within(y, want, (err + pair + n.abs() * rel) * 1.01 + rounding(want, t) * 1.01)
        if w is None:
            assert torch.equal(y, c.cider_rope(x, pos, freq, interleaved=interleaved, scale=scale))
    at, of = slots[kept].long() % page, slots[kept].long() // page
    place = ref.v_place(D, G).to("cuda")
    for x, codes, scales, order in ((seen, cache.k_codes, cache.k_scale, None), (v, cache.v_codes, cache.v_scale, place)):
        want, s = ref.int4_rule(x[kept], G)
        got = ref.unpack(codes[of, :, at]).long()
        assert torch.equal(got if order is None else got[..., order], want)
        assert torch.equal(scales[of, :, :, at], s)
    untouched = torch.ones(pages, page, dtype=torch.bool, device="cuda")
    untouched[of, at] = False
    for a, b, tok in zip(cache, before, (2, 3, 2, 3)):
        a, b = (a, b) if tok == 2 else (a.transpose(2, 3), b.transpose(2, 3))
        assert torch.equal(a.transpose(1, 2)[untouched], b.transpose(1, 2)[untouched])
    # and back, the same slot twice, slots outside as zeros
    again = torch.cat((slots, slots[:1]))
    rk, rv = c.cider_kv4_read(cache, again, out_dtype=t)
    inside = torch.where((again >= 0) & (again < pages * page), again, 0)
    wk, wv = ref.stored_rows(cache, inside)
    ok = (again == inside)[:, None, None]
    for got, want in ((rk, wk), (rv, wv)):
        want = torch.where(ok, want, torch.zeros_like(want))
        assert torch.equal(got, want.float().to(t))   # one fp32 product, then one rounding


def test_append_in_place_and_from_fused_rows():
    """q, k and v as slices of the projections' rows, q written back in place."""
    c, g, T = cider(), gen(11), 50
    for D, gs in ((64, 0), (128, 64)):
        rows = rnd(g, T, 6 + 2 + 2, D, t=torch.bfloat16)
        freq, _ = c.rope_frequencies(D)
        pos = torch.arange(T, device="cuda").to(torch.int32)
        slots = torch.arange(T, device="cuda").to(torch.int32)
        a, b = c.kv4_cache(4, 2, 16, D, gs), c.kv4_cache(4, 2, 16, D, gs)
        parts = [rows[:, :6].contiguous(), rows[:, 6:8].contiguous(), rows[:, 8:].contiguous()]
        want = c.cider_kv4_append(a, parts[1], parts[2], slots, q=parts[0], positions=pos, inv_freq=freq)
        kv = rows[:, 6:].clone()
        view = rows[:, :6]
        got = c.cider_kv4_append(b, rows[:, 6:8], rows[:, 8:], slots, q=view, positions=pos, inv_freq=freq, q_out=view)
        assert got.data_ptr() == rows.data_ptr() and torch.equal(rows[:, :6], want) and torch.equal(rows[:, 6:], kv)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,gs", GROUPS)
def test_append_values_at_the_borders(D, gs, dtype):
    """Ties between codes, zeros, the type's smallest and largest values; what is not finite leaves a NaN scale."""
    c, t, g = cider(), DT[dtype], gen(5)
    fin, G = torch.finfo(t), D // gs if gs else 1
    x = torch.randint(-14, 15, (24, 2, D), generator=g, device="cuda").to(t) / 2      # 7 * x / max on half-integers
    x[..., ::32] = 7
    x[1] = 0
    x[2] *= fin.smallest_normal / 8                                                   # denormals
    x[3] = (x[3].float() / 7 * fin.max).to(t)
    x[4] = torch.where(x[4] == 7, x[4], -x[4])
    x[5] = -0.0
    x[6] = fin.smallest_normal * fin.eps
    cache = c.kv4_cache(2, 2, 16, D, gs)
    slots = torch.arange(24, device="cuda").to(torch.int32)
    bad = x.clone()
    bad[8, 0, 3], bad[9, 1, D - 1], bad[10, 0, 40] = float("nan"), float("inf"), -float("inf")
    c.cider_kv4_append(cache, bad, bad, slots)
    codes, s = ref.int4_rule(x, G)
    hit = torch.zeros(24, 2, G, dtype=torch.bool, device="cuda")
    hit[8, 0, 3 * G // D] = hit[9, 1, G - 1] = hit[10, 0, 40 * G // D] = True
    codes = torch.where(hit.repeat_interleave(D // G, -1), 0, codes)
    at, of = slots.long() % 16, slots.long() // 16
    for got, scale, order in ((cache.k_codes, cache.k_scale, None), (cache.v_codes, cache.v_scale, ref.v_place(D, G).cuda())):
        got = ref.unpack(got[of, :, at]).long()
        assert torch.equal(got if order is None else got[..., order], codes)
        scale = scale[of, :, :, at]
        assert torch.equal(scale.isnan(), hit) and torch.equal(scale[~hit], s[~hit])


@pytest.mark.parametrize("dtype,interleaved", [("fp16", False), ("bf16", True)])
def test_results_past_the_cache(dtype, interleaved):
    """Results of 64 MB and more are stored another way: the same values as in parts."""
    c, t, g = cider(), DT[dtype], gen(6)
    T, Hq, Hkv, D = 9000, 32, 16, 128
    q, k, v = rnd(g, T, Hq, D, t=t), rnd(g, T, Hkv, D, t=t), rnd(g, T, Hkv, D, t=t)
    assert 2 * q.numel() >= 64 << 20 and 4 * k.numel() >= 64 << 20
    freq, _ = c.rope_frequencies(D)
    pos, slots = torch.arange(T, device="cuda").to(torch.int32), torch.arange(T, device="cuda").to(torch.int32)
    kw = dict(inv_freq=freq, interleaved=interleaved)
    y = c.cider_rope(q, pos, **kw)
    whole, parts = c.kv4_cache(71, Hkv, 128, D, 64), c.kv4_cache(71, Hkv, 128, D, 64)
    out = c.cider_kv4_append(whole, k, v, slots, q=q, positions=pos, **kw)
    rows = c.cider_kv4_read(whole, slots, out_dtype=t)
    for lo in range(0, T, 3000):
        at = slice(lo, lo + 3000)
        p, s = pos[at].clone(), slots[at].clone()
        assert torch.equal(c.cider_rope(q[at], p, **kw), y[at])
        assert torch.equal(c.cider_kv4_append(parts, k[at], v[at], s, q=q[at], positions=p, **kw), out[at])
        for a, b in zip(c.cider_kv4_read(whole, s, out_dtype=t), rows):
            assert torch.equal(a, b[at])
    assert all(torch.equal(a, b) for a, b in zip(whole, parts)) and torch.equal(out, y)


# ---- attention --------------------------------------------------------------

def filled(g, c, pages, Hkv, page, D, gs, t):
    """A cache as quantization leaves it: bells of codes, scales of a spread."""
    G = D // gs if gs else 1
    code = lambda: torch.randn(pages, Hkv, page, D, generator=g, device="cuda").mul_(2.6).round_().clamp_(-7, 7)  # noqa: E731
    scale = lambda: 0.3 + 0.3 * torch.rand(pages, Hkv, G, page, generator=g, device="cuda")   # noqa: E731
    return c.KV4Cache(ref.pack(code()), scale(), ref.pack(code()), scale())


def setup(c, g, lens, counts, Hq, Hkv, D, gs, page, t, spare=3, extra_pages=0):
    B = len(lens)
    most = max(1, -(-max(max(lens), 1) // page)) + extra_pages
    pages = sum(-(-max(L, 0) // page) for L in lens) + spare
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, most), -7, dtype=torch.int32, device="cuda")      # never used where there are no tokens
    done = 0
    for b, L in enumerate(lens):
        n = -(-max(L, 0) // page)
        table[b, :n] = order[done:done + n]
        done += n
    cache = filled(g, c, pages, Hkv, page, D, gs, t)
    ends = [sum(counts[:i]) for i in range(B + 1)]
    q = rnd(g, ends[-1], Hq, D, t=t, scale=1.5)
    return q, cache, table, ends


def check(y, q, cache, table, lens, ends, causal=True, window=0, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    want, bound, (typical, eps) = ref.attention(q, cache, table, lens, ends, causal, window, scale)
    rows = slice(0, ends[-1])
    within(y[rows], want[rows], bound[rows])
    # and over all elements the errors add up as independent ones do
    fin = ~want.isnan()
    err = (y.double() - want)[fin].norm()
    # (a result below the type's normal range is rounded to its smallest step)
    least = torch.finfo(q.dtype).tiny * torch.finfo(q.dtype).eps / 2
    allowed = 3 * typical[fin].norm() + eps * want[fin].norm() + least * int(fin.sum()) ** 0.5
    assert float(err) <= float(allowed) + 1e-12, (float(err), float(allowed))


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# lengths, queries of each sequence (None: one each), query heads, key/value heads, page size, causal, window
ATTEND = [
    ([1], None, 1, 1, 16, True, 0),
    ([15, 16, 17, 31, 32, 33], None, 4, 2, 16, True, 0),
    ([0, 5, 0, 129, 1000, 1], None, 6, 3, 16, True, 0),
    ([2000], None, 16, 8, 16, True, 0),
    ([777, 64], None, 20, 1, 64, True, 0),                       # more rows than one tile
    ([300, 900], None, 33, 3, 128, True, 100),
    ([100, 200], None, 8, 8, 32, True, 1),                       # a window of the token itself
    ([500, 31], None, 4, 4, 1024, False, 64),
    ([40, 300, 7], [5, 3, 7], 4, 2, 16, True, 0),                # a few drafted tokens
    ([90, 300, 4], [2, 3, 9], 8, 2, 32, True, 50),               # more queries than tokens
    ([100], [0], 4, 2, 16, True, 0),
    ([600, 0, 20], [0, 4, 2], 4, 2, 64, False, 0),
    ([200], [200], 4, 4, 16, True, 0),                           # whole prompts
    ([333, 65, 64, 129], [333, 65, 64, 129], 6, 2, 32, True, 0),
    ([700, 500], [150, 77], 8, 1, 16, True, 0),
    ([700, 1200], [150, 400], 3, 3, 128, True, 130),
    ([2100], [130], 8, 4, 64, True, 0),                          # the next part of a long one
    ([257, 300], [257, 90], 4, 2, 16, False, 0),
    ([100, 150], [190, 150], 4, 2, 16, True, 0),                 # rows before the first token
    ([1500], [140], 2, 2, 32, False, 200),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,gs", GROUPS)
@pytest.mark.parametrize("lens,counts,Hq,Hkv,page,causal,window", ATTEND)
def test_attention(lens, counts, Hq, Hkv, page, causal, window, D, gs, dtype):
    c, t, g = cider(), DT[dtype], gen(sum(lens) + D + gs)
    one = counts or [1] * len(lens)
    q, cache, table, ends = setup(c, g, lens, one, Hq, Hkv, D, gs, page, t)
    T = ends[-1]
    tail = torch.full((T + 3, Hq, D), 5.0, dtype=t, device="cuda")   # rows behind the last sequence
    if counts is None:
        y = c.cider_kv4_attention(q, cache, table, i32(lens), causal=causal, window=window)
    else:
        qq = torch.cat((q, torch.full((3, Hq, D), float("nan"), dtype=t, device="cuda")))
        y = c.cider_kv4_attention(qq, cache, table, i32(lens), query_offsets=i32(ends), causal=causal, window=window, y=tail)
        assert bool((y[T:] == 5).all())
        y = y[:T]
    if T:
        check(y, q, cache, table, lens, ends, causal, window)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 2, 1), (8, 2, 70)])
def test_same_rows_in_either_form(Hq, Hkv, n, dtype):
    """Queries with offsets, without, and from strided rows: the same bits where the plan is the same."""
    c, t, g = cider(), DT[dtype], gen(n)
    lens = [500, 900, 333]
    q, cache, table, ends = setup(c, g, lens, [n] * 3, Hq, Hkv, 128, 64, 32, t)
    a = c.cider_kv4_attention(q, cache, table, i32(lens))
    b = c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=i32(ends))
    check(a, q, cache, table, lens, ends)
    check(b, q, cache, table, lens, ends)
    rows = torch.full((3 * n, Hq + 4, 128), float("nan"), dtype=t, device="cuda")
    rows[:, 2:2 + Hq] = q
    assert torch.equal(c.cider_kv4_attention(rows[:, 2:2 + Hq], cache, table, i32(lens)), a)
    flip = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(c.cider_kv4_attention(flip, cache, table, i32(lens)), a)


@pytest.mark.parametrize("n,Hq", [(1, 4), (100, 4)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_nothing_hidden_is_used(n, Hq, dtype):
    """NaN and infinite scales in pages' ends, other pages, before a window and behind a row's position; page ids that are
    none, in places that no row sees."""
    c, t, g = cider(), DT[dtype], gen(n + 1)
    lens, counts = [300, 261], [n, n]
    for window in (0, 40):
        q, cache, table, ends = setup(c, g, lens, counts, Hq, 2, 128, 64, 32, t, extra_pages=2)
        wild = [a.clone() for a in cache]
        used = torch.zeros(cache.k_codes.shape[0], 32, dtype=torch.bool, device="cuda")
        for b, L in enumerate(lens):
            first = max(0, L - n - window + 1) if window else 0
            at = torch.arange(first, L, device="cuda")
            used[table[b].long()[at // 32], at % 32] = True
        hidden = ~used[:, None, None, :].expand_as(cache.k_scale)
        wild[1][hidden], wild[3][hidden] = float("nan"), float("inf")
        wild[3][:, 1][hidden[:, 1]] = float("nan")
        want = c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=i32(ends), window=window)
        t2 = table.clone()
        t2[:, -2:] = torch.tensor([1 << 30, -(1 << 31)], device="cuda").to(torch.int32)
        if window:
            t2[0, 0], t2[1, 0] = (1 << 31) - 1, -5       # pages given back
        got = c.cider_kv4_attention(q, c.KV4Cache(*wild), t2, i32(lens), query_offsets=i32(ends), window=window)
        assert torch.equal(want, got)
        check(got, q, cache, table, lens, ends, window=window)


@pytest.mark.parametrize("D,gs", GROUPS)
def test_nothing_hidden_is_used_of_small_pages(D, gs):
    """Windows that begin inside a page of 16, with infinite scales before them."""
    c, g = cider(), gen(D + gs)
    for n, window in ((3, 9), (90, 21), (90, 40)):
        lens, ends = [333, 500], [0, n, 2 * n]
        q, cache, table, _ = setup(c, g, lens, [n, n], 4, 2, D, gs, 16, torch.float16)
        wild = [a.clone() for a in cache]
        for b, L in enumerate(lens):
            for at in range(L - n - window + 1):
                for side in (1, 3):
                    wild[side][int(table[b, at // 16]), :, :, at % 16] = float("inf") if at % 2 else 1e30
        got = c.cider_kv4_attention(q, c.KV4Cache(*wild), table, i32(lens), window=window)
        assert torch.equal(got, c.cider_kv4_attention(q, cache, table, i32(lens), window=window))
        check(got, q, cache, table, lens, ends, window=window)


@pytest.mark.parametrize("n", [3, 90, 1500])
@pytest.mark.parametrize("side", [1, 3])
def test_an_infinite_scale_reaches_only_rows_that_see_it(n, side):
    """The rows before it, in the same tile too, are as without it (a maximum may be raised at another step); those behind
    an infinite scale of V are not finite."""
    c, g = cider(), gen(n)
    lens = [n + 40, 200 + n]
    q, cache, table, ends = setup(c, g, lens, [n] * 2, 4, 2, 128, 64, 16, torch.bfloat16)
    want, bound, _ = ref.attention(q, cache, table, lens, ends, True, 0, 128 ** -0.5)
    at = lens[1] - n // 2 - 1
    wild = [a.clone() for a in cache]
    wild[side][int(table[1, at // 16]), 1, 0, at % 16] = float("inf")
    y = c.cider_kv4_attention(q, c.KV4Cache(*wild), table, i32(lens))
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[ends[1] + at - (lens[1] - n):, 2:, : 128 if side == 1 else 64] = True
    within(y[~hit], want[~hit], bound[~hit])
    if side == 3:
        assert not bool(y[hit].isfinite().any())


@pytest.mark.parametrize("n", [1, 90])
def test_a_bad_token_reaches_only_rows_that_see_it(n):
    """A NaN scale of K or V at one token: rows that see it are NaN, the others have the bits they had."""
    c, g = cider(), gen(n)
    lens = [200, 200, 300]
    q, cache, table, ends = setup(c, g, lens, [n] * 3, 4, 2, 64, 32, 16, torch.float16)
    want = c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=i32(ends))
    for side in (1, 3):
        wild = [a.clone() for a in cache]
        at = 160 if n > 1 else 50
        wild[side][int(table[1, at // 16]), 1, 0, at % 16] = float("nan")
        y = c.cider_kv4_attention(q, c.KV4Cache(*wild), table, i32(lens), query_offsets=i32(ends))
        hit = torch.zeros_like(y, dtype=torch.bool)
        first = ends[1] + max(0, at - (200 - n))
        if side == 1:
            hit[first:ends[2], 2:] = True
        else:
            hit[first:ends[2], 2:, :32] = True           # the dimensions of that group
        assert torch.equal(y.isnan() & hit, hit)
        assert torch.equal(y[~hit], want[~hit])


@pytest.mark.parametrize("n", [1, 80])
def test_missing_pages_are_not_seen(n):
    c, g = cider(), gen(9)
    lens = [400, 150]
    q, cache, table, ends = setup(c, g, lens, [n, n], 4, 2, 128, 0, 16, torch.bfloat16)
    table[0, 3], table[0, 11], table[1, :] = -1, cache.k_codes.shape[0], -3      # the second sequence has none at all
    y = c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=i32(ends))
    check(y, q, cache, table, lens, ends)
    assert not bool(y[n:].any())


def test_lengths_and_offsets_out_of_range():
    """Lengths below 0 and past the table, offsets that do not ascend: clamped, every access in bounds."""
    c, g = cider(), gen(10)
    for n in (2, 70):
        lens, counts = [64, 64, 64], [n, n, n]
        q, cache, table, ends = setup(c, g, lens, counts, 4, 2, 64, 0, 16, torch.float16)
        y = c.cider_kv4_attention(q, cache, table, i32([-5, 1 << 30, 64]), query_offsets=i32(ends))
        check(y, q, cache, table, [0, 64, 64], ends)
        out = torch.full_like(q, 3.0)
        c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=i32([-4, n, n - 1, 1 << 30]), y=out)
        # 0 .. n, then nothing (it would descend), then n - 1 .. T: that row comes twice
        assert bool(out.isfinite().all())
        first = c.cider_kv4_attention(q[:n].contiguous(), cache, table[:1], i32([64]), query_offsets=i32([0, n]))
        check(first, q[:n], cache, table, [64], [0, n])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_values_of_any_size(dtype):
    """Scales of V from the type's smallest to its largest, in one sequence and alone; large and tiny scores."""
    c, t, g = cider(), DT[dtype], gen(12)
    for n in (1, 70):
        for power in (-20, 0, 12) if dtype == "fp16" else (-110, -20, 0, 12, 100):
            lens = [400]
            q, cache, table, ends = setup(c, g, lens, [n], 4, 2, 128, 64, 16, t)
            cache.v_scale.mul_(2.0 ** power)
            y = c.cider_kv4_attention(q, cache, table, i32(lens))
            check(y, q, cache, table, lens, ends)
        # growing along the sequence: the units follow
        q, cache, table, ends = setup(c, g, [400], [n], 4, 2, 128, 0, 16, t)
        for i, p in enumerate(table[0].tolist()):
            cache.v_scale[p] *= 2.0 ** (i / 3 - 6)
        check(c.cider_kv4_attention(q, cache, table, i32([400])), q, cache, table, [400], ends)
        # scores that grow by thousands from page to page, and scores of nearly nothing
        for f in (50.0, 2.0 ** -10):
            q, cache, table, ends = setup(c, g, [400], [n], 4, 2, 128, 0, 16, t)
            for i, p in enumerate(table[0].tolist()):
                cache.k_scale[p] *= f * (i + 1) / 4
            check(c.cider_kv4_attention(q, cache, table, i32([400])), q, cache, table, [400], ends)
        q, cache, table, ends = setup(c, g, [400], [n], 4, 2, 128, 0, 16, t)
        check(c.cider_kv4_attention(q, cache, table, i32([400]), softmax_scale=-0.05), q, cache, table, [400], ends, scale=-0.05)
        check(c.cider_kv4_attention(q, cache, table, i32([400]), softmax_scale=0.0), q, cache, table, [400], ends, scale=0.0)


@pytest.mark.parametrize("B,Hq,Hkv,D,n,L", [(1, 16, 8, 128, 1, 20000), (2, 4, 1, 256, 1, 40000), (1, 2, 1, 64, 100, 9000),
                                            (300, 2, 1, 64, 1, 90), (130, 2, 2, 64, 3, 60), (3, 16, 16, 128, 600, 700)])
def test_attention_long_and_many(B, Hq, Hkv, D, n, L):
    """Long contexts over many workgroups, more sequences than a wave has lanes."""
    c, g = cider(), gen(B)
    lens = [max(0, L - 17 * b % (L + 1)) for b in range(B)]
    counts = [n if n == 1 or b % 5 else 0 for b in range(B)] if B > 100 else [n] * B
    q, cache, table, ends = setup(c, g, lens, counts, Hq, Hkv, D, 0, 64, torch.bfloat16)
    offsets = None if n == 1 else i32(ends)
    y = c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=offsets)
    check(y, q, cache, table, lens, ends)


# lengths, queries of each sequence, query heads, key/value heads, page size, causal, window
LARGE = [
    ([1100, 3000], [1100, 1024], 8, 1, 64, True, 0),             # more than 8192 rows of a key/value head, no whole prompts
    ([6000], [1030], 2, 2, 16, True, 0),                         # from 1024 rows on a long cache: parts to join
    ([6000, 100, 0, 4000], [2050, 100, 0, 1025], 2, 1, 32, True, 900),
    ([2500], [1100], 1, 1, 128, False, 333),
    ([40000], [40], 1, 1, 1024, True, 0),                        # more than eight parts
    ([8300], [8300], 1, 1, 64, True, 0),                         # a whole prompt
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,gs", GROUPS)
@pytest.mark.parametrize("lens,counts,Hq,Hkv,page,causal,window", LARGE)
def test_attention_large_tiles(lens, counts, Hq, Hkv, page, causal, window, D, gs, dtype):
    c, g = cider(), gen(sum(lens) + D + gs)
    q, cache, table, ends = setup(c, g, lens, counts, Hq, Hkv, D, gs, page, DT[dtype])
    y = c.cider_kv4_attention(q, cache, table, i32(lens), query_offsets=i32(ends), causal=causal, window=window)
    check(y, q, cache, table, lens, ends, causal, window)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,gs", GROUPS)
@pytest.mark.parametrize("B,L,window", [(9, 5000, 0), (70, 900, 0), (70, 900, 200), (300, 400, 0), (3, 9000, 3000)])
def test_attention_shares_of_a_ragged_batch(B, L, window, D, gs, dtype):
    """Few rows of sequences of all lengths: workgroups end one, have some of their own and begin another; sequences
    without queries or tokens between them."""
    c, g = cider(), gen(B + L + D)
    lens = [0 if b % 11 == 5 else 1 + (b * 7919 + 13 * b * b) % L for b in range(B)]
    lens[B // 2] = L
    counts = [0 if b % 7 == 3 else 1 + b % 3 for b in range(B)]
    q, cache, table, ends = setup(c, g, lens, counts, 6, 2, D, gs, 32, DT[dtype])
    y = torch.full((ends[-1] + 2, 6, D), 5.0, dtype=DT[dtype], device="cuda")
    qq = torch.cat((q, q[:2]))
    c.cider_kv4_attention(qq, cache, table, i32(lens), query_offsets=i32(ends), window=window, y=y)
    assert bool((y[ends[-1]:] == 5).all())
    check(y[:ends[-1]], q, cache, table, lens, ends, window=window)


def test_a_cache_past_32_bits():
    """Codes and scales behind 4 GiB: the pages in use are the last ones."""
    c, g = cider(), gen(13)
    pages, Hkv, page, D = 33 * 1024, 8, 128, 256                  # 4.1 GiB of codes each
    cache = c.KV4Cache(torch.empty(pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda"),
                       torch.empty(pages, Hkv, 4, page, device="cuda"),
                       torch.empty(pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda"),
                       torch.empty(pages, Hkv, 4, page, device="cuda"))
    assert cache.k_codes.numel() > 1 << 32
    T = 300
    ids = i32([pages - 1, pages - 3, pages - 2])
    at = torch.arange(T, device="cuda")
    slots = (ids[at // page] * page + at % page).to(torch.int32)
    k, v = rnd(g, T, Hkv, D, t=torch.bfloat16), rnd(g, T, Hkv, D, t=torch.bfloat16)
    c.cider_kv4_append(cache, k, v, slots)
    small = c.kv4_cache(3, Hkv, page, D, 64)
    for a, b in zip(small, cache):
        a.copy_(b[ids.long()])
    other = c.kv4_cache(3, Hkv, page, D, 64)
    c.cider_kv4_append(other, k, v, at.to(torch.int32))
    for a, b in zip(small, other):
        if a.dtype == torch.uint8:
            assert torch.equal(a.transpose(1, 2).flatten(0, 1)[:T], b.transpose(1, 2).flatten(0, 1)[:T])
    for a, b in zip(c.cider_kv4_read(cache, slots), c.cider_kv4_read(other, at.to(torch.int32))):
        assert torch.equal(a, b)
    q = rnd(g, T, Hkv, D, t=torch.bfloat16)
    for n in (1, T):
        y = c.cider_kv4_attention(q[:n], cache, ids.view(1, 3), i32([T]))
        z = c.cider_kv4_attention(q[:n], other, i32([[0, 1, 2]]), i32([T]))
        assert torch.equal(y, z)


# ---- as they are used -------------------------------------------------------

def block_inputs(c, g, T, K, Hq, Hkv, D, t):
    x = rnd(g, T, K, t=t)
    w = rnd(g, (Hq + 2 * Hkv) * D, K, t=t, scale=K ** -0.5)
    wo = rnd(g, K, Hq * D, t=t, scale=(Hq * D) ** -0.5)
    return (*c.cider_quant_act(x), *c.cider_quant_weight(w), *c.cider_quant_weight(wo))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_block_prompt_then_tokens(dtype):
    """A prompt in two parts and then single tokens through w8a8_attention give what one whole prompt gives, and both
    what the parts give one after another."""
    c, t, g = cider(), DT[dtype], gen(21)
    K, Hq, Hkv, D, page, L = 512, 8, 2, 64, 16, 75
    freq, _ = c.rope_frequencies(D)
    xq, sx, wq, sw, woq, swo = block_inputs(c, g, L, K, Hq, Hkv, D, t)
    nq, nk = rnd(g, D, t=t, mean=1.0, scale=0.1), rnd(g, D, t=t, mean=1.0, scale=0.1)
    table = torch.randperm(8, generator=g, device="cuda").to(torch.int32).view(1, 8)
    pos = torch.arange(L, device="cuda")
    slots = (table[0].long()[pos // page] * page + pos % page).to(torch.int32)
    kw = dict(inv_freq=freq, q_norm=nq, k_norm=nk, out_dtype=t)

    def part(cache, lo, hi):
        return c.w8a8_attention(xq[lo:hi], sx[lo:hi].clone(), wq, sw, woq, swo, cache, slots[lo:hi].clone(), table,
                                i32([hi]), Hq, positions=pos[lo:hi].to(torch.int32), **kw)
    whole_cache, cache = c.kv4_cache(8, Hkv, page, D, 32), c.kv4_cache(8, Hkv, page, D, 32)
    whole = part(whole_cache, 0, L)
    # by hand
    q, k, v = c.cider_w8a8_gemm_split(xq, sx, wq, sw, [Hq * D, Hkv * D, Hkv * D], out_dtype=t)
    other = c.kv4_cache(8, Hkv, page, D, 32)
    q2 = c.cider_kv4_append(other, k.view(L, Hkv, D), v.view(L, Hkv, D), slots, q=q.view(L, Hq, D), positions=pos.to(torch.int32),
                            inv_freq=freq, q_norm=nq, k_norm=nk)
    a = c.cider_kv4_attention(q2, other, table, i32([L]))
    check(a, q2, other, table, [L], [0, L])
    aq, sa = c.cider_quant_act(a.view(L, -1))
    assert torch.equal(c.cider_w8a8_gemm(aq, sa, woq, swo, out_dtype=t), whole)
    assert all(torch.equal(x, y) for x, y in zip(whole_cache, other))
    rows = [part(cache, 0, 40), part(cache, 40, 70)] + [part(cache, i, i + 1) for i in range(70, L)]
    assert all(torch.equal(x, y) for x, y in zip(whole_cache, cache))      # the same tokens, the same codes
    # rows from other tiles' sums: the attention's bound, then codes of 1/127 that may differ by one
    got = torch.cat(rows)
    assert float((got.double() - whole.double()).norm() / whole.double().norm()) < 0.01


def test_block_captured_and_replayed():
    """One decode step of a block captured; replays for other lengths, slots, pages and rows equal the eager step, with
    eager work between them."""
    c, t, g = cider(), torch.bfloat16, gen(22)
    B, K, Hq, Hkv, D, page = 5, 512, 8, 2, 128, 16
    freq, _ = c.rope_frequencies(D)
    xq, sx, wq, sw, woq, swo = block_inputs(c, g, 4 * B, K, Hq, Hkv, D, t)
    table = torch.randperm(B * 20, generator=g, device="cuda").to(torch.int32).view(B, 20)
    cache = filled(g, c, B * 20, Hkv, page, D, 64, t)
    eager = c.KV4Cache(*(a.clone() for a in cache))
    x, s = xq[:B].clone(), sx[:B].clone()
    lens, slots, pos = i32([1] * B), i32([0] * B), i32([0] * B)

    def step(into):
        return c.w8a8_attention(x, s, wq, sw, woq, swo, into, slots, table, lens, Hq, positions=pos, inv_freq=freq, out_dtype=t)

    def place(i):
        L = [20 + 37 * ((b + i) % B) + i for b in range(B)]
        lens.copy_(i32(L))
        pos.copy_(lens - 1)
        at = pos.long()
        slots.copy_((table[torch.arange(B, device="cuda"), at // page].long() * page + at % page).to(torch.int32))
        x.copy_(xq[i * B:(i + 1) * B])
        s.copy_(sx[i * B:(i + 1) * B])

    place(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c.KV4Cache(*(a.clone() for a in cache)))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(cache)
    for i in (1, 2, 3, 1):
        place(i)
        graph.replay()
        got = y.clone()
        want = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
        assert all(torch.equal(a, b) for a, b in zip(cache, eager)), i


def test_two_graphs_with_a_workspace_each_and_two_streams():
    c, g = cider(), gen(23)
    cases = []
    for i in range(2):
        lens = [3000 - 500 * i, 800]
        q, cache, table, ends = setup(c, g, lens, [1, 1], 8, 2, 128, 0, 32, torch.float16)
        n = c.cider_kv4_attention_workspace_size(2, 2, 8, 2, 128, table.shape[1] * 32)
        assert n > 0
        cases.append((q, cache, table, i32(lens), torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)))
    want = [c.cider_kv4_attention(q, k, tb, ln) for q, k, tb, ln, _, _ in cases]
    graphs = []
    for q, k, tb, ln, ws, y in cases:
        c.cider_kv4_attention(q, k, tb, ln, workspace=ws, y=y)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.cider_kv4_attention(q, k, tb, ln, workspace=ws, y=y)
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for case in cases:
            case[4].fill_(255)                     # NaN partial results
            case[5].zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for w, case in zip(want, cases):
            assert torch.equal(case[5], w)
    # a stream that is not the current one: outputs and temporaries belong to it
    for _ in range(3):
        outs = [c.cider_kv4_attention(*case[:4], stream=st) for case, st in zip(cases, streams)]
        torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(1)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("n,Hq", [(1, 4), (90, 4)])
def test_repeats_are_the_same_bits(n, Hq):
    c, g = cider(), gen(24)
    lens = [2500, 1800, 90]
    q, cache, table, ends = setup(c, g, lens, [n] * 3, Hq, 2, 128, 64, 32, torch.bfloat16)
    want = c.cider_kv4_attention(q, cache, table, i32(lens))
    for _ in range(20):
        assert torch.equal(c.cider_kv4_attention(q, cache, table, i32(lens)), want)


def test_empty_calls():
    c = cider()
    cache = c.kv4_cache(2, 2, 16, 64)
    none = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    freq, _ = c.rope_frequencies(64)
    assert c.cider_rope(none, ids, freq).shape == (0, 4, 64)
    assert c.cider_kv4_append(cache, kv, kv, ids, q=none, positions=ids, inv_freq=freq).shape == (0, 4, 64)
    assert c.cider_kv4_read(cache, ids)[0].shape == (0, 2, 64)
    y = c.cider_kv4_attention(none, cache, torch.zeros(3, 1, dtype=torch.int32, device="cuda"), i32([0, 1, 2]),
                              query_offsets=i32([0, 0, 0, 0]))
    assert y.shape == (0, 4, 64)
    # no pages at all: every row is zeros
    q = torch.ones(3, 4, 64, dtype=torch.float16, device="cuda")
    y = c.cider_kv4_attention(q, cache, torch.zeros(3, 0, dtype=torch.int32, device="cuda"), i32([4, 1, 2]))
    assert not bool(y.any())


def test_refusals_of_the_binding():
    c, g = cider(), gen(25)
    cache = c.kv4_cache(2, 2, 16, 64)
    q, k = rnd(g, 2, 4, 64, t=torch.float16), rnd(g, 2, 2, 64, t=torch.float16)
    ids, freq = i32([0, 1]), c.rope_frequencies(64)[0]
    table = i32([[0], [1]])
    for call in (
        lambda: c.cider_rope(q.cpu(), ids, freq), lambda: c.cider_rope(q.float(), ids, freq),
        lambda: c.cider_rope(q, ids.long(), freq), lambda: c.cider_rope(q, ids, freq.float()),
        lambda: c.cider_rope(q, ids[:1], freq), lambda: c.cider_rope(q.transpose(1, 2), ids, freq),
        lambda: c.cider_rope(q, ids, freq, y=q.to(torch.bfloat16)), lambda: c.cider_rope(q, ids, freq, y=q[:, :2]),
        lambda: c.cider_kv4_append(cache, k, k, ids.long()), lambda: c.cider_kv4_append(cache, k, k.to(torch.bfloat16), ids),
        lambda: c.cider_kv4_append(cache, k[:, :1], k, ids), lambda: c.cider_kv4_append(cache, k, k, ids, positions=ids),
        lambda: c.cider_kv4_append(cache, k, k, ids, inv_freq=freq), lambda: c.cider_kv4_append(cache, k, k, ids, q_out=q),
        lambda: c.cider_kv4_append(cache, k, k, ids, q=q, q_norm=freq),
        lambda: c.cider_kv4_append(c.KV4Cache(cache[0], cache[1][:1], *cache[2:]), k, k, ids),
        lambda: c.cider_kv4_read(cache, ids, k=torch.empty(2, 2, 64, device="cuda")),
        lambda: c.cider_kv4_read(cache, ids.long()),
        lambda: c.cider_kv4_attention(q[:, :3], cache, table, ids), lambda: c.cider_kv4_attention(q, cache, table, ids.long()),
        lambda: c.cider_kv4_attention(q, cache, table[:1], ids), lambda: c.cider_kv4_attention(q, cache, table, ids, window=-1),
        lambda: c.cider_kv4_attention(q, cache, table, ids, query_offsets=ids),
        lambda: c.cider_kv4_attention(q[..., :32], cache, table, ids),
        lambda: c.cider_kv4_attention(rnd(g, 3, 4, 64, t=torch.float16), cache, table, ids),
        lambda: c.cider_kv4_attention(q, cache, i32([[0] * 512] * 2), ids, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: c.cider_kv4_attention(q, cache, table, ids, softmax_scale=float("inf")),
    ):
        with pytest.raises((TypeError, ValueError, c.CiderError)):
            call()
