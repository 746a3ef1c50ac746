"""The routing plan and the products grouped by expert against plain forms in
64 bits: the plan exactly, the plain products bit for bit (exact integers, two
fp32 products, one rounding), the gated products within the bound of their
fp32 steps plus half a step of the output type."""
import numpy as np
import pytest

from tests.test_gpu_parity import cider

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# ---- plan ------------------------------------------------------------------

def plain_plan(ids, E):
    flat = ids.reshape(-1).astype(np.int64)
    kept = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(kept, flat, E), kind="stable")
    n = int(kept.sum())
    rows = np.full(flat.size, -1, np.int64)
    rows[:n] = order[:n]
    slots = np.full(flat.size, -1, np.int64)
    slots[order[:n]] = np.arange(n)
    counts = np.bincount(flat[kept], minlength=E)
    return np.concatenate([[0], np.cumsum(counts)]), rows, slots.reshape(ids.shape)


def check_plan(c, ids, E, **kw):
    got = c.cider_moe_plan(torch.from_numpy(ids).cuda(), E, **kw)
    torch.cuda.synchronize()
    for name, g, o in zip(("offsets", "rows", "slots"), got, plain_plan(ids, E)):
        assert np.array_equal(g.cpu().numpy(), o), (name, ids.shape, E)


@pytest.mark.parametrize("T,k,E", [(0, 2, 5), (1, 1, 1), (1, 8, 64), (3, 3, 7), (63, 1, 2), (65, 2, 512), (129, 8, 128),
                                   (1024, 8, 64), (1025, 8, 40), (2049, 8, 511), (5000, 3, 96), (40000, 8, 128)])
def test_plan(T, k, E):
    c = cider()
    rng = np.random.default_rng(T * 31 + E)
    check_plan(c, rng.integers(0, E, (T, k)).astype(np.int32), E)
    ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)          # some of no expert
    ids[rng.random((T, k)) < 0.05] = np.int32(-2 ** 31)
    ids[rng.random((T, k)) < 0.05] = np.int32(2 ** 31 - 1)
    check_plan(c, ids, E)


@pytest.mark.parametrize("T", [40, 3000])
def test_plan_one_expert_or_none(T):
    c = cider()
    check_plan(c, np.full((T, 4), 6, np.int32), 7)
    check_plan(c, np.full((T, 4), -1, np.int32), 7)
    check_plan(c, np.full((T, 4), 7, np.int32), 7)


def test_plan_beyond_the_largest_grid_of_chunks():
    c = cider()
    rng = np.random.default_rng(3)
    check_plan(c, rng.integers(-1, 300, (600001, 1)).astype(np.int32), 299)


# ---- grouped products ---------------------------------------------------------

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def unpack(w):
    return torch.stack(((w & 15).to(torch.int16) - 8, (w >> 4).to(torch.int16) - 8), -1).flatten(-2)


def make(counts, N, K, bits, seed, T=None, k=1):
    """Codes, scales and offsets; with T, a gather index of T rows."""
    rng = np.random.default_rng(seed)
    E, P = len(counts), int(sum(counts))
    xr = P if T is None else T
    q = lambda *s: torch.from_numpy(np.clip(np.rint(rng.standard_normal(s) * 40), -127, 127).astype(np.int8))  # noqa: E731
    x = q(xr, K)
    sx = torch.from_numpy((0.01 + 0.03 * rng.random(xr)).astype(np.float32))
    if bits == 8:
        w, s = q(E, N, K), 6e-4
    else:
        nib = rng.integers(1, 16, (E, N, K)).astype(np.uint8)       # codes -7 .. 7
        w, s = torch.from_numpy(nib[..., 0::2] | (nib[..., 1::2] << 4)), 6e-3
    sw = torch.from_numpy((s * (0.5 + rng.random((E, N)))).astype(np.float32))
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    idx = None if T is None else torch.from_numpy(rng.integers(0, T * k, P).astype(np.int32))
    return x, sx, w, sw, off, idx


def plain_values(x, sx, w, sw, off, idx, div, bits):
    """v [P', N] as the fp32 two-step on exact sums, on the CPU."""
    codes = w if bits == 8 else unpack(w)
    out = []
    for e in range(w.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        src = torch.arange(lo, hi) if idx is None else idx[lo:hi].long() // div
        acc = x[src].double() @ codes[e].double().t()               # exact: |acc| < 2^31
        out.append((acc.to(torch.float32) * sx[src][:, None]) * sw[e])
    return torch.cat(out) if out else torch.empty(0, w.shape[1])


def call(c, bits, gated, x, sx, w, sw, off, idx, div, **kw):
    fn = getattr(c, f"cider_w{bits}a8_grouped_{'swiglu' if gated else 'gemm'}")
    return fn(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), off.cuda(), row_index=None if idx is None else idx.cuda(),
              row_div=div, **kw)


def assert_gated(y, v, dtype):
    n = v.shape[1] // 2
    g, u = v[:, :n].double(), v[:, n:].double()
    o = g * torch.sigmoid(g) * u
    # fp32 steps of the activation: (8 + |g|) 2^-23 relative; then half a step
    # of the output type, or of its smallest number
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    bound = o.abs() * (half + (8 + g.abs()) * 2.0 ** -23 * (1 + half)) + tiny + u.abs() * 2.0 ** -118
    off = (y.double().cpu() - o).abs() - bound
    assert y.shape == o.shape and bool((off <= 0).all()), float(off.max())


COUNTS = {
    "one": [1], "single rows": [1] * 8, "holes": [0, 5, 0, 0, 17, 1, 0], "edges": [16, 15, 17, 64, 63, 65, 0, 128],
    "large": [129, 0, 300, 257, 1, 700], "skewed": [0] * 63 + [400] + [1, 2],
    "many": [(7 * e) % 5 for e in range(500)], "many large": [60 + 9 * (e % 8) for e in range(70)]}


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("name,N,K", [("one", 16, 32), ("one", 1, 160), ("single rows", 200, 1024), ("holes", 136, 96),
                                      ("holes", 67, 672), ("edges", 264, 416), ("edges", 1003, 128),
                                      ("large", 520, 288), ("large", 321, 1152), ("skewed", 96, 64), ("many", 40, 64),
                                      ("many large", 72, 96)])
def test_grouped_is_the_dense_arithmetic(name, N, K, bits, dtype):
    c = cider()
    for T, k in ((None, 1), (37, 3)):
        a = make(COUNTS[name], N, K, bits, seed=len(name) + N, T=T, k=k)
        y = call(c, bits, False, *a, k, out_dtype=DT[dtype])
        o = plain_values(*a, k, bits).to(DT[dtype])
        assert torch.equal(y.cpu().view(torch.int16), o.view(torch.int16)), (T, k)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("name,N,K", [("one", 2, 32), ("single rows", 416, 1024), ("holes", 130, 672),
                                      ("edges", 528, 416), ("large", 1040, 288), ("large", 202, 1152),
                                      ("many", 80, 64), ("many large", 144, 96)])
def test_swiglu(name, N, K, bits, dtype):
    c = cider()
    for T, k in ((None, 1), (37, 3)):
        a = make(COUNTS[name], N, K, bits, seed=len(name) + N, T=T, k=k)
        y = call(c, bits, True, *a, k, out_dtype=DT[dtype])
        assert_gated(y, plain_values(*a, k, bits), DT[dtype])


# Experts of many rows: several units per block, remainders of every size,
# tiles cut by N, K that ends inside a stage (the fewest stages among them)
MANY_ROWS = {
    "remainders": [255, 257, 512, 0, 17, 1025, 16, 100], "one expert": [1500],
    "uneven": [0, 0, 3000, 1, 0, 259], "three hundred": [90 + (13 * e) % 60 for e in range(300)],
    "exact": [256, 512, 256, 768]}


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("name,N,K", [("remainders", 1288, 512), ("remainders", 528, 1120), ("one expert", 2320, 544),
                                      ("uneven", 272, 704), ("three hundred", 48, 512), ("exact", 1024, 640)])
def test_experts_of_many_rows(name, N, K, bits, dtype):
    c = cider()
    for T, k, gated in ((None, 1, False), (211, 2, True)):
        a = make(MANY_ROWS[name], N, K, bits, seed=N + K, T=T, k=k)
        v = plain_values(*a, k, bits)
        y = call(c, bits, gated, *a, k, out_dtype=DT[dtype])
        if gated:
            assert_gated(y, v, DT[dtype])
        else:
            assert torch.equal(y.cpu().view(torch.int16), v.to(DT[dtype]).view(torch.int16))


# Launches wide enough for the larger tiles (128 x 256, 256 x 192, 256 x 256
# rows by columns), remainders of several sizes, N that ends inside a tile and
# off the 16-byte store path, one to four stages of K
WIDE = [([1399, 0, 1601], 5000, 160), ([1399, 3, 1598], 5003, 400), ([250, 513, 0, 380, 400, 127, 900, 430], 2560, 288),
        ([2300, 200], 8008, 112), ([3000, 1000], 6000, 240), ([1200], 12301, 400), ([511, 2189, 16], 6160, 512)]


@pytest.mark.parametrize("bits,dtype", [(8, "bf16"), (8, "fp16"), (4, "fp16")])
@pytest.mark.parametrize("counts,N,K", WIDE)
def test_wide_launches(counts, N, K, bits, dtype):
    c = cider()
    K = -(-K // 32) * 32 if bits == 4 else K
    a = make(counts, N, K, bits, seed=N)
    y = call(c, bits, False, *a, 1, out_dtype=DT[dtype])
    v = plain_values(*a, 1, bits)
    assert torch.equal(y.cpu().view(torch.int16), v.to(DT[dtype]).view(torch.int16))
    if bits == 8 and dtype == "fp16":
        return
    a = make(counts, 2 * N, K, bits, seed=N + 1, T=500, k=2)
    assert_gated(call(c, bits, True, *a, 2, out_dtype=DT[dtype]), plain_values(*a, 2, bits), DT[dtype])


def test_swiglu_of_large_gates():
    """Gates far in both tails: silu is 0 on the left and the identity on the right."""
    c = cider()
    x = torch.full((4, 32), 127, dtype=torch.int8)
    w = torch.zeros(1, 32, 32, dtype=torch.int8)
    w[0, :8], w[0, 8:16], w[0, 16:] = 127, -127, 1
    sx = torch.tensor([1e-4, 1e-3, 1e-2, 1.0])
    sw = torch.full((1, 32), 1e-3)
    off = torch.tensor([0, 4], dtype=torch.int32)
    for t in (torch.float16, torch.bfloat16):
        y = c.cider_w8a8_grouped_swiglu(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), off.cuda(), out_dtype=t)
        v = plain_values(x, sx, w, sw, off, None, 1, 8)
        assert float(v.abs().max()) > 400.0
        assert_gated(y, v, t)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,K", [([3, 0, 9], 96), ([40, 70, 0], 96), ([200, 0, 310], 96), ([200, 0, 310], 640)])
def test_rows_behind_the_last_group_stay(counts, K, gated):
    c = cider()
    a = make(counts + [7], 64, K, 8, seed=5)
    x, sx, w, sw, off, _ = a
    off = off[:-1].contiguous()                                    # the last 7 rows belong to no expert
    w, sw = w[:-1].contiguous(), sw[:-1].contiguous()
    n = 32 if gated else 64
    y = torch.full((x.shape[0], n), 7.5, dtype=torch.float16, device="cuda")
    call(c, 8, gated, x, sx, w, sw, off, None, 1, y=y)
    torch.cuda.synchronize()
    assert bool((y[int(off[-1]):] == 7.5).all()) and not bool((y[:int(off[-1])] == 7.5).all())


def test_no_group_has_rows():
    c = cider()
    x, sx, w, sw, _, _ = make([4, 4], 32, 64, 8, seed=6)
    y = torch.full((8, 32), 7.5, dtype=torch.float16, device="cuda")
    c.cider_w8a8_grouped_gemm(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), torch.zeros(3, dtype=torch.int32).cuda(), y=y)
    torch.cuda.synchronize()
    assert bool((y == 7.5).all())


@pytest.mark.parametrize("counts,K", [([5, 9], 128), ([90, 100], 128), ([300, 290], 128), ([300, 290], 512)])
def test_sources_out_of_range_give_zeros(counts, K):
    c = cider()
    x, sx, w, sw, off, idx = make(counts, 48, K, 8, seed=7, T=20, k=2)
    idx[::3] = -1
    idx[1::5] = 40                                                   # // 2 = 20: past the last row
    idx[2::7] = 2 ** 31 - 1
    y = call(c, 8, False, x, sx, w, sw, off, idx, 2).cpu()
    bad = (idx < 0) | (idx >= 40)
    o = plain_values(x, sx, w, sw, off, torch.where(bad, 0, idx), 2, 8).to(torch.float16)
    o[bad] = 0.0
    assert torch.equal(y, o)


def test_same_rows_many_times_and_empty_x():
    c = cider()
    x, sx, w, sw, off, idx = make([30, 0, 41], 40, 64, 8, seed=8, T=1, k=1)
    y = call(c, 8, False, x, sx, w, sw, off, idx, 1)
    assert torch.equal(y.cpu(), plain_values(x, sx, w, sw, off, idx, 1, 8).to(torch.float16))
    none = torch.empty(0, 64, dtype=torch.int8), torch.empty(0)
    y = call(c, 8, False, *none, w, sw, off, idx, 1)
    assert not bool(y.any())


@pytest.mark.parametrize("n,K", [(64, 64), (300, 64), (300, 512)])
def test_offsets_out_of_order_stay_inside_the_buffers(n, K):
    """Clamped, whatever they hold; rows past P are never written."""
    c = cider()
    x, sx, w, sw, _, _ = make([n, n], 64, K, 8, seed=9)
    back = torch.full((2 * n + 2, 64), 3.0, dtype=torch.float16, device="cuda")
    for off in ([0, 5 * n, 2 * n], [-7, n, 10 ** 9], [2 ** 31 - 1, 0, -2 ** 31], [n + 10, 20, 2 * n]):
        c.cider_w8a8_grouped_gemm(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(),
                                  torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda(), y=back[:2 * n])
        torch.cuda.synchronize()
        assert bool((back[2 * n:] == 3.0).all())


def test_one_expert_is_the_dense_gemm():
    c = cider()
    x, sx, w, sw, off, _ = make([333], 640, 512, 8, seed=10)
    y = call(c, 8, False, x, sx, w, sw, off, None, 1)
    o = c.cider_w8a8_gemm(x.cuda(), sx.cuda(), w[0].cuda(), sw[0].cuda(), 0)
    assert torch.equal(y, o)


def test_weights_past_4_gib_of_offsets():
    """Experts behind 2^32 bytes of weights (9 experts of 512 MiB)."""
    c = cider()
    E, N, K = 9, 4096, 131072
    w = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    w[:, :, 0] = torch.arange(1, E + 1, dtype=torch.int8, device="cuda")[:, None]
    w[:, :, K - 1] = 1
    x = torch.zeros(E, K, dtype=torch.int8, device="cuda")
    x[:, 0], x[:, K - 1] = 2, 5
    one = torch.ones(E, N, device="cuda")
    y = c.cider_w8a8_grouped_gemm(x, torch.ones(E, device="cuda"), w, one,
                                  torch.arange(E + 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, (2.0 * torch.arange(1, E + 1, device="cuda") + 5)[:, None].expand(E, N).to(torch.float16))


@pytest.mark.parametrize("gated", [False, True])
def test_rows_past_4_gib_of_offsets(gated):
    """The last rows of 2.2 GB of codes and 4.6 GB of outputs are what they are alone."""
    c = cider()
    P, K, N = 1100000, 2048, 4200 if gated else 2100
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    x = torch.zeros(P, K, dtype=torch.int8, device="cuda")
    x[-700:] = codes(700, K)
    sx, w, sw = torch.full((P,), 0.01, device="cuda"), codes(2, N, K), torch.full((2, N), 1e-4, device="cuda")
    fn = c.cider_w8a8_grouped_swiglu if gated else c.cider_w8a8_grouped_gemm
    y = fn(x, sx, w, sw, torch.tensor([0, P - 300, P], dtype=torch.int32, device="cuda"), out_dtype=torch.bfloat16)
    o = fn(x[-700:].contiguous(), sx[:700], w, sw, torch.tensor([0, 400, 700], dtype=torch.int32, device="cuda"),
           out_dtype=torch.bfloat16)
    assert torch.equal(y[-700:], o) and not bool(y[:-700].any())


def test_grouped_refuses_other_tensors():
    c = cider()
    x, sx, w, sw, off, idx = (t if t is None else t.cuda() for t in make([3, 4], 32, 64, 8, seed=11, T=5))
    with pytest.raises(ValueError):
        c.cider_w8a8_grouped_gemm(x, sx, w, sw, off[:-1], row_index=idx)
    with pytest.raises(TypeError):
        c.cider_w8a8_grouped_gemm(x, sx, w, sw, off.long(), row_index=idx)
    with pytest.raises(ValueError):
        c.cider_w8a8_grouped_gemm(x, sx, w.transpose(1, 2), sw, off, row_index=idx)
    with pytest.raises(TypeError):
        c.cider_w8a8_grouped_gemm(x, sx, w, sw, off.cpu(), row_index=idx)
    with pytest.raises(ValueError):
        c.cider_w8a8_grouped_swiglu(x, sx, w[:, :31].contiguous(), sw[:, :31].contiguous(), off, row_index=idx)
    with pytest.raises(c.CiderError):
        c.cider_w8a8_grouped_gemm(x, sx, w, sw, off, row_index=idx, row_div=0)
    with pytest.raises(ValueError):
        c.cider_w8a8_grouped_gemm(x, sx, w, sw, off, row_index=idx, y=torch.empty(8, 32, dtype=torch.float16,
                                                                                  device="cuda"))


# ---- a run of them, as they are used ------------------------------------------

def moe_weights(E, I, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = cider()
    gu = (0.02 * torch.randn(E, 2 * I, H, generator=g, device="cuda")).to(torch.bfloat16)
    dn = (0.02 * torch.randn(E, H, I, generator=g, device="cuda")).to(torch.bfloat16)
    q = lambda w: tuple(t.view(w.shape[0], w.shape[1], *t.shape[1:]) for t in c.cider_quant_weight(w.flatten(0, 1), 8))  # noqa: E731
    return q(gu), q(dn)


def block(c, x, ids, weights, nw, gu, dn):
    """norm -> experts -> weighted sum into the residual -> next norm's codes."""
    _, x_q, x_s = c.cider_norm_quant(x, norm_weight=nw)
    rows, slots = c.w8a8_moe(x_q, x_s, ids, *gu, *dn, out_dtype=x.dtype)
    return c.cider_norm_quant(x, rows, nw, slots=slots, weights=weights)


def plain_block(x, ids, weights, nw, gu, dn, eps=1e-6):
    d = lambda q: q[0].double() * q[1].double()[..., None]        # noqa: E731
    gu, dn, x = d(gu), d(dn), x.double()
    norm = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * nw.double()   # noqa: E731
    quant = lambda v: (lambda s: torch.round(v / s) * s)(v.abs().amax(1, keepdim=True) / 127)   # noqa: E731
    n = quant(norm(x))
    out = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < gu.shape[0]:
                continue
            v = gu[e] @ n[t]
            g, u = v.chunk(2)
            a = (g * torch.sigmoid(g) * u).to(torch.bfloat16).double()
            out[t] += weights[t, j].double() * (dn[e] @ quant(a[None])[0])
    return x + out


@pytest.mark.parametrize("T", [1, 5, 70])
def test_expert_block(T):
    c = cider()
    E, I, H, k = 6, 96, 256, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    gu, dn = moe_weights(E, I, H, 20)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32)
    ids[T // 2, 1] = -1
    w = torch.rand(T, k, generator=g, device="cuda")
    nw = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    h, x_q, x_s = block(c, x, ids, w, nw, gu, dn)
    o = plain_block(x, ids, w, nw, gu, dn)
    # the block's part of h: codes one step off where a value lies on a border
    # (1/127 of a row's largest value, here at most 3 of them), plus bf16
    # roundings of a, of the expert rows and of h, each half a step
    part = (o - x.double()).norm(dim=1)
    off = (h.double() - o).norm(dim=1)
    assert bool((off <= 2 ** -8 * o.norm(dim=1) + 0.03 * part).all()), float((off / part).max())
    assert x_q.shape == (T, H) and x_s.shape == (T,)


def test_expert_block_captured_and_replayed():
    """One capture serves other routings of as many tokens; every replay is the eager result."""
    c = cider()
    E, I, H, k, T = 6, 96, 256, 3, 40
    gu, dn = moe_weights(E, I, H, 21)
    nw = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(c, x, ids, w, nw, gu, dn)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(c, x, ids, w, nw, gu, dn)
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        ids.copy_(torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32))
        w.copy_(torch.rand(T, k, generator=g, device="cuda"))
        if seed == 2:
            ids[:, 1] = -1
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        eager = block(c, x, ids, w, nw, gu, dn)
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a, b), seed


def test_grouped_on_another_stream():
    c = cider()
    x, sx, w, sw, off, idx = (t if t is None else t.cuda() for t in make([50, 0, 120], 256, 512, 8, seed=12, T=64, k=2))
    o = c.cider_w8a8_grouped_gemm(x, sx, w, sw, off, row_index=idx, row_div=2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = c.cider_w8a8_grouped_gemm(x, sx, w, sw, off, row_index=idx, row_div=2, stream=s)
    ids = torch.randint(0, 5, (3000, 4), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    plan = c.cider_moe_plan(ids, 5, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, o)
    for a, b in zip(plan, c.cider_moe_plan(ids, 5)):
        assert torch.equal(a, b)


def test_expert_block_of_no_tokens():
    c = cider()
    gu, dn = moe_weights(4, 32, 64, 22)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    h, x_q, x_s = block(c, x, ids, torch.empty(0, 2, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda"),
                        gu, dn)
    torch.cuda.synchronize()
    assert h.shape == x_q.shape == (0, 64) and x_s.shape == (0,)


@pytest.mark.parametrize("T", [1, 33])
def test_expert_rows_of_packed_weights(T):
    """w8a8_moe on packed int4 experts is its parts, one expert's rows after another on the dense entries."""
    c = cider()
    E, I, H, k = 5, 160, 224, 2
    rng = np.random.default_rng(T)
    x, sx, gu, sgu, _, _ = (t if t is None else t.cuda() for t in make([T] + [0] * (E - 1), 2 * I, H, 4, seed=30))
    _, _, dn, sdn, _, _ = (t if t is None else t.cuda() for t in make([1] + [0] * (E - 1), H, I, 4, seed=31))
    ids = torch.from_numpy(rng.permuted(np.tile(np.arange(E), (T, 1)), axis=1)[:, :k].astype(np.int32)).cuda()
    y, slots = c.w8a8_moe(x, sx, ids, gu, sgu, dn, sdn, out_dtype=torch.bfloat16)
    offsets, rows, slots2 = c.cider_moe_plan(ids, E)
    assert torch.equal(slots, slots2)
    a = c.cider_w4a8_grouped_swiglu(x, sx, gu, sgu, offsets, row_index=rows, row_div=k, out_dtype=torch.bfloat16)
    a_q, a_s = c.cider_quant_act(a, 0)
    off = offsets.tolist()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            part = [t[lo:hi].clone() for t in (a_q, a_s)]
            o = c.cider_w4a8_gemm(*part, dn[e].clone(), sdn[e].clone(), out_dtype=torch.bfloat16)
            assert torch.equal(y[lo:hi], o), e


def test_two_streams_at_once():
    """Blocks in flight together on two streams, each with its own outputs and workspaces: the results of either alone."""
    c = cider()
    E, I, H, k, T = 6, 96, 256, 3, 3500
    gu, dn = moe_weights(E, I, H, 23)
    nw = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    inputs, alone = [], []
    for seed in (0, 1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        ids = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32)
        inputs.append((x, ids, torch.rand(T, k, generator=g, device="cuda")))
        alone.append([t.clone() for t in block(c, *inputs[-1], nw, gu, dn)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(block(c, *inputs[i], nw, gu, dn))
    torch.cuda.synchronize()
    for i in (0, 1):
        for run in got[i]:
            for a, b in zip(run, alone[i]):
                assert torch.equal(a, b), i


def test_captured_plan_with_a_workspace():
    """Two captured plans of more ids than one launch takes, replayed by turns for new ids."""
    c = cider()
    T, k, E = 4000, 4, 50
    need = c.cider_moe_plan_workspace_size(T, k, E)
    assert need > 0
    both = []
    for _ in range(2):
        ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        c.cider_moe_plan(ids, E, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = c.cider_moe_plan(ids, E, workspace=ws)
        both.append((ids, graph, out))
    rng = np.random.default_rng(40)
    for _ in range(3):
        new = [rng.integers(-1, E, (T, k)).astype(np.int32) for _ in both]
        for (ids, graph, _), n in zip(both, new):
            ids.copy_(torch.from_numpy(n))
            graph.replay()
        torch.cuda.synchronize()
        for (_, _, out), n in zip(both, new):
            for a, o in zip(out, plain_plan(n, E)):
                assert np.array_equal(a.cpu().numpy(), o)


def test_repeats_are_bit_identical():
    c = cider()
    E, I, H, k, T = 6, 96, 256, 3, 900
    gu, dn = moe_weights(E, I, H, 24)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    nw = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    first = block(c, x, ids, w, nw, gu, dn)
    for _ in range(20):
        for a, b in zip(first, block(c, x, ids, w, nw, gu, dn)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n", [2, 70])
def test_packed_sums_of_the_largest_codes(n):
    """The longest K of packed weights with every code at its end (-128 and 127 times nibbles 0 and 15): exact, as the
    dense entry's."""
    c = cider()
    K, N = 131040, 48
    x = torch.full((n, K), -128, dtype=torch.int8, device="cuda")
    x[1::2] = 127
    w = torch.zeros(1, N, K // 2, dtype=torch.uint8, device="cuda")
    w[:, 1::2] = 255
    sx, sw = torch.full((n,), 2.0 ** -12, device="cuda"), torch.ones(1, N, device="cuda")
    y = c.cider_w4a8_grouped_gemm(x, sx, w, sw, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    v = (x[:, :1].double() * torch.tensor([-8.0, 7.0], device="cuda").repeat(N // 2) * K).to(torch.float32)
    assert torch.equal(y, (v * 2.0 ** -12).to(torch.float16))
    assert torch.equal(y, c.cider_w4a8_gemm(x, sx, w[0], sw[0]))
    with pytest.raises(c.CiderError):
        c.cider_w4a8_grouped_gemm(torch.cat((x, x[:, :32]), 1), sx, torch.cat((w, w[..., :16]), 2), sw,
                                  torch.tensor([0, n], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("P,E,share", [(800001, 40, 2048), (1100001, 299, 4096), (2500003, 7, 8192), (2300001, 512, 8192),
                                       (9001, 1, 0)])
def test_plan_of_grown_chunks(P, E, share):
    """More ids than the largest grid has usual chunks for: blocks take more than `share` ids each (asserted by the
    workspace, so that another choice of chunks cannot pass this by). Beyond 8192 a wave walks its ids in several
    rounds, the last of them partial."""
    c = cider()
    blocks = c.cider_moe_plan_workspace_size(P, 1, E) // (4 * E)
    assert blocks > 1 and blocks * share < P
    rng = np.random.default_rng(P)
    ids = rng.integers(-1, E + 1, (P, 1)).astype(np.int32)
    check_plan(c, ids, E)
    ids[:] = np.sort(ids, 0)                                       # whole chunks of one expert, all dropped ids at the ends
    check_plan(c, ids, E)


# Launches of the larger tiles again, in every type: by the rule of tiles the plain
# products take 128 x 256, 128 x 256, 256 x 192 and 256 x 256 (rows by columns), the
# gated ones 256 x 192, 256 x 256, 256 x 256 and 128 x 256.
LARGE = [([1399, 3, 1598], 5003, 160), ([1300, 1200], 2500, 96), ([2300, 200], 8008, 128), ([2000, 0, 2000], 6000, 288)]


def gated_off(y, v, dtype):
    """How far gated rows are outside assert_gated's bound, on the GPU."""
    n = v.shape[1] // 2
    g, u = v[:, :n].double(), v[:, n:].double()
    o = g * torch.sigmoid(g) * u
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    bound = o.abs() * (half + (8 + g.abs()) * 2.0 ** -23 * (1 + half)) + tiny + u.abs() * 2.0 ** -118
    return float(((y.double() - o).abs() - bound).max())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,N,K", LARGE)
def test_large_tiles(counts, N, K, gated, bits, dtype):
    """In place and gathered, with sources out of range, and rows behind the last group left as they were."""
    c, t = cider(), DT[dtype]
    n = 2 * N if gated else N
    for T in (None, 500):
        x, sx, w, sw, off, idx = (v if v is None else v.cuda() for v in make(counts, n, K, bits, seed=N, T=T, k=2))
        P = int(off[-1])
        bad = torch.zeros(P, dtype=torch.bool, device="cuda")
        if idx is None:
            x, sx = torch.cat((x, x[:7])), torch.cat((sx, sx[:7]))
        else:
            idx[::3], idx[1::5], idx[2::7] = -1, 1000, 2 ** 31 - 1   # 1000 // 2: past the last row
            bad = (idx < 0) | (idx >= 1000)
            idx = torch.cat((idx, idx[:7]))
        y = torch.full((P + 7, N), 7.5, dtype=t, device="cuda")
        call(c, bits, gated, x, sx, w, sw, off, idx, 2, y=y)
        v = plain_values(x, sx, w, sw, off.cpu(), None if idx is None else torch.where(bad, 0, idx[:P]), 2, bits)
        v[bad] = 0.0
        assert bool((y[P:] == 7.5).all()) and not bool(y[:P][bad].any())
        if gated:
            assert gated_off(y[:P], v, t) <= 0, T
        else:
            assert torch.equal(y[:P].view(torch.int16), v.to(t).view(torch.int16)), T


@pytest.mark.parametrize("gated", [False, True])
def test_large_tiles_of_offsets_out_of_order(gated):
    """Clamped, whatever they hold; rows past P are never written."""
    c = cider()
    n, N, K = 2000, 6000, 96
    x, sx, w, sw, _, _ = (v if v is None else v.cuda() for v in make([n, n], 2 * N if gated else N, K, 8, seed=9))
    back = torch.full((2 * n + 2, N), 3.0, dtype=torch.float16, device="cuda")
    fn = c.cider_w8a8_grouped_swiglu if gated else c.cider_w8a8_grouped_gemm
    for off in ([0, 5 * n, 2 * n], [-7, n, 10 ** 9], [2 ** 31 - 1, 0, -2 ** 31], [n + 10, 20, 2 * n], [0, 0, 0]):
        fn(x, sx, w, sw, torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda(), y=back[:2 * n])
        torch.cuda.synchronize()
        assert bool((back[2 * n:] == 3.0).all())


def test_plan_refuses_other_workspaces():
    c = cider()
    ids = torch.zeros(3000, 4, dtype=torch.int32, device="cuda")
    need = c.cider_moe_plan_workspace_size(3000, 4, 9)
    with pytest.raises(TypeError):
        c.cider_moe_plan(ids, 9, workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(ValueError):
        c.cider_moe_plan(ids, 9, workspace=torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(c.CiderError):
        c.cider_moe_plan(ids, 9, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    wide = torch.empty(need // 4, dtype=torch.int32, device="cuda")  # any element type
    assert int(c.cider_moe_plan(ids, 9, workspace=wide)[0][1]) == 12000


def test_sizes_past_32_bits_are_refused():
    c = cider()
    with pytest.raises(ValueError):
        c.cider_moe_plan(torch.zeros(4, 1, dtype=torch.int32, device="cuda"), (1 << 32) + 8)
    x, sx, w, sw, off, idx = (v.cuda() for v in make([3, 4], 32, 64, 8, seed=11, T=5))
    for div in (1 << 31, (1 << 32) + 1, 1 - (1 << 32), -1):
        with pytest.raises((ValueError, c.CiderError)):
            c.cider_w8a8_grouped_gemm(x, sx, w, sw, off, row_index=idx, row_div=div)
    y = c.cider_w8a8_grouped_gemm(x, sx, w, sw, off, row_index=idx, row_div=(1 << 31) - 1)   # all of them row 0
    o = c.cider_w8a8_grouped_gemm(x, sx, w, sw, off, row_index=torch.zeros_like(idx))
    assert torch.equal(y, o)


def test_captured_blocks_that_make_their_own_workspace():
    """Two captured blocks of more ids than one launch takes, replayed by turns between eager calls."""
    c = cider()
    E, I, H, k, T = 6, 64, 128, 3, 3100
    gu, dn = moe_weights(E, I, H, 25)
    nw = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    assert c.cider_moe_plan_workspace_size(T, k, E) > 0
    both = []
    for _ in range(2):
        x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
        block(c, x, ids, w, nw, gu, dn)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block(c, x, ids, w, nw, gu, dn)
        both.append((x, ids, w, graph, out))
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for x, ids, w, graph, _ in both:
            x.copy_(torch.randn(T, H, generator=g, device="cuda"))
            ids.copy_(torch.randint(-1, E + 1, (T, k), generator=g, device="cuda"))
            w.copy_(torch.rand(T, k, generator=g, device="cuda"))
            graph.replay()
        eager = [block(c, x, ids, w, nw, gu, dn) for x, ids, w, _, _ in both]
        torch.cuda.synchronize()
        for (_, _, _, _, out), o in zip(both, eager):
            for a, b in zip(out, o):
                assert torch.equal(a, b), seed


def test_nan_in_what_nothing_reads():
    """Rows, scales and experts that no group names, and the weights of dropped slots, may hold NaN."""
    c = cider()
    x, sx, w, sw, off, idx = (v.cuda() for v in make([5, 0, 9], 48, 64, 8, seed=13, T=20, k=1))
    idx = idx.remainder(10)                                          # rows 10 .. 19 are read by no one
    y = c.cider_w8a8_grouped_gemm(x, sx, w, sw, off, row_index=idx)
    sx2, sw2 = sx.clone(), sw.clone()
    sx2[10:], sw2[1] = float("nan"), float("nan")
    rows = torch.cat((c.cider_w8a8_grouped_gemm(x, sx2, w, sw2, off, row_index=idx), torch.full_like(y[:4], float("nan"))))
    assert torch.equal(rows[:14], y)
    slots = torch.tensor([[0, -1, 13], [-5, 18, 99], [7, 7, -1]], dtype=torch.int32, device="cuda")
    wt = torch.rand(3, 3, device="cuda")
    there = (slots >= 0) & (slots < 18)
    a = c.cider_norm_quant(None, rows, slots=slots, weights=torch.where(there, wt, float("nan")))[0]
    b = c.cider_norm_quant(None, rows, slots=slots, weights=torch.where(there, wt, 0.0))[0]
    assert torch.equal(a, b) and bool(a.isfinite().all()) and not bool(a[1].any())
