"""The boundary between two blocks (cider_norm_quant) and the way back from
codes (cider_dequant_act) against plain forms in 64 bits."""
import numpy as np
import pytest

from tests.test_gpu_parity import cider

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24   # half a step of fp32


def rms_error(K):
    """Relative error of a row's 1 / sqrt(mean of squares + eps) in fp32: the
    sum of positive terms in a tree of K / 256 sequential adds, 6 levels of a
    wave and 3 of the workgroup (each fma rounds once: one more), halved by the
    root; then the division by K, + eps, the root and the division."""
    return ((K / 256 + 8) + 6 + 4) / 2 * U + 4 * U


def reference(x, block, slots, weights, post, gate, rows_per_gate, alpha, eps):
    """h before its rounding, in 64 bits, and the bound of the fp32 steps."""
    d = lambda t: t.double()   # noqa: E731
    M, K = (x if x is not None else slots if slots is not None else block).shape[0], block.shape[1]
    if slots is not None:
        k = slots.shape[1]
        ok = (slots >= 0) & (slots < block.shape[0])
        rows = d(block)[torch.where(ok, slots, 0).long()] * (d(weights) * ok)[..., None]
        p, err = rows.sum(1), k * U * rows.abs().sum(1)
    else:
        p, err = d(block), torch.zeros(M, K, dtype=torch.float64, device=block.device)
    if post is not None:
        r = 1.0 / torch.sqrt((p * p).mean(1, keepdim=True) + eps)
        # an error of p changes the mean square by twice its relative size at
        # most, so the root by once
        rel = rms_error(K) + err.norm(dim=1, keepdim=True) / p.norm(dim=1, keepdim=True).clamp(min=1e-300)
        err = (err + p.abs() * (rel + 2 * U)) * r * d(post).abs() * 1.001
        p = p * r * d(post)
    if gate is not None:
        g = d(gate).reshape(-1, K)[(torch.arange(M, device=block.device) // rows_per_gate) if rows_per_gate else
                                   torch.zeros(M, dtype=torch.long, device=block.device)]
        err = err * g.abs() + (g * p).abs() * U
        p = g * p
    h = alpha * p + (d(x) if x is not None else 0.0)
    return h, abs(alpha) * err + h.abs() * U


def check_norm(h, nw, eps, gs, x_q, x_s, normed=None):
    """Codes, scales and normed rows against the stored h, as n is defined."""
    M, K = h.shape
    h, w = h.double(), nw.double()
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w
    rel = rms_error(K) + 2 * U                                       # and the two products
    g = gs or K
    nn = n.view(M, K // g, g)
    s = nn.abs().amax(2) / 127
    got_s = x_s.double().view(M, K // g)
    assert bool(((got_s - s).abs() <= s * (rel + 2 * U) + 2.0 ** -149).all())
    # code = rint(fl(n~ / s~)): half a unit, plus 127 times the relative errors
    # of n~, s~ and the quotient
    quotient = torch.where(s[..., None] > 0, nn / s[..., None], torch.zeros_like(nn))
    off = (x_q.double().view(M, K // g, g) - quotient).abs()
    assert float(off.max()) <= 0.5 + 127 * (2 * rel + 4 * U)
    assert int(x_q.abs().max()) <= 127
    if normed is not None:
        half = torch.finfo(normed.dtype).eps / 2
        tiny = torch.finfo(normed.dtype).tiny * torch.finfo(normed.dtype).eps / 2
        assert bool(((normed.double() - n).abs() <= n.abs() * (half + rel * 1.01) + tiny).all())


def rnd(g, *shape, t, scale=1.0, mean=0.0):
    return (mean + scale * torch.randn(*shape, generator=g, device="cuda")).to(t)


SIZES = [(1, 1), (3, 5), (2, 8), (5, 64), (4, 130), (7, 512), (5, 520), (9, 1024), (3, 1032), (1, 2048), (6, 2056),
         (2, 4096), (3, 5120), (2, 8192), (2, 8200), (3, 8195), (1, 20480), (300, 384)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_residual_norm_and_codes(M, K, dtype):
    c, t = cider(), DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(M * 7 + K)
    x, block = rnd(g, M, K, t=t, scale=3.0), rnd(g, M, K, t=t)
    nw, post = rnd(g, K, t=t, scale=0.1, mean=1.0), rnd(g, K, t=t, scale=0.1, mean=1.0)
    gate1, gates = rnd(g, K, t=t), rnd(g, -(-M // 2), K, t=t)
    for gs in (0, 64, 128):
        if gs and K % gs:
            continue
        for kw in (dict(), dict(post_weight=post), dict(gate=gate1, alpha=0.25),
                   dict(post_weight=post, gate=gates, rows_per_gate=2, alpha=-1.5)):
            normed = torch.empty_like(x)
            h, x_q, x_s = c.cider_norm_quant(x, block, nw, group_size=gs, eps=1e-5, normed=normed, **kw)
            o, err = reference(x, block, None, None, kw.get("post_weight"), kw.get("gate"),
                               kw.get("rows_per_gate", 0), kw.get("alpha", 1.0), 1e-5)
            half = torch.finfo(t).eps / 2
            tiny = torch.finfo(t).tiny * torch.finfo(t).eps / 2
            assert bool(((h.double() - o).abs() <= o.abs() * half + err * (1 + half) + tiny).all()), (gs, list(kw))
            check_norm(h, nw, 1e-5, gs, x_q, x_s, normed)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,k", [(1, 2048, 8), (5, 64, 1), (6, 1000, 3), (9, 77, 2), (4, 512, 64), (3, 4096, 5),
                                   (2, 8192, 8), (2, 9000, 2), (70, 640, 6)])
def test_weighted_sum_of_expert_rows(M, K, k, dtype):
    c, t = cider(), DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(M + K)
    R = M * k + 3
    x, block = rnd(g, M, K, t=t), rnd(g, R, K, t=t)
    nw, post = rnd(g, K, t=t, scale=0.1, mean=1.0), rnd(g, K, t=t, scale=0.1, mean=1.0)
    w = torch.rand(M, k, generator=g, device="cuda")
    slots = torch.randint(0, R, (M, k), generator=g, device="cuda", dtype=torch.int32)
    slots[0, 0] = -1                                                   # dropped, and out of range
    slots[-1, -1] = R
    if M > 2:
        slots[1] = -1                                                  # a row without any expert
    for kw in (dict(), dict(post_weight=post, alpha=0.5)):
        h, x_q, x_s = c.cider_norm_quant(x, block, nw, slots=slots, weights=w, **kw)
        o, err = reference(x, block, slots, w, kw.get("post_weight"), None, 0, kw.get("alpha", 1.0), 1e-6)
        half = torch.finfo(t).eps / 2
        tiny = torch.finfo(t).tiny * torch.finfo(t).eps / 2
        assert bool(((h.double() - o).abs() <= o.abs() * half + err * (1 + half) + tiny).all()), list(kw)
        check_norm(h, nw, 1e-6, 0, x_q, x_s)
        if M > 2:
            assert torch.equal(h[1], x[1])
    # the sum alone: no residual, no norm
    h, x_q, x_s = c.cider_norm_quant(None, block, slots=slots, weights=w)
    o, err = reference(None, block, slots, w, None, None, 0, 1.0, 1e-6)
    assert x_q is None and x_s is None
    assert bool(((h.double() - o).abs() <= o.abs() * half + err * (1 + half) + tiny).all())


# more rows than are resident at once, where rows of some sizes share a workgroup
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(1025, 1024), (1027, 520), (1026, 2560), (1027, 2056), (1025, 512), (1030, 4096)])
def test_many_rows(M, K, dtype):
    test_residual_norm_and_codes(M, K, dtype)
    test_weighted_sum_of_expert_rows(M, K, 3, dtype)


@pytest.mark.parametrize("K", [96, 2048, 4000, 9000, 33])
def test_norm_alone_and_in_place(K):
    c, t = cider(), torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(K)
    x, block, nw = rnd(g, 11, K, t=t), rnd(g, 11, K, t=t), rnd(g, K, t=t, mean=1.0, scale=0.2)
    h, x_q, x_s = c.cider_norm_quant(x, norm_weight=nw)
    assert h is x
    check_norm(x, nw, 1e-6, 0, x_q, x_s)
    copy = torch.empty_like(x)
    h2, q2, s2 = c.cider_norm_quant(x, norm_weight=nw, h=copy)
    assert torch.equal(copy, x) and torch.equal(q2, x_q) and torch.equal(s2, x_s)
    o = c.cider_norm_quant(x, block, nw)
    mine = x.clone()
    got = c.cider_norm_quant(mine, block, nw, h=mine)
    assert got[0] is mine
    for a, b in zip(got, o):
        assert torch.equal(a, b)


@pytest.mark.parametrize("K", [64, 100, 512, 2048, 8192, 9216])
@pytest.mark.parametrize("gs", [0, 64])
def test_rows_and_groups_of_zeros(K, gs):
    c = cider()
    if gs and K % gs:
        pytest.skip("groups divide K")
    for t in (torch.float16, torch.bfloat16):
        x = torch.zeros(3, K, dtype=t, device="cuda")
        x[1, :] = 1.0
        x[1, :64 if gs else 1] = 0.0
        h, q, s = c.cider_norm_quant(x, x.clone(), torch.ones(K, dtype=t, device="cuda"), group_size=gs,
                                     post_weight=torch.ones(K, dtype=t, device="cuda"))
        assert not bool(q[0].any()) and not bool(s[0].any()) and not bool(h[0].any())
        check_norm(h, torch.ones(K, dtype=t, device="cuda"), 1e-6, gs, q, s)
        assert not bool(q[1, :64 if gs else 1].any())


@pytest.mark.parametrize("t,big,small", [(torch.float16, 60000.0, 2.0 ** -24), (torch.bfloat16, 1e17, 1e-36)])
def test_largest_and_smallest_values(t, big, small):
    """No overflow of the fp32 squares, and subnormal rows quantize by the rule."""
    c = cider()
    g = torch.Generator(device="cuda").manual_seed(1)
    sign = torch.sign(torch.randn(4, 1024, generator=g, device="cuda"))
    for v in (big, small):
        x = (sign * v * (0.5 + 0.5 * torch.rand(4, 1024, generator=g, device="cuda"))).to(t)
        nw = torch.ones(1024, dtype=t, device="cuda")
        _, q, s = c.cider_norm_quant(x, norm_weight=nw)
        check_norm(x, nw, 1e-6, 0, q, s)


def test_codes_follow_the_quantizer_on_representable_norms():
    """Where n is exact in the 16-bit type (constant rows, eps lost), the codes
    and scales are cider_quant_act's on the normed row."""
    c = cider()
    x = torch.full((4, 1024), 2.0, dtype=torch.float16, device="cuda")
    w = torch.linspace(-2, 2, 1025, device="cuda")[:1024].to(torch.float16)
    for gs in (0, 64, 128):
        _, q, s = c.cider_norm_quant(x, norm_weight=w, eps=1e-30, group_size=gs)
        q2, s2 = c.cider_quant_act(w.expand(4, 1024).contiguous(), gs)
        assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,gs", [(1, 1, 0), (3, 33, 0), (2, 16, 0), (17, 48, 0), (5, 1000, 0), (4, 192, 64),
                                    (9, 384, 128), (200, 2560, 0), (64, 2560, 128), (1, 133120, 0)])
def test_dequant(M, K, gs, dtype):
    c, t = cider(), DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(K)
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(M, K // gs if gs else 1, generator=g, device="cuda") * 0.1
    y = c.cider_dequant_act(q, s if gs else s[:, 0].contiguous(), gs, out_dtype=t)
    o = (q.float() * s.repeat_interleave(gs or K, 1)).to(t)           # one fp32 product, one rounding
    assert torch.equal(y.view(torch.int16), o.view(torch.int16))


def test_dequant_inverts_the_quantizer():
    c = cider()
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(50, 640, generator=g, device="cuda").to(torch.float16)
    for gs in (0, 64, 128):
        q, s = c.cider_quant_act(x, gs)
        y = c.cider_dequant_act(q, s, gs)
        step = s.view(50, -1).repeat_interleave(gs or 640, 1).double()
        # half a code, the quotient's and the scale's fp32 roundings on at most
        # 127 codes, and half a step of fp16
        bound = step * (0.5 + 127 * 2 * U) + y.double().abs() * 2.0 ** -11 + 2.0 ** -25
        assert bool(((y.double() - x.double()).abs() <= bound).all())


def test_norm_refuses_other_tensors():
    c = cider()
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    nw = torch.ones(64, dtype=torch.float16, device="cuda")
    slots = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for kw in (dict(norm_weight=nw.bfloat16()), dict(norm_weight=nw, block=x.bfloat16()), dict(norm_weight=nw.cpu())):
        with pytest.raises(TypeError):
            c.cider_norm_quant(x, **kw)
    for kw in (dict(norm_weight=nw[:32]), dict(norm_weight=nw, block=x[:3]), dict(norm_weight=nw, slots=slots),
               dict(norm_weight=nw, group_size=48), dict(norm_weight=nw, block=x, weights=torch.zeros(4, 2).cuda()),
               dict(block=x, gate=torch.zeros(3, 64, dtype=torch.float16, device="cuda"), rows_per_gate=2),
               dict(norm_weight=nw, block=x.t().contiguous().t()), dict(block=x, x_q=x.to(torch.int8))):
        with pytest.raises(ValueError):
            c.cider_norm_quant(x, **kw)
    with pytest.raises(ValueError):
        c.cider_norm_quant()
    with pytest.raises(c.CiderError):
        c.cider_norm_quant(x, norm_weight=nw, eps=0.0)
    with pytest.raises(c.CiderError):
        c.cider_norm_quant(x, x, nw, slots=torch.zeros(4, 65, dtype=torch.int32, device="cuda"),
                           weights=torch.zeros(4, 65, device="cuda"))
    assert np.prod(c.cider_norm_quant(x[:0], norm_weight=nw)[1].shape) == 0


@pytest.mark.parametrize("M,K", [(600000, 4096), (150000, 16392), (600000, 4097)])
def test_rows_past_32_bits_of_offsets(M, K):
    """The last rows of more than 2^31 elements are what they are alone."""
    c, t = cider(), torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.zeros(M, K, dtype=t, device="cuda")
    nw = rnd(g, K, t=t, mean=1.0, scale=0.2)
    x[-5:] = rnd(g, 5, K, t=t)
    tail = x[-5:].clone()
    h, q, s = c.cider_norm_quant(x, x, nw, h=x)                      # in place: 2 x
    y = c.cider_dequant_act(q, s, out_dtype=t)
    h1, q1, s1 = c.cider_norm_quant(tail, tail, nw)
    assert torch.equal(h[-5:], h1) and torch.equal(q[-5:], q1) and torch.equal(s[-5:], s1)
    assert torch.equal(y[-5:], c.cider_dequant_act(q1, s1, out_dtype=t))
    assert not bool(q[:7].any()) and not bool(s[:-5].any())
    # expert rows from the same depth
    slots = torch.tensor([[M - 1, M - 3], [M - 2, 0]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[4, 2], [3, 5]], dtype=torch.int32, device="cuda")   # row 5: none, as row 0 of x is zeros
    w = torch.rand(2, 2, generator=g, device="cuda")
    a = c.cider_norm_quant(None, h, nw, slots=slots, weights=w)
    b = c.cider_norm_quant(None, h1, nw, slots=near, weights=w)
    for i, j in zip(a, b):
        assert torch.equal(i, j)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(9, 512), (9, 2048), (9, 2112), (9, 8192), (9, 9088), (9, 77), (1030, 1024), (1031, 2560)])
def test_rows_that_overflow_do_not_vanish(M, K, dtype):
    """A residual that is not finite, or whose squares overflow fp32, gives NaN scales and normed rows in every form;
    the rows beside it are what they are without it."""
    c, t = cider(), DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(K)
    x, block, nw = rnd(g, M, K, t=t), rnd(g, M, K, t=t), rnd(g, K, t=t, mean=1.0, scale=0.2)
    bad = {1: float("nan"), 3: float("inf"), 4: float("-inf"), M - 2: 60000.0 if dtype == "fp16" else 3e30}
    wild, wild_block = x.clone(), block.clone()
    for row, v in bad.items():
        wild[row, K // 3] = v
    wild_block[M - 2, K // 3] = bad[M - 2]                             # 120000 in fp16; 3.6e61 squared in bf16
    hit = torch.zeros(M, dtype=torch.bool, device="cuda")
    hit[list(bad)] = True
    for gs in (0, 64, 128):
        if gs and K % gs:
            continue
        n0, n1 = torch.empty_like(x), torch.empty_like(x)
        a = c.cider_norm_quant(x, block, nw, group_size=gs, normed=n0)
        b = c.cider_norm_quant(wild, wild_block, nw, group_size=gs, normed=n1)
        assert bool(b[2][hit].isnan().all()) and bool(n1[hit].isnan().all()) and not bool(b[1][hit].any()), gs
        assert bool(c.cider_dequant_act(b[1], b[2], gs)[hit].isnan().all())
        for i, j in zip((*a, n0), (*b, n1)):
            assert torch.equal(i[~hit], j[~hit]), gs
        # in the block alone, before its own norm: the residual's row is NaN
        h, q, s = c.cider_norm_quant(x, wild if dtype == "bf16" else torch.where(hit[:, None], wild * 2, wild), nw,
                                     post_weight=nw, group_size=gs)
        assert bool(h[hit].isnan().all()) and bool(s[hit].isnan().all()) and not bool(q[hit].any())
        assert bool(h[~hit].isfinite().all()) and bool(s[~hit].isfinite().all())
        # a weight that is NaN reaches the scales it enters
        lost = nw.clone()
        lost[K - 1] = float("nan")
        _, _, s = c.cider_norm_quant(x, block, lost, group_size=gs)
        assert bool((s.view(M, -1)[:, -1]).isnan().all()) and bool((s.view(M, -1)[:, :-1]).isfinite().all())


@pytest.mark.parametrize("M,K", [(0, 64), (1, 64), (3, 77), (2, 9000)])
def test_no_expert_rows_at_all(M, K):
    """A rank whose experts got no token: an empty block adds nothing to any row."""
    c, t = cider(), torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(K)
    x, nw = rnd(g, M, K, t=t), rnd(g, K, t=t, mean=1.0, scale=0.2)
    block = torch.empty(0, K, dtype=t, device="cuda")
    slots, w = torch.full((M, 2), -1, dtype=torch.int32, device="cuda"), torch.ones(M, 2, device="cuda")
    for kw in (dict(), dict(post_weight=nw)):
        h, q, s = c.cider_norm_quant(x, block, nw, slots=slots, weights=w, **kw)
        assert torch.equal(h, x)
        for a, b in zip((q, s), c.cider_norm_quant(x, norm_weight=nw)[1:]):
            assert torch.equal(a, b)
    h, _, _ = c.cider_norm_quant(None, block, slots=slots, weights=w)
    assert h.shape == (M, K) and not bool(h.any())
