"""The operators between the q/k/v projections and the output projection of a
quantized decoder, as workloads: rotary positions, writing keys and values
into a paged cache held in 4 bits, and attention over that cache.

Each case can run in its plain form (elementary torch operations in 32 bits,
angles in 64) or, with `own` set, through libcider's entry points. Sizes are
generic or those of this repository's own configurations (16 query heads and
8 key/value heads of 128).

Operators, by a case's "op":

* rope: x [T, H, D] (a view into the fused projections' rows where "fused")
  rotated by its tokens' positions, half or interleaved pairs, the first "rd"
  dimensions of each head, frequencies scaled for long contexts where "factor".
* append: per-head norms of q and k, their rotation, and k and v quantized to
  4 bits into their slots of the cache; the stored values are read back.
* attend: softmax(scale * q k^T) v over each sequence's pages: "n" queries at
  the end of up to "L" tokens (both ragged over the batch where "ragged"),
  causal, within a window where "window".

The cache: codes c in -7 .. 7 as nibbles c + 8, two per byte, low nibble first,
k_codes and v_codes uint8 [pages, Hkv, page, D / 2], scales fp32
[pages, Hkv, G, page] for G = D / group groups. A head's dimensions lie in
order in k_codes; in v_codes as [16][G][D / 16 / G], so that each sixteenth of
a row holds as many of every group.
"""
import math

import torch

own = False


def listed():
    return [
        # one decode step of 16 requests
        {"name": "rope decode", "op": "rope", "T": 16, "H": 16, "D": 128, "rd": 128, "interleaved": False, "factor": 1.0,
         "far": 8192, "fused": False, "dtype": "bf16"},
        # q and k of a long prompt, in the projections' rows; half of each head, positions past the trained length
        {"name": "rope prompt", "op": "rope", "T": 16384, "H": 24, "D": 128, "rd": 64, "interleaved": True, "factor": 8.0,
         "far": 1000000, "fused": True, "dtype": "fp16"},
        # one decode step of 32 requests: the launch
        {"name": "append decode", "op": "append", "T": 32, "Hq": 16, "Hkv": 8, "D": 128, "rd": 128, "interleaved": False,
         "factor": 1.0, "far": 32768, "group": 0, "page": 16, "norm": True, "dtype": "bf16"},
        # small heads, odd counts, padded tokens that have no slot
        {"name": "append odd", "op": "append", "T": 1003, "Hq": 9, "Hkv": 3, "D": 64, "rd": 32, "interleaved": True,
         "factor": 4.0, "far": 100000, "group": 32, "page": 32, "norm": False, "dtype": "fp16"},
        # a long prompt
        {"name": "append prompt", "op": "append", "T": 16384, "Hq": 16, "Hkv": 8, "D": 128, "rd": 128,
         "interleaved": False, "factor": 1.0, "far": 16384, "group": 64, "page": 64, "norm": True, "dtype": "bf16"},
        # one request's next token: latency
        {"name": "attend one token", "op": "attend", "B": 1, "n": 1, "L": 2000, "Hq": 16, "Hkv": 8, "D": 128, "group": 0,
         "page": 16, "window": 0, "ragged": 0.0, "dtype": "fp16"},
        # a served batch of requests of all lengths
        {"name": "attend batch", "op": "attend", "B": 64, "n": 1, "L": 8192, "Hq": 16, "Hkv": 8, "D": 128, "group": 64,
         "page": 64, "window": 0, "ragged": 0.9, "dtype": "bf16"},
        # two very long contexts
        {"name": "attend long", "op": "attend", "B": 2, "n": 1, "L": 131072, "Hq": 32, "Hkv": 8, "D": 128, "group": 0,
         "page": 128, "window": 0, "ragged": 0.3, "dtype": "fp16"},
        # a few drafted tokens of each request, large heads, small groups, a window
        {"name": "attend drafts", "op": "attend", "B": 24, "n": 5, "L": 5000, "Hq": 8, "Hkv": 2, "D": 256, "group": 64,
         "page": 32, "window": 3000, "ragged": 0.5, "dtype": "bf16"},
        # the next part of a long prompt
        {"name": "attend chunk", "op": "attend", "B": 1, "n": 512, "L": 32768, "Hq": 16, "Hkv": 8, "D": 128, "group": 0,
         "page": 64, "window": 0, "ragged": 0.0, "dtype": "bf16"},
        # several prompts of small heads and groups at once
        {"name": "attend prompts", "op": "attend", "B": 5, "n": 1501, "L": 1777, "Hq": 12, "Hkv": 4, "D": 64, "group": 32,
         "page": 16, "window": 0, "ragged": 0.6, "dtype": "fp16"},
        # one long prompt: the matrix cores
        {"name": "attend prompt", "op": "attend", "B": 1, "n": 8192, "L": 8192, "Hq": 16, "Hkv": 8, "D": 128, "group": 0,
         "page": 128, "window": 0, "ragged": 0.0, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    D = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["fp16", "bf16"])
    rotary = {"rd": rng.choice([D, D, D // 2, D // 4]), "interleaved": rng.random() < 0.4,
              "factor": rng.choice([1.0, 1.0, 4.0, 16.0]), "far": _log_int(rng, 1000, 1000000)}
    if op == "rope":
        D = rng.choice([64, 96, 128, 256])
        H = _log_int(rng, 1, 40)
        T = min(_log_int(rng, 1, 16384), (48 << 20) // (H * D))
        return {"op": op, "T": T, "H": H, "D": D, **rotary, "rd": min(D, rotary["rd"]), "fused": rng.random() < 0.5,
                "dtype": dtype}
    Hkv = _log_int(rng, 1, 10)
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([0, 32, 64]) if D < 256 else rng.choice([0, 64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        T = min(_log_int(rng, 1, 16384), (64 << 20) // ((Hq + 2 * Hkv) * D))
        return {"op": op, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, **rotary, "group": group, "page": page,
                "norm": rng.random() < 0.5, "dtype": dtype}
    while True:
        B, L = _log_int(rng, 1, 64), _log_int(rng, 1, 131072)
        n = 1 if rng.random() < 0.5 else _log_int(rng, 1, 4096)
        if n <= L and B * n * L * Hq <= 1 << 28 and B * L * Hkv * D <= 1 << 28 and (n < 8 or n * L * B * Hq * D <= 1 << 35):
            return {"op": op, "B": B, "n": n, "L": L, "Hq": Hq, "Hkv": Hkv, "D": D, "group": group, "page": page,
                    "window": rng.choice([0, 0, 0, max(1, L // 3)]), "ragged": rng.choice([0.0, 0.5, 1.0]),
                    "dtype": dtype}


def _dtype(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _groups(case):
    return case["D"] // case["group"] if case["group"] else 1


def _frequencies(case):
    """The rotation's frequencies and the factor of its cosines and sines:
    theta^(-2i/rd); scaled for contexts `factor` times the trained 8192 by
    dividing the frequencies that turn less than once over it, keeping those
    that turn more than 32 times, and blending those between."""
    rd, theta, factor, trained = case["rd"], 1e6, case["factor"], 8192.0
    freq = [theta ** (-2.0 * i / rd) for i in range(rd // 2)]
    if factor == 1.0:
        return freq, 1.0
    at = lambda turns: rd * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rd - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(rd // 2)]
    return [f / factor * r + f * (1.0 - r) for f, r in zip(freq, ramp)], 0.1 * math.log(factor) + 1.0


def _lengths(case):
    """Tokens and queries of each sequence, largest first; a wholly ragged batch ends in an empty one."""
    B, L, n = case["B"], case["L"], case["n"]
    part = [1.0 - case["ragged"] * b / max(B - 1, 1) for b in range(B)]
    lens = [int(L * p) for p in part]
    return lens, [n if n == 1 else max(1, min(int(n * p), k)) for p, k in zip(part, lens)]


def _pack(codes):
    """Codes [..., D] -> nibbles [..., D / 2], low nibble first."""
    nib = (codes + 8).to(torch.uint8).unflatten(-1, (-1, 2))
    return nib[..., 0] | (nib[..., 1] << 4)


def _unpack(packed):
    return torch.stack(((packed & 15).float() - 8.0, (packed >> 4).float() - 8.0), dim=-1).flatten(-2)


def _v_order(x, G):
    """A head's dimensions in the order of v_codes, and back."""
    return x.unflatten(-1, (G, 16, -1)).transpose(-3, -2).flatten(-3)


def _v_back(x, G):
    return x.unflatten(-1, (16, G, -1)).transpose(-3, -2).flatten(-3)


def _quantize(x, G):
    """fp32 rows [..., D] -> codes [..., D] and scales [..., G]: the library's
    int4 rule. 16-bit values often lie on a border between two codes, so both
    quotients are the correctly rounded fp32 ones (formed in 64 bits; torch
    divides by a number through its reciprocal)."""
    x = x.unflatten(-1, (G, -1))
    scale = (x.abs().amax(-1).double() / 7.0).float()
    codes = torch.where(scale[..., None] > 0, torch.round((x.double() / scale[..., None].double()).float()),
                        torch.zeros_like(x)).clamp(-7, 7)
    return codes.flatten(-2), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s, t, D = {"case": dict(case)}, _dtype(case), case["D"]
    if case["op"] != "attend":
        T, freq = case["T"], _frequencies(case)
        s["inv_freq"], s["scale"] = torch.tensor(freq[0], dtype=torch.float64, device="cuda"), freq[1]
        first = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
        if T <= 64:  # a decode step: every request at a place of its own
            s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda").to(torch.int32)
    if case["op"] == "rope":
        s["rows"] = rnd(T, case["H"] + (8 if case["fused"] else 0), D).to(t)
        s["x"] = s["rows"][:, :case["H"]]
        return s
    Hq, Hkv, G, page = case["Hq"], case["Hkv"], _groups(case), case["page"]
    if case["op"] == "append":
        # the projections' rows: some channels of k are much larger than the others
        s["q"], s["v"] = rnd(T, Hq, D).to(t), rnd(T, Hkv, D).to(t)
        s["k"] = (rnd(T, Hkv, D) * (1.0 + 4.0 * (rnd(Hkv, D) > 2.0))).to(t)
        s["q_norm"] = (1.0 + 0.1 * rnd(D)).to(t) if case["norm"] else None
        s["k_norm"] = (1.0 + 0.1 * rnd(D)).to(t) if case["norm"] else None
        pages = -(-T // page) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(T, device="cuda")
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        shape = (pages, Hkv, page, D // 2)
        s["cache"] = [torch.zeros(shape, dtype=torch.uint8, device="cuda"), torch.zeros(pages, Hkv, G, page, device="cuda"),
                      torch.zeros(shape, dtype=torch.uint8, device="cuda"), torch.zeros(pages, Hkv, G, page, device="cuda")]
        return s
    lens, queries = _lengths(case)
    order = torch.randperm(case["B"], generator=g, device="cuda").tolist()
    lens, queries = [lens[i] for i in order], [queries[i] for i in order]
    most = max(1, -(-max(lens) // page))
    pages = case["B"] * most + 2
    s["page_table"] = torch.randperm(pages, generator=g, device="cuda")[:case["B"] * most].to(torch.int32).view(-1, most)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ends = [sum(queries[:i]) for i in range(case["B"] + 1)]
    s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda") if case["n"] > 1 else None
    s["most_queries"] = max(queries)  # the plain form's padding
    s["q"] = (1.5 * rnd(ends[-1], Hq, D)).to(t)
    # keys and values as quantization leaves them: bells of codes, scales around a typical row's
    code = lambda: (rnd(pages, Hkv, page, D).mul_(2.6).round_().clamp_(-7, 7)).to(torch.int8)  # noqa: E731
    scale = lambda: 0.35 + 0.1 * torch.rand(pages, Hkv, G, page, generator=g, device="cuda")  # noqa: E731
    k_codes = _pack(code())
    k_scale = scale()
    v_codes = _pack(code())
    s["cache"] = [k_codes, k_scale, v_codes, scale()]
    return s


# ---- the plain forms --------------------------------------------------------

def _plain_rotate(x, s):
    """fp32 x [T, H, D] rotated by its tokens' positions."""
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = (torch.cos(angle) * s["scale"]).float()[:, None], (torch.sin(angle) * s["scale"]).float()[:, None]
    r, rest = x[..., :c["rd"]], x[..., c["rd"]:]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = r[..., :c["rd"] // 2], r[..., c["rd"] // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((r, rest), dim=-1)


def _plain_norm(x, weight, eps=1e-6):
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()


def _plain_append(s):
    c, t, G = s["case"], _dtype(s["case"]), _groups(s["case"])
    k_codes, k_scale, v_codes, v_scale = s["cache"]
    q = _plain_rotate(_plain_norm(s["q"].float(), s["q_norm"]), s).to(t)
    k = _plain_rotate(_plain_norm(s["k"].float(), s["k_norm"]), s).to(t)
    page, at = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    codes, scale = _quantize(k.float(), G)
    k_codes[page, :, at], k_scale[page, :, :, at] = _pack(codes), scale
    codes, scale = _quantize(s["v"].float(), G)
    v_codes[page, :, at], v_scale[page, :, :, at] = _pack(_v_order(codes, G)), scale
    k = (_unpack(k_codes[page, :, at]).unflatten(-1, (G, -1)) * k_scale[page, :, :, at][..., None]).flatten(-2).to(t)
    v = _v_back(_unpack(v_codes[page, :, at]), G)
    return {"q": q, "k": k, "v": (v.unflatten(-1, (G, -1)) * v_scale[page, :, :, at][..., None]).flatten(-2).to(t)}


def _plain_attend(s):
    c, G = s["case"], _groups(s["case"])
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    k_codes, k_scale, v_codes, v_scale = s["cache"]
    table, lens = s["page_table"].long(), s["lengths"].long()
    tokens = table.shape[1] * c["page"]

    def rows(codes, scale, back):
        x = _unpack(codes[table])                                       # [B, pages, Hkv, page, D]
        x = (_v_back(x, G) if back else x).unflatten(-1, (G, -1)) * scale[table].transpose(-1, -2)[..., None]
        return x.flatten(-2).transpose(1, 2).reshape(B, Hkv, tokens, D)

    n = s["most_queries"]
    if s["offsets"] is None:
        start, count = torch.arange(B, device="cuda"), torch.ones(B, dtype=torch.long, device="cuda")
    else:
        start, count = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    i = torch.arange(n, device="cuda")
    real = i < count[:, None]                                           # [B, n]
    q = s["q"].float()[torch.where(real, start[:, None] + i, 0)]        # [B, n, Hq, D]
    q = q.view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = torch.matmul(q, rows(k_codes, k_scale, False).transpose(-1, -2)) * D ** -0.5
    place = (lens - count)[:, None] + i                                 # [B, n]
    key = torch.arange(tokens, device="cuda")
    seen = key <= place[..., None]
    if c["window"]:
        seen &= key > place[..., None] - c["window"]
    score = score.view(B, Hkv, Hq // Hkv, n, tokens).masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)                    # rows that see nothing: zeros
    y = torch.matmul(p.view(B, Hkv, -1, tokens), rows(v_codes, v_scale, True))
    y = y.view(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return y[real].to(_dtype(c))


# ---- one pass ---------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        from w8a8_online_quantized_amd import cider
        if c["op"] == "rope":
            return cider.cider_rope(s["x"], s["positions"], s["inv_freq"], interleaved=c["interleaved"], scale=s["scale"])
        cache = cider.KV4Cache(*s["cache"])
        if c["op"] == "append":
            q = cider.cider_kv4_append(cache, s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"],
                                       inv_freq=s["inv_freq"], interleaved=c["interleaved"], rope_scale=s["scale"],
                                       q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6)
            k, v = cider.cider_kv4_read(cache, s["slots"], out_dtype=_dtype(c))
            return {"q": q, "k": k, "v": v}
        return cider.cider_kv4_attention(s["q"], cache, s["page_table"], s["lengths"], query_offsets=s["offsets"],
                                         window=c["window"])
    if c["op"] == "rope":
        return _plain_rotate(s["x"].float(), s).to(_dtype(c))
    return _plain_append(s) if c["op"] == "append" else _plain_attend(s)


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        return {"bytes": 4 * case["T"] * case["H"] * D + 4 * case["T"] + 4 * case["rd"],
                "flops": 3 * case["T"] * case["H"] * case["rd"]}
    stored = D + 8 * _groups(case)  # one token's keys and values of a head
    if case["op"] == "append":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        # q, k and v in, q out, the codes written, and the same read back into rows
        return {"bytes": T * (4 * Hq * D + 4 * Hkv * D + 8) + T * Hkv * (2 * stored + 4 * D), "flops": 12 * T * (Hq + 2 * Hkv) * D}
    lens, queries = _lengths(case)
    seen = keys = 0
    for k, n in zip(lens, queries):
        w = case["window"] or k
        # query i of n sees min(k - n + 1 + i, w) keys
        free = max(0, min(n, w - (k - n)))
        seen += (free * (k - n + 1) + free * (free - 1) // 2 + (n - free) * w) if k else 0
        keys += min(k, w + n - 1)
    return {"bytes": keys * case["Hkv"] * stored + 4 * sum(queries) * case["Hq"] * D + 4 * keys // case["page"],
            "flops": 4.0 * seen * case["Hq"] * D}


def exact(case, seed):
    """The definitions in 64 bits: complex rotations, one row of scales and one sequence after another."""
    s = prepare(case, seed)
    D, t = case["D"], _dtype(case)

    def turned(x):
        rd = case["rd"]
        turn = torch.polar(torch.full_like(s["inv_freq"], s["scale"]).expand(case["T"], -1).contiguous(),
                           s["positions"].double().outer(s["inv_freq"]))[:, None]
        r = x[..., :rd]
        pairs = r.unflatten(-1, (-1, 2)) if case["interleaved"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat((z, x[..., rd:]), -1)

    if case["op"] == "rope":
        return turned(s["x"].double())
    G = _groups(case)
    if case["op"] == "append":
        def normed(x, w):
            x = x.double()
            return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()

        def stored(x):
            # the library's rule: the scale is an fp32 number, and so is the quotient that is rounded to a code
            out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
            for first in range(0, D, D // G):
                part = x[..., first:first + D // G].double()
                step = (part.abs().amax(-1, keepdim=True) / 7).float().double()
                code = torch.round((part / step.clamp(min=1e-300)).float()).double()
                out[..., first:first + D // G] = code.clamp(-7, 7) * step
            return out

        return {"q": turned(normed(s["q"], s["q_norm"])), "k": stored(turned(normed(s["k"], s["k_norm"])).to(t)),
                "v": stored(s["v"])}
    k_codes, k_scale, v_codes, v_scale = s["cache"]
    lens = s["lengths"].tolist()
    ends = list(range(case["B"] + 1)) if s["offsets"] is None else s["offsets"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    per = case["Hq"] // case["Hkv"]
    pos_v = torch.arange(D, device="cuda").view(G, 16, -1).permute(1, 0, 2).reshape(-1).argsort()  # where a dimension lies
    for b, length in enumerate(lens):
        if not length:
            continue
        ids = s["page_table"][b, : -(-length // case["page"])].long()
        place = length - (ends[b + 1] - ends[b]) + torch.arange(ends[b + 1] - ends[b], device="cuda")
        key = torch.arange(length, device="cuda")
        hidden = key[None] > place[:, None]
        if case["window"]:
            hidden |= key[None] <= place[:, None] - case["window"]
        for h in range(case["Hkv"]):
            def side(codes, scale, order):
                raw = codes[ids, h].reshape(-1, D // 2)[:length]
                x = torch.empty(length, D, dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = raw.bitwise_and(15).double() - 8, raw.bitwise_right_shift(4).double() - 8
                if order is not None:
                    x = x[:, order]
                return x * scale[ids, h].transpose(1, 2).reshape(-1, G)[:length].double().repeat_interleave(D // G, 1)
            k, v = side(k_codes, k_scale, None), side(v_codes, v_scale, pos_v)
            for j in range(h * per, (h + 1) * per):
                a = (s["q"][ends[b]:ends[b + 1], j].double() @ k.t()) / math.sqrt(D)
                out[ends[b]:ends[b + 1], j] = torch.softmax(a.masked_fill(hidden, -math.inf), -1) @ v
    return out
