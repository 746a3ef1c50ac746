"""Plain forms in 64 bits of the attention block's operators, and the bounds of
their fp32 steps. Used by the GPU tests; nothing here calls the library."""
import math

import torch

U = 2.0 ** -24   # half a step of fp32


def pack(codes):
    nib = (codes + 8).to(torch.uint8)
    return nib[..., 0::2] | (nib[..., 1::2] << 4)


def unpack(packed):
    out = torch.empty(*packed.shape[:-1], 2 * packed.shape[-1], dtype=torch.float64, device=packed.device)
    out[..., 0::2], out[..., 1::2] = (packed & 15).double() - 8, (packed >> 4).double() - 8
    return out


def v_place(D, G):
    """Where each dimension of a head lies in a row of v_codes, from the header's formula."""
    per = D // 16 // G
    at = torch.empty(D, dtype=torch.long)
    for g in range(G):
        for u in range(16):
            for r in range(per):
                at[g * (D // G) + u * per + r] = (u * G + g) * per + r
    return at


def stored_rows(cache, slots):
    """fp64 k, v [n, Hkv, D] of slots inside the cache."""
    k_codes, k_scale, v_codes, v_scale = cache
    page_size, G = k_codes.shape[2], k_scale.shape[2]
    page, at = slots.long() // page_size, slots.long() % page_size
    k, v = unpack(k_codes[page, :, at]), unpack(v_codes[page, :, at])
    D = k.shape[-1]
    v = v[..., v_place(D, G).to(v.device)]
    return (k * k_scale[page, :, :, at].double().repeat_interleave(D // G, -1),
            v * v_scale[page, :, :, at].double().repeat_interleave(D // G, -1))


def rotate(x, positions, inv_freq, interleaved, scale):
    x = x.double().clone()
    n = inv_freq.numel()
    a = positions.double()[:, None] * inv_freq
    c, s = (torch.cos(a) * scale)[:, None], (torch.sin(a) * scale)[:, None]
    iu = torch.arange(n, device=x.device) * (2 if interleaved else 1)
    iw = iu + (1 if interleaved else n)
    u, w = x[..., iu], x[..., iw]
    x[..., iu], x[..., iw] = u * c - w * s, w * c + u * s
    return x


def rotation_error(x, inv_freq, interleaved, scale):
    """Bound of the fp32 steps of a rotation of fp64 rows x: the cosines are off
    by the remainder's rounding (half a turn's 2^-25 turns: pi * 2^-24 rad), the
    functions' 4 steps and the factor's rounding, then two products and a sum."""
    n = inv_freq.numel()
    err = torch.zeros_like(x)
    iu = torch.arange(n, device=x.device) * (2 if interleaved else 1)
    iw = iu + (1 if interleaved else n)
    size = (x[..., iu].abs() + x[..., iw].abs()) * abs(scale)
    err[..., iu] = err[..., iw] = size * (math.pi + 8 + 1 + 3) * U + 1e-12 * size
    return err


def int4_rule(x, G):
    """Codes and fp32 scales of 16-bit rows [..., D]: s = fl(max / 7), code = rint(fl(x / s))."""
    x = x.float().double().unflatten(-1, (G, -1))
    s = (x.abs().amax(-1) / 7).float()
    code = torch.round((x / s.double().clamp(min=1e-300)[..., None]).float())
    code = torch.where(s[..., None] > 0, code, torch.zeros_like(code)).clamp(-7, 7)
    return code.flatten(-2).long(), s


def attention(q, cache, page_table, lengths, offsets, causal, window, scale):
    """y in 64 bits and a bound of the kernel's error per element (before and
    with the rounding of y). Pages outside the cache are not seen."""
    k_codes, k_scale, v_codes, v_scale = cache
    n_pages, Hkv, page_size, half = k_codes.shape
    T, Hq, D = q.shape
    per = Hq // Hkv
    B = len(lengths)
    y = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    bound, typical = torch.zeros_like(y), torch.zeros_like(y)
    # codes enter the products as 128 + n (bf16) or 64 + n (fp16; V always), n below 16,
    # and the sums start at what is too much, 136 or 72: the largest operand and the
    # offset's part. The matrix core may cut a sum where fp32 would round it: 2 U.
    reach, reach_v = (2 * 279.0 if q.dtype == torch.bfloat16 else 2 * 151.0), 2 * 151.0
    for b in range(B):
        lo, hi = offsets[b], offsets[b + 1]
        n, L = hi - lo, min(max(lengths[b], 0), page_table.shape[1] * page_size)
        if n == 0 or L == 0:
            continue
        ids = page_table[b, : -(-L // page_size)].long()
        ok = (ids >= 0) & (ids < n_pages)
        at = torch.arange(L, device=q.device)
        there = ok[at // page_size]
        slots = torch.where(ok, ids, 0)[at // page_size] * page_size + at % page_size
        k, v = stored_rows(cache, slots)
        sk = k_scale[slots // page_size, :, :, slots % page_size].double().amax(-1)    # [L, Hkv]
        sv = v_scale[slots // page_size, :, :, slots % page_size].double().amax(-1)
        pos = L - n + torch.arange(n, device=q.device)
        seen = there[None].expand(n, L).clone()
        if causal:
            seen &= at[None] <= pos[:, None]
        if window:
            seen &= at[None] > pos[:, None] - window
        k, v, sk, sv = (torch.where(seen.any(0).view(-1, *[1] * (t.dim() - 1)), t, torch.zeros_like(t)) for t in (k, v, sk, sv))
        for h in range(Hq):
            g = h // per
            qh = q[lo:hi, h].double()
            s = scale * (qh @ k[:, g].t())
            s = s.masked_fill(~seen, -math.inf)
            top = s.amax(1, keepdim=True).clamp(min=-1e300)
            p = torch.exp(s - top)
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
            y[lo:hi, h] = p @ v[:, g]
            # a score is a sum of D products of 16-bit numbers, exact in fp32, of at
            # most |q| * reach * s_k (2 U included), then its scaling and the difference to the maximum
            one = abs(scale) * qh.abs().sum(1, keepdim=True) * reach * sk[:, g][None] * U
            worst = one * (D + 8) + (s.masked_fill(~seen, 0).abs() + 16) * 4 * U
            usual = one / math.sqrt(D) * 3 + (s.masked_fill(~seen, 0).abs() + 16) * 4 * U
            # the weights: their own rounding to fp16 (eps 2^-10, so at most half of it,
            # 2^-11; as independent errors about 2^-12; or half its smallest step
            # where they are small: 2^-25 times at most twice the largest scale), and
            # twice the scores' errors (numerator and sum)
            A, S = p @ v[:, g].abs(), (p @ sv[:, g:g + 1])
            tiny = 2.0 ** -24 * 15 * L * sv[:, g].max() * 2.0 ** -8
            w = (p * worst).amax(1, keepdim=True), (p * usual * usual).sum(1, keepdim=True).sqrt()
            e = (p * worst) @ v[:, g].abs() + A * (p * worst).sum(1, keepdim=True)
            # sums over the tokens
            sums = reach_v * S * (L / 4 + 64) * U
            bound[lo:hi, h] = e + A * (2.0 ** -11 + (L / 4 + 64) * U) + sums + tiny
            typical[lo:hi, h] = (p.square() @ v[:, g].square()).sqrt() * 2.0 ** -12 + A * (2.0 ** -20 + w[1]) + \
                reach_v * S * math.sqrt(L + 64) * U + tiny
    eps = torch.finfo(q.dtype).eps / 2
    small = torch.finfo(q.dtype).tiny * torch.finfo(q.dtype).eps / 2
    return y, bound * 1.01 + y.abs() * eps + small, (typical, eps)
