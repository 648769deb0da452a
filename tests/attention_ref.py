"""Plain 64-bit references of the rotary, 4-bit cache and attention operators (torch / numpy, from the definitions)."""
import math

import numpy as np
import torch

from tests import nvfp4_ref


def angles(far, rot, base=10000.0):
    """fp32 [far, rot]: cosines then sines, from 64-bit angles."""
    inv = base ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(far)[:, None] * inv
    return torch.from_numpy(np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32))


def pair_of(rot, pairs):
    """Indexes of the first and second elements of the rotated pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)


def rope(x, w, pos, table, eps, pairs):
    """float64 [T, heads, D]; positions must be inside the table."""
    x = x.double()
    y = x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    y = y.clone()
    at = table.double()[pos.long()]
    rot = at.shape[1]
    c, s = at[:, None, :rot // 2], at[:, None, rot // 2:]
    a, b = pair_of(rot, pairs)
    ya, yb = y[..., a], y[..., b]
    y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y


def rope_grad(dy, x, w, pos, table, eps, pairs):
    """(dx, dw) in 64 bits by the formula."""
    d, x = dy.double().clone(), x.double()
    at = table.double()[pos.long()]
    rot = at.shape[1]
    c, s = at[:, None, :rot // 2], at[:, None, rot // 2:]
    a, b = pair_of(rot, pairs)
    da, db = d[..., a], d[..., b]
    d[..., a], d[..., b] = da * c + db * s, db * c - da * s
    if w is None:
        return d, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    g = d * w.double()
    return r * (g - x * r * r * (g * x).mean(-1, keepdim=True)), (d * x * r).sum((0, 1))


def put(pages, page_size, slots, k, v, kg, vg):
    """Rows k, v [T, heads, D] (numpy float32) quantised into `pages` (numpy uint8 [n, heads, page / 16, 18 D]), one
    token after the other."""
    D = k.shape[2]
    for t, slot in enumerate(slots):
        if not 0 <= slot < pages.shape[0] * page_size:
            continue
        p, o = divmod(int(slot), page_size)
        tile, i = divmod(o, 16)
        for x, g, code_at, sf_at in ((k, kg, 0, 16 * D), (v, vg, 8 * D, 17 * D)):
            code, sf = nvfp4_ref.quantize(x[t], g)
            pages[p, :, tile, code_at + i * (D // 2):code_at + (i + 1) * (D // 2)] = nvfp4_ref.pack(code)
            pages[p, :, tile, sf_at + i * (D // 16):sf_at + (i + 1) * (D // 16)] = sf


def cached(pages, which):
    """float64 [n, heads, page, D] that K (0) or V (1) of `pages` (torch uint8, any device) stands for, without its
    global scale; NaN where a scale factor is."""
    n, heads, tiles, wide = pages.shape
    D = wide // 18
    dev = pages.device
    code = pages[..., which * 8 * D:(which + 1) * 8 * D].reshape(n, heads, tiles, 16, D // 2)
    sf = pages[..., (16 + which) * D:(17 + which) * D].reshape(n, heads, tiles, 16, D // 16)
    f4 = torch.tensor(np.concatenate((nvfp4_ref.F4, -nvfp4_ref.F4)), device=dev)
    v = f4[torch.stack((code & 15, code >> 4), -1).flatten(-2).int()]
    step = torch.tensor(nvfp4_ref.E4M3, device=dev)[(sf & 127).int()]
    return (v * step.repeat_interleave(16, -1)).view(n, heads, tiles * 16, D)


def attention(q, pages, kg, vg, table, lens, cu, scale, causal=True, window=0):
    """(out, lse, slack_out, slack_lse) in 64 bits; the slacks bound the kernel's error but for the output's rounding.

    A score's error: exact products, at most D + 4 fp32 additions and factors of 2^-23 of the sum of magnitudes each.
    exp: that error, 2^-21 of its own; rounding to fp16 2^-11 (2^-25 of the maximum for the smallest).  The sums of
    the softmax are in fp32, of positive terms: 2^-18 covers those of the longest call here."""
    T, hq, D = q.shape
    page = pages.shape[2] * 16
    heads = pages.shape[1]
    G = hq // heads
    out, slack = torch.zeros(T, hq, D, dtype=torch.float64, device=q.device), torch.zeros(T, hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=q.device)
    slack_lse = torch.zeros(T, hq, dtype=torch.float64, device=q.device)
    kc, vc = cached(pages, 0) / kg, cached(pages, 1) / vg
    for b in range(len(lens)):
        q0, q1 = (int(cu[b]), int(cu[b + 1])) if cu is not None else (b, b + 1)
        L, m = int(lens[b]), q1 - q0
        L = min(L, table.shape[1] * page)
        if m == 0 or L <= 0:
            continue
        ids = table[b, :-(-L // page)].long()
        here = ((ids >= 0) & (ids < pages.shape[0])).repeat_interleave(page)[:L]
        ids = torch.where((ids >= 0) & (ids < pages.shape[0]), ids, 0)
        j = torch.arange(L, device=q.device)
        at = L - m + torch.arange(m, device=q.device).view(-1, 1)
        sees = here.expand(m, L)
        if causal:
            sees = sees & (j <= at)
        if window:
            sees = sees & (j > at - window)
        for h in range(heads):
            k = torch.nan_to_num(kc[ids, h].reshape(-1, D)[:L])
            v = torch.where(sees.any(0).unsqueeze(1), vc[ids, h].reshape(-1, D)[:L], 0.0)
            x = q[q0:q1, h * G:(h + 1) * G].double()
            s = torch.einsum("mgd,jd->mgj", x, k) * scale
            no = ~sees.view(m, 1, L)
            mag = torch.einsum("mgd,jd->mgj", x.abs(), k.abs()).masked_fill_(no, 0.0).amax(-1) * scale
            es = (D + 4) * 2.0 ** -23 * mag + 2.0 ** -20
            s.masked_fill_(no, -math.inf)
            total = torch.logsumexp(s, -1)
            p = torch.where(sees.any(1).view(m, 1, 1), (s - total.unsqueeze(-1)).exp(), 0.0)
            out[q0:q1, h * G:(h + 1) * G] = torch.einsum("mgj,jd->mgd", p, v)
            lse[q0:q1, h * G:(h + 1) * G] = total
            each = 2.0 ** -11 + 2.0 ** -18 + 2 * es
            tiny = 2.0 ** -24 / p.amax(-1, keepdim=True).clamp(min=1e-30) * p.amax(-1, keepdim=True)
            slack[q0:q1, h * G:(h + 1) * G] = each.unsqueeze(-1) * torch.einsum("mgj,jd->mgd", p, v.abs()) + \
                tiny * p.amax(-1, keepdim=True) * v.abs().sum(0)
            slack_lse[q0:q1, h * G:(h + 1) * G] = es + 2.0 ** -18 + 2.0 ** -22 * total.abs().nan_to_num(posinf=0.0)
    return out, lse, slack, slack_lse
