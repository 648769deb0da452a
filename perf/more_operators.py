"""Measured cases of the rotary, 4-bit cache and attention operators, with their plain forms.

Four operators, in the order in which an attention layer uses them:

  rope    each head's RMSNorm of queries and keys and the rotation by position, in one pass
  grad    the gradient of `rope`
  append  `rope` whose keys, with the values, go into a paged NVFP4 cache; and the cache read back
  attend  attention of queries over the cache: single tokens, a few of each sequence, whole prompts

`own` chooses between the plain form (elementary torch operations, fp32) and the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
F4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of E2M1
TILE = 16                                       # tokens of a tile of the cache


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the decoded tokens of one tensor-parallel shard of 8 query heads and one key head: latency
        dict(name="rope_decode", op="rope", T=16, hq=8, hk=1, D=128, rot=128, pairs=False, far=32768),
        # a long prompt, all heads of a layer, an odd number of tokens, half of each head rotated
        dict(name="rope_prompt", op="rope", T=16383, hq=64, hk=8, D=128, rot=64, pairs=False, far=32768),
        # a short sequence of a training step, neighbours rotated together
        dict(name="grad_short", op="grad", T=77, hq=32, hk=4, D=64, rot=64, pairs=True, far=4096),
        # a training step's tokens
        dict(name="grad_batch", op="grad", T=8192, hq=64, hk=8, D=128, rot=128, pairs=False, far=8192),
        # a decode batch's keys and values put into the cache
        dict(name="append_decode", op="append", T=64, hq=64, hk=8, D=128, rot=128, pairs=False, far=32768, page=64),
        # a prompt's, into small pages
        dict(name="append_prompt", op="append", T=16384, hq=64, hk=8, D=128, rot=128, pairs=False, far=32768, page=16),
        # one token of one sequence on one shard's heads: latency
        dict(name="attend_one", op="attend", B=1, n=1, L=1024, hq=8, hk=1, D=128, page=64, window=0, mix=0),
        # a decode batch of sequences of very different lengths, some of them still empty
        dict(name="attend_decode", op="attend", B=64, n=1, L=16384, hq=64, hk=8, D=128, page=64, window=0, mix=1),
        # one token far into a long document, one shard's heads
        dict(name="attend_long", op="attend", B=1, n=1, L=131072, hq=8, hk=1, D=128, page=128, window=0, mix=0),
        # a few proposed tokens of each sequence checked at once, narrow heads, a sliding window
        dict(name="attend_few", op="attend", B=16, n=5, L=4096, hq=40, hk=8, D=64, page=16, window=1024, mix=2),
        # pieces of several prompts, each after what the cache holds already
        dict(name="attend_chunk", op="attend", B=5, n=1024, L=6144, hq=64, hk=8, D=128, page=64, window=0, mix=3),
        # a whole prompt, an odd number of tokens
        dict(name="attend_prompt", op="attend", B=1, n=8191, L=8191, hq=64, hk=8, D=128, page=64, window=0, mix=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "grad", "append", "attend", "attend", "attend"))
    hk = rng.choice((1, 2, 4, 8))
    hq = hk * rng.choice((1, 2, 4, 5, 8))
    D = rng.choice((64, 128))
    if op != "attend":
        most = (8192 if op == "grad" else 16384) * 72 * 128 // ((hq + hk) * D)
        c = dict(op=op, T=_log(rng, 1, min(32768, most)), hq=hq, hk=hk, D=D, rot=rng.choice((32, 64, D)),
                 pairs=rng.choice((False, True)), far=_log(rng, 1024, 65536))
        if op == "append":
            c["page"] = rng.choice((16, 32, 64, 128))
        return c
    page = rng.choice((16, 32, 64, 128))
    window = rng.choice((0, 0, _log(rng, 16, 8192)))
    mix = rng.randint(0, 1 << 20)
    kind = rng.choice(("one", "few", "many"))
    if kind == "many":
        n = _log(rng, 17, 4096)
        B = _log(rng, 1, max(1, min(8, 4096 // n)))
        L = n + _log(rng, 1, 4096)
    else:
        n = 1 if kind == "one" else rng.randint(2, 12)
        B = _log(rng, 1, 64)
        L = max(n, _log(rng, 16, min(131072, 32 * 16384 // B)))
    return dict(op=op, B=B, n=n, L=L, hq=hq, hk=hk, D=D, page=page, window=window, mix=mix)


def _lengths(c):
    """(new tokens, cached tokens with them) of each sequence; mix 0: all the longest."""
    B, n, L = c["B"], c["n"], c["L"]
    if c["mix"] == 0:
        return [n] * B, [L] * B
    r = random.Random(c["mix"])
    new = [n if n == 1 else r.randint(1, n) for _ in range(B)]
    all_ = [min(L, max(m, int(L * r.random() ** 1.5))) for m in new]
    new[r.randrange(B)], all_[r.randrange(B)] = n, L
    all_ = [max(a, m) for a, m in zip(all_, new)]
    for b in range(B):  # some sequences hold nothing yet (decode batches are padded with them)
        if n == 1 and all_[b] < L and r.random() < 0.05:
            all_[b] = 0
    return new, all_


def _seen(m, length, window):
    """(query, key) pairs of m new tokens that end at `length`, and the keys that any of them sees."""
    pairs, first = 0, length
    lo, hi = max(0, length - m), length  # positions of the queries, those below 0 left out
    if lo >= hi:
        return 0, 0
    if not window:
        return (lo + 1 + hi) * (hi - lo) // 2, length
    full = max(lo, min(hi, window))  # queries from here on see `window` keys
    pairs = (lo + 1 + full) * (full - lo) // 2 + (hi - full) * window
    first = max(0, lo - window + 1)
    return pairs, length - first


def work(case):
    c = case
    if c["op"] == "attend":
        new, lens = _lengths(c)
        seen = [_seen(m, n, c["window"]) for m, n in zip(new, lens)]
        rows = sum(new) * c["hq"]
        return {"bytes": sum(k for _, k in seen) * c["hk"] * c["D"] * 9 / 8 + 4 * rows * c["D"] + 4 * rows,
                "flops": 4 * sum(p for p, _ in seen) * c["hq"] * c["D"]}
    T, D, heads = c["T"], c["D"], c["hq"] + c["hk"]
    table = 4 * min(T, c["far"]) * c["rot"] + 4 * T
    if c["op"] == "rope":
        return {"bytes": 4 * T * heads * D + table, "flops": 8 * T * heads * D}
    if c["op"] == "grad":  # x, dy and dx, and the weights' gradients
        return {"bytes": 6 * T * heads * D + table + 8 * D, "flops": 16 * T * heads * D}
    # append: q twice, k and v once, the cache written and read, k and v read back
    kv = 2 * T * c["hk"] * D
    return {"bytes": 4 * T * c["hq"] * D + 2 * kv + 2 * kv * 9 / 16 + 2 * kv + table + 4 * T,
            "flops": 8 * T * heads * D + 4 * kv}


# ---------------------------------------------------------------------------
# NVFP4 in plain torch
# ---------------------------------------------------------------------------

def _encode(x, g):
    """(codes 0..15 as uint8, scale factors as e4m3 [.., D/16]) of bf16 rows [.., D]."""
    v = x.float().unflatten(-1, (-1, 16))
    sf = (g * (v.abs().amax(-1) / torch.full_like(g, 6.0))).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = sf.float()
    es = torch.where(d != 0, g / d, torch.zeros_like(d))
    n = v * es.unsqueeze(-1)
    a = n.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * ((n < 0) | ((n == 0) & torch.signbit(n)) & (d != 0).unsqueeze(-1)).to(torch.uint8)
    return code.flatten(-2), sf


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _decode(packed, sf, dtype=torch.float32):
    """code * scale factor (exact) of packed codes and their e4m3 scale factors [.., D/16]."""
    table = torch.tensor(F4 + tuple(-v for v in F4), dtype=dtype, device=packed.device)
    v = table[torch.stack((packed & 15, packed >> 4), -1).int()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * sf.to(dtype).unsqueeze(-1)).flatten(-2)


def _global_scale(x, gen):
    """A calibrated global scale: room for amax up to a factor that other data asked for."""
    room = 1.0 + 0.3 * torch.rand(1, generator=gen, device=DEV)
    return (448.0 * 6.0) / (room * x.abs().amax().float().clamp(min=1e-30))


# The cache is uint8 [pages, heads, page / 16, 18 D]: in the last dimension, for 16 tokens, the codes of K
# [16, D / 2] and of V, then the scale factors of K [16, D / 16] and of V.
def _put(pages, slots, page, k, v, kg, vg):
    """Rows k and v [T, heads, D] quantised into the cache's slots; a negative one gets nothing."""
    n, heads, tiles, wide = pages.shape
    D = wide // 18
    flat = pages.view(n * heads * tiles, wide)
    use = slots >= 0
    s = slots[use].long()
    row = ((s // page).unsqueeze(1) * heads + torch.arange(heads, device=DEV)) * tiles + ((s % page) // TILE).unsqueeze(1)
    t = (s % TILE).view(-1, 1, 1)
    for x, g, code_at, sf_at in ((k, kg, 0, 16 * D), (v, vg, 8 * D, 17 * D)):
        code, sf = _encode(x[use], g)
        half = torch.arange(D // 2, device=DEV)
        flat[row.unsqueeze(2), code_at + t * (D // 2) + half] = _pack(code)
        flat[row.unsqueeze(2), sf_at + t * (D // 16) + torch.arange(D // 16, device=DEV)] = sf.view(torch.uint8)


def _parts(tiles, D):
    """K and V (codes, scale factors) [.., 16, ..] of the cache's tiles [.., 18 D]."""
    lead = tiles.shape[:-1]
    at = lambda lo, n: tiles[..., lo:lo + 16 * n].reshape(*lead, 16, n)  # noqa: E731
    return ((at(0, D // 2), at(16 * D, D // 16).contiguous().view(torch.float8_e4m3fn)),
            (at(8 * D, D // 2), at(17 * D, D // 16).contiguous().view(torch.float8_e4m3fn)))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _heads(T, heads, D, gen, tail):
    """bf16 [T, heads, D] as a projection leaves it: a view of wider rows, a few columns that stand out."""
    x = torch.randn(T, heads * D + tail, generator=gen, device=DEV)
    x *= torch.where(torch.rand(x.shape[1], generator=gen, device=DEV) < 0.01, 6.0, 1.0)
    return x.bfloat16()[:, :heads * D].unflatten(1, (heads, D))


def _angles(far, rot):
    """cos | sin of every position, fp32 [far, rot], from 64-bit angles."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(far, dtype=torch.float64, device=DEV).unsqueeze(1) * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    c, gen = case, torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    hq, hk, D = c["hq"], c["hk"], c["D"]
    if c["op"] == "attend":
        return _prepare_attend(c, s, gen)
    T = c["T"]
    s["q"], s["k"] = _heads(T, hq, D, gen, hk * D), _heads(T, hk, D, gen, 64)
    s["qw"] = (0.5 + torch.rand(D, generator=gen, device=DEV)).bfloat16()
    s["kw"] = (0.5 + torch.rand(D, generator=gen, device=DEV)).bfloat16()
    s["table"] = _angles(c["far"], c["rot"])
    if T <= 128:  # decoded tokens, each of its own sequence
        s["pos"] = torch.randint(0, c["far"], (T,), generator=gen, device=DEV).int()
    else:         # sequences one after the other
        first = int(torch.randint(0, c["far"], (1,), generator=gen, device=DEV))
        s["pos"] = ((torch.arange(T, device=DEV) + first) % c["far"]).int()
    if c["op"] == "grad":
        s["dqo"] = torch.randn(T, hq, D, generator=gen, device=DEV).bfloat16()
        s["dko"] = torch.randn(T, hk, D, generator=gen, device=DEV).bfloat16()
    if c["op"] == "append":
        s["v"] = _heads(T, hk, D, gen, 64)
        n = -(-T // c["page"]) + 3
        s["pages"] = torch.zeros(n, hk, c["page"] // TILE, 18 * D, dtype=torch.uint8, device=DEV)
        order = torch.randperm(n, generator=gen, device=DEV)
        at = torch.arange(T, device=DEV)
        s["slots"] = (order[at // c["page"]] * c["page"] + at % c["page"]).int()
        s["slots"][torch.rand(T, generator=gen, device=DEV) < 0.02] = -1  # padding: not kept
        s["kg"] = (448.0 * 6.0) / (12.0 + 4.0 * torch.rand(1, generator=gen, device=DEV))
        s["vg"] = _global_scale(s["v"], gen)
        s["ko"], s["vo"] = (torch.zeros(T, hk, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    return s


def _prepare_attend(c, s, gen):
    B, hq, hk, D, page = c["B"], c["hq"], c["hk"], c["D"], c["page"]
    new, lens = _lengths(c)
    s["new"], s["lens"] = new, lens
    most = max(1, -(-max(lens) // page))
    used = [-(-n // page) for n in lens]
    total = sum(used) + 2
    order = torch.randperm(total, generator=gen, device=DEV).int()
    s["table"] = torch.full((B, most), -1, dtype=torch.int32, device=DEV)
    at = torch.tensor([[b, i] for b in range(B) for i in range(used[b])], device=DEV).view(-1, 2)
    s["table"][at[:, 0], at[:, 1]] = order[:len(at)]
    s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["cu"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    # keys and values as a model leaves them, quantised: keys with columns that stand out
    shape = (total * hk * (page // TILE), TILE, D)
    s["pages"] = torch.empty(shape[0], 18 * D, dtype=torch.uint8, device=DEV)
    for i, code_at in enumerate((0, 8 * D)):
        x = torch.randn(shape, generator=gen, device=DEV)
        if i == 0:
            x *= torch.where(torch.rand(D, generator=gen, device=DEV) < 0.03, 4.0, 1.0)
        x = x.bfloat16()
        s["kg" if i == 0 else "vg"] = g = _global_scale(x, gen)
        code, sf = _encode(x, g)
        s["pages"][:, code_at:code_at + 8 * D] = _pack(code).flatten(1)
        s["pages"][:, (16 + i) * D:(17 + i) * D] = sf.view(torch.uint8).flatten(1)
    s["pages"] = s["pages"].view(total, hk, page // TILE, 18 * D)
    s["q"] = (1.5 * torch.randn(sum(new), hq, D, generator=gen, device=DEV)).bfloat16()
    # where the queries of a padded batch [B, longest] are
    longest = max(new)
    i = torch.arange(longest, device=DEV)
    s["live"] = i < torch.tensor(new, device=DEV).unsqueeze(1)
    s["row"] = torch.where(s["live"], s["cu"][:B].long().unsqueeze(1) + i, 0)
    return s


# ---------------------------------------------------------------------------
# one pass: the library's calls
# ---------------------------------------------------------------------------

def _calls(s):
    import reduce_residual_rmsnorm_gb300 as ts

    c, op = s["case"], s["case"]["op"]
    if op == "attend":
        cache = ts.KVCache(s["pages"], s["kg"], s["vg"])
        out, lse = ts.ts_nvfp4_attention(s["q"], cache, s["table"], s["kv_lens"], None if c["n"] == 1 else s["cu"],
                                         max_q=c["n"], window=c["window"], return_lse=True, launch_with_pdl=True)
        return {"out": out, "lse": lse}
    common = (s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["table"], EPS)
    if op == "rope":
        q, k = ts.ts_qk_norm_rope(*common, interleaved=c["pairs"], launch_with_pdl=True)
        return {"q": q, "k": k}
    if op == "grad":
        dq, dk, dqw, dkw = ts.ts_qk_norm_rope_grad(s["dqo"], s["dko"], *common, interleaved=c["pairs"],
                                                   launch_with_pdl=True)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    cache = ts.KVCache(s["pages"], s["kg"], s["vg"])
    q, _ = ts.ts_qk_norm_rope(*common, interleaved=c["pairs"], v=s["v"], cache=cache, slots=s["slots"],
                              launch_with_pdl=True)
    ts.ts_kv_cache_read(cache, s["slots"], k_out=s["ko"], v_out=s["vo"], launch_with_pdl=True)
    return {"q": q, "k": s["ko"], "v": s["vo"]}


# ---------------------------------------------------------------------------
# one pass: the plain form
# ---------------------------------------------------------------------------

def _turn(x, cos, sin, rot, pairs, back=False):
    """The first `rot` columns of x [T, heads, D] rotated by each token's angles (backwards for the gradient)."""
    cos, sin = cos.unsqueeze(1), (-sin if back else sin).unsqueeze(1)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    return torch.cat((torch.stack((u, w), -1).flatten(-2) if pairs else torch.cat((u, w), -1), x[..., rot:]), -1)


def _normed(x, w):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r * w.float()


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "attend":
        return _plain_attend(s)
    rot, pairs = c["rot"], c["pairs"]
    at = s["table"][s["pos"].long()]
    cos, sin = at[:, :rot // 2], at[:, rot // 2:]
    if op == "grad":
        return dict(zip(("dq", "dqw", "dk", "dkw"), (*_grad(s["dqo"], s["q"], s["qw"], cos, sin, rot, pairs),
                                                     *_grad(s["dko"], s["k"], s["kw"], cos, sin, rot, pairs))))
    q = _turn(_normed(s["q"], s["qw"]), cos, sin, rot, pairs).bfloat16()
    k = _turn(_normed(s["k"], s["kw"]), cos, sin, rot, pairs).bfloat16()
    if op == "rope":
        return {"q": q, "k": k}
    _put(s["pages"], s["slots"], c["page"], k, s["v"], s["kg"], s["vg"])
    # the rows read back
    heads, D, page = c["hk"], c["D"], c["page"]
    kept = (s["slots"] >= 0).view(-1, 1, 1)
    slot = s["slots"].clamp(min=0).long()
    tiles = s["pages"][slot // page, :, (slot % page) // TILE]
    t = (slot % TILE).view(-1, 1, 1, 1).expand(-1, heads, 1, 1)
    for (codes, sf), g, out in zip(_parts(tiles, D), (s["kg"], s["vg"]), (s["ko"], s["vo"])):
        codes = codes.gather(2, t.expand(-1, -1, 1, D // 2)).squeeze(2)
        sf = sf.view(torch.uint8).gather(2, t.expand(-1, -1, 1, D // 16)).squeeze(2).view(torch.float8_e4m3fn)
        out.copy_(torch.where(kept, (_decode(codes, sf) / g).bfloat16(), out))
    return {"q": q, "k": s["ko"], "v": s["vo"]}


def _grad(dy, x, w, cos, sin, rot, pairs):
    d = _turn(dy.float(), cos, sin, rot, pairs, back=True)
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    g = d * w.float()
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    return dx.bfloat16(), (d * x * r).sum((0, 1))


def _plain_attend(s):
    c = s["case"]
    B, hq, hk, D, page = c["B"], c["hq"], c["hk"], c["D"], c["page"]
    # every sequence's keys and values in a padded batch [B, hk, keys, D]
    tiles = s["pages"][s["table"].clamp(min=0).long()].transpose(1, 2)
    keys = s["table"].shape[1] * page
    (kc, ks), (vc, vs) = _parts(tiles, D)
    k = _decode(kc, ks).reshape(B, hk, keys, D) / s["kg"]
    v = _decode(vc, vs).reshape(B, hk, keys, D) / s["vg"]
    longest = s["row"].shape[1]
    q = s["q"][s["row"]].float().view(B, longest, hk, hq // hk, D).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).view(B, hk, hq // hk, longest, keys) * (1 / math.sqrt(D))
    new = s["cu"][1:] - s["cu"][:-1]
    at = (s["kv_lens"] - new).view(B, 1, 1) + torch.arange(longest, device=DEV).view(1, -1, 1)
    j = torch.arange(keys, device=DEV)
    sees = j <= at
    if c["window"]:
        sees = sees & (j > at - c["window"])
    score.masked_fill_(~sees.view(B, 1, 1, longest, keys), -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).view(B, hk, hq // hk, longest, D) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    return {"out": out.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["live"]].bfloat16(),
            "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[s["live"]]}


def run(state):
    if own:
        return _calls(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest(v, grid):
    """The nearest value of an ascending grid to each v >= 0, ties to the even index, the last one above the end."""
    hi = torch.searchsorted(grid, v.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up = (grid[hi] - v < v - grid[lo]) | ((grid[hi] - v == v - grid[lo]) & (hi % 2 == 0))
    return torch.where(up | (lo == hi), grid[hi], grid[lo])


def _quantized64(x, g):
    """The values of rows by the definition: sf = e4m3(g amax / 6), e2m1(x g / sf) sf / g."""
    steps = torch.tensor([(f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)) for e in range(16) for f in range(8)][:127],
                         dtype=torch.float64, device=DEV)
    f4 = torch.tensor(F4, dtype=torch.float64, device=DEV)
    v = x.double().reshape(-1, 16)
    sf = _nearest(g.double() * v.abs().amax(1) / 6, steps).unsqueeze(1)
    by = torch.where(sf > 0, g.double() / sf, 0.0)
    return (_nearest(v.abs() * by, f4) * torch.sign(v) * sf / g.double()).reshape(x.shape)


def _turned64(x, w, table, pos, rot, pairs):
    """Norm and rotation of [T, heads, D] as complex numbers."""
    y = x.double()
    y = y / (y.square().sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * w.double()
    at = table[pos.long()].double()
    turn = torch.complex(at[:, :rot // 2], at[:, rot // 2:]).unsqueeze(1)
    first = list(range(0, rot, 2)) if pairs else list(range(rot // 2))
    second = [i + 1 for i in first] if pairs else [i + rot // 2 for i in first]
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _values64(tile_rows, D, which):
    """The values [n, 16, D] of K (0) or V (1) that tiles [n, 18 D] hold, without their global scale."""
    n = tile_rows.shape[0]
    byte = tile_rows[:, which * 8 * D:(which + 1) * 8 * D].reshape(n, 16, D // 2).long()
    code = torch.stack((byte % 16, byte // 16), -1).view(n, 16, D)
    e, f = (code // 2) % 4, code % 2
    mag = torch.where(e == 0, f * 0.5, (2 + f).double() * torch.pow(2.0, (e - 2).double()))
    sf = tile_rows[:, (16 + which) * D:(17 + which) * D].reshape(n, 16, D // 16).long()
    step = torch.where(sf // 8 == 0, (sf % 8) * 2.0 ** -9, (8 + sf % 8).double() * torch.pow(2.0, (sf // 8 - 10).double()))
    return torch.where(code >= 8, -mag, mag) * step.repeat_interleave(16, 2)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "attend":
        return _exact_attend(c, s)
    a = (s["table"], s["pos"], c["rot"], c["pairs"])
    if c["op"] == "grad":
        got = {}
        for n, x, w, d in (("q", s["q"], s["qw"], s["dqo"]), ("k", s["k"], s["kw"], s["dko"])):
            x, w = x.double().requires_grad_(), w.double().requires_grad_()
            at = s["table"][s["pos"].long()].double().unsqueeze(1)
            cos, sin = at.chunk(2, -1)
            y = x * (x.square().mean(-1, keepdim=True) + EPS).pow(-0.5) * w
            d, rot = d.double(), c["rot"]
            if c["pairs"]:
                one, two, d1, d2 = y[..., 0:rot:2], y[..., 1:rot:2], d[..., 0:rot:2], d[..., 1:rot:2]
            else:
                one, two, d1, d2 = y[..., :rot // 2], y[..., rot // 2:rot], d[..., :rot // 2], d[..., rot // 2:rot]
            loss = ((one * cos - two * sin) * d1).sum() + ((two * cos + one * sin) * d2).sum() + (y[..., rot:] * d[..., rot:]).sum()
            got["d" + n], got["d" + n + "w"] = torch.autograd.grad(loss, (x, w))
        return got
    q, k = _turned64(s["q"], s["qw"], *a), _turned64(s["k"], s["kw"], *a)
    if c["op"] == "rope":
        return {"q": q, "k": k}
    kept = (s["slots"] >= 0).view(-1, 1, 1)
    return {"q": q, "k": torch.where(kept, _quantized64(k.bfloat16(), s["kg"]), 0.0),
            "v": torch.where(kept, _quantized64(s["v"], s["vg"]), 0.0)}


def _exact_attend(c, s):
    hq, hk, D, page, window = c["hq"], c["hk"], c["D"], c["page"], c["window"]
    G = hq // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    row = 0
    for b, (m, L) in enumerate(zip(s["new"], s["lens"])):
        for h in range(hk if L else 0):
            tiles = s["pages"][s["table"][b, :-(-L // page)].long(), h].reshape(-1, 18 * D)
            k = _values64(tiles, D, 0).view(-1, D)[:L] / s["kg"].double()
            v = _values64(tiles, D, 1).view(-1, D)[:L] / s["vg"].double()
            for i0 in range(0, m, 1024):  # (a part of the queries at a time)
                i1 = min(m, i0 + 1024)
                q = s["q"][row + i0:row + i1, h * G:(h + 1) * G].double()
                at = L - m + torch.arange(i0, i1, device=DEV).view(-1, 1, 1)
                j = torch.arange(L, device=DEV)
                no = j > at
                if window:
                    no = no | (j <= at - window)
                score = (q.reshape(-1, D) @ k.t() / math.sqrt(D)).view(i1 - i0, G, L).masked_fill_(no, -math.inf)
                some = (~no).any(-1)
                total = torch.logsumexp(score, -1)
                p = torch.where(some.unsqueeze(-1), (score - total.unsqueeze(-1)).exp(), 0.0)
                out[row + i0:row + i1, h * G:(h + 1) * G] = (p.view(-1, L) @ v).view(-1, G, D)
                lse[row + i0:row + i1, h * G:(h + 1) * G] = total
        row += m
    return {"out": out, "lse": lse}
