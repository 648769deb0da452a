"""Measured cases of the NVFP4 and expert-routing operators, with their plain forms.

Six operators, in the order in which a mixture-of-experts layer on NVFP4 weights uses them:

  quantize  bf16 rows to NVFP4 codes and scale factors, and the values read back
  gemm      the product of two NVFP4 matrices
  dispatch  token rows sorted by expert (as bf16, or as NVFP4)
  experts   each expert's NVFP4 product with its own rows
  combine   the experts' rows weighted and summed back into token order
  grad      the gradient of `combine`

`own` chooses between the plain form (elementary torch operations, fp32) and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
F4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of E2M1
LINEAR, SWIZZLED_128x4, SWIZZLED_8x4 = "linear", "128x4", "8x4"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoded token quantised ahead of a projection: latency
        dict(name="quantize_one_token", op="quantize", T=1, K=4096, layout=LINEAR),
        # a long prompt's activations, in the layout the product reads
        dict(name="quantize_prompt", op="quantize", T=16384, K=5120, layout=SWIZZLED_128x4),
        # a projection of one decoded token: the weights' bytes and latency
        dict(name="gemm_one_token", op="gemm", M=1, N=4096, K=4096),
        # the largest projection, an odd number of tokens
        dict(name="gemm_prompt", op="gemm", M=8191, N=7168, K=7168),
        # a decode batch's rows sorted by expert
        dict(name="dispatch_decode", op="dispatch", T=16, k=8, E=64, total=64, H=7168, fp4=False),
        # a prompt's rows sorted by expert and quantised on the way
        dict(name="dispatch_prompt_fp4", op="dispatch", T=4096, k=8, E=64, total=64, H=7168, fp4=True),
        # a decode batch through the experts: every chosen expert's weights are read for a row or a few
        dict(name="experts_decode", op="experts", T=16, k=8, E=64, total=64, N=4096, K=7168),
        # a prompt through half of the experts (the others live on another rank)
        dict(name="experts_prompt", op="experts", T=8192, k=8, E=32, total=64, N=4096, K=7168),
        # a decode batch's rows weighted and summed
        dict(name="combine_decode", op="combine", T=16, k=8, E=64, total=64, H=7168),
        # a prompt's rows weighted and summed
        dict(name="combine_prompt", op="combine", T=8192, k=8, E=64, total=64, H=7168),
        # a short sequence of a training step, an odd number of tokens
        dict(name="grad_short", op="grad", T=77, k=6, E=40, total=40, H=4096),
        # a training step's tokens
        dict(name="grad_batch", op="grad", T=4096, k=8, E=64, total=64, H=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, of):
    return min(hi, max(lo, (_log(rng, lo, hi) + of // 2) // of * of))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "dispatch", "experts", "combine", "grad"))
    if op == "quantize":
        K = _multiple(rng, 64, 8192, 16)
        return dict(op=op, T=_log(rng, 1, min(16384, 16384 * 5120 // K)), K=K,
                    layout=rng.choice((LINEAR, SWIZZLED_128x4, SWIZZLED_8x4)))
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 8191), N=_multiple(rng, 64, 7168, 8), K=_multiple(rng, 64, 7168, 32))
    E = _log(rng, 4, 64)
    k = rng.randint(1, min(8, E))
    total = E * rng.choice((1, 1, 2))
    if op == "experts":
        return dict(op=op, T=_log(rng, 1, 4096), k=k, E=E, total=total, N=_multiple(rng, 128, 4096, 8),
                    K=_multiple(rng, 128, 7168, 32))
    if op == "dispatch":
        return dict(op=op, T=_log(rng, 1, 4096), k=k, E=E, total=total, H=_multiple(rng, 128, 7168, 16),
                    fp4=rng.choice((False, True)))
    return dict(op=op, T=_log(rng, 1, 8192 if op == "combine" else 4096), k=k, E=E, total=total,
                H=_multiple(rng, 128, 7168, 8))


def _up(n, m):
    return (n + m - 1) // m * m


def _sf_bytes(T, K, layout):
    if layout == LINEAR:
        return T * (K // 16)
    return _up(T, 128 if layout == SWIZZLED_128x4 else 8) * _up(K // 16, 4)


def _held(c):
    """The expected number of (token, slot) entries whose expert is held here."""
    return c["T"] * c["k"] * c["E"] / c["total"]


def work(case):
    c = case
    if c["op"] == "quantize":  # read bf16, write codes and scale factors, read them, write bf16
        n, f4 = c["T"] * c["K"], c["T"] * c["K"] / 2 + _sf_bytes(c["T"], c["K"], c["layout"])
        return {"bytes": 4 * n + 2 * f4, "flops": 4 * n}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * K * 9 / 16 + 2 * M * N, "flops": 2 * M * N * K}
    n = _held(c)
    if c["op"] == "dispatch":
        H, ids = c["H"], 4 * c["T"] * c["k"]
        rows = n * H * 9 / 16 * 2 + 2 * n * H if c["fp4"] else 2 * n * H
        return {"bytes": 2 * c["T"] * H + rows + 3 * ids, "flops": 3 * n * H if c["fp4"] else 0}
    if c["op"] == "experts":
        touched = c["E"] * (1 - (1 - 1 / c["total"]) ** (c["T"] * c["k"]))
        return {"bytes": (n + touched * c["N"]) * c["K"] * 9 / 16 + 2 * n * c["N"], "flops": 2 * n * c["N"] * c["K"]}
    entries = 8 * c["T"] * c["k"]
    if c["op"] == "combine":
        return {"bytes": 2 * n * c["H"] + 2 * c["T"] * c["H"] + entries, "flops": 2 * n * c["H"]}
    # grad: dout once, y once, dy once, the weights and their gradient
    return {"bytes": 2 * c["T"] * c["H"] + 4 * n * c["H"] + 12 * c["T"] * c["k"], "flops": 3 * n * c["H"]}


# ---------------------------------------------------------------------------
# NVFP4 in plain torch
# ---------------------------------------------------------------------------

def _swizzle(sf, layout):
    """Scale factors [T, K/16] in a layout's order, padding 0."""
    T, n = sf.shape
    if layout == LINEAR:
        return sf
    tile = 128 if layout == SWIZZLED_128x4 else 8
    p = torch.zeros(_up(T, tile), _up(n, 4), dtype=sf.dtype, device=sf.device)
    p[:T, :n] = sf
    if layout == SWIZZLED_128x4:
        q = p.view(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    else:
        q = p.view(-1, 8, p.shape[1] // 4, 4).permute(0, 2, 1, 3)
    return q.reshape(p.shape)


def _unswizzle(buf, T, n, layout):
    """The inverse of _swizzle, for one buffer or a batch [E, rows, columns] of them."""
    if layout == LINEAR:
        return buf
    lead, (R, C) = buf.shape[:-2], buf.shape[-2:]
    if layout == SWIZZLED_128x4:
        p = buf.reshape(-1, R // 128, C // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    else:
        p = buf.reshape(-1, R // 8, C // 4, 8, 4).permute(0, 1, 3, 2, 4)
    return p.reshape(*lead, R, C)[..., :T, :n]


def _encode(x, g):
    """(codes 0..15 as uint8 [T, K], scale factors as e4m3 [T, K/16]) of bf16 rows."""
    v = x.float().view(x.shape[0], -1, 16)
    amax = v.abs().amax(-1)
    sf = (g * (amax / torch.full_like(g, 6.0))).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = sf.float()
    es = torch.where(d != 0, g / d, torch.zeros_like(d))
    n = v * es.unsqueeze(-1)
    a = n.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * ((n < 0) | ((n == 0) & torch.signbit(n)) & (d != 0).unsqueeze(-1)).to(torch.uint8)
    return code.view(x.shape), sf


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(packed, dtype=torch.float32):
    """The E2M1 values [.., K] of packed codes [.., K/2]."""
    table = torch.tensor(F4 + tuple(-v for v in F4), dtype=dtype, device=packed.device)
    both = torch.stack((packed & 15, packed >> 4), -1)
    return table[both.long()].flatten(-2)


def _decode(packed, sf, dtype=torch.float32):
    """code * scale factor (exact) of packed codes and their e4m3 scale factors [.., K/16]."""
    v = _values(packed, dtype)
    return (v.unflatten(-1, (-1, 16)) * sf.to(dtype).unsqueeze(-1)).flatten(-2)


def _global_scale(x, gen):
    """A calibrated global scale: room for amax up to a factor that other data asked for."""
    room = 1.0 + 0.3 * torch.rand(1, generator=gen, device=DEV)
    return (448.0 * 6.0) / (room * x.abs().amax().float().clamp(min=1e-30))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _activations(T, H, gen):
    """bf16 rows as a norm leaves them: about unit, with a few columns that stand out."""
    x = torch.randn(T, H, generator=gen, device=DEV)
    x *= torch.where(torch.rand(H, generator=gen, device=DEV) < 0.002, 20.0, 1.0)
    return x.bfloat16()


def _fp4_matrix(rows, K, gen, weights):
    """A quantised matrix as a program holds it: packed codes, swizzled scale factors, 1 / its global scale."""
    x = (torch.randn(rows, K, generator=gen, device=DEV) / math.sqrt(K)).bfloat16() if weights else _activations(rows, K, gen)
    g = _global_scale(x, gen)
    code, sf = _encode(x, g)
    return _pack(code), _swizzle(sf.view(torch.uint8), SWIZZLED_128x4), 1.0 / g


def _routing(c, gen):
    """int32 ids [T, k] of distinct experts, some of them busier than others; -1 where the expert is not held here."""
    logits = torch.randn(c["T"], c["total"], generator=gen, device=DEV)
    logits += 0.7 * torch.randn(c["total"], generator=gen, device=DEV)
    w, ids = logits.topk(c["k"], dim=1)
    ids = torch.where(ids < c["E"], ids, -1).int()
    return ids.contiguous(), torch.softmax(w, 1).contiguous()


def _capacity(c, align):
    n = c["T"] * c["k"]
    return _up(n + min(n, c["E"]) * (align - 1), align)


def _sorted_rows(ids, E, align, cap):
    """The stable order of the entries by expert, each expert's rows starting at a multiple of `align`."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    count = (key.unsqueeze(0) == torch.arange(E, device=ids.device).unsqueeze(1)).sum(1)
    padded = (count + align - 1) // align * align
    start = torch.cat((torch.zeros(1, dtype=torch.long, device=ids.device), padded.cumsum(0)))
    first = torch.cat((count.new_zeros(1), count.cumsum(0)))  # without padding
    e = key[order]
    place = torch.arange(T * k, device=ids.device) - first[e]
    dest = torch.where(e < E, start[e.clamp(max=E - 1)] + place, -1)
    row_of = torch.empty_like(flat).scatter_(0, order, dest)
    src = torch.full((cap + 1,), -1, dtype=torch.int32, device=ids.device)
    src[torch.where(dest >= 0, dest, cap)] = torch.where(dest >= 0, order, -1).int()
    return row_of.int().view(T, k), src[:cap].contiguous(), start.int(), count.int()


def prepare(case, seed):
    c, gen = case, torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quantize":
        s["x"] = _activations(c["T"], c["K"], gen)
        s["g"] = _global_scale(s["x"], gen)
        return s
    if c["op"] == "gemm":
        s["a"], s["a_sf"], ra = _fp4_matrix(c["M"], c["K"], gen, False)
        s["b"], s["b_sf"], rb = _fp4_matrix(c["N"], c["K"], gen, True)
        s["alpha"] = ra * rb
        return s
    s["ids"], s["w"] = _routing(c, gen)
    if c["op"] == "dispatch":
        align = 128 if c["fp4"] else 1
        cap = _capacity(c, align)
        s["x"] = _activations(c["T"], c["H"], gen)
        s["g"] = _global_scale(s["x"], gen)
        s["out"] = torch.zeros(cap, c["H"], dtype=torch.bfloat16, device=DEV)
        if c["fp4"]:
            s["codes"] = torch.zeros(cap, c["H"] // 2, dtype=torch.uint8, device=DEV)
            s["sf"] = torch.zeros(cap, _up(c["H"] // 16, 4), dtype=torch.uint8, device=DEV)
        return s
    align = 128 if c["op"] == "experts" else 1
    cap = _capacity(c, align)
    s["rows"] = _sorted_rows(s["ids"], c["E"], align, cap)
    if c["op"] == "experts":
        s["longest"] = max(1, int(s["rows"][3].max()))
        x = _activations(c["T"], c["K"], gen)
        g = _global_scale(x, gen)
        code, sf = _encode(x, g)
        src = s["rows"][1].long()
        token = torch.where(src >= 0, src // c["k"], 0)
        s["a"], s["a_sf"] = _pack(code)[token], _swizzle(sf.view(torch.uint8)[token], SWIZZLED_128x4)
        E, N, K = c["E"], c["N"], c["K"]
        s["b"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
        s["b_sf"] = torch.empty(E, _up(N, 128), _up(K // 16, 4), dtype=torch.uint8, device=DEV)
        s["alpha"] = torch.empty(E, device=DEV)
        for e in range(E):
            s["b"][e], s["b_sf"][e], r = _fp4_matrix(N, K, gen, True)
            s["alpha"][e] = (r / g)[0]
        s["out"] = torch.zeros(cap, N, dtype=torch.bfloat16, device=DEV)
        return s
    s["y"] = torch.randn(cap, c["H"], generator=gen, device=DEV).bfloat16()
    if c["op"] == "grad":
        s["dout"] = torch.randn(c["T"], c["H"], generator=gen, device=DEV).bfloat16()
        s["dy"] = torch.zeros(cap, c["H"], dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass: the library's calls
# ---------------------------------------------------------------------------

def _calls(s):
    import reduce_residual_rmsnorm_gb300 as ts

    c, op = s["case"], s["case"]["op"]
    if op == "quantize":
        layout = {LINEAR: ts.SFLayout.LINEAR, SWIZZLED_128x4: ts.SFLayout.SWIZZLED_128x4,
                  SWIZZLED_8x4: ts.SFLayout.SWIZZLED_8x4}[c["layout"]]
        codes, sf = ts.ts_nvfp4_quantize(s["x"], s["g"], sf_layout=layout, launch_with_pdl=True)
        v = ts.ts_nvfp4_dequantize(codes, sf, s["g"], sf_layout=layout, launch_with_pdl=True)
        return {"values": v, "scale": sf.view(torch.float8_e4m3fn)}
    if op == "gemm":
        return {"out": ts.ts_nvfp4_gemm(s["a"], s["a_sf"], s["b"], s["b_sf"], s["alpha"], launch_with_pdl=True)}
    if op == "dispatch":
        rows = ts.ts_moe_sort(s["ids"], c["E"], row_align=128 if c["fp4"] else 1, launch_with_pdl=True)
        got = {"row_of": rows.row_of, "row_src": rows.row_src, "start": rows.expert_start, "count": rows.expert_count}
        if not c["fp4"]:
            ts.ts_moe_dispatch(s["x"], rows, out=s["out"], launch_with_pdl=True)
            return dict(got, out=s["out"])
        ts.ts_moe_dispatch(s["x"], rows, s["g"], quant_out=s["codes"], scale_out=s["sf"],
                           sf_layout=ts.SFLayout.SWIZZLED_128x4, launch_with_pdl=True)
        ts.ts_nvfp4_dequantize(s["codes"], s["sf"], s["g"], sf_layout=ts.SFLayout.SWIZZLED_128x4,
                               row_src=rows.row_src, out=s["out"], launch_with_pdl=True)
        return dict(got, out=s["out"], scale=s["sf"].view(torch.float8_e4m3fn))
    rows = ts.MoERows(*s["rows"])
    if op == "experts":
        return {"out": ts.ts_nvfp4_grouped_gemm(s["a"], s["a_sf"], s["b"], s["b_sf"], s["alpha"], rows,
                                                out=s["out"], launch_with_pdl=True)}
    if op == "combine":
        return {"out": ts.ts_moe_combine(s["y"], rows, s["w"], launch_with_pdl=True)}
    _, dw = ts.ts_moe_combine_grad(s["dout"], s["y"], rows, s["w"], dy=s["dy"], launch_with_pdl=True)
    return {"dy": s["dy"], "dw": dw}


# ---------------------------------------------------------------------------
# one pass: the plain form
# ---------------------------------------------------------------------------

def _e4m3(buf):
    return buf.view(torch.float8_e4m3fn).float()


def _read_back(code, sf, g):
    return (_decode(_pack(code), sf) / g).bfloat16()


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "quantize":
        code, sf = _encode(s["x"], s["g"])
        return {"values": _read_back(code, sf, s["g"]),
                "scale": _swizzle(sf.view(torch.uint8), c["layout"]).view(torch.float8_e4m3fn)}
    if op == "gemm":
        a = _decode(s["a"], _e4m3(_unswizzle(s["a_sf"], c["M"], c["K"] // 16, SWIZZLED_128x4)))
        b = _decode(s["b"], _e4m3(_unswizzle(s["b_sf"], c["N"], c["K"] // 16, SWIZZLED_128x4)))
        return {"out": (torch.matmul(a, b.t()) * s["alpha"]).bfloat16()}
    if op == "dispatch":
        align = 128 if c["fp4"] else 1
        row_of, src, start, count = _sorted_rows(s["ids"], c["E"], align, s["out"].shape[0])
        got = {"row_of": row_of, "row_src": src, "start": start, "count": count}
        used = (src >= 0).unsqueeze(1)
        token = torch.where(src >= 0, src.long() // c["k"], 0)
        if not c["fp4"]:
            s["out"].copy_(torch.where(used, s["x"][token], s["out"]))
            return dict(got, out=s["out"])
        code, sf = _encode(s["x"], s["g"])
        s["out"].copy_(torch.where(used, _read_back(code, sf, s["g"])[token], s["out"]))
        sf = torch.where(used, sf.view(torch.uint8)[token], 0)
        return dict(got, out=s["out"], scale=_swizzle(sf, SWIZZLED_128x4).view(torch.float8_e4m3fn))
    row_of, src, start, count = s["rows"]
    if op == "experts":
        # every expert's rows padded to the longest's number of them, one batched product
        E, N, K = c["E"], c["N"], c["K"]
        at = torch.arange(s["longest"], device=DEV)
        live = at < count.unsqueeze(1)
        row = torch.where(live, start[:E].unsqueeze(1) + at, 0).long()
        a = _decode(s["a"], _e4m3(_unswizzle(s["a_sf"], s["a"].shape[0], K // 16, SWIZZLED_128x4)))
        b = _decode(s["b"], _e4m3(_unswizzle(s["b_sf"], N, K // 16, SWIZZLED_128x4)))
        y = torch.bmm(a[row], b.transpose(1, 2)) * s["alpha"].view(E, 1, 1)
        s["out"][row[live]] = y[live].bfloat16()
        return {"out": s["out"]}
    held = row_of >= 0
    y = torch.where(held.unsqueeze(2), s["y"][row_of.clamp(min=0).long()].float(), 0.0)
    if op == "combine":
        return {"out": (s["w"].unsqueeze(2) * y).sum(1).bfloat16()}
    d = s["dout"].float().unsqueeze(1)
    s["dy"][row_of[held].long()] = (s["w"].unsqueeze(2) * d).bfloat16()[held]
    return {"dy": s["dy"], "dw": (d * y).sum(2)}


def run(state):
    if own:
        return _calls(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _matrix64(packed, sf_buf):
    """The values [rows, K] that packed codes and 128x4-swizzled scale factors stand for, by the byte offsets' formula."""
    rows, K = packed.shape[0], packed.shape[1] * 2
    m = torch.arange(rows, device=DEV).unsqueeze(1)
    k = torch.arange(K // 16, device=DEV).unsqueeze(0)
    wide = (K // 16 + 3) // 4
    at = ((m // 128) * wide + k // 4) * 512 + (m % 32) * 16 + ((m % 128) // 32) * 4 + k % 4
    byte = sf_buf.reshape(-1)[at].long()
    sf = torch.where(byte >> 3 == 0, (byte & 7) * 2.0 ** -9,
                     (8 + (byte & 7)).double() * torch.pow(2.0, ((byte >> 3) - 10).double()))
    half = torch.empty(rows, K, dtype=torch.long, device=DEV)
    half[:, 0::2], half[:, 1::2] = packed & 15, packed >> 4
    e, f = (half >> 1) & 3, half & 1
    mag = torch.where(e == 0, f * 0.5, (2 + f).double() * torch.pow(2.0, (e - 2).double()))
    return torch.where(half >= 8, -mag, mag) * sf.repeat_interleave(16, 1)


def _nearest(v, grid):
    """The nearest value of an ascending grid to each v >= 0, ties to the even index, the last one above the end."""
    hi = torch.searchsorted(grid, v).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up = (grid[hi] - v < v - grid[lo]) | ((grid[hi] - v == v - grid[lo]) & (hi % 2 == 0))
    return torch.where(up | (lo == hi), grid[hi], grid[lo])


def _quantized64(x, g):
    """(values, scale factors) of rows by the definition: sf = e4m3(g amax / 6), e2m1(x g / sf) sf / g."""
    steps = torch.tensor([(f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)) for e in range(16) for f in range(8)][:127],
                         dtype=torch.float64, device=DEV)
    f4 = torch.tensor(F4, dtype=torch.float64, device=DEV)
    v = x.double().reshape(x.shape[0], -1, 16)
    sf = _nearest(g.double() * v.abs().amax(2) / 6, steps)
    by = torch.where(sf > 0, g.double() / sf, 0.0).unsqueeze(2)
    code = _nearest(v.abs() * by, f4) * torch.sign(v)
    return (code * sf.unsqueeze(2) / g.double()).reshape(x.shape), sf


def _laid_out(sf, layout):
    """Scale factors [T, n] put at their byte offsets, one by one."""
    T, n = sf.shape
    if layout == LINEAR:
        return sf
    m, k = torch.arange(T, device=DEV).unsqueeze(1), torch.arange(n, device=DEV).unsqueeze(0)
    wide = (n + 3) // 4
    if layout == SWIZZLED_128x4:
        at = ((m // 128) * wide + k // 4) * 512 + (m % 32) * 16 + ((m % 128) // 32) * 4 + k % 4
        rows = (T + 127) // 128 * 128
    else:
        at = ((m // 8) * wide + k // 4) * 32 + (m % 8) * 4 + k % 4
        rows = (T + 7) // 8 * 8
    buf = torch.zeros(rows * wide * 4, dtype=sf.dtype, device=DEV)
    buf[at.reshape(-1)] = sf.reshape(-1)
    return buf.view(rows, wide * 4)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        v, sf = _quantized64(s["x"], s["g"])
        return {"values": v, "scale": _laid_out(sf, c["layout"])}
    if c["op"] == "gemm":
        return {"out": torch.mm(_matrix64(s["a"], s["a_sf"]), _matrix64(s["b"], s["b_sf"]).t()) * s["alpha"].double()}
    T, k, E = c["T"], c["k"], c["E"]
    ids = s["ids"].cpu().tolist()
    if c["op"] == "dispatch":
        align, cap, H = 128 if c["fp4"] else 1, s["out"].shape[0], c["H"]
        of = [[] for _ in range(E)]
        for t in range(T):
            for j in range(k):
                if 0 <= ids[t][j] < E:
                    of[ids[t][j]].append(t * k + j)
        row_of, src, start = [-1] * (T * k), [-1] * cap, [0]
        for e in range(E):
            for i, n in enumerate(of[e]):
                row_of[n], src[start[-1] + i] = start[-1] + i, n
            start.append(start[-1] + (len(of[e]) + align - 1) // align * align)
        whole = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        got = {"row_of": whole(row_of).view(T, k), "row_src": whole(src), "start": whole(start),
               "count": whole([len(o) for o in of])}
        at = torch.tensor([r for r in range(cap) if src[r] >= 0], dtype=torch.long, device=DEV)
        token = torch.tensor([v // k for v in src if v >= 0], dtype=torch.long, device=DEV)
        out = torch.zeros(cap, H, dtype=torch.float64, device=DEV)
        if not c["fp4"]:
            out[at] = s["x"].double()[token]
            return dict(got, out=out)
        v, sf = _quantized64(s["x"], s["g"])
        out[at] = v[token]
        rows_sf = torch.zeros(cap, H // 16, dtype=torch.float64, device=DEV)
        rows_sf[at] = sf[token]
        return dict(got, out=out, scale=_laid_out(rows_sf, SWIZZLED_128x4))
    start, count = s["rows"][2].tolist(), s["rows"][3].tolist()
    if c["op"] == "experts":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for e in range(E):
            if count[e]:
                r0 = start[e]  # a multiple of 128: the expert's scale factors begin on a tile row
                a = _matrix64(s["a"][r0:r0 + count[e]], s["a_sf"][r0:])
                out[r0:r0 + count[e]] = torch.mm(a, _matrix64(s["b"][e], s["b_sf"][e]).t()) * s["alpha"][e].double()
        return {"out": out}
    row_of, y, w = s["rows"][0].long(), s["y"].double(), s["w"].double()
    out = torch.zeros(T, c["H"], dtype=torch.float64, device=DEV)
    if c["op"] == "combine":
        for j in range(k):
            t = (row_of[:, j] >= 0).nonzero().squeeze(1)
            out[t] += w[t, j].unsqueeze(1) * y[row_of[t, j]]
        return {"out": out}
    d = s["dout"].double()
    dy = torch.zeros(y.shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        t = (row_of[:, j] >= 0).nonzero().squeeze(1)
        dy[row_of[t, j]] = w[t, j].unsqueeze(1) * d[t]
        dw[t, j] = (d[t] * y[row_of[t, j]]).sum(1)
    return {"dy": dy, "dw": dw}
