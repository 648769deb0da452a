"""Plain 64-bit NVFP4 and expert-routing references for the tests (numpy / torch, written from the definitions)."""
import numpy as np
import torch

F4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(f / 8) * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7) for e in range(16) for f in range(8)])
E4M3[127] = np.nan


def up(n, m):
    return (n + m - 1) // m * m


def sf_places(T, n, layout):
    """Byte offset of scale factor (t, j) and the buffer's shape, layout 0 128x4, 1 8x4, 2 linear."""
    m, k = np.arange(T)[:, None], np.arange(n)[None, :]
    if layout == 2:
        return m * n + k, (T, n)
    w = up(n, 4) // 4
    if layout == 0:
        return ((m // 128) * w + k // 4) * 512 + (m % 32) * 16 + ((m % 128) // 32) * 4 + k % 4, (up(T, 128), 4 * w)
    return ((m // 8) * w + k // 4) * 32 + (m % 8) * 4 + k % 4, (up(T, 8), 4 * w)


def lay_out(sf, layout, fill=0):
    """Scale-factor bytes [T, n] in a layout; other bytes are `fill`."""
    at, shape = sf_places(*sf.shape, layout)
    buf = np.full(shape[0] * shape[1], fill, np.uint8)
    buf[at] = sf
    return buf.reshape(shape)


def pick(buf, T, n, layout):
    at, shape = sf_places(T, n, layout)
    assert tuple(buf.shape) == shape, (buf.shape, shape)
    return np.ascontiguousarray(buf).reshape(-1)[at]


def unpack(codes):
    out = np.empty((*codes.shape[:-1], codes.shape[-1] * 2), np.uint8)
    out[..., 0::2], out[..., 1::2] = codes & 15, codes >> 4
    return out


def pack(nibbles):
    return (nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)).astype(np.uint8)


def values(codes, sf):
    """float64 e2m1 * e4m3 of packed codes [.., K/2] and scale-factor bytes [.., K/16]."""
    n = unpack(codes)
    v = np.where(n >= 8, -F4[n & 7], F4[n & 7])
    return v * np.repeat(E4M3[sf & 127], 16, axis=-1)


def nearest(v, grid):
    """Index of the nearest grid value, ties to the even index, for v >= 0."""
    hi = np.clip(np.searchsorted(grid, v), 0, len(grid) - 1)
    lo = np.clip(hi - 1, 0, None)
    dh, dl = grid[hi] - v, v - grid[lo]
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo).astype(np.uint8)


def quantize(x, g):
    """(nibbles [T, K], scale-factor bytes [T, K/16]) of float values by the definition, each step rounded to fp32."""
    f = np.float32
    x = np.asarray(x, f)
    b = x.reshape(x.shape[0], -1, 16)
    with np.errstate(over="ignore"):
        amax = np.abs(b).max(-1)
        sf = nearest(np.minimum((f(g) * (amax / f(6))).astype(f).astype(np.float64), 448.0), E4M3[:127])
        d = E4M3[sf].astype(f)
        es = np.divide(f(g), d, out=np.zeros_like(d), where=d != 0)
        n = (b * es[..., None]).astype(f)
    code = nearest(np.minimum(np.abs(n), 6).astype(np.float64), F4)
    code = code | np.where(np.signbit(n) & (d != 0)[..., None], 8, 0).astype(np.uint8)
    return code.reshape(x.shape), sf


def sort_rows(ids, E, align, cap):
    """(row_of, row_src, start, count) of ids [T, k] by the definition, one entry after the other."""
    T, k = ids.shape
    of = [[] for _ in range(E)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            of[e].append(i)
    row_of, src, start = np.full(T * k, -1, np.int32), np.full(cap, -1, np.int32), [0]
    for e in range(E):
        for j, i in enumerate(of[e]):
            row_of[i] = start[-1] + j
            src[start[-1] + j] = i
        start.append(start[-1] + up(len(of[e]), align))
    return row_of.reshape(T, k), src, np.array(start, np.int32), np.array([len(o) for o in of], np.int32)


def random_nvfp4(rows, K, seed, dev, sf_codes=None):
    """Random codes [rows, K/2], scale-factor bytes [rows, K/16] (from `sf_codes`, else a spread of finite ones),
    on the CPU, and both on `dev` with the scale factors in the 128x4 layout."""
    r = np.random.RandomState(seed)
    codes = r.randint(0, 256, (rows, K // 2)).astype(np.uint8)
    sf = np.asarray(sf_codes, np.uint8)[r.randint(0, len(sf_codes), (rows, K // 16))] if sf_codes is not None else \
        r.randint(40, 90, (rows, K // 16)).astype(np.uint8)
    return codes, sf, torch.from_numpy(codes).to(dev), torch.from_numpy(lay_out(sf, 0)).to(dev)


# 2^-1, 1, 2, 4 and 1.5: with E2M1 values every product is a multiple of 2^-4
EXACT_SF = [6 << 3, 7 << 3, 8 << 3, 9 << 3, (7 << 3) | 4]
