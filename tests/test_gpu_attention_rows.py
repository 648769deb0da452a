"""Rows of queries and bounds that attention may meet at the ends of their ranges, in each way to split the work."""
import math

import numpy as np
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from tests import attention_ref as ref
from tests.test_gpu_attention import _cache, _close, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


# queries and lengths of the sequences: units by clusters (of 8, 16 and 32 rows), by even shares, on the fifth-generation
# tensor cores in one piece and in shares
FORMS = {"cluster": ([1, 1, 1, 1], [300, 17, 0, 1]), "cluster16": ([3, 2, 0, 4], [150, 40, 9, 2]), "cluster32": ([7, 8, 5], [90, 200, 3]),
         "shares": ([1, 1, 1], [17000, 33, 700]), "shares32": ([6, 8, 3], [17001, 40, 1]), "prompt": ([70, 130, 20], [200, 150, 10]),
         "prompt_shares": ([40, 33], [20001, 300])}


def _call(dev, q, cache, table, lens, new, scale=None, **args):
    """(out, lse) and the reference's four."""
    cu = np.concatenate(([0], np.cumsum(new)))
    got = pkg.ts_nvfp4_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=dev), torch.from_numpy(cu).int().to(dev),
                                 max_q=max(new), scale=scale, return_lse=True, **args)
    real = 1 / math.sqrt(q.shape[2]) if scale is None else float(torch.tensor(scale, dtype=torch.float32))
    return got, ref.attention(q, cache.pages, cache.k_scale.double(), cache.v_scale.double(), table, lens, cu, real,
                              args.get("causal", True), args.get("window", 0))


def _check(got, want):
    out, lse, slack, slack_lse = want
    _close(got[0], out, slack, "out")
    none = torch.isinf(lse)
    assert torch.equal(torch.isneginf(got[1]), none)
    assert bool(((got[1].double() - lse).abs()[~none] <= slack_lse[~none]).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("k_scale,scale,spread", [(1e7, None, 4e4), (300.0, 1e-30, 1.0), (300.0, 1e-45, 1.0), (1e7, 1e-37, 3e37),
                                                  (1e30, None, 1e25), (300.0, 1e-38, 1e36)])
@pytest.mark.parametrize("form", FORMS)
def test_rows_of_zeros_and_tiny_factors(dev, form, k_scale, scale, spread, window, D):
    """A row of zeros (padding) sees the mean of V, whatever the other rows, the scales and the mask are; so does any row
    whose scores all come out at zero."""
    new, lens = FORMS[form]
    cache, table = _cache(dev, lens, 2, D, 32, 5)
    cache = pkg.KVCache(cache.pages, torch.tensor([k_scale], device=dev), cache.v_scale)
    if len(lens) > 1 and lens[1] > 32:
        table[1, 1] = -1  # a page that is not there
    q = _rand((sum(new), 8, D), dev, 3, spread)
    q[::2, 1::3] = 0.0
    q[1::2, ::5] = 0.0
    got, want = _call(dev, q, cache, table, lens, new, scale, window=window)
    _check(got, want)
    assert bool(torch.isfinite(got[0]).all()) and not bool(torch.isnan(got[1]).any())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 30 + 1, 2 ** 30])
def test_windows_that_bound_nothing(dev, window, D):
    """Windows beyond every length give the bits of none, also where queries stand in front of the first key."""
    for new, lens in (([20, 150, 3], [10, 100, 2]), ([600, 40], [300, 20]), ([5, 3, 7], [3, 1, 50]), ([2, 4], [1, 2])):
        cache, table = _cache(dev, lens, 2, D, 32, 5)
        q = _rand((sum(new), 8, D), dev, 3)
        args = dict(cu_q=torch.tensor([0, *np.cumsum(new)], dtype=torch.int32, device=dev), max_q=max(new), return_lse=True)
        kv = torch.tensor(lens, dtype=torch.int32, device=dev)
        want, got = (pkg.ts_nvfp4_attention(q, cache, table, kv, window=w, **args) for w in (0, window))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("v_scale", [1e36, 1e30, 1e-30])
@pytest.mark.parametrize("form", FORMS)
def test_scales_of_values(dev, form, v_scale, D):
    """Values of any magnitude that their scale gives come out, however large the sum of a row is."""
    new, lens = FORMS[form]
    cache, table = _cache(dev, lens, 2, D, 32, 5)
    cache = pkg.KVCache(cache.pages, cache.k_scale, torch.tensor([v_scale], device=dev))
    q = _rand((sum(new), 8, D), dev, 3, 0.01)  # (nearly equal weights: a sum as large as the length)
    _check(*_call(dev, q, cache, table, lens, new))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [18.62, 21.62, 22.62, 24.62, 26.62])
@pytest.mark.parametrize("new,lens", [([1] * 20, [3000] * 20), ([4] * 20, [2500] * 20), ([200], [20000]), ([40], [33000])],
                         ids=["single", "few", "prompt", "prompt_far"])
def test_one_key_that_outweighs_the_others(dev, new, lens, far, D):
    """A key with the weight of 2^far others and no value of its own: the output is made of the small weights.

    A weight is rounded to fp16 as 2^7 times its part of the largest: 2^-11 of it, or 2^-25 / 2^7 of the largest where it
    is subnormal.  The scores' error and the fp32 sums' as in the reference's bounds."""
    hk, G, page = 2, 4, 64
    g = torch.Generator(device=dev).manual_seed(1)
    one = torch.ones(1, device=dev)
    used = [-(-n // page) for n in lens]
    cache = pkg.ts_kv_cache(sum(used), hk, D, one, 1700 * one, page_size=page, device=dev)
    table = torch.arange(sum(used), device=dev).int().view(len(lens), -1)
    slots = (table.long().repeat_interleave(page, 1) * page + torch.arange(page, device=dev).repeat(used[0]))[:, :lens[0]].int().flatten()
    k = torch.zeros(len(lens), lens[0], hk, D, dtype=torch.bfloat16, device=dev)
    v = (0.5 + torch.rand(k.shape, generator=g, device=dev)).bfloat16()
    k[:, 0, :, 0], v[:, 0] = 6.0, 0.0  # (6 is exact in the cache)
    flat = torch.zeros(1, 16, device=dev)
    flat[:, :8] = 1.0
    k, v = k.flatten(0, 1), v.flatten(0, 1)
    pkg.ts_qk_norm_rope(k, k, None, None, torch.zeros(len(k), dtype=torch.int32, device=dev), flat, v=v, cache=cache, slots=slots)
    q = torch.randn(sum(new), hk * G, D, generator=g, device=dev).bfloat16()
    q[..., 0] = 1.0
    scale = far * math.log(2.0) / 6.0
    got, (out, lse, _, slack_lse) = _call(dev, q, cache, table, lens, new, scale)
    values = ref.cached(cache.pages, 1) / 1700.0
    at = 0
    for b, n in enumerate(new):
        all_v = values[table[b].long()].transpose(0, 1).flatten(1, 2)[:, :lens[b]].abs().cumsum(1)  # [hk, keys, D]
        seen = all_v[:, lens[b] - n:lens[b]].transpose(0, 1).repeat_interleave(G, 1)                # of each query
        rows = slice(at, at + n)
        top = torch.exp(scale * 6.0 - lse[rows]).unsqueeze(-1)
        es = (D + 4) * 2.0 ** -23 * scale * 6.0 + 2.0 ** -20
        slack = (2.0 ** -11 + 2.0 ** -18 + 2 * es) * out[rows].abs() + 2.0 ** -32 * top * seen
        _close(got[0][rows], out[rows], slack, "out")
        at += n
    assert bool(((got[1].double() - lse).abs() <= slack_lse).all())
    assert float(out.abs().min()) > 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [1e6, -1e6, 1e8, 4e8, -4e8, 1e9, 3e12, -3e12, 1e30])
@pytest.mark.parametrize("form", FORMS)
def test_scores_of_any_size(dev, form, size, D):
    """Scores whose neighbouring fp32 are far apart: alike they weigh alike, and where one key has twice the others', it
    (or, below zero, the others) has all the weight.  Weights are then equal or zero, so that fp16 and the sums cost
    2^-11 and 2^-16 of the output at most."""
    hk, G, page = 2, 4, 32
    new, lens = FORMS[form]
    g = torch.Generator(device=dev).manual_seed(3)
    one = torch.ones(1, device=dev)
    used = [-(-n // page) for n in lens]
    cache = pkg.ts_kv_cache(max(1, sum(used)), hk, D, one, 1700 * one, page_size=page, device=dev)
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32, device=dev)
    flat = torch.zeros(1, 16, device=dev)
    flat[:, :8] = 1.0
    for b, n in enumerate(lens):
        if n == 0:
            continue
        table[b, :used[b]] = sum(used[:b]) + torch.arange(used[b], device=dev).int()
        k = torch.zeros(n, hk, D, dtype=torch.bfloat16, device=dev)
        k[..., 0] = 3.0
        k[n // 3, 1, 0] = 6.0  # (the first head's keys are all alike)
        v = (0.5 + torch.rand(n, hk, D, generator=g, device=dev)).bfloat16()
        at = torch.arange(n, device=dev)
        slots = (table[b].long()[at // page] * page + at % page).int()
        pkg.ts_qk_norm_rope(k, k, None, None, torch.zeros(n, dtype=torch.int32, device=dev), flat, v=v, cache=cache, slots=slots)
    q = torch.zeros(sum(new), hk * G, D, dtype=torch.bfloat16, device=dev)
    q[..., 0] = size / (3 * 0.125)
    got, _ = _call(dev, q, cache, table, lens, new, 0.125)
    # the scores less their largest, which 64 bits hold whatever their size (lse would lose the logarithm of the sum)
    values, at = ref.cached(cache.pages, 1) / 1700.0, 0
    s0 = float(q[0, 0, 0]) * 0.125 * 3.0 if len(q) else 0.0
    for n, m, ids in zip(lens, new, table):
        for i in range(m):
            seen = max(n - m + i + 1, 0)
            out, lse = got[0][at + i].unflatten(0, (hk, G)), got[1][at + i].view(hk, G)
            if seen == 0:
                assert bool((out == 0).all() and torch.isneginf(lse).all())
                continue
            s = torch.full((hk, seen), s0, dtype=torch.float64, device=dev)
            if n // 3 < seen:
                s[1, n // 3] *= 2
            v = values[ids[:-(-seen // page)].long()].transpose(0, 1).flatten(1, 2)[:, :seen]
            want = torch.einsum("hj,hjd->hd", torch.softmax(s, 1), v).unsqueeze(1)
            _close(out, want.expand(out.shape), (2.0 ** -11 + 2.0 ** -16) * want, "out")
            # (scale, log2 e and the products: a few roundings of the score)
            total = torch.logsumexp(s, 1, keepdim=True)
            assert bool(((lse.double() - total).abs() <= 2.0 ** -21 * total.abs() + 2.0 ** -16).all())
        at += m
