"""The rotary call's rounding, and the runs of heads that it takes together in long calls."""
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def _formula(x, w, pos, table, pairs):
    """The documented order in fp32, an operation at a time: the squares in 32 sums that are added in pairs,
    n = (x r) w, then (a c - b s, b c + a s), then bf16."""
    n = x.float()
    D = x.shape[-1]
    if w is not None:
        sums = torch.zeros(*x.shape[:-1], 32, device=x.device)
        for j in range(0, D, 32):
            part = n[..., j:j + 32].square()
            sums[..., :part.shape[-1]] += part
        while sums.shape[-1] > 1:
            sums = sums[..., 0::2] + sums[..., 1::2]
        n = n * torch.rsqrt(sums * (1.0 / D) + EPS) * w.float()
    at = table[pos.long()]
    rot = at.shape[1]
    c, s = at[:, None, :rot // 2], at[:, None, rot // 2:]
    a, b = ref.pair_of(rot, pairs)
    na, nb = n[..., a], n[..., b]
    y = n.clone()
    y[..., a], y[..., b] = na * c - nb * s, nb * c + na * s
    return y.bfloat16()


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("D,rot", [(256, 256), (128, 128), (128, 64), (64, 64), (32, 16), (16, 16), (48, 32), (80, 80), (144, 64), (208, 208)])
def test_bits_of_the_documented_order(dev, D, rot, norm, pairs):
    """Keys and the cache bit for bit.  The queries hold whole numbers up to 7: their squares' sum, at most 49 * 256, is exact
    in fp32 in any order."""
    T, hq, hk, page, far = 2000, 8, 8, 64, 700
    g = torch.Generator(device=dev).manual_seed(D + rot)
    q = torch.randint(-7, 8, (T, hq, D), generator=g, device=dev).bfloat16()
    k, v = ((2.0 * torch.randn(T, hk, D, generator=g, device=dev)).bfloat16() for _ in range(2))
    qw, kw = ((0.5 + torch.rand(D, generator=g, device=dev)).bfloat16() if norm else None for _ in range(2))
    pos = torch.randint(0, far, (T,), generator=g, device=dev).int()
    table = ref.angles(far, rot).to(dev)
    slots = torch.randperm(-(-T // page) * page, generator=g, device=dev)[:T].int()
    scales = torch.tensor([300.0], device=dev), torch.tensor([411.0], device=dev)
    cache = pkg.ts_kv_cache(-(-T // page), hk, D, *scales, page_size=page, device=dev)
    plain = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, interleaved=pairs)
    kept = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, interleaved=pairs, v=v, cache=cache, slots=slots, k_out=torch.empty_like(k))
    for x, w, got in ((q, qw, (plain[0], kept[0])), (k, kw, (plain[1], kept[1]))):
        want = _formula(x, w, pos, table, pairs)
        assert all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for o in got)
    pages = torch.zeros_like(cache.pages).cpu().numpy()
    ref.put(pages, page, slots.cpu().numpy(), _formula(k, kw, pos, table, pairs).float().cpu().numpy(), v.float().cpu().numpy(), 300.0, 411.0)
    assert torch.equal(cache.pages.cpu(), torch.from_numpy(pages))


@pytest.mark.parametrize("pairs", [False, True])
def test_columns_that_are_not_turned_stay(dev, pairs):
    """Bit for bit without a norm, whatever they hold: zeros keep their sign, infinities stay."""
    T, h, D, rot = 50, 3, 64, 32
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(T, h, D, generator=g, device=dev).bfloat16()
    x[..., 33::7], x[..., 35::9], x[..., 40::11] = -0.0, float("inf"), float("-inf")
    pos = torch.arange(T, device=dev).int()
    got = pkg.ts_qk_norm_rope(x, x, None, None, pos, ref.angles(T, rot).to(dev), EPS, interleaved=pairs)
    for y in got:
        assert torch.equal(y[..., rot:].view(torch.int16), x[..., rot:].contiguous().view(torch.int16))
        assert bool(torch.isfinite(y[..., :rot]).all())


# (tokens, query heads, key heads, D): runs of 5 heads, then of 16 (tokens * heads * lanes of a row / (152 * 1024), at
# most 16), the last one of a token shorter; as many blocks of keys as of queries, more and fewer
RUNS = [(5700, 6, 6, 64), (4100, 13, 13, 128), (16000, 20, 3, 64), (16000, 2, 19, 64), (33000, 17, 1, 128)]


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("T,hq,hk,D", RUNS)
def test_long_calls_as_short_ones(dev, T, hq, hk, D, kept):
    """Long calls take several heads of a token together; a token's bits are those of a call of few tokens, and of its
    formula (a sample of the tokens, the first and last among them)."""
    g = torch.Generator(device=dev).manual_seed(T)
    q, k, v = (torch.randn(T, h, D, generator=g, device=dev).bfloat16() for h in (hq, hk, hk))
    qw, kw = ((0.5 + torch.rand(D, generator=g, device=dev)).bfloat16() for _ in range(2))
    pos, table = torch.randint(0, 700, (T,), generator=g, device=dev).int(), ref.angles(700, D).to(dev)
    at = torch.cat((torch.randperm(T, generator=g, device=dev)[:46], torch.tensor([0, T - 1], device=dev)))
    one, page = torch.tensor([300.0], device=dev), 64
    more, few = {}, {}
    if kept:
        caches = [pkg.ts_kv_cache(-(-T // page), hk, D, one, one, page_size=page, device=dev) for _ in range(2)]
        slots = torch.arange(T, device=dev).int()
        more = dict(v=v, cache=caches[0], slots=slots, k_out=torch.empty_like(k))
        few = dict(v=v[at], cache=caches[1], slots=slots[at], k_out=torch.empty_like(k[at]))
    long = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, **more)
    short = pkg.ts_qk_norm_rope(q[at], k[at], qw, kw, pos[at], table, EPS, **few)
    assert all(torch.equal(a[at], b) for a, b in zip(long, short))
    assert torch.equal(long[1].view(torch.int16), _formula(k, kw, pos, table, False).view(torch.int16))
    want = ref.rope(q, qw, pos, table, EPS, False)
    # a sum of D squares and ten roundings, of terms up to sqrt(2) of the largest; bf16
    assert bool(((long[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + (D + 16) * 2.0 ** -23 * want.abs().amax(-1, keepdim=True)).all())
    if kept:
        got, want = (pkg.ts_kv_cache_read(c, slots[at]) for c in caches)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        codes, sf = pkg.ts_nvfp4_quantize(long[1].reshape(T * hk, D), one)
        values = pkg.ts_nvfp4_dequantize(codes, sf, one).view(T, hk, D)
        assert torch.equal(pkg.ts_kv_cache_read(caches[0], slots)[0].view(torch.int16), values.view(torch.int16))
