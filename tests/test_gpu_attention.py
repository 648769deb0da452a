"""The rotary, 4-bit cache and attention operators on a GPU against the plain 64-bit references.

Tolerances: an output's rounding to bf16 is at most 2^-8 of it (half a step); what comes before is counted where it is
used.  Where the result is bits (the cache, the cache read back) it is compared bit for bit."""
import math

import numpy as np
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from tests import attention_ref as ref
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def _rand(shape, dev, seed, scale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device=dev)).bfloat16()


def _rope_inputs(dev, T, hq, hk, D, rot, far=700, seed=0, strided=True):
    """q, k, v as columns of one matrix of rows (strided) or on their own, weights, positions, the table."""
    w = (hq + 2 * hk) * D
    if strided:
        rows = _rand((T, w + 24), dev, seed, 2.0)
        q, k, v = (rows[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    else:
        q, k, v = (_rand((T, h, D), dev, seed + i, 2.0) for i, h in enumerate((hq, hk, hk)))
    g = torch.Generator(device=dev).manual_seed(seed + 9)
    qw, kw = ((0.5 + torch.rand(D, generator=g, device=dev)).bfloat16() for _ in range(2))
    pos = torch.randint(0, far, (T,), generator=g, device=dev).int()
    return q, k, v, qw, kw, pos, ref.angles(far, rot).to(dev)


def _close(got, want, slack, what):
    """|got - want| <= 2^-8 |want| + slack, and the same infinities."""
    err = (got.double() - want).abs()
    over = err > 2.0 ** -8 * want.abs() + slack
    assert not bool((over | torch.isnan(err) & ~(torch.isinf(want) & (got == want))).any()), \
        (what, float((err - 2.0 ** -8 * want.abs() - slack).max()))


SHAPES = [(1, 1, 1, 16, 16), (3, 2, 1, 32, 16), (5, 3, 3, 48, 32), (17, 8, 1, 128, 128), (9, 40, 8, 64, 32), (2, 5, 5, 80, 48),
          (33, 6, 2, 256, 64), (70, 4, 2, 112, 112), (600, 64, 8, 128, 64)]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,hq,hk,D,rot", SHAPES)
def test_norm_rope(dev, T, hq, hk, D, rot, norm, pairs):
    q, k, _, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, seed=T + D)
    if not norm:
        qw = kw = None
    qo, ko = Guarded((T, hq, D), torch.bfloat16, dev), Guarded((T, hk, D), torch.bfloat16, dev)
    got = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, interleaved=pairs, q_out=qo.t, k_out=ko.t)
    assert got[0].data_ptr() == qo.t.data_ptr() and got[1].data_ptr() == ko.t.data_ptr()
    for x, w, o in ((q, qw, qo), (k, kw, ko)):
        want = ref.rope(x, w, pos, table, EPS, pairs)
        # the norm: a sum of D squares and five roundings; the turn: three of terms up to sqrt(2) of the largest
        slack = (D + 16) * 2.0 ** -24 * 2 * want.abs().amax(-1, keepdim=True)
        _close(o.t, want, slack, "out")
        assert o.intact()


@pytest.mark.parametrize("pairs", [False, True])
def test_norm_rope_in_place_and_one_row_alike(dev, pairs):
    """In place in the columns of one matrix; a token's bits do not depend on the others (short and long calls)."""
    T, hq, hk, D, rot = 900, 8, 2, 128, 64
    q, k, v, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, seed=3)
    want = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, interleaved=pairs)
    few = pkg.ts_qk_norm_rope(q[100:103], k[100:103], qw, kw, pos[100:103], table, EPS, interleaved=pairs, launch_with_pdl=True)
    assert all(torch.equal(a[100:103], b) for a, b in zip(want, few))
    kept = v.clone()
    got = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, interleaved=pairs, q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)


def test_norm_rope_leaves_out_bad_positions(dev):
    T, hq, hk, D, rot = 40, 4, 2, 64, 64
    q, k, v, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, far=50, seed=4)
    bad = torch.zeros(T, dtype=torch.bool, device=dev)
    for t, p in ((0, -1), (7, 50), (8, 2 ** 31 - 1), (39, -2 ** 31)):
        pos[t], bad[t] = p, True
    qo, ko = torch.full_like(q, 7.0).contiguous(), torch.full_like(k, 7.0).contiguous()
    pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, q_out=qo, k_out=ko)
    good = pkg.ts_qk_norm_rope(q, k, qw, kw, torch.where(bad, 0, pos), table, EPS)
    for o, w in zip((qo, ko), good):
        assert bool((o[bad] == 7.0).all()) and torch.equal(o[~bad], w[~bad])
    # in the gradient such a token's rows stay, and add nothing to the weights
    dq, dk = torch.full_like(qo, 7.0), torch.full_like(ko, 7.0)
    dy = _rand((T, hq, D), dev, 5), _rand((T, hk, D), dev, 6)
    _, _, dqw, dkw = pkg.ts_qk_norm_rope_grad(*dy, q, k, qw, kw, pos, table, EPS, dq=dq, dk=dk)
    keep = ~bad
    want = pkg.ts_qk_norm_rope_grad(*(d[keep].contiguous() for d in dy), q[keep], k[keep], qw, kw, pos[keep], table, EPS)
    assert bool((dq[bad] == 7.0).all() and (dk[bad] == 7.0).all())
    assert torch.equal(dq[keep], want[0]) and torch.equal(dk[keep], want[1])
    assert torch.allclose(dqw, want[2], rtol=1e-5, atol=1e-4) and torch.allclose(dkw, want[3], rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,hq,hk,D,rot", SHAPES)
def test_norm_rope_grad(dev, T, hq, hk, D, rot, norm, pairs):
    q, k, _, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, seed=T + D + 1)
    if not norm:
        qw = kw = None
    dys = _rand((T, hq, D), dev, 11), _rand((T, hk, D), dev, 12)
    dq, dk = Guarded((T, hq, D), torch.bfloat16, dev), Guarded((T, hk, D), torch.bfloat16, dev)
    _, _, dqw, dkw = pkg.ts_qk_norm_rope_grad(*dys, q, k, qw, kw, pos, table, EPS, interleaved=pairs, dq=dq.t, dk=dk.t)
    for x, w, dy, dx, dw in ((q, qw, dys[0], dq, dqw), (k, kw, dys[1], dk, dkw)):
        want, want_w = ref.rope_grad(dy, x, w, pos, table, EPS, pairs)
        # sums of D terms and a few roundings, of terms no larger than r |g| (1 + |x r|^2)
        big = want.abs().amax(-1, keepdim=True)
        if norm:
            r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + EPS)
            big = (r * 4 * dy.double().abs().amax(-1, keepdim=True) * (1 + (x.double() * r).abs().amax(-1, keepdim=True) ** 2))
        _close(dx.t, want, (D + 16) * 2.0 ** -24 * 2 * big, "dx")
        assert dx.intact()
        if norm:
            # fp32 sums of T * heads terms: each term's error and at most 2 sqrt(n) partial sums' steps, of magnitudes' sum
            r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + EPS)
            mag = (2 * dy.double().abs().amax(-1, keepdim=True) * (x.double() * r).abs()).sum((0, 1))
            assert bool(((dw.double() - want_w).abs() <= (D + 64) * 2.0 ** -24 * mag).all())
        else:
            assert dw is None


def test_norm_rope_grad_against_differences(dev):
    """The formula itself: the reference's gradient equals central differences of the reference's forward."""
    T, h, D, rot = 3, 2, 32, 16
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(T, h, D, generator=g, dtype=torch.float64), 0.5 + torch.rand(D, generator=g, dtype=torch.float64)
    dy, pos, table = torch.randn(T, h, D, generator=g, dtype=torch.float64), torch.tensor([5, 0, 77]), ref.angles(100, rot)
    for pairs in (False, True):
        dx, dw = ref.rope_grad(dy, x, w, pos, table, EPS, pairs)
        for i in (0, 7, 17, 40, 100, 191):
            e = torch.zeros_like(x).view(-1)
            e[i] = 1e-5
            up, down = (ref.rope(x + s * e.view(x.shape), w, pos, table, EPS, pairs) for s in (1, -1))
            assert abs(float(((up - down) * dy).sum() / 2e-5 - dx.view(-1)[i])) < 1e-8
        for j in (0, 9, 31):
            e = torch.zeros_like(w)
            e[j] = 1e-5
            up, down = (ref.rope(x, w + s * e, pos, table, EPS, pairs) for s in (1, -1))
            assert abs(float(((up - down) * dy).sum() / 2e-5 - dw[j])) < 1e-8


def test_norm_rope_grad_in_place_and_empty(dev):
    T, hq, hk, D, rot = 300, 6, 2, 64, 32
    q, k, _, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, seed=8)
    dq, dk = _rand((T, hq, D), dev, 1), _rand((T, hk, D), dev, 2)
    want = pkg.ts_qk_norm_rope_grad(dq, dk, q, k, qw, kw, pos, table, EPS)
    got = pkg.ts_qk_norm_rope_grad(dq, dk, q, k, qw, kw, pos, table, EPS, dq=dq, dk=dk, launch_with_pdl=True)
    assert got[0].data_ptr() == dq.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))
    _, _, dqw, dkw = pkg.ts_qk_norm_rope_grad(dq[:0], dk[:0], q[:0], k[:0], qw, kw, pos[:0], table, EPS,
                                              dq_weight=torch.ones(D, device=dev))
    assert bool((dqw == 0).all() and (dkw == 0).all())


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rot", [(37, 6, 2, 64, 32), (9, 3, 1, 48, 16), (2000, 40, 5, 128, 128)])
def test_norm_rope_grad_leaves_out_bad_positions(dev, T, hq, hk, D, rot, pairs):
    """Rows behind a batch's end (positions below zero or past the table) may hold anything: NaN there
    reaches neither the weights' gradient nor another row."""
    q, k, _, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, seed=9)
    dq, dk = _rand((T, hq, D), dev, 1), _rand((T, hk, D), dev, 2)
    out = torch.arange(T, device=dev) % 3 == 1
    pos = torch.where(out, torch.where(torch.arange(T, device=dev) % 2 == 0, -1, table.shape[0]).to(pos.dtype), pos)
    keep = ~out
    want = pkg.ts_qk_norm_rope_grad(dq[keep], dk[keep], q[keep].contiguous(), k[keep].contiguous(), qw, kw, pos[keep].contiguous(),
                                    table, EPS, interleaved=pairs)
    for t in (dq, dk, q, k):
        t[out] = float("nan")
    to = [torch.full((T, h, D), 3.0, dtype=torch.bfloat16, device=dev) for h in (hq, hk)]
    got = pkg.ts_qk_norm_rope_grad(dq, dk, q, k, qw, kw, pos, table, EPS, interleaved=pairs, dq=to[0], dk=to[1])
    for i in (0, 1):
        assert torch.equal(got[i][keep], want[i]) and bool((to[i][out] == 3.0).all())
        # the same terms in another order: twice a sum's error, of the magnitudes' sum (at most sqrt(n) more than the sum's own)
        x, dy = ((q, dq), (k, dk))[i]
        r = torch.rsqrt(x[keep].double().square().mean(-1, keepdim=True) + EPS)
        mag = (2 * dy[keep].double().abs().amax(-1, keepdim=True) * (x[keep].double() * r).abs()).sum((0, 1))
        assert bool(((got[2 + i].double() - want[2 + i].double()).abs() <= 2 * (D + 64) * 2.0 ** -24 * mag).all())


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,hq,hk,D,rot,page", [(1, 1, 1, 16, 16, 16), (5, 3, 1, 48, 32, 48), (40, 8, 2, 128, 64, 16),
                                                (70, 5, 5, 64, 64, 64), (9, 2, 2, 80, 16, 32), (3, 4, 2, 256, 256, 16),
                                                (1500, 8, 8, 128, 128, 128)])
def test_cache_write_and_read(dev, T, hq, hk, D, rot, page):
    """Every byte of the cache against the definition (quantising the kernel's own bf16 keys), the other bytes as they
    were; the cache read back as ts_nvfp4_dequantize reads the same rows."""
    q, k, v, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, seed=T)
    n = T // page + 3
    g = torch.Generator(device=dev).manual_seed(1)
    slots = torch.randperm(n * page, generator=g, device=dev)[:T].int()
    if T > 4:
        slots[1], slots[T // 2], slots[T - 1], pos[2] = -1, n * page, -2 ** 31, -5
    kg, vg = torch.tensor([300.0], device=dev), torch.tensor([411.0], device=dev)
    old = torch.randint(0, 255, (n, hk, page // 16, 18 * D), generator=g, device=dev).to(torch.uint8)
    cache = pkg.KVCache(old.clone(), kg, vg)
    ko = torch.zeros(T, hk, D, dtype=torch.bfloat16, device=dev)
    both = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, v=v, cache=cache, slots=slots, k_out=ko)
    assert both[1].data_ptr() == ko.data_ptr()
    plain = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, q_out=torch.zeros_like(q).contiguous(), k_out=torch.zeros_like(ko))
    live = pos >= 0
    assert torch.equal(both[0][live], plain[0][live]) and torch.equal(ko, plain[1])
    want = old.cpu().numpy()
    kept = torch.where(live, slots, -1).cpu().numpy()
    ref.put(want, page, kept, ko.float().cpu().numpy(), v.float().cpu().numpy(), 300.0, 411.0)
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    # without k_out the same bytes
    alone = pkg.KVCache(old.clone(), kg, vg)
    assert pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, v=v, cache=alone, slots=slots)[1] is None
    assert torch.equal(alone.pages, cache.pages)
    kr, vr = (Guarded((T, hk, D), torch.bfloat16, dev) for _ in range(2))
    pkg.ts_kv_cache_read(cache, slots, k_out=kr.t, v_out=vr.t)
    for x, got, gs in ((ko, kr, kg), (v, vr, vg)):
        codes, sf = pkg.ts_nvfp4_quantize(x.reshape(T * hk, D).contiguous(), gs)
        values = pkg.ts_nvfp4_dequantize(codes, sf, gs).view(T, hk, D)
        ok = live & (slots >= 0) & (slots < n * page)
        assert torch.equal(got.t[ok].view(torch.int16), values[ok].view(torch.int16))
        out = ~((slots >= 0) & (slots < n * page))
        assert bool((got.t[out].view(torch.int16) == -23131).all())  # 0xA5A5: as it was
        assert got.intact()


def test_cache_beyond_4_gib(dev):
    """A cache whose offsets pass 32 bits, written, read and attended at its end."""
    D, hk, page, n = 128, 8, 128, 33000  # 4.9e9 bytes
    pages = torch.zeros(n, hk, page // 16, 18 * D, dtype=torch.uint8, device=dev)
    one = torch.tensor([448.0], device=dev)
    cache = pkg.KVCache(pages, one, one)
    T = 200
    q, k, v, qw, kw, pos, table = _rope_inputs(dev, T, 8, hk, D, 64, seed=5)
    ids = torch.tensor([[n - 1, n - 2]], dtype=torch.int32, device=dev)
    at = torch.arange(T, device=dev)
    slots = (ids[0].long()[at // page] * page + at % page).int()
    qo, ko = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table, EPS, v=v, cache=cache, slots=slots, k_out=torch.empty_like(k).contiguous())
    kr, vr = pkg.ts_kv_cache_read(cache, slots)
    small = pkg.KVCache(pages[n - 2:].clone(), one, one)
    s2 = slots - (n - 2) * page
    assert all(torch.equal(a, b) for a, b in zip((kr, vr), pkg.ts_kv_cache_read(small, s2)))
    assert float((kr.float() - ko.float()).norm() / ko.float().norm()) < 0.2
    lens = torch.tensor([T], dtype=torch.int32, device=dev)
    assert torch.equal(pkg.ts_nvfp4_attention(qo[-1:], cache, ids, lens), pkg.ts_nvfp4_attention(qo[-1:], small, ids - (n - 2), lens))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def test_one_slot_for_many_tokens(dev):
    """Tokens with the same slot leave the bytes of one or another of them there, and nothing elsewhere."""
    T, hk, D, page = 300, 2, 64, 16
    _, k, v, _, kw, pos, table = _rope_inputs(dev, T, hk, hk, D, D, seed=12)
    g = torch.tensor([300.0], device=dev)
    apart = pkg.ts_kv_cache(-(-T // page), hk, D, g, g, page_size=page, device=dev)
    one = pkg.ts_kv_cache(2, hk, D, g, g, page_size=page, device=dev)
    one.pages.fill_(0xA5)
    for cache, slots in ((apart, torch.arange(T, device=dev).int()), (one, torch.full((T,), 21, dtype=torch.int32, device=dev))):
        pkg.ts_qk_norm_rope(k, k, kw, kw, pos, table, EPS, v=v, cache=cache, slots=slots)

    def token(pages, slot):  # [heads, bytes of the slot]
        tile = pages[slot // page, :, slot % page // 16]
        i = slot % 16
        return torch.cat([tile[:, o + i * n:o + (i + 1) * n] for o, n in ((0, D // 2), (8 * D, D // 2), (16 * D, D // 16), (17 * D, D // 16))], 1)

    theirs, got = torch.stack([token(apart.pages, t) for t in range(T)]), token(one.pages, 21)
    assert bool((theirs == got).any(0).all())
    rest = one.pages.clone()
    rest[1, :, 0] = 0xA5
    others = [token(one.pages, s) for s in range(16, 32) if s != 21]
    assert bool((rest == 0xA5).all()) and all(bool((o == 0xA5).all()) for o in others)


def _cache(dev, lens, hk, D, page, seed, spread=1.0):
    """A cache whose unused slots hold NaN scale factors, pages in random order; table [B, most + 1], ids of no page
    behind the used ones."""
    r = np.random.RandomState(seed)
    used = [-(-n // page) for n in lens]
    n = max(1, sum(used))
    pages = torch.full((n, hk, page // 16, 18 * D), 0xFF, dtype=torch.uint8, device=dev)
    order = r.permutation(n)
    table = np.full((len(lens), max(used, default=0) + 1), -1, np.int32)
    table[:, -1] = 2 ** 31 - 1
    kg, vg = torch.tensor([300.0], device=dev), torch.tensor([200.0], device=dev)
    cache, i = pkg.KVCache(pages, kg, vg), 0
    ones = torch.zeros(1, 16, device=dev)
    ones[:, :8] = 1.0  # no rotation
    for b, L in enumerate(lens):
        if L == 0:
            continue
        table[b, :used[b]] = order[i:i + used[b]]
        i += used[b]
        at = torch.arange(L, device=dev)
        ids = torch.from_numpy(table[b]).to(dev).long()
        slots = (ids[at // page] * page + at % page).int()
        k, v = _rand((L, hk, D), dev, seed + 7 * b, spread), _rand((L, hk, D), dev, seed + 7 * b + 1)
        k[..., ::13] *= 3
        pkg.ts_qk_norm_rope(k, k, None, None, torch.zeros(L, dtype=torch.int32, device=dev), ones, v=v, cache=cache, slots=slots)
    return cache, torch.from_numpy(table).to(dev)


def _check_attention(dev, new, lens, hq, hk, D, page, seed=0, causal=True, window=0, max_q=None, gap=0, scale=None, qscale=1.0):
    """One call against the reference, rows in front of, between and behind the sequences left as they were."""
    cache, table = _cache(dev, lens, hk, D, page, seed)
    B = len(lens)
    T = sum(new) + gap
    q = _rand((T, hq, D), dev, seed + 3, 1.3 * qscale)
    cu = np.concatenate(([0], np.cumsum(new)))
    kv = torch.tensor(lens, dtype=torch.int32, device=dev)
    single = gap == 0 and all(n == 1 for n in new)
    cut = None if single else torch.from_numpy(cu).int().to(dev)
    out, lse = Guarded((T, hq, D), torch.bfloat16, dev), Guarded((T, hq), torch.float32, dev)
    real = 1 / math.sqrt(D) if scale is None else scale
    args = dict(scale=scale, causal=causal, window=window, max_q=max_q)
    pkg.ts_nvfp4_attention(q, cache, table, kv, cut, out=out.t, lse=lse.t, **args)
    want, want_lse, slack, slack_lse = ref.attention(q, cache.pages, cache.k_scale.double(), cache.v_scale.double(), table, lens, cu,
                                                     real, causal, window)
    n = int(cu[-1])
    _close(out.t[:n], want[:n], slack[:n], "out")
    got = lse.t[:n].double()
    inf = torch.isinf(want_lse[:n])
    assert torch.equal(torch.isneginf(got), inf)
    assert bool(((got - want_lse[:n]).abs()[~inf] <= slack_lse[:n][~inf]).all()), float((got - want_lse[:n]).abs()[~inf].max())
    assert bool((out.t[:n][inf] == 0).all())
    assert bool((out.t[n:].contiguous().view(torch.int16) == -23131).all() and (lse.t[n:].view(torch.int32) == -1515870811).all())
    assert out.intact() and lse.intact()
    again = pkg.ts_nvfp4_attention(q, cache, table, kv, cut, return_lse=True, launch_with_pdl=True,
                                   out=out.t.clone(), lse=lse.t.clone(), **args)
    assert torch.equal(again[0][:n], out.t[:n]) and torch.equal(again[1][:n], lse.t[:n])


HEADS = [(1, 1), (2, 1), (5, 1), (8, 1), (8, 8), (16, 1), (40, 8), (24, 1)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", HEADS)
def test_single_tokens(dev, hq, hk, D):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 130, 1, 400, 0, 1000, 33]
    _check_attention(dev, [1] * len(lens), lens, hq, hk, D, 64 if hk == 1 else 16, seed=hq)


@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_pages(dev, page):
    _check_attention(dev, [1, 1, 1, 1, 1], [page - 1, page, page + 1, 3 * page + 7, 5], 8, 2, 128, page, seed=page)


@pytest.mark.parametrize("D,L,hq,hk", [(128, 40000, 8, 1), (64, 70001, 4, 2), (128, 9999, 32, 2), (128, 131072, 1, 1)])
def test_one_long_sequence(dev, D, L, hq, hk):
    """One sequence over every block, joined."""
    _check_attention(dev, [1], [L], hq, hk, D, 128, seed=1)


@pytest.mark.parametrize("B", [255, 256, 257, 600, 1025])
def test_many_sequences(dev, B):
    r = np.random.RandomState(B)
    lens = [int(v) for v in r.randint(0, 90, B)]
    lens[B // 3], lens[-1] = 3000, 700
    _check_attention(dev, [1] * B, lens, 4, 2, 64, 32, seed=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 16, 100])
@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 1), (10, 2), (16, 16)])
def test_a_few_queries(dev, hq, hk, window, D):
    """Queries in front of the first key (a length below the number of queries) see nothing."""
    new, lens = [3, 1, 5, 0, 7, 2, 4, 6], [200, 0, 3, 50, 7, 17, 1, 1500]
    _check_attention(dev, new, lens, hq, hk, D, 16, seed=hq + window, window=window, max_q=7, gap=3)


# (sequences, key heads, query heads of each, queries, keys at most): units of up to 8, 16 and 32 rows, as
# many as take clusters of 8, 4, 2 and 1 blocks, and one more than take any; then keys that are too many for a
# cluster, with few units (joined by large blocks) and with many
SPLITS = [(19, 2, 8, 1, 700), (39, 1, 5, 1, 700), (77, 1, 8, 1, 300), (51, 3, 4, 1, 300), (61, 5, 8, 1, 300),
          (19, 1, 8, 2, 700), (20, 1, 4, 4, 300), (39, 1, 8, 2, 300), (77, 1, 6, 2, 300), (51, 3, 8, 2, 200),
          (19, 1, 5, 5, 700), (20, 1, 8, 3, 300), (13, 3, 16, 2, 300), (77, 1, 4, 8, 300), (51, 3, 5, 4, 200),
          (1, 1, 8, 1, 8192), (4, 1, 8, 1, 8193), (5, 1, 8, 1, 16384),
          (2, 1, 8, 1, 17000), (2, 2, 8, 2, 17000), (3, 2, 5, 5, 17000), (12, 2, 8, 1, 17000), (6, 3, 8, 3, 17000)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,hk,group,n,most", SPLITS)
def test_every_split_of_few_rows(dev, B, hk, group, n, most, D):
    r = np.random.RandomState(B + n)
    lens = [int(v) for v in r.randint(0, min(most, 600), B)]
    lens[B // 2], lens[-1] = most, 1
    new = [n] * B
    if n > 1:
        new[0], new[B // 3] = 0, 1
    _check_attention(dev, new, lens, hk * group, hk, D, 16, seed=B, max_q=n, gap=1 if n > 1 else 0, window=150 if most == 200 else 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [31, 32, 33, 34, 47, 48, 49, 50])
def test_rows_at_the_change_of_kernels(dev, rows, D):
    """Up to 32 (D = 64: 48) (query, head) pairs of a key head go one way, more another."""
    _check_attention(dev, [rows, 1, rows - 1], [300, 40, 2100], 2, 2, D, 48, seed=rows, max_q=rows)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(49, 1), (64, 1), (130, 2), (1024, 1)])
def test_single_tokens_of_many_heads(dev, hq, hk, D):
    """More heads to a key head than the kernel of few rows takes."""
    _check_attention(dev, [1] * 5, [1, 0, 129, 700, 33], hq, hk, D, 16, seed=hq)


@pytest.mark.parametrize("rows", [1, 40])
def test_lengths_beyond_the_table(dev, rows):
    """A length counts as far as its table goes, which may be nowhere."""
    D, page = 64, 32
    lens = [64, 90, 5]
    cache, table = _cache(dev, lens, 2, D, page, 4)
    table = table[:, :2].contiguous()
    cu = torch.tensor([0, rows, 2 * rows, 3 * rows], dtype=torch.int32, device=dev)
    q = _rand((3 * rows, 4, D), dev, 1)

    def call(table, lens):
        return pkg.ts_nvfp4_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=dev), cu, max_q=rows, return_lse=True)

    want, got = call(table, [64, 64, 5]), call(table, [65, 2 ** 31 - 1, 5])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for t, n in ((table[:, :0].contiguous(), [3, 2 ** 31 - 1, 0]), (table, [0, -1, -2 ** 31])):
        out, lse = call(t, n)
        assert bool((out == 0).all() and torch.isneginf(lse).all())


@pytest.mark.parametrize("rows", [1, 5, 70])
def test_pages_shared_by_sequences(dev, rows):
    """Sequences with a common beginning may have its pages in common."""
    D, page, L = 128, 32, 500
    cache, table = _cache(dev, [L], 2, D, page, 8)
    table = table.expand(3, -1).contiguous()
    lens = torch.tensor([L, 300, L], dtype=torch.int32, device=dev)
    q = _rand((3 * rows, 8, D), dev, 2)
    cu = torch.arange(4, device=dev).int() * rows
    out, lse = pkg.ts_nvfp4_attention(q, cache, table, lens, cu, max_q=rows, return_lse=True)
    want, want_lse, slack, slack_lse = ref.attention(q, cache.pages, cache.k_scale.double(), cache.v_scale.double(), table, lens.tolist(),
                                                     cu.tolist(), 1 / math.sqrt(D), True, 0)
    _close(out, want, slack, "out")
    assert bool(((lse.double() - want_lse).abs() <= slack_lse).all())


def test_two_calls_at_once(dev):
    """Calls on two streams, each with a workspace of its own, and captured ones that share one in turn, give the bits of
    calls on their own: each way to split the work."""
    D, hk, page = 128, 2, 16
    lens = [17000, 300, 0, 2500]
    cache, table = _cache(dev, lens, hk, D, page, 3)
    kv = torch.tensor(lens, dtype=torch.int32, device=dev)
    side, calls = torch.cuda.Stream(), []
    for new in ([1, 1, 1, 1], [4, 0, 1, 2], [200, 30, 5, 300]):
        q = _rand((sum(new), 8, D), dev, len(calls))
        cu = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32, device=dev)
        bytes_ = pkg.library().ts_nvfp4_attention_workspace(4, 8, hk, D, max(new), table.shape[1] * page, 0)
        assert bytes_ > 0
        args = dict(cu_q=cu, max_q=max(new), return_lse=True)
        calls.append((q, args, [torch.full((bytes_,), 0xA5, dtype=torch.uint8, device=dev) for _ in range(2)]))
    want = [pkg.ts_nvfp4_attention(q, cache, table, kv, **args) for q, args, _ in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for q, args, spaces in calls:
            got.append([pkg.ts_nvfp4_attention(q, cache, table, kv, workspace=spaces[0], launch_with_pdl=True, **args),
                        pkg.ts_nvfp4_attention(q, cache, table, kv, workspace=spaces[1], stream=side, **args)])
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        for out, lse in pair:
            assert torch.equal(out, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])
    shared = max((spaces[0] for _, _, spaces in calls), key=lambda t: t.numel())
    graph, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for q, args, _ in calls + calls:
            outs.append(pkg.ts_nvfp4_attention(q, cache, table, kv, workspace=shared, launch_with_pdl=True, **args))
    for _ in range(2):
        for out, lse in outs:
            out.fill_(3.0)
            lse.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for i, (out, lse) in enumerate(outs):
            assert torch.equal(out, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])


def test_not_causal(dev):
    _check_attention(dev, [4, 1, 3, 2], [100, 9, 2, 0], 6, 2, 128, 32, causal=False, max_q=4)


@pytest.mark.parametrize("max_q", [1, 2, 4, 1000])
def test_any_max_q(dev, max_q):
    """The bound chooses a kernel, not the result."""
    _check_attention(dev, [9, 1, 30], [300, 17, 31], 8, 2, 128, 64, max_q=max_q, gap=2)


@pytest.mark.parametrize("qscale", [1e-30, 1e-4, 30.0, 1e30])
def test_scales_of_queries(dev, qscale):
    """Rows of any magnitude go through fp16; a wide spread of scores moves the maximum often."""
    _check_attention(dev, [1, 1, 2], [700, 40, 300], 8, 2, 64, 32, qscale=qscale, scale=0.125 / max(qscale / 30, 1.0) if qscale > 1 else None,
                     max_q=2)


def test_pages_outside_the_cache_are_not_seen(dev):
    hq, hk, D, page, L = 8, 2, 128, 32, 500
    cache, table = _cache(dev, [L], hk, D, page, 3)
    kv = torch.tensor([L], dtype=torch.int32, device=dev)
    table[0, 2], table[0, 7], table[0, 15] = -3, cache.pages.shape[0], 2 ** 31 - 1
    q = _rand((1, hq, D), dev, 4)
    got, lse = pkg.ts_nvfp4_attention(q, cache, table, kv, return_lse=True)
    want, want_lse, slack, slack_lse = ref.attention(q, cache.pages, cache.k_scale.double(), cache.v_scale.double(), table, [L], None,
                                                     1 / math.sqrt(D))
    _close(got, want, slack, "out")
    assert bool(((lse - want_lse).abs() <= slack_lse).all())
    table[:] = -1  # none at all
    got, lse = pkg.ts_nvfp4_attention(q, cache, table, kv, return_lse=True)
    assert bool((got == 0).all() and torch.isneginf(lse).all())
    # lengths beyond the table, and negative ones
    kv[0] = 2 ** 31 - 1
    assert bool((pkg.ts_nvfp4_attention(q, cache, table, kv) == 0).all())
    kv[0] = -5
    assert bool((pkg.ts_nvfp4_attention(q, cache, table, kv) == 0).all())


def test_not_a_number_shows(dev):
    """A NaN or an infinity in a query's row makes that row NaN and no other."""
    cache, table = _cache(dev, [300, 300], 1, 64, 16, 3)
    kv = torch.tensor([300, 300], dtype=torch.int32, device=dev)
    q = _rand((2, 4, 64), dev, 4)
    good = pkg.ts_nvfp4_attention(q, cache, table, kv)
    q[0, 1, 5], q[1, 2, 9] = math.nan, math.inf
    got, lse = pkg.ts_nvfp4_attention(q, cache, table, kv, return_lse=True)
    bad = torch.zeros(2, 4, dtype=torch.bool, device=dev)
    bad[0, 1] = bad[1, 2] = True
    assert bool(torch.isnan(got[bad]).all() and torch.isnan(lse[bad]).all()) and torch.equal(got[~bad], good[~bad])


def test_strides_streams_and_graphs(dev):
    """A decode step (rotate, keep, attend) on columns of wider matrices, on another stream, captured and replayed on new
    inputs, equals the calls on their own; the workspace is given, and two graphs that run in turn share it."""
    B, hq, hk, D, page, far = 6, 8, 2, 128, 16, 400
    cache, table = _cache(dev, [300, 40, 0, 17, 250, 99], hk, D, page, 6)
    lens = torch.tensor([301, 41, 1, 18, 251, 100], dtype=torch.int32, device=dev)
    need = int(lens.max() + page - 1) // page
    extra = torch.full((B, 1), -1, dtype=torch.int32, device=dev)
    pages = torch.cat((cache.pages, torch.full((B, *cache.pages.shape[1:]), 0xFF, dtype=torch.uint8, device=dev)))
    table = torch.cat((table[:, :need], extra), 1).contiguous()
    for b in range(B):  # a page of its own for each sequence's new token, where it begins one
        at = int(lens[b] - 1) // page
        if int(table[b, at]) < 0 or int(table[b, at]) >= cache.pages.shape[0]:
            table[b, at] = cache.pages.shape[0] + b
    cache = pkg.KVCache(pages, cache.k_scale, cache.v_scale)
    rows, qw, kw, angles = torch.empty(B, (hq + 2 * hk) * D + 8, dtype=torch.bfloat16, device=dev), _rand((D,), dev, 1), _rand((D,), dev, 2), ref.angles(far, D).to(dev)
    pos = (lens - 1).int()
    slots = (table.gather(1, (pos // page).long().unsqueeze(1)).squeeze(1) * page + pos % page).int()
    space = torch.full((max(16, pkg.library().ts_nvfp4_attention_workspace(B, hq, hk, D, 1, table.shape[1] * page, 0)),), 0xA5, dtype=torch.uint8, device=dev)

    def step(out, stream=None):
        q, k, v = (rows[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
        qo, _ = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, angles, EPS, v=v, cache=cache, slots=slots, launch_with_pdl=True, stream=stream)
        return pkg.ts_nvfp4_attention(qo, cache, table, lens, out=out[:, :hq * D].unflatten(1, (hq, D)), workspace=space,
                                      return_lse=True, launch_with_pdl=True, stream=stream)

    side = torch.cuda.Stream()
    outs = [torch.zeros(B, hq * D + 16, dtype=torch.bfloat16, device=dev) for _ in range(3)]
    rows.copy_(_rand(rows.shape, dev, 20))
    torch.cuda.synchronize()
    step(outs[0], side)
    side.synchronize()
    graphs, lses = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, o in zip(graphs, outs[1:]):
        with torch.cuda.graph(g):
            lses.append(step(o)[1])
    for seed in (30, 31):
        rows.copy_(_rand(rows.shape, dev, seed))
        for o in outs[1:]:
            o.fill_(3.0)
        graphs[0].replay()
        graphs[1].replay()
        _, lse = step(outs[0])
        torch.cuda.synchronize()
        assert torch.equal(outs[1][:, :hq * D], outs[0][:, :hq * D]) and torch.equal(outs[2], outs[1])
        assert torch.equal(lses[0], lse) and torch.equal(lses[1], lse)
        assert bool((outs[1][:, hq * D:] == 3.0).all())
    q = pkg.ts_qk_norm_rope(rows[:, :hq * D].unflatten(1, (hq, D)), rows[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D)), qw, kw, pos, angles, EPS)[0]
    want, _, slack, _ = ref.attention(q, cache.pages, cache.k_scale.double(), cache.v_scale.double(), table, lens.tolist(), None, 1 / math.sqrt(D))
    _close(outs[1][:, :hq * D].view(B, hq, D), want, slack, "out")


def test_refusals_on_tensors(dev):
    cache, table = _cache(dev, [20], 2, 64, 16, 1)
    q, kv = _rand((1, 4, 64), dev, 1), torch.tensor([20], dtype=torch.int32, device=dev)
    good = pkg.ts_nvfp4_attention(q, cache, table, kv)
    assert good.shape == q.shape
    with pytest.raises(ValueError, match="head_dim"):
        pkg.ts_nvfp4_attention(_rand((1, 4, 128), dev, 1), cache, table, kv)
    with pytest.raises(ValueError, match="cu_q"):
        pkg.ts_nvfp4_attention(_rand((2, 4, 64), dev, 1), cache, table, kv)
    with pytest.raises(ValueError, match="contiguous heads"):
        pkg.ts_nvfp4_attention(q.transpose(1, 2), cache, table, kv)
    with pytest.raises(ValueError, match="workspace"):
        pkg.ts_nvfp4_attention(q, cache, table, kv, max_q=100, workspace=torch.zeros(64, dtype=torch.uint8, device=dev))
    with pytest.raises(TypeError, match="int32"):
        pkg.ts_nvfp4_attention(q, cache, table, kv.long())
    with pytest.raises(pkg.TsError, match="multiple of the cache"):
        pkg.ts_nvfp4_attention(_rand((1, 3, 64), dev, 1), cache, table, kv)
    with pytest.raises(pkg.TsError, match="scale"):
        pkg.ts_nvfp4_attention(q, cache, table, kv, scale=-1.0)
    with pytest.raises(TypeError, match="CUDA tensor"):
        pkg.ts_nvfp4_attention(q.cpu().pin_memory(), cache, table, kv)
    with pytest.raises(pkg.TsError, match="overlaps"):
        pkg.ts_nvfp4_attention(q, cache, table, kv, out=q)
    k = _rand((1, 2, 64), dev, 2)
    pos, angles = torch.zeros(1, dtype=torch.int32, device=dev), ref.angles(4, 64).to(dev)
    with pytest.raises(ValueError, match="need a cache"):
        pkg.ts_qk_norm_rope(q, k, None, None, pos, angles, v=k)
    with pytest.raises(TypeError, match="slots"):
        pkg.ts_qk_norm_rope(q, k, None, None, pos, angles, v=k, cache=cache)
    with pytest.raises(pkg.TsError, match="rot"):
        pkg.ts_qk_norm_rope(q, k, None, None, pos, ref.angles(4, 24).to(dev))
    with pytest.raises(pkg.TsError, match="together"):
        pkg.ts_qk_norm_rope(q, k, k[0, 0], None, pos, angles)


def test_rope_on_pinned_host_buffers(dev):
    """The rotary calls read and write page-locked host memory themselves, with the same bits."""
    T, hq, hk, D, rot = 20, 4, 2, 64, 32
    q, k, v, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, strided=False)
    want = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, table)
    h = [t.cpu().pin_memory() for t in (q, k, qw, kw, pos, table)]
    got = pkg.ts_qk_norm_rope(*h)
    torch.cuda.synchronize()
    assert not got[0].is_cuda and all(torch.equal(a, b.cpu()) for a, b in zip(got, want))


def test_norm_rope_grad_on_pinned_host_buffers(dev):
    """So does the gradient, whose rows are copied to shared memory ahead."""
    T, hq, hk, D, rot = 300, 4, 2, 64, 32
    q, k, _, qw, kw, pos, table = _rope_inputs(dev, T, hq, hk, D, rot, strided=False)
    dq, dk = _rand((T, hq, D), dev, 1), _rand((T, hk, D), dev, 2)
    want = pkg.ts_qk_norm_rope_grad(dq, dk, q, k, qw, kw, pos, table)
    h = [t.cpu().pin_memory() for t in (dq, dk, q, k, qw, kw, pos, table)]
    before = torch.cuda.memory_stats()["allocated_bytes.all.allocated"]
    got = pkg.ts_qk_norm_rope_grad(*h)
    # (the workspace is on the GPU: host memory given back early could be another tensor's while the kernels run)
    assert torch.cuda.memory_stats()["allocated_bytes.all.allocated"] - before >= pkg.library().ts_qk_norm_rope_grad_workspace(D)
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b.cpu()) for a, b in zip(got, want))


# ---------------------------------------------------------------------------
# many rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L,hq,hk", [(17, 17, 1, 1), (20, 100, 1, 1), (32, 32, 4, 4), (130, 130, 1, 1), (129, 400, 2, 1), (300, 300, 8, 2),
                                       (257, 1000, 5, 1), (64, 5000, 16, 2), (1000, 1111, 3, 3), (2050, 2050, 8, 1)])
def test_prompts(dev, n, L, hq, hk, D):
    _check_attention(dev, [n], [L], hq, hk, D, 64, seed=n, max_q=n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 100, 128, 700])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_ragged_prompts(dev, page, window, D):
    """Lengths of none, of fewer keys than queries, ends inside tiles and pages; rows behind the last sequence."""
    new, lens = [100, 0, 1, 257, 33, 64, 700, 5], [100, 50, 300, 200, 0, 2000, 813, 3]
    _check_attention(dev, new, lens, 8, 2, D, page, seed=page + window, window=window, max_q=700, gap=5)


def test_prompts_not_causal(dev):
    _check_attention(dev, [150, 20, 90], [600, 1000, 0], 6, 2, 128, 32, causal=False, max_q=150)
    _check_attention(dev, [40, 300], [70, 129], 2, 2, 64, 32, causal=False, max_q=300, gap=1)


def test_a_few_queries_far_into_a_document(dev):
    """Few rows over many keys: one unit's keys over every block."""
    _check_attention(dev, [9], [50000], 8, 1, 128, 128, max_q=9)
    _check_attention(dev, [33], [20001], 10, 2, 64, 64, max_q=33)


@pytest.mark.parametrize("B", [256, 300, 700])
def test_prompts_of_many_sequences(dev, B):
    r = np.random.RandomState(B)
    new = [int(v) for v in r.randint(0, 25, B)]
    new[0], new[B // 2] = 60, 41
    lens = [m + int(v) for m, v in zip(new, r.randint(0, 60, B))]
    _check_attention(dev, new, lens, 4, 2, 64, 16, seed=2, max_q=60)


def test_prompt_scales(dev):
    for qscale, scale in ((1e-30, None), (30.0, 0.125), (1e30, 4e-30)):
        _check_attention(dev, [40, 130], [700, 400], 8, 2, 64, 32, qscale=qscale, scale=scale, max_q=130)


def test_prompt_pages_outside_the_cache_are_not_seen(dev):
    hq, hk, D, page, L, n = 8, 2, 128, 32, 500, 60
    cache, table = _cache(dev, [L], hk, D, page, 3)
    kv, cu = torch.tensor([L], dtype=torch.int32, device=dev), torch.tensor([0, n], dtype=torch.int32, device=dev)
    table[0, 2], table[0, 7], table[0, 14] = -3, cache.pages.shape[0], 2 ** 31 - 1
    q = _rand((n, hq, D), dev, 4)
    got, lse = pkg.ts_nvfp4_attention(q, cache, table, kv, cu, return_lse=True)
    want, want_lse, slack, slack_lse = ref.attention(q, cache.pages, cache.k_scale.double(), cache.v_scale.double(), table, [L], [0, n],
                                                     1 / math.sqrt(D))
    _close(got, want, slack, "out")
    assert bool(((lse - want_lse).abs() <= slack_lse).all())
    table[:] = -1
    got, lse = pkg.ts_nvfp4_attention(q, cache, table, kv, cu, return_lse=True)
    assert bool((got == 0).all() and torch.isneginf(lse).all())


def test_prompt_not_a_number_shows(dev):
    cache, table = _cache(dev, [300], 1, 64, 16, 3)
    kv, cu = torch.tensor([300], dtype=torch.int32, device=dev), torch.tensor([0, 50], dtype=torch.int32, device=dev)
    q = _rand((50, 4, 64), dev, 4)
    good = pkg.ts_nvfp4_attention(q, cache, table, kv, cu)
    q[10, 1, 5], q[44, 2, 9] = math.nan, math.inf
    got, lse = pkg.ts_nvfp4_attention(q, cache, table, kv, cu, return_lse=True)
    bad = torch.zeros(50, 4, dtype=torch.bool, device=dev)
    bad[10, 1] = bad[44, 2] = True
    assert bool(torch.isnan(got[bad]).all() and torch.isnan(lse[bad]).all()) and torch.equal(got[~bad], good[~bad])
    assert pkg.ts_stalled_waits() == 0


def test_lists_of_queries_that_do_not_fit(dev):
    """cu_q outside the rows or descending: clamped, never followed; other rows stay."""
    cache, table = _cache(dev, [300, 300, 300], 1, 64, 16, 3)
    kv = torch.tensor([300] * 3, dtype=torch.int32, device=dev)
    q = _rand((50, 4, 64), dev, 4)
    for max_q in (2, 40):
        for cu in ([0, 20, 10, 60], [-5, 3, 2 ** 31 - 1, 7], [40, 50, 50, 0]):
            out = torch.full_like(q, 7.0)
            pkg.ts_nvfp4_attention(q, cache, table, kv, torch.tensor(cu, dtype=torch.int32, device=dev), max_q=max_q, out=out)
            torch.cuda.synchronize()
            used = torch.zeros(50, dtype=torch.bool)
            for lo, hi in zip(cu[:-1], cu[1:]):
                lo, hi = max(0, min(50, lo)), min(50, hi)
                used[lo:max(lo, hi)] = True
            assert bool((out[~used.to(dev)] == 7.0).all()) and not bool((out[used.to(dev)] == 7.0).all(-1).any())
