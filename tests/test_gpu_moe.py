"""GPU parity of the expert-routing operators against plain references, and the layer they make together.

Indices are compared exactly, copies bit for bit.  combine: fp32 fused
multiply-adds over k slots, rounded once: within half a bf16 step (2^-8 of the
value) plus k * 2^-24 of the terms' magnitude.  Its gradient: dy within half a
bf16 step of the fp32 product (2^-24), dweights an fp32 sum of H products:
H / 8 / 256 steps of 8 per thread and the tree over 256 threads lose at most
(H / 256 + 16) * 2^-24 of the terms' magnitude.
"""
import numpy as np
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from tests import nvfp4_ref as ref
from tests.gpu_util import FILL, Guarded, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def _ids(T, k, E, seed=0, stray=True):
    """Ids [T, k], some outside 0..E-1, some twice in a token."""
    r = np.random.RandomState(seed)
    ids = r.randint(0, E, (T, k)).astype(np.int32)
    if stray:
        ids[r.rand(T, k) < 0.1] = -1
        ids[r.rand(T, k) < 0.05] = E + 3
    return ids


SORT = [(1, 1, 1, 1), (1, 8, 64, 128), (5, 3, 7, 1), (16, 8, 64, 128), (77, 6, 40, 8), (33, 64, 1024, 1),
        (1000, 8, 256, 128), (1025, 8, 33, 256), (1500, 7, 1000, 3), (8192, 8, 64, 128), (20000, 3, 5, 1)]


@pytest.mark.parametrize("T,k,E,align", SORT)
def test_sort(dev, T, k, E, align):
    ids = _ids(T, k, E, T)
    cap = pkg.ts_moe_rows(T, k, E, align) + 5
    bufs = [Guarded(s, torch.int32, dev) for s in ((T, k), (cap,), (E + 1,), (E,))]
    rows = pkg.MoERows(*(b.t for b in bufs))
    pkg.ts_moe_sort(torch.from_numpy(ids).to(dev), E, row_align=align, rows=rows)
    torch.cuda.synchronize()
    assert all(b.intact() for b in bufs)
    for got, want, name in zip(rows, ref.sort_rows(ids, E, align, cap), pkg.MoERows._fields):
        assert np.array_equal(host(got), want), name


@pytest.mark.parametrize("T,k,E,align", [(512, 8, 1024, 128), (513, 8, 1, 1), (2049, 2, 2, 128), (16384, 8, 17, 128), (40000, 5, 1024, 256)])
def test_sort_around_its_forms(dev, T, k, E, align):
    """Entries up to and beyond what 8 blocks take, and beyond what the registers hold."""
    test_sort(dev, T, k, E, align)


@pytest.mark.parametrize("ids", ([[0] * 40] * 300, [[-1] * 4] * 9, [[7] * 2] * 5000), ids=("one", "none", "last"))
def test_sort_one_sided(dev, ids):
    ids = np.array(ids, np.int32)
    rows = pkg.ts_moe_sort(torch.from_numpy(ids).to(dev), 8, row_align=128)
    for got, want in zip(rows, ref.sort_rows(ids, 8, 128, rows.row_src.numel())):
        assert np.array_equal(host(got), want)


def test_sort_no_tokens(dev):
    rows = pkg.ts_moe_sort(torch.empty(0, 4, dtype=torch.int32, device=dev), 9, row_align=128)
    assert host(rows.expert_start).tolist() == [0] * 10 and host(rows.expert_count).tolist() == [0] * 9


def _rows(dev, T, k, E, align=1, seed=0, stray=True):
    return pkg.ts_moe_sort(torch.from_numpy(_ids(T, k, E, seed, stray)).to(dev), E, row_align=align)


MOVE = [(1, 1, 1, 8), (3, 2, 4, 24), (16, 8, 64, 7168), (77, 6, 40, 4096), (130, 3, 5, 1040), (40, 17, 30, 520),
        (9, 64, 80, 264), (1, 8, 9, 65536)]


@pytest.mark.parametrize("T,k,E,H", MOVE)
def test_dispatch(dev, T, k, E, H):
    rows = _rows(dev, T, k, E)
    wide = torch.randn(T, H + 16).bfloat16().to(dev)
    x = wide[:, 8:8 + H]  # a strided view
    out = Guarded((rows.row_src.numel(), H), torch.bfloat16, dev)
    pkg.ts_moe_dispatch(x, rows, out=out.t)
    torch.cuda.synchronize()
    assert out.intact()
    src = host(rows.row_src)
    want = np.full((len(src), H), FILL << 8 | FILL, np.uint16)
    want[src >= 0] = host(x)[src[src >= 0] // k]
    assert np.array_equal(host(out.t), want)


@pytest.mark.parametrize("layout", (0, 1, 2))
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 16), (5, 2, 3, 48), (16, 8, 64, 7168), (77, 6, 40, 1040), (33, 20, 9, 256)])
def test_dispatch_nvfp4(dev, T, k, E, H, layout):
    """The bits of ts_nvfp4_quantize in every entry's row; other rows are left."""
    rows = _rows(dev, T, k, E, 128)
    x, g = torch.randn(T, H).bfloat16().to(dev), torch.tensor([211.0], device=dev)
    n = rows.row_src.numel()
    codes, sf = Guarded((n, H // 2), torch.uint8, dev), Guarded(pkg.sf_shape(n, H, layout), torch.uint8, dev)
    pkg.ts_moe_dispatch(x, rows, g, quant_out=codes.t, scale_out=sf.t, sf_layout=layout)
    torch.cuda.synchronize()
    assert codes.intact() and sf.intact()
    code, s = ref.quantize(x.float().cpu().numpy(), 211.0)
    src = host(rows.row_src)
    live = src >= 0
    want = np.full((n, H // 2), FILL, np.uint8)
    want[live] = ref.pack(code)[src[live] // k]
    assert np.array_equal(host(codes.t), want)
    at, shape = ref.sf_places(n, H // 16, layout)
    want = np.full(shape[0] * shape[1], FILL, np.uint8)
    if layout != 2:
        pad, _ = ref.sf_places(n, ref.up(H // 16, 4), layout)
        want[pad[live]] = 0
    want[at[live]] = s[src[live] // k]
    assert np.array_equal(host(sf.t), want.reshape(shape))


@pytest.mark.parametrize("weighted", (True, False))
@pytest.mark.parametrize("T,k,E,H", MOVE)
def test_combine(dev, T, k, E, H, weighted):
    rows = _rows(dev, T, k, E)
    n = rows.row_src.numel()
    y = torch.randn(n, H + 8).bfloat16().to(dev)[:, :H]
    y[(rows.row_src < 0).to(dev)] = float("nan")  # rows without an entry are not read
    w = torch.rand(T, k, device=dev)
    w[rows.row_of < 0] = float("inf")  # nor are the weights of entries without a row
    out = Guarded((T, H + 8), torch.bfloat16, dev)
    pkg.ts_moe_combine(y, rows, w if weighted else None, out=out.t[:, :H])
    torch.cuda.synchronize()
    assert out.intact() and (host(out.t)[:, H:] == (FILL << 8 | FILL)).all()
    held = (rows.row_of >= 0).unsqueeze(2)
    terms = torch.where(held, y.double()[rows.row_of.clamp(min=0).long()], 0.0)
    if weighted:
        terms = terms * torch.where(held, w.double().unsqueeze(2), 0.0)
    want, mag = terms.sum(1), terms.abs().sum(1)
    assert ((out.t[:, :H].double() - want).abs() <= 2.0 ** -8 * want.abs() + k * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("T,k,E,H", MOVE)
def test_combine_grad(dev, T, k, E, H):
    rows = _rows(dev, T, k, E)
    n = rows.row_src.numel()
    y = torch.randn(n, H).bfloat16().to(dev)
    d = torch.randn(T, H + 24).bfloat16().to(dev)[:, 16:16 + H]
    w = torch.rand(T, k, device=dev)
    dy, dw = Guarded((n, H), torch.bfloat16, dev), Guarded((T, k), torch.float32, dev)
    pkg.ts_moe_combine_grad(d, y, rows, w, dy=dy.t, dweights=dw.t)
    torch.cuda.synchronize()
    assert dy.intact() and dw.intact()
    held = rows.row_of >= 0
    at = rows.row_of[held].long()
    want = (w.double().unsqueeze(2) * d.double().unsqueeze(1))[held]
    got = dy.t[at].double()
    assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -24) * want.abs()).all()
    left = torch.ones(n, dtype=torch.bool)
    left[at.cpu()] = False
    assert (host(dy.t)[left.numpy()] == (FILL << 8 | FILL)).all()
    terms = torch.where(held.unsqueeze(2), y.double()[rows.row_of.clamp(min=0).long()], 0.0) * d.double().unsqueeze(1)
    assert (dw.t[~held] == 0).all()
    assert ((dw.t.double() - terms.sum(2)).abs() <= (H / 256 + 16) * 2.0 ** -24 * terms.abs().sum(2)).all()


def test_combine_grad_by_differences(dev):
    """dweights against the loss's differences in 64 bits, dy against autograd of the plain sum."""
    T, k, E, H = 6, 3, 5, 64
    rows = _rows(dev, T, k, E, stray=False)
    y = torch.randn(rows.row_src.numel(), H).bfloat16().to(dev)
    d, w = torch.randn(T, H).bfloat16().to(dev), torch.rand(T, k, device=dev)
    dy, dw = pkg.ts_moe_combine_grad(d, y, rows, w)
    at = rows.row_of.long()

    def loss(ww, yy):
        return ((ww.unsqueeze(2) * yy[at]).sum(1) * d.double()).sum()

    w64, y64 = w.double().requires_grad_(), y.double().requires_grad_()
    loss(w64, y64).backward()
    assert ((dy.double() - y64.grad).abs() <= 2.0 ** -7 * y64.grad.abs()).all()
    for t, j in ((0, 0), (3, 2), (5, 1)):
        step = torch.zeros(T, k, dtype=torch.float64, device=dev)
        step[t, j] = 0.5
        diff = loss(w.double() + step, y.double()) - loss(w.double() - step, y.double())
        assert abs(float(diff) - float(dw[t, j])) <= 1e-4 * H


def test_dispatch_and_combine_are_adjoint(dev):
    """<dispatch(x), y> == <x, combine(y)> without weights, both sums in 64 bits."""
    T, k, E, H = 50, 4, 11, 128
    rows = _rows(dev, T, k, E)
    x = torch.randint(-4, 5, (T, H)).bfloat16().to(dev)
    y = torch.randint(-4, 5, (rows.row_src.numel(), H)).bfloat16().to(dev)
    out = torch.zeros_like(y)
    pkg.ts_moe_dispatch(x, rows, out=out)
    back = pkg.ts_moe_combine(y, rows)
    assert float((out.double() * y.double()).sum()) == float((x.double() * back.double()).sum())


def test_bad_indices_are_skipped(dev):
    """Entries outside the buffers are neither read nor written."""
    T, k, H = 4, 3, 64
    bad = torch.tensor([[0, 7, -5], [2, 1 << 30, 1], [-(1 << 31), 3, 8], [4, 5, 6]], dtype=torch.int32, device=dev)
    rows = pkg.MoERows(bad, torch.zeros(7, dtype=torch.int32, device=dev), None, None)
    x = torch.randn(T, H).bfloat16().to(dev)
    out = Guarded((7, H), torch.bfloat16, dev)
    pkg.ts_moe_dispatch(x, rows, out=out.t)
    codes, sf = Guarded((7, H // 2), torch.uint8, dev), Guarded(pkg.sf_shape(7, H, 0), torch.uint8, dev)
    pkg.ts_moe_dispatch(x, rows, torch.ones(1, device=dev), quant_out=codes.t, scale_out=sf.t, sf_layout=0)
    w = torch.ones(T, k, device=dev)
    got = pkg.ts_moe_combine(out.t, rows, w)
    dy = Guarded((7, H), torch.bfloat16, dev)
    _, dw = pkg.ts_moe_combine_grad(x, out.t, rows, w, dy=dy.t)
    torch.cuda.synchronize()
    assert out.intact() and codes.intact() and sf.intact() and dy.intact()
    token = {0: 0, 2: 1, 1: 1, 3: 2, 4: 3, 5: 3, 6: 3}
    for r, t in token.items():
        assert torch.equal(out.t[r], x[t]) and torch.equal(dy.t[r], x[t])
    n = torch.tensor([1.0, 2.0, 1.0, 3.0], device=dev)
    assert torch.equal(got, (x.float() * n.unsqueeze(1)).bfloat16())
    assert (dw[(bad < 0) | (bad >= 7)] == 0).all()


def test_rows_past_32_bit_offsets(dev):
    """Rows more than 2^31 elements behind the first are moved, summed and differentiated."""
    n, H, T = 34000, 65536, 2
    row_of = torch.tensor([[n - 1, 0], [n - 3, n - 2]], dtype=torch.int32, device=dev)
    rows = pkg.MoERows(row_of, torch.empty(n, dtype=torch.int32, device=dev), None, None)
    x, w = torch.randn(T, H).bfloat16().to(dev), torch.ones(T, 2, device=dev)
    y = torch.empty(n, H, dtype=torch.bfloat16, device=dev)
    pkg.ts_moe_dispatch(x, rows, out=y)
    for t in range(T):
        for j in range(2):
            assert torch.equal(y[int(row_of[t, j])], x[t])
    assert torch.equal(pkg.ts_moe_combine(y, rows, w), (2 * x.float()).bfloat16())
    dy = torch.empty_like(y)
    _, dw = pkg.ts_moe_combine_grad(x, y, rows, w, dy=dy)
    assert torch.equal(dy[n - 1], x[0]) and torch.equal(dy[n - 2], x[1])
    dots = x.double().square().sum(1, keepdim=True)
    assert ((dw.double() - dots).abs() <= (H / 256 + 16) * 2.0 ** -24 * dots).all()
    g = torch.tensor([100.0], device=dev)
    codes, sf = pkg.ts_moe_dispatch(x, rows, g, sf_layout=2)
    q, s = pkg.ts_nvfp4_quantize(x, g)
    assert torch.equal(codes[n - 1], q[0]) and torch.equal(sf[n - 2], s[1])


def test_pinned_host_buffers_and_another_stream(dev):
    T, k, E, H = 19, 3, 7, 136
    ids = _ids(T, k, E, 3)
    x, w = torch.randn(T, H).bfloat16(), torch.rand(T, k)
    rows = pkg.ts_moe_sort(torch.from_numpy(ids).to(dev), E)
    out = pkg.ts_moe_dispatch(x.to(dev), rows, out=torch.zeros(rows.row_src.numel(), H, dtype=torch.bfloat16, device=dev))
    want = pkg.ts_moe_combine(out, rows, w.to(dev))
    wdy, wdw = pkg.ts_moe_combine_grad(x.to(dev), out, rows, w.to(dev), dy=torch.zeros_like(out))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    xh, wh = x.pin_memory(), w.pin_memory()
    hrows = pkg.ts_moe_sort(torch.from_numpy(ids).pin_memory(), E, stream=s)
    hout = torch.zeros(hrows.row_src.numel(), H, dtype=torch.bfloat16).pin_memory()
    pkg.ts_moe_dispatch(xh, hrows, out=hout, stream=s.cuda_stream)
    got = pkg.ts_moe_combine(hout, hrows, wh, stream=s)
    hdy = torch.zeros_like(hout).pin_memory()
    _, hdw = pkg.ts_moe_combine_grad(xh, hout, hrows, wh, dy=hdy, stream=s)
    s.synchronize()
    for a, b in zip((*rows, out, want, wdy, wdw), (*hrows, hout, got, hdy, hdw)):
        assert b.is_pinned() and torch.equal(a.cpu(), b)


def test_outputs_belong_to_the_given_stream(dev):
    """A new output comes from the memory of the stream that writes it, not from what the current stream has just freed
    with work still queued on it."""
    T, k, E, H = 64, 2, 4, 4096
    rows = _rows(dev, T, k, E, stray=False)
    x = torch.randn(T, H).bfloat16().to(dev)
    y = torch.zeros(rows.row_src.numel(), H, dtype=torch.bfloat16, device=dev)
    pkg.ts_moe_dispatch(x, rows, out=y)
    want = pkg.ts_moe_combine(y, rows).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for _ in range(20):
            junk = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
            torch.cuda._sleep(2_000_000)
            junk.fill_(-1.0)  # queued behind the sleep
            del junk
            got = pkg.ts_moe_combine(y, rows, stream=stream)
            s.synchronize()
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_refusals_of_tensors(dev):
    """What the binding refuses (types, shapes, places) and what the library does (sizes), before any launch."""
    f, ids = torch.ones(1, device=dev), torch.zeros(3, 2, dtype=torch.int32, device=dev)
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device=dev)
    q, s = pkg.ts_nvfp4_quantize(x, f, sf_layout=0)
    rows = pkg.ts_moe_sort(ids, 4)
    y, w = torch.zeros(6, 64, dtype=torch.bfloat16, device=dev), torch.ones(3, 2, device=dev)
    for err, call in (
            (TypeError, lambda: pkg.ts_nvfp4_quantize(x.half(), f)), (TypeError, lambda: pkg.ts_nvfp4_quantize(x.float(), f)),
            (TypeError, lambda: pkg.ts_nvfp4_quantize(x, 1.0)), (TypeError, lambda: pkg.ts_nvfp4_quantize(x.cpu(), f)),
            (ValueError, lambda: pkg.ts_nvfp4_quantize(x.t(), f)), (ValueError, lambda: pkg.ts_nvfp4_quantize(x[0], f)),
            (ValueError, lambda: pkg.ts_nvfp4_quantize(x, torch.ones(2, device=dev))),
            (ValueError, lambda: pkg.ts_nvfp4_quantize(x, f, row_src=ids)),
            (ValueError, lambda: pkg.ts_nvfp4_quantize(x, f, quant_out=q.new_empty(3, 33))),
            (ValueError, lambda: pkg.ts_nvfp4_quantize(x, f, scale_out=s, sf_layout=1)),
            (TypeError, lambda: pkg.ts_nvfp4_quantize(x, f, stream="s")),
            (pkg.TsError, lambda: pkg.ts_nvfp4_quantize(x[:, :40], f)), (pkg.TsError, lambda: pkg.ts_nvfp4_quantize(x, f, sf_layout=5)),
            (pkg.TsError, lambda: pkg.ts_nvfp4_quantize(x[:, 1:49], f)),
            (ValueError, lambda: pkg.ts_nvfp4_dequantize(q, s, f)), (ValueError, lambda: pkg.ts_nvfp4_dequantize(q[0], s, f)),
            (ValueError, lambda: pkg.ts_nvfp4_gemm(q, s, q[:, :16].contiguous(), s, f)),
            (ValueError, lambda: pkg.ts_nvfp4_gemm(q, s[:64], q, s, f)), (TypeError, lambda: pkg.ts_nvfp4_gemm(q.cpu().pin_memory(), s, q, s, f)),
            (pkg.TsError, lambda: pkg.ts_nvfp4_gemm(q, s, q, s, f)),  # N = 3
            (ValueError, lambda: pkg.ts_nvfp4_gemm(q, s, q, s, f, out=x)),
            (TypeError, lambda: pkg.ts_moe_sort(ids.long(), 4)), (ValueError, lambda: pkg.ts_moe_sort(ids[0], 4)),
            (ValueError, lambda: pkg.ts_moe_sort(ids, 0)), (ValueError, lambda: pkg.ts_moe_sort(ids, 2000)),
            (pkg.TsError, lambda: pkg.ts_moe_sort(ids, 4, row_align=128, rows=rows)),
            (ValueError, lambda: pkg.ts_moe_sort(ids, 5, rows=rows)),
            (ValueError, lambda: pkg.ts_moe_dispatch(x[:2], rows)), (ValueError, lambda: pkg.ts_moe_dispatch(x, rows, out=y[:5])),
            (ValueError, lambda: pkg.ts_moe_dispatch(x, rows, f, out=y)), (ValueError, lambda: pkg.ts_moe_dispatch(x, rows, quant_out=q)),
            (pkg.TsError, lambda: pkg.ts_moe_dispatch(y[3:6], rows, out=y)),  # overlap
            (ValueError, lambda: pkg.ts_moe_combine(y, rows, w[:2])), (TypeError, lambda: pkg.ts_moe_combine(y, rows, w.double())),
            (ValueError, lambda: pkg.ts_moe_combine_grad(x[:2], y, rows, w)),
            (ValueError, lambda: pkg.ts_moe_combine_grad(x, y, rows, w, dy=y[:4])),
            (pkg.TsError, lambda: pkg.ts_moe_combine_grad(x, y, rows, w, dy=y)),
            (ValueError, lambda: pkg.ts_nvfp4_grouped_gemm(q, s, q, s, f, rows))):
        with pytest.raises(err) as e:
            call()
        assert str(e.value)


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------

def _layer(p, ids, w, stream=None):
    """norm + quantise -> sort -> dispatch -> gate-up product -> silu -> quantise -> down product -> combine."""
    kw = dict(launch_with_pdl=True, stream=stream)
    pkg.ts_fused_reduce_norm(1, p["parts"], p["res"], p["gamma"], 1e-6, residual_out=p["res_out"], norm_out=p["norm"], **kw)
    rows = pkg.ts_moe_sort(ids, p["E"], row_align=128, **kw)
    a, asf = pkg.ts_moe_dispatch(p["norm"], rows, p["g1"], **kw)
    h = pkg.ts_nvfp4_grouped_gemm(a, asf, p["w1"], p["w1_sf"], p["alpha1"], rows, **kw)
    gate, lin = h.float().chunk(2, 1)
    act = (torch.nn.functional.silu(gate) * lin).bfloat16()
    b, bsf = pkg.ts_nvfp4_quantize(act, p["g2"], row_src=rows.row_src, sf_layout=0, **kw)
    y = pkg.ts_nvfp4_grouped_gemm(b, bsf, p["w2"], p["w2_sf"], p["alpha2"], rows, **kw)
    return pkg.ts_moe_combine(y, rows, w, **kw), rows, act


def _params(dev, T, H, F, E, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().to(dev)  # noqa: E731
    p = {"E": E, "parts": rnd(2, T, H), "res": rnd(T, H), "gamma": torch.ones(H, dtype=torch.bfloat16, device=dev),
         "res_out": torch.empty(T, H, dtype=torch.bfloat16, device=dev),
         "norm": torch.empty(T, H, dtype=torch.bfloat16, device=dev),
         "g1": torch.tensor([400.0], device=dev), "g2": torch.tensor([300.0], device=dev)}
    for name, (N, K), gin in (("w1", (2 * F, H), "g1"), ("w2", (H, F), "g2")):
        w = [pkg.ts_nvfp4_quantize((rnd(N, K) / K ** 0.5).contiguous(), torch.tensor([2000.0], device=dev), sf_layout=0)
             for _ in range(E)]
        p[name], p[name + "_sf"] = torch.stack([q for q, _ in w]), torch.stack([s for _, s in w])
        p["alpha" + name[1]] = (1.0 / (2000.0 * p[gin])).expand(E).contiguous()
        p[name + "_v"] = torch.stack([pkg.ts_nvfp4_dequantize(q, s, torch.ones(1, device=dev), sf_layout=0) for q, s in w])
    return p


@pytest.mark.parametrize("T,k,E", [(1, 2, 4), (19, 3, 6), (300, 4, 8)])
def test_layer(dev, T, k, E):
    """The chain against the same chain in 64 bits on the operators' own quantised inputs: each product within the
    tolerance of its rounding, so the sum of k weighted rows within k + 1 half steps of bf16 of its terms."""
    H, F = 256, 192
    p = _params(dev, T, H, F, E)
    ids = torch.from_numpy(_ids(T, k, E, 1, stray=False)).to(dev)
    w = torch.rand(T, k, device=dev)
    out, rows, act = _layer(p, ids, w)
    torch.cuda.synchronize()
    assert pkg.ts_stalled_waits() == 0
    live = (rows.row_src >= 0).nonzero().squeeze(1)
    expert = ids.reshape(-1)[rows.row_src[live].long()].long()
    b, bsf = pkg.ts_nvfp4_quantize(act, p["g2"], row_src=rows.row_src, sf_layout=0)
    one = torch.ones(1, device=dev)
    bv = pkg.ts_nvfp4_dequantize(b, bsf, one, sf_layout=0)[live].double()  # exact: 6 bits
    y = torch.zeros(rows.row_src.numel(), H, dtype=torch.float64, device=dev)
    y[live] = torch.einsum("rk,rnk->rn", bv, p["w2_v"].double()[expert]) * float(p["alpha2"][0])
    terms = w.double().unsqueeze(2) * y[rows.row_of.long()]
    want, mag = terms.sum(1), terms.abs().sum(1)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * mag).all()
    # and the first product, from the norm
    a, asf = pkg.ts_moe_dispatch(p["norm"], rows, p["g1"])
    av = pkg.ts_nvfp4_dequantize(a, asf, one, sf_layout=0)[live].double()
    h = torch.einsum("rk,rnk->rn", av, p["w1_v"].double()[expert]) * float(p["alpha1"][0])
    gate, lin = h.chunk(2, 1)
    a64 = torch.nn.functional.silu(gate) * lin
    assert ((act[live].double() - a64).abs() <= 2.0 ** -5 * (gate.abs() + 1) * (lin.abs() + 2.0 ** -6)).all()


def test_layer_in_a_graph(dev):
    """Captured once, replayed on other routings and tokens of the same buffers: the bits of the direct calls."""
    T, k, E, H, F = 40, 4, 8, 256, 192
    p = _params(dev, T, H, F, E)
    ids = torch.from_numpy(_ids(T, k, E, 2)).to(dev)
    w = torch.rand(T, k, device=dev)
    s = torch.cuda.Stream()
    _layer(p, ids, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        out, _, _ = _layer(p, ids, w)
    for seed in (3, 4, 5):
        ids.copy_(torch.from_numpy(_ids(T, k, E, seed)))
        p["parts"].copy_(torch.randn(2, T, H).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        want, _, _ = _layer(p, ids, w)
        assert torch.equal(out, want)
