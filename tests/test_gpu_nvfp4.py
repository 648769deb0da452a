"""GPU parity of the NVFP4 operators against plain 64-bit references.

Codes and scale factors are compared bit for bit (every step is one fp32
rounding, which the reference repeats).  The product is compared exactly where
every partial sum is an fp32 value, and else within

  |got - want| <= 2^-8 |want| + 2^-20 sum_k |a b|

half a bf16 step of the result (bf16 keeps 8 bits: 2^-8 of the value covers the
step at the next binade), and the fp32 sum over K: products of two E2M1 and two
E4M3 values have 12 bits and are exact; each 64-element instruction's sum is
held to fp32 with at most 2^-22 of the terms' magnitude lost (alignment to the
largest term with at least 22 bits), and the losses of K/64 instructions on a
running sum add up to less than four times that for random signs.
"""
import numpy as np
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from tests import nvfp4_ref as ref
from tests.gpu_util import FILL, Guarded, host
from tests.helpers import f32_of_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def no_stalls(dev):
    yield
    assert pkg.ts_stalled_waits() == 0


def _x(T, K, seed=0, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g)
    if spread:
        x *= torch.exp2(torch.randint(-12, 6, (T, K), generator=g).float())
        x[:, : 16] = 0  # a block of zeros
    return x.bfloat16()


# ---------------------------------------------------------------------------
# quantise and read back
# ---------------------------------------------------------------------------

ROWS = [(1, 16), (1, 4096), (3, 32), (7, 48), (5, 64), (130, 112), (9, 240), (33, 1024), (2, 1040), (300, 2064),
        (1, 65536), (17, 7168)]


@pytest.mark.parametrize("layout", (0, 1, 2))
@pytest.mark.parametrize("T,K", ROWS)
def test_quantize_bits(dev, T, K, layout):
    x = _x(T, K, seed=T + K)
    for g in (1.0, 300.7, 3e-3):
        q = Guarded((T, K // 2), torch.uint8, dev)
        s = Guarded(pkg.sf_shape(T, K, layout), torch.uint8, dev)
        pkg.ts_nvfp4_quantize(x.to(dev), torch.tensor([g], device=dev), quant_out=q.t, scale_out=s.t, sf_layout=layout)
        torch.cuda.synchronize()
        assert q.intact() and s.intact()
        code, sf = ref.quantize(x.float().numpy(), g)
        assert np.array_equal(host(s.t), ref.lay_out(sf, layout))
        assert np.array_equal(host(q.t), ref.pack(code))


def test_quantize_matches_the_fused_pattern(dev):
    """The bits that kARResidualRMSNormOutFP4Quant writes for its norm_out."""
    T, H = 70, 1024
    g = torch.tensor([250.0], device=dev)
    outs = pkg.new_outputs(5, T, H, dev, sf_layout=0)
    pkg.ts_fused_reduce_norm(5, [_x(T, H, 1, False).to(dev)], _x(T, H, 2, False).to(dev),
                             torch.ones(H, dtype=torch.bfloat16, device=dev), 1e-6, g, sf_layout=0, **outs)
    q, s = pkg.ts_nvfp4_quantize(outs["norm_out"], g, sf_layout=0)
    assert torch.equal(q, outs["quant_out"]) and torch.equal(s, outs["scale_out"])


def test_quantize_infinite_and_tiny_values(dev):
    x = torch.zeros(4, 32).bfloat16()
    x[0, 3], x[0, 20] = float("inf"), -float("inf")
    x[1, 0] = torch.finfo(torch.bfloat16).max
    x[1, 17] = -torch.finfo(torch.bfloat16).max
    x[2, 1] = 2.0 ** -133  # subnormal
    x[3, :] = -0.0
    q, s = pkg.ts_nvfp4_quantize(x.to(dev), torch.ones(1, device=dev), sf_layout=2)
    code, sf = ref.unpack(host(q)), host(s)
    assert (sf[:2] == 126).all() and (sf[2:] == 0).all()  # saturated; too small for a scale factor
    assert code[0, 3] == 7 and code[0, 20] == 15 and code[1, 0] == 7 and code[1, 17] == 15
    assert (code[2:] == 0).all()


@pytest.mark.parametrize("layout", (0, 1, 2))
@pytest.mark.parametrize("T,K", ROWS)
def test_dequantize(dev, T, K, layout):
    r = np.random.RandomState(T + K)
    codes = r.randint(0, 256, (T, K // 2)).astype(np.uint8)
    sf = r.randint(0, 127, (T, K // 16)).astype(np.uint8)
    g = np.float32(3.7)
    out = Guarded((T, K + 8), torch.bfloat16, dev)
    pkg.ts_nvfp4_dequantize(torch.from_numpy(codes).to(dev), torch.from_numpy(ref.lay_out(sf, layout, 255)).to(dev),
                            torch.tensor([g], device=dev), sf_layout=layout, out=out.t[:, :K])
    torch.cuda.synchronize()
    assert out.intact()
    got = f32_of_bf16(host(out.t)).astype(np.float64)
    assert (host(out.t)[:, K:] == (FILL << 8 | FILL)).all()
    want = ref.values(codes, sf) / float(g)
    # half a bf16 step, and the fp32 quotient and product (2^-24 each)
    assert (np.abs(got[:, :K] - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want)).all()


def test_rows_without_an_entry_are_left(dev):
    T, K = 37, 96
    src = torch.arange(T, dtype=torch.int32)
    src[::3] = -1
    x, g = _x(T, K, 3), torch.ones(1, device=dev)
    x[0] = float("nan")  # not read
    codes = torch.full((T, K // 2), 0x5A, dtype=torch.uint8, device=dev)
    sf = torch.full(pkg.sf_shape(T, K, 0), 0x5A, dtype=torch.uint8, device=dev)
    pkg.ts_nvfp4_quantize(x.to(dev), g, row_src=src.to(dev), quant_out=codes, scale_out=sf, sf_layout=0)
    code, s = ref.quantize(torch.nan_to_num(x).float().numpy(), 1.0)
    want_c, want_s = ref.pack(code), np.full(tuple(sf.shape), 0x5A, np.uint8)
    want_c[::3] = 0x5A
    at, _ = ref.sf_places(T, K // 16, 0)
    live = (src >= 0).numpy()
    want_s.reshape(-1)[at[live]] = s[live]
    pad, _ = ref.sf_places(T, ref.up(K // 16, 4), 0)
    want_s.reshape(-1)[pad[live][:, K // 16:]] = 0
    assert np.array_equal(host(codes), want_c) and np.array_equal(host(sf), want_s)
    out = torch.full((T, K), 7.0, dtype=torch.bfloat16, device=dev)
    pkg.ts_nvfp4_dequantize(codes, sf, g, sf_layout=0, row_src=src.to(dev), out=out)
    assert (out[::3] == 7.0).all() and not (out[1::3] == 7.0).all()


def test_strided_rows_and_pinned_host_buffers(dev):
    """Rows of a wider matrix, and buffers in page-locked host memory, give the bits of contiguous device rows."""
    wide = _x(21, 400, 4)
    x, g = wide[:, 16:16 + 240], torch.tensor([37.0])
    q, s = pkg.ts_nvfp4_quantize(x.contiguous().to(dev), g.to(dev), sf_layout=1)
    q2, s2 = pkg.ts_nvfp4_quantize(wide.to(dev)[:, 16:16 + 240], g.to(dev), sf_layout=1)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    q3, s3 = pkg.ts_nvfp4_quantize(wide.pin_memory()[:, 16:16 + 240], g.pin_memory(), sf_layout=1)
    v3 = pkg.ts_nvfp4_dequantize(q3, s3, g.pin_memory(), sf_layout=1)
    torch.cuda.synchronize()
    assert q3.is_pinned() and torch.equal(q.cpu(), q3) and torch.equal(s.cpu(), s3)
    assert torch.equal(pkg.ts_nvfp4_dequantize(q, s, g.to(dev), sf_layout=1).cpu(), v3)


def test_rows_past_32_bit_offsets(dev):
    """More than 2^31 elements in and out: the last rows are those of a small call."""
    T, K = 33000, 65536
    x = torch.empty(T, K, dtype=torch.bfloat16, device=dev)
    tail = _x(3, K, 9).to(dev)
    x[-3:] = tail
    g = torch.tensor([5.0], device=dev)
    q, s = pkg.ts_nvfp4_quantize(x, g)
    q1, s1 = pkg.ts_nvfp4_quantize(tail, g)
    assert torch.equal(q[-3:], q1) and torch.equal(s[-3:], s1)
    pkg.ts_nvfp4_dequantize(q, s, g, out=x)
    assert torch.equal(x[-3:], pkg.ts_nvfp4_dequantize(q1, s1, g))


# ---------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------

def _want(a, asf, b, bsf, dev):
    av = torch.from_numpy(ref.values(a, asf)).to(dev)
    bv = torch.from_numpy(ref.values(b, bsf)).to(dev)
    return av @ bv.t(), av.abs() @ bv.abs().t()


GEMM = [(1, 8, 32), (1, 128, 64), (2, 16, 96), (5, 136, 160), (31, 72, 256), (32, 264, 288), (33, 128, 512),
        (64, 200, 64), (65, 520, 1056), (100, 256, 320), (128, 384, 2048), (129, 128, 256), (130, 8, 32),
        (200, 136, 1120), (257, 264, 512), (385, 640, 96), (1000, 1032, 544), (7, 4096, 4096), (4, 264, 1024), (9, 512, 2080),
        (40, 200, 2048), (61, 8192, 3104), (70, 1032, 5152), (128, 264, 6400), (97, 72, 1056)]


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm_exact(dev, M, N, K):
    """Scale factors that are small powers of two (and 1.5): every sum is exact, so the output is the rounded one."""
    a, asf, ta, tas = ref.random_nvfp4(M, K, M + K, dev, ref.EXACT_SF)
    b, bsf, tb, tbs = ref.random_nvfp4(N, K, N + K + 1, dev, ref.EXACT_SF)
    want, mag = _want(a, asf, b, bsf, dev)
    assert float(mag.max()) * 16 < 2 ** 24  # exact in fp32
    out = Guarded((M, N + 8), torch.bfloat16, dev)
    pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, torch.tensor([0.5], device=dev), out=out.t[:, :N])
    torch.cuda.synchronize()
    assert out.intact() and (host(out.t)[:, N:] == (FILL << 8 | FILL)).all()
    assert torch.equal(out.t[:, :N], (want * 0.5).float().bfloat16())


@pytest.mark.parametrize("M,N,K", [(1, 4096, 7168), (16, 2112, 7168), (48, 1024, 2048), (127, 264, 4064),
                                   (300, 520, 7168), (2048, 2112, 1536)])
def test_gemm_random(dev, M, N, K):
    a, asf, ta, tas = ref.random_nvfp4(M, K, 1, dev)
    b, bsf, tb, tbs = ref.random_nvfp4(N, K, 2, dev)
    alpha = torch.tensor([1.7e-3], device=dev)
    want, mag = _want(a, asf, b, bsf, dev)
    want, mag = want * alpha.double(), mag * alpha.double()
    got = pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, alpha, launch_with_pdl=True).double()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * mag).all()


@pytest.mark.parametrize("M,N,K", [(97, 8, 5152), (128, 2112, 5152), (129, 520, 2848), (256, 1000, 3104), (257, 2112, 5408),
                                   (300, 136, 4096), (512, 2048, 5152), (700, 264, 2912), (1000, 1032, 5152)])
def test_gemm_exact_over_two_pairs(dev, M, N, K):
    """Few tiles with a long K, of odd and even steps."""
    test_gemm_exact(dev, M, N, K)


@pytest.mark.parametrize("M,N,K", [(257, 7200, 544), (512, 7168, 96), (1024, 5000, 160), (1500, 7168, 288), (2048, 5120, 1056)])
def test_gemm_exact_in_tiles_of_192(dev, M, N, K):
    """Tiles that begin in the middle of 128 rows of scale factors, the last one whole and not."""
    test_gemm_exact(dev, M, N, K)


def test_gemm_over_two_pairs_replayed(dev):
    """The same call twice in a graph, on two streams, gives the bits of the direct call."""
    sets = []
    for i in range(2):
        _, _, ta, tas = ref.random_nvfp4(300, 4128, 10 + i, dev)
        _, _, tb, tbs = ref.random_nvfp4(1032, 4128, 20 + i, dev)
        sets.append((ta, tas, tb, tbs, torch.ones(1, device=dev)))
    direct = [pkg.ts_nvfp4_gemm(*s) for s in sets]
    outs = [[torch.empty_like(d) for d in direct] for _ in range(2)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(main), torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        for stream, to in zip((main, side), outs):
            for _ in range(4):
                for s, o in zip(sets, to):
                    pkg.ts_nvfp4_gemm(*s, out=o, launch_with_pdl=True, stream=stream)
        main.wait_stream(side)
    for _ in range(3):
        for o in outs[0] + outs[1]:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for to in outs:
            for o, d in zip(to, direct):
                assert torch.equal(o, d)
    assert pkg.ts_stalled_waits() == 0


@pytest.mark.parametrize("M", (90, 1500))
def test_gemm_out_past_32_bit_offsets(dev, M):
    """An output whose last rows lie more than 2^31 elements behind the first."""
    N, K, ldo = 72, 64, (1 << 31) // 80 if M == 90 else (1 << 31) // 1400
    ldo = ldo // 8 * 8
    a, asf, ta, tas = ref.random_nvfp4(M, K, 3, dev, ref.EXACT_SF)
    b, bsf, tb, tbs = ref.random_nvfp4(N, K, 4, dev, ref.EXACT_SF)
    out = torch.empty(M, ldo, dtype=torch.bfloat16, device=dev)[:, :N]
    assert (M - 1) * out.stride(0) > 1 << 31
    pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, torch.ones(1, device=dev), out=out)
    want, _ = _want(a, asf, b, bsf, dev)
    assert torch.equal(out, want.float().bfloat16())


def test_gemm_reads_no_scale_factor_of_other_rows(dev):
    """NaN scale factors in the padding rows, and rows of NaN scale factors, stay in their own rows and columns."""
    for M, N in ((5, 24), (70, 136), (300, 264)):
        a, asf, ta, tas = ref.random_nvfp4(M, 160, 1, dev, ref.EXACT_SF)
        b, bsf, tb, tbs = ref.random_nvfp4(N, 160, 2, dev, ref.EXACT_SF)
        asf[M // 2], bsf[3] = 127, 127
        live = np.zeros((ref.up(M, 128), 12), bool)
        at, _ = ref.sf_places(ref.up(M, 128), 12, 0)
        buf = np.full(at.size, 127, np.uint8)
        at_live, _ = ref.sf_places(M, 12, 0)
        buf[at_live[:, 10:]] = 0  # the padding columns are zero by definition
        buf[at_live[:, :10]] = asf
        tas = torch.from_numpy(buf.reshape(live.shape)).to(dev)
        tbs = torch.from_numpy(ref.lay_out(bsf, 0)).to(dev)
        got = pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, torch.ones(1, device=dev))
        want, _ = _want(a, np.where(asf == 127, 0, asf), b, np.where(bsf == 127, 0, bsf), dev)
        want = want.float().bfloat16()
        bad = torch.zeros(M, N, dtype=torch.bool, device=dev)
        bad[M // 2], bad[:, 3] = True, True
        assert got[bad].isnan().all() and torch.equal(got[~bad], want[~bad])


def test_gemm_no_rows(dev):
    z = torch.empty(0, 32, dtype=torch.uint8, device=dev)
    b = torch.zeros(16, 32, dtype=torch.uint8, device=dev)
    out = pkg.ts_nvfp4_gemm(z, torch.empty(0, 4, dtype=torch.uint8, device=dev), b,
                            torch.zeros(128, 4, dtype=torch.uint8, device=dev), torch.ones(1, device=dev))
    assert out.shape == (0, 16)


def test_gemm_many_calls_and_replays(dev):
    """Calls one after the other with programmatic dependent launch, and a graph of them replayed on new inputs."""
    shapes = [(1, 512, 512), (40, 512, 512), (300, 512, 512), (100, 512, 512)]
    sets = []
    for i, (M, N, K) in enumerate(shapes):
        _, _, ta, tas = ref.random_nvfp4(M, K, 10 + i, dev)
        _, _, tb, tbs = ref.random_nvfp4(N, K, 20 + i, dev)
        sets.append((ta, tas, tb, tbs, torch.ones(1, device=dev)))
    direct = [pkg.ts_nvfp4_gemm(*s) for s in sets]
    outs = [torch.empty_like(d) for d in direct]
    s0 = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s0):
        with torch.cuda.graph(g, stream=s0):
            for s, o in zip(sets, outs):
                pkg.ts_nvfp4_gemm(*s, out=o, launch_with_pdl=True)
    for _ in range(5):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, d in zip(outs, direct):
            assert torch.equal(o, d)
    for s in sets:  # new contents of the same buffers
        s[0].copy_(s[0].flip(0))
    direct = [pkg.ts_nvfp4_gemm(*s) for s in sets]
    g.replay()
    torch.cuda.synchronize()
    for o, d in zip(outs, direct):
        assert torch.equal(o, d)


def test_gemm_two_streams_at_once(dev):
    _, _, ta, tas = ref.random_nvfp4(500, 1024, 1, dev)
    _, _, tb, tbs = ref.random_nvfp4(1024, 1024, 2, dev)
    one = torch.ones(1, device=dev)
    want = pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, one)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in range(12)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, one, out=o, stream=streams[i % 3])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


# ---------------------------------------------------------------------------
# the experts' products
# ---------------------------------------------------------------------------

def _grouped(dev, counts, N, K, tokens_hint=None, starts=None):
    E = len(counts)
    start = [0]
    for c in counts:
        start.append(start[-1] + ref.up(c, 128))
    rows = start[-1] + 128
    a, asf, ta, tas = ref.random_nvfp4(rows, K, 5, dev, ref.EXACT_SF)
    bs = [ref.random_nvfp4(N, K, 50 + e, dev, ref.EXACT_SF) for e in range(E)]
    tb, tbs = torch.stack([b[2] for b in bs]), torch.stack([b[3] for b in bs])
    alpha = torch.tensor([2.0 ** (e % 3) for e in range(E)], device=dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    hint = sum(counts) if tokens_hint is None else tokens_hint
    r = pkg.MoERows(torch.empty(hint, 1, dtype=torch.int32, device=dev), torch.empty(rows, dtype=torch.int32, device=dev),
                    i32(start if starts is None else starts), i32(counts))
    out = Guarded((rows, N), torch.bfloat16, dev)
    pkg.ts_nvfp4_grouped_gemm(ta, tas, tb, tbs, alpha, r, out=out.t, launch_with_pdl=True)
    torch.cuda.synchronize()
    assert out.intact()
    want = torch.full((rows, N), FILL << 8 | FILL, dtype=torch.int32, device=dev).to(torch.int16).view(torch.bfloat16)
    for e, c in enumerate(counts):
        s = start[e]
        if c and (starts is None or (starts[e] == s)):
            w, mag = _want(a[s:s + c], asf[s:s + c], bs[e][0], bs[e][1], dev)
            assert float(mag.max()) * 16 < 2 ** 24
            want[s:s + c] = (w * alpha[e].double()).float().bfloat16()
    assert torch.equal(out.t.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("hint", (None, 1, 100000), ids=("by-count", "few", "many"))
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 32), ([0, 0, 0], 128, 64), ([3, 0, 1, 7], 136, 160), ([128, 127, 129, 0, 1], 264, 96),
    ([33, 64, 65, 100, 0, 2], 384, 512), ([300, 0, 513, 5], 200, 288), ([255, 256, 257, 31, 32, 224, 225], 520, 320),
    ([1000, 161, 0, 448], 1032, 1024)], ids=str)
def test_grouped(dev, counts, N, K, hint):
    _grouped(dev, counts, N, K, hint)


def test_one_row_of_any_stride(dev):
    """A single row of a wider buffer, whose stride is no multiple of 8."""
    g = torch.ones(1, device=dev)
    x = torch.randn(1, 77, device=dev).bfloat16()
    q, s = pkg.ts_nvfp4_quantize(x[:, :64], g, sf_layout=pkg.SFLayout.SWIZZLED_128x4)
    want_q, want_s = pkg.ts_nvfp4_quantize(x[:, :64].contiguous(), g, sf_layout=pkg.SFLayout.SWIZZLED_128x4)
    assert torch.equal(q, want_q) and torch.equal(s, want_s)
    wide = torch.zeros(1, 77, dtype=torch.bfloat16, device=dev)
    pkg.ts_nvfp4_gemm(q, s, q.expand(8, -1).contiguous(), s, g, out=wide[:, :8])
    assert torch.equal(wide[:, :1], pkg.ts_nvfp4_gemm(q, s, q.expand(8, -1).contiguous(), s, g)[:, :1])
    assert not wide[:, 8:].any()


@pytest.mark.parametrize("hint", (1, 100000), ids=("few", "many"))
@pytest.mark.parametrize("counts,N", [([5000], 520), ([1, 2049, 1025, 4097, 2048], 776)], ids=str)
def test_grouped_many_tokens(dev, counts, N, hint):
    """More tiles of tokens than pass over the weights together."""
    _grouped(dev, counts, N, 96, hint)


def test_grouped_many_experts(dev):
    r = np.random.RandomState(0)
    _grouped(dev, [int(v) for v in r.randint(0, 4, 300)], 72, 64)


def test_grouped_shared_rows(dev):
    """Experts that share rows, more of them than rows have tiles, stay inside the buffers."""
    E, rows, N, K = 300, 1024, 64, 64
    a, asf, ta, tas = ref.random_nvfp4(rows, K, 5, dev, ref.EXACT_SF)
    b, bsf, tb, tbs = ref.random_nvfp4(N, K, 6, dev, ref.EXACT_SF)
    i32 = lambda v: torch.full((v[0],), v[1], dtype=torch.int32, device=dev)  # noqa: E731
    for hint in (1, 100000):
        r = pkg.MoERows(torch.empty(hint, 1, dtype=torch.int32, device=dev), i32((rows, 0)), i32((E + 1, 0)), i32((E, rows)))
        out = Guarded((rows, N), torch.bfloat16, dev)
        pkg.ts_nvfp4_grouped_gemm(ta, tas, tb.expand(E, -1, -1).contiguous(), tbs.expand(E, -1, -1).contiguous(),
                                  torch.ones(E, device=dev), r, out=out.t)
        torch.cuda.synchronize()
        assert out.intact()
        assert torch.equal(out.t, _want(a, asf, b, bsf, dev)[0].float().bfloat16())
    assert pkg.ts_stalled_waits() == 0


def test_grouped_skips_bad_starts(dev):
    """An expert that does not start on a multiple of 128, or does not lie inside the rows, is skipped."""
    _grouped(dev, [5, 6, 7, 8], 64, 64, starts=[0, 64, 1 << 20, -128, 0])
