"""Calls behind a kernel that lets them start early and writes their inputs only at its end: they read none of them
before.  Products behind one that holds the stream for longer than a wait inside a product may take (4e9 cycles, about
2 s): the product waits for it, and its own waits begin afterwards."""
import ctypes
import os
import subprocess

import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from reduce_residual_rmsnorm_gb300 import build as libbuild
from tests import nvfp4_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HOLD_NS = 3_000_000_000


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def hold(dev, tmp_path_factory):
    out = tmp_path_factory.mktemp("hold") / "libpdl_hold.so"
    subprocess.check_call([libbuild.nvcc(), *libbuild.ARCH, *libbuild.NVCC_FLAGS, "-shared", "-cudart", "static",
                           os.path.join(ROOT, "tests", "pdl_hold.cu"), "-o", str(out)])
    lib = ctypes.CDLL(str(out))
    lib.pdl_hold.argtypes = [ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
    lib.pdl_hold.restype = ctypes.c_int

    def run(ns, src, dst):
        assert src.is_contiguous() and dst.is_contiguous() and src.nbytes == dst.nbytes
        assert lib.pdl_hold(ns, src.data_ptr(), dst.data_ptr(), src.nbytes, torch.cuda.current_stream().cuda_stream) == 0

    return run


# few tokens: alone, K over a cluster, 128 columns; pairs: alone, K over two of them
@pytest.mark.parametrize("M,N,K", [(3, 136, 96), (3, 256, 4096), (90, 264, 5152), (300, 520, 320), (256, 264, 5408)])
def test_product_outwaits_the_kernel_before(dev, hold, M, N, K):
    _, _, ta, tas = ref.random_nvfp4(M, K, 1, dev)
    _, _, tb, tbs = ref.random_nvfp4(N, K, 2, dev)
    one = torch.ones(1, device=dev)
    want = pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, one)
    late = torch.zeros_like(ta)  # the codes are there when the kernel before ends
    out = torch.full_like(want, float("nan"))
    torch.cuda.synchronize()
    hold(HOLD_NS, ta, late)
    pkg.ts_nvfp4_gemm(late, tas, tb, tbs, one, out=out, launch_with_pdl=True)
    torch.cuda.synchronize()
    assert pkg.ts_stalled_waits() == 0
    assert torch.equal(out, want)


def _late(hold, tensors):
    """Copies of the tensors that hold zeros until a kernel, queued here, ends after 20 ms; the next call may start at once."""
    at, offsets = 0, []
    for t in tensors:
        offsets.append(at)
        at = (at + t.nbytes + 255) // 256 * 256
    src = torch.zeros(at, dtype=torch.uint8, device=tensors[0].device)
    dst = torch.zeros_like(src)
    part = lambda buf, o, t: buf[o:o + t.nbytes].view(t.dtype).view(t.shape)  # noqa: E731
    for o, t in zip(offsets, tensors):
        part(src, o, t).copy_(t)
    torch.cuda.synchronize()
    hold(20_000_000, src, dst)
    return [part(dst, o, t) for o, t in zip(offsets, tensors)]


def _check(got, want):
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("T,K", [(1, 64), (300, 2048), (700, 272)])
def test_rows_read_nothing_early(dev, hold, T, K):
    torch.manual_seed(T)
    x, g = torch.randn(T, K, device=dev).bfloat16(), torch.tensor([37.0], device=dev)
    src = torch.arange(T, dtype=torch.int32, device=dev)
    q, s = pkg.ts_nvfp4_quantize(x, g, sf_layout=0)
    want = [q, s], [pkg.ts_nvfp4_dequantize(q, s, g, sf_layout=0)]
    live = torch.zeros_like(s)  # padding rows are not written with row_src
    lx, lg, lsrc = _late(hold, (x, g, src))
    got = pkg.ts_nvfp4_quantize(lx, lg, row_src=lsrc, scale_out=live, sf_layout=0, launch_with_pdl=True)
    _check(got, want[0])
    lq, ls, lg, lsrc = _late(hold, (q, s, g, src))
    _check([pkg.ts_nvfp4_dequantize(lq, ls, lg, row_src=lsrc, sf_layout=0, launch_with_pdl=True)], want[1])


@pytest.mark.parametrize("T,k,E,H", [(1, 2, 4, 64), (70, 3, 5, 1040), (300, 11, 16, 512), (2000, 8, 64, 128)])
def test_routing_reads_nothing_early(dev, hold, T, k, E, H):
    torch.manual_seed(T)
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device=dev)
    x, w, g = torch.randn(T, H, device=dev).bfloat16(), torch.rand(T, k, device=dev), torch.tensor([50.0], device=dev)
    rows = pkg.ts_moe_sort(ids, E)
    n = rows.row_src.numel()
    zeros = lambda: torch.zeros(n, H, dtype=torch.bfloat16, device=dev)  # noqa: E731
    codes = lambda: dict(quant_out=torch.zeros(n, H // 2, dtype=torch.uint8, device=dev),  # noqa: E731
                         scale_out=torch.zeros(n, H // 16, dtype=torch.uint8, device=dev), sf_layout=2)
    y = pkg.ts_moe_dispatch(x, rows, out=zeros())
    q = pkg.ts_moe_dispatch(x, rows, g, **codes())
    out = pkg.ts_moe_combine(y, rows, w)
    dy, dw = pkg.ts_moe_combine_grad(x, y, rows, w, dy=zeros())
    late, = _late(hold, (ids,))
    _check(pkg.ts_moe_sort(late, E, launch_with_pdl=True), rows)
    lx, of = _late(hold, (x, rows.row_of))
    _check([pkg.ts_moe_dispatch(lx, rows._replace(row_of=of), out=zeros(), launch_with_pdl=True)], [y])
    outs = codes()
    lx, of, lg = _late(hold, (x, rows.row_of, g))
    _check(pkg.ts_moe_dispatch(lx, rows._replace(row_of=of), lg, launch_with_pdl=True, **outs), q)
    ly, of, lw = _late(hold, (y, rows.row_of, w))
    _check([pkg.ts_moe_combine(ly, rows._replace(row_of=of), lw, launch_with_pdl=True)], [out])
    to = zeros()
    lx, ly, of, lw = _late(hold, (x, y, rows.row_of, w))
    _check(pkg.ts_moe_combine_grad(lx, ly, rows._replace(row_of=of), lw, dy=to, launch_with_pdl=True), [dy, dw])


@pytest.mark.parametrize("M,N,K", [(3, 136, 96), (3, 256, 4096), (40, 24576, 256), (300, 520, 320), (256, 264, 5408)])
def test_product_reads_nothing_early(dev, hold, M, N, K):
    _, _, ta, tas = ref.random_nvfp4(M, K, 1, dev)
    _, _, tb, tbs = ref.random_nvfp4(N, K, 2, dev)
    alpha = torch.tensor([0.37], device=dev)
    want = pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, alpha)
    _check([pkg.ts_nvfp4_gemm(*_late(hold, (ta, tas, tb, tbs, alpha)), launch_with_pdl=True)], [want])


@pytest.mark.parametrize("hint", (1, 100000), ids=("few", "many"))
def test_grouped_reads_nothing_early(dev, hold, hint):
    counts, N, K = [130, 0, 300, 5], 264, 288
    start = [0, 256, 256, 640, 768]
    E, rows = len(counts), start[-1]
    _, _, ta, tas = ref.random_nvfp4(rows, K, 5, dev)
    bs = [ref.random_nvfp4(N, K, 50 + e, dev) for e in range(E)]
    tb, tbs = torch.stack([b[2] for b in bs]), torch.stack([b[3] for b in bs])
    alpha = torch.arange(E, device=dev) + 0.5
    first, count = (torch.tensor(v, dtype=torch.int32, device=dev) for v in (start, counts))
    of = torch.empty(hint, 1, dtype=torch.int32, device=dev)
    want, got = (torch.zeros(rows, N, dtype=torch.bfloat16, device=dev) for _ in range(2))
    pkg.ts_nvfp4_grouped_gemm(ta, tas, tb, tbs, alpha, pkg.MoERows(of, None, first, count), out=want)
    la, las, lb, lbs, lalpha, lfirst, lcount = _late(hold, (ta, tas, tb, tbs, alpha, first, count))
    pkg.ts_nvfp4_grouped_gemm(la, las, lb, lbs, lalpha, pkg.MoERows(of, None, lfirst, lcount), out=got, launch_with_pdl=True)
    _check([got], [want])
