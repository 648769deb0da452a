"""Product kernels whose waits run out: every block ends in time and counts the wait, writes nothing but right values
inside the output, leaves nothing in flight towards the shared memory that it gives back, and the next call is right.

The kernels are built for it once more, with waits that run out at a chosen time after a block's start (every role of
a block gives up there, wherever it is in its work) and a limit of 1 ms for what is in flight then."""
import ctypes
import os
import subprocess

import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from reduce_residual_rmsnorm_gb300 import build as libbuild
from tests import nvfp4_ref as ref
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NEVER = 1 << 62


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def probe(dev, tmp_path_factory):
    out = tmp_path_factory.mktemp("give_up") / "libgive_up_probe.so"
    subprocess.check_call([libbuild.nvcc(), *libbuild.ARCH, *libbuild.NVCC_FLAGS, "-shared", "-cudart", "static",
                           os.path.join(ROOT, "tests", "give_up_probe.cu"), "-o", str(out)])
    lib = ctypes.CDLL(str(out))
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.set_run_out.argtypes = [i64]
    lib.stalls.argtypes = [vp]
    lib.squat.argtypes = [vp, vp]
    lib.product.argtypes = [vp] * 7 + [i64] * 5 + [vp, i64, vp]
    return lib


def _stalls(lib):
    n = ctypes.c_uint32(0)
    assert lib.stalls(ctypes.byref(n)) == 0
    return n.value


def _sweep(dev, lib, call, out, want):
    """`call` with waits that run out ever later, until none does."""
    bad = torch.zeros(1, dtype=torch.int32, device=dev)
    stream = torch.cuda.current_stream().cuda_stream
    fill = out.t.clone()
    ran_out = []
    try:
        for cycles in [*range(0, 12000, 250), *range(12000, 60000, 2000), NEVER]:
            out.t.copy_(fill)
            before = _stalls(lib)
            assert lib.set_run_out(cycles) == 0
            assert call(stream) == 0 and lib.squat(bad.data_ptr(), stream) == 0
            ran_out.append(_stalls(lib) - before)  # (waits for the device)
            got = out.t.view(torch.int16)
            assert ((got == want.view(torch.int16)) | (got == fill.view(torch.int16))).all(), cycles
            assert out.intact() and int(bad) == 0, cycles
            if ran_out[-1] == 0:
                assert torch.equal(got, want.view(torch.int16)), cycles
    finally:
        assert lib.set_run_out(NEVER) == 0
    assert ran_out[0] > 0 and ran_out[-1] == 0
    return ran_out


# few tokens: alone, K over a cluster, several tiles a block, 128 columns; pairs: one and many tiles, 192 and 256 rows
# of weights, K over two pairs
@pytest.mark.parametrize("M,N,K", [(3, 136, 96), (3, 256, 4096), (40, 24576, 1056), (90, 264, 5152), (300, 520, 320),
                                   (2048, 5120, 1056), (4096, 7168, 2080), (256, 264, 5408)])
def test_dense(dev, probe, M, N, K):
    _, _, ta, tas = ref.random_nvfp4(M, K, 1, dev)
    _, _, tb, tbs = ref.random_nvfp4(N, K, 2, dev)
    one = torch.ones(1, device=dev)
    want = pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, one)
    out = Guarded((M, N), torch.bfloat16, dev)
    _sweep(dev, probe, lambda stream: probe.product(ta.data_ptr(), tas.data_ptr(), tb.data_ptr(), tbs.data_ptr(),
                                                    one.data_ptr(), None, None, 0, M, 0, N, K, out.t.data_ptr(), N, stream),
           out, want)


@pytest.mark.parametrize("hint", (1, 100000), ids=("few", "many"))
def test_grouped(dev, probe, hint):
    counts, N, K = [300, 0, 513, 5, 128], 1032, 1056
    E, start = len(counts), [0]
    for c in counts:
        start.append(start[-1] + ref.up(c, 128))
    rows = start[-1]
    _, _, ta, tas = ref.random_nvfp4(rows, K, 5, dev)
    bs = [ref.random_nvfp4(N, K, 50 + e, dev) for e in range(E)]
    tb, tbs = torch.stack([b[2] for b in bs]), torch.stack([b[3] for b in bs])
    alpha = torch.ones(E, device=dev)
    first, count = (torch.tensor(v, dtype=torch.int32, device=dev) for v in (start, counts))
    out = Guarded((rows, N), torch.bfloat16, dev)
    want = out.t.clone()
    pkg.ts_nvfp4_grouped_gemm(ta, tas, tb, tbs, alpha,
                              pkg.MoERows(torch.empty(hint, 1, dtype=torch.int32, device=dev), None, first, count), out=want)
    _sweep(dev, probe, lambda stream: probe.product(ta.data_ptr(), tas.data_ptr(), tb.data_ptr(), tbs.data_ptr(),
                                                    alpha.data_ptr(), first.data_ptr(), count.data_ptr(), E, rows, hint, N, K,
                                                    out.t.data_ptr(), N, stream), out, want)
