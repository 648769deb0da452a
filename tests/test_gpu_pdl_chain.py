"""Products behind a kernel that lets them start early and then holds the stream for longer than a wait inside a
product may take (4e9 cycles, about 2 s): the product waits for it, and its own waits begin afterwards."""
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
