"""Where the buffers of the products may be: operands and output, which the tensor copy engine reads and writes, on the
GPU; alpha and the experts' starts and counts there or in page-locked host memory."""
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from tests import nvfp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("M", (3, 90, 300))
def test_dense(dev, M):
    N, K = 136, 96
    _, _, ta, tas = ref.random_nvfp4(M, K, 1, dev)
    _, _, tb, tbs = ref.random_nvfp4(N, K, 2, dev)
    alpha = torch.tensor([0.3])
    want = pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, alpha.to(dev))
    assert torch.equal(pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, alpha.pin_memory()), want)
    with pytest.raises(TypeError, match="out must be a CUDA tensor"):
        pkg.ts_nvfp4_gemm(ta, tas, tb, tbs, alpha.to(dev), out=torch.empty(M, N, dtype=torch.bfloat16).pin_memory())


@pytest.mark.parametrize("hint", (1, 100000))
def test_grouped(dev, hint):
    N, K, E, rows = 136, 96, 2, 256
    _, _, ta, tas = ref.random_nvfp4(rows, K, 1, dev)
    bs = [ref.random_nvfp4(N, K, 2 + e, dev) for e in range(E)]
    tb, tbs = torch.stack([b[2] for b in bs]), torch.stack([b[3] for b in bs])
    alpha, start, count = torch.tensor([0.3, 0.7]), torch.tensor([0, 128, 256]).int(), torch.tensor([7, 100]).int()
    of = torch.empty(hint, 1, dtype=torch.int32, device=dev)
    outs = []
    for place in (lambda t: t.to(dev), lambda t: t.pin_memory()):
        outs.append(torch.zeros(rows, N, dtype=torch.bfloat16, device=dev))
        pkg.ts_nvfp4_grouped_gemm(ta, tas, tb, tbs, place(alpha), pkg.MoERows(of, None, place(start), place(count)), out=outs[-1])
    assert torch.equal(*outs)
    with pytest.raises(TypeError, match="out must be a CUDA tensor"):
        pkg.ts_nvfp4_grouped_gemm(ta, tas, tb, tbs, alpha.to(dev), pkg.MoERows(of, None, start.to(dev), count.to(dev)),
                                  out=torch.empty(rows, N, dtype=torch.bfloat16).pin_memory())
