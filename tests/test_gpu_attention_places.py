"""Where the attention calls put what they are not given."""
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def test_the_cache_read_back_is_where_the_cache_is(dev):
    T, hk, D, page = 20, 2, 64, 16
    g = torch.Generator(device=dev).manual_seed(0)
    k, v = (torch.randn(T, hk, D, generator=g, device=dev).bfloat16() for _ in range(2))
    one = torch.tensor([300.0], device=dev)
    cache = pkg.ts_kv_cache(2, hk, D, one, one, page_size=page, device=dev)
    slots = torch.randperm(2 * page, generator=g, device=dev)[:T].int()
    pkg.ts_qk_norm_rope(k, k, None, None, torch.zeros_like(slots), ref.angles(1, D).to(dev), v=v, cache=cache, slots=slots)
    want = pkg.ts_kv_cache_read(cache, slots)
    host = pkg.KVCache(cache.pages.cpu().pin_memory(), one, one)
    for c, s, on_gpu in ((cache, slots.cpu().pin_memory(), True), (host, slots, False), (host, slots.cpu().pin_memory(), False)):
        got = pkg.ts_kv_cache_read(c, s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert a.is_cuda == on_gpu and (on_gpu or a.is_pinned())
            assert torch.equal(a.cpu(), b.cpu())


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one device: the current one and the tensors' are the same")
def test_a_new_workspace_is_on_the_device_that_the_call_runs_on(dev):
    """Rows in host memory with lists on a device that is not the current one: the call runs there."""
    T, h, D = 30, 2, 64
    other = torch.device("cuda:1")
    g = torch.Generator().manual_seed(0)
    dq, dk, q, k = (torch.randn(T, h, D, generator=g).bfloat16().pin_memory() for _ in range(4))
    w, pos, table = torch.ones(D).bfloat16().to(other), torch.arange(T).int().to(other), ref.angles(T, D).to(other)
    with torch.cuda.device(0):
        before = torch.cuda.memory_stats(other)["allocation.all.allocated"]
        pkg.ts_qk_norm_rope_grad(dq, dk, q, k, w, w, pos, table)
        torch.cuda.synchronize(other)
        assert torch.cuda.memory_stats(other)["allocation.all.allocated"] > before
