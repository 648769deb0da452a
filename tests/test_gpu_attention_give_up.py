"""Prompt attention whose waits run out: every block ends in time and counts the wait, writes nothing outside its outputs
and workspace (and where a unit is one block's alone, nothing wrong), leaves nothing in flight towards the memory that it gives back, and the next call is right.

As tests/test_gpu_give_up.py has it for the product kernels."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from reduce_residual_rmsnorm_gb300 import build as libbuild
from tests.gpu_util import Guarded
from tests.test_gpu_attention import _cache, _rand

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
    out = tmp_path_factory.mktemp("give_up") / "libattention_give_up_probe.so"
    subprocess.check_call([libbuild.nvcc(), *libbuild.ARCH, *libbuild.NVCC_FLAGS, "-shared", "-cudart", "static",
                           os.path.join(ROOT, "tests", "attention_give_up_probe.cu"), "-o", str(out)])
    lib = ctypes.CDLL(str(out))
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.set_run_out.argtypes = [i64]
    lib.stalls.argtypes = [vp]
    lib.workspace.argtypes, lib.workspace.restype = [i64], i64
    lib.squat.argtypes = [vp, vp]
    lib.attend.argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, i64, i64, vp, vp, vp, i64, vp, ctypes.c_float, vp, vp, vp, ctypes.c_int, vp]
    return lib


def _stalls(lib):
    n = ctypes.c_uint32(0)
    assert lib.stalls(ctypes.byref(n)) == 0
    return n.value


# (queries, lengths, query heads, key heads, D, whether every unit is one block's alone): 152 units of 256 rows and 4
# steps, one a block; units over several blocks, some of one tile of rows, with many steps and few
CASES = [([32] * 19, [500] * 19, 64, 8, 128, True), ([64] * 19, [500] * 19, 32, 8, 64, True), ([300, 20, 1], [5000, 100, 30], 8, 2, 128, False),
         ([17, 700], [20000, 900], 10, 2, 64, False)]


@pytest.mark.parametrize("new,lens,hq,hk,D,alone", CASES)
def test_prompts(dev, probe, new, lens, hq, hk, D, alone):
    page, T, B = 32, sum(new), len(new)
    cache, table = _cache(dev, lens, hk, D, page, 3)
    q = _rand((T, hq, D), dev, 1)
    cu, kv = (torch.tensor(v, dtype=torch.int32, device=dev) for v in ([0, *np.cumsum(new)], lens))
    want = pkg.ts_nvfp4_attention(q, cache, table, kv, cu, max_q=max(new), return_lse=True)
    out, lse = Guarded((T, hq, D), torch.bfloat16, dev), Guarded((T, hq), torch.float32, dev)
    space = Guarded((probe.workspace(D),), torch.uint8, dev)
    bad = torch.zeros(1, dtype=torch.int32, device=dev)
    stream = torch.cuda.current_stream().cuda_stream
    fills = out.t.clone(), lse.t.clone()
    ran_out = []

    def attend(join):
        return probe.attend(q.data_ptr(), T, hq, cu.data_ptr(), B, cache.pages.data_ptr(), cache.pages.shape[0], page, hk, D,
                            cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), table.data_ptr(), table.shape[1], kv.data_ptr(),
                            1 / math.sqrt(D), out.t.data_ptr(), lse.t.data_ptr(), space.t.data_ptr(), join, stream)

    try:
        for cycles in [*range(0, 40000, 500), *range(40000, 200000, 8000), NEVER]:
            out.t.copy_(fills[0])
            lse.t.copy_(fills[1])
            before = _stalls(probe)
            assert probe.set_run_out(cycles) == 0
            assert attend(0) == 0 and probe.squat(bad.data_ptr(), stream) == 0 and attend(1) == 0
            ran_out.append(_stalls(probe) - before)  # (waits for the device)
            assert out.intact() and lse.intact() and space.intact() and int(bad) == 0, cycles
            for got, right, fill, bits in ((out.t, want[0], fills[0], torch.int16), (lse.t, want[1], fills[1], torch.int32)):
                same = got.view(bits) == right.view(bits)
                assert not alone or bool((same | (got.view(bits) == fill.view(bits))).all()), cycles
                assert ran_out[-1] != 0 or bool(same.all()), cycles
    finally:
        assert probe.set_run_out(NEVER) == 0
    assert ran_out[0] > 0 and ran_out[-1] == 0 and 0 < sum(n > 0 for n in ran_out) < len(ran_out)
    again = pkg.ts_nvfp4_attention(q, cache, table, kv, cu, max_q=max(new), return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(again, want)) and pkg.ts_stalled_waits() == 0
