"""The kernels whose inputs may be outputs of the kernel before read none of them through the non-coherent path: its
loads are for memory that nothing writes while the kernel runs, and a dependent launch begins before the writes."""
import os
import re

import pytest

from reduce_residual_rmsnorm_gb300 import build as libbuild


@pytest.mark.parametrize("name", ("moe_rows.cu", "nvfp4_rows.cu", "nvfp4_gemm.cu", "tcgen05.cuh"))
def test_no_load_through_the_non_coherent_path(name):
    with open(os.path.join(libbuild.CSRC, name), encoding="utf-8") as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert re.findall(r"__ldg|ld_keep|ld\.global\S*\.nc|__restrict__", code) == []
