"""What of the attention kernels' ordering can be read in their sources only: no run shows that it is missing."""
import os
import re

import pytest

from reduce_residual_rmsnorm_gb300 import build as libbuild


def _code(name):
    with open(os.path.join(libbuild.CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ("rope_rows.cu", "attn_few.cu", "attn_prompt.cu", "attn_util.cuh", "f32x2.cuh", "async_copy.cuh"))
def test_no_load_through_the_non_coherent_path(name):
    """As tests/test_pdl_loads.py has it for the other kernels whose inputs the kernel before may have written."""
    assert re.findall(r"__ldg|ld_keep|ld\.global\S*\.nc|__restrict__", _code(name)) == []


def test_what_lanes_wrote_is_ordered_before_one_of_them_arrives():
    """The copying warp's lanes write where a step's tiles lie; one lane's arrival hands it over.  A vote between them orders
    no memory."""
    code = _code("attn_prompt.cu")
    written = code.index("seen[it & 3][lane] = in;")
    arrived = code.index("mbar_expect_tx(", written)
    assert "__syncwarp();" in code[written:arrived]
