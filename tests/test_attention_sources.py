"""What of the attention kernels' ordering can be read in their sources only: no run shows that it is missing."""
import os
import re
import subprocess

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


def test_the_prompt_kernel_is_launched_with_the_registers_that_its_roles_divide(tmp_path):
    """Its warps take 192, 72 and 56 of the 128 registers a thread that a block of 512 is launched with; with fewer,
    the division would wait for ever (the launch refuses it), and the build is the place to see that."""
    cmd = [libbuild.nvcc(), *libbuild.ARCH, *libbuild.NVCC_FLAGS, "-Xptxas", "-v", "-c", os.path.join(libbuild.CSRC, "attn_prompt.cu"),
           "-o", str(tmp_path / "attn_prompt.o")]
    log = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    used = re.findall(r"Compiling entry function '\S*attn_prompt_kernel\S*'.*?Used (\d+) registers", log, flags=re.S)
    assert used == ["128", "128"]
