"""A scale-factor layout that is none is refused before anything else, also one that is a layout in its low 32 bits: the
binding would size the outputs by the number that it was given and the library write by the other."""
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from reduce_residual_rmsnorm_gb300 import build as libbuild

BAD_PATTERN = -1


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()


def _calls(device):
    f, x = torch.ones(1, device=device), torch.zeros(4, 64, device=device).bfloat16()
    q, s = torch.zeros(4, 32, dtype=torch.uint8, device=device), torch.zeros(8, 4, dtype=torch.uint8, device=device)
    rows = pkg.MoERows(torch.zeros(4, 1, dtype=torch.int32, device=device), torch.zeros(4, dtype=torch.int32, device=device),
                       None, None)
    return (lambda v: pkg.ts_nvfp4_quantize(x, f, sf_layout=v), lambda v: pkg.ts_nvfp4_dequantize(q, s, f, sf_layout=v),
            lambda v: pkg.ts_moe_dispatch(x, rows, f, sf_layout=v))


LAYOUTS = (3, -1, 1 << 32, (1 << 32) + 1, (1 << 32) + 2, -(1 << 32), 1 << 62)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_refused_without_a_gpu(layout):
    for call in _calls("cpu"):
        with pytest.raises(pkg.TsError) as e:
            call(layout)
        assert e.value.status == BAD_PATTERN and str(layout) in str(e.value)


def test_no_number():
    for call in _calls("cpu"):
        with pytest.raises(TypeError):
            call("linear")
        with pytest.raises(OverflowError):
            call(1 << 64)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_refused(layout):
    for call in _calls("cuda:0"):
        with pytest.raises(pkg.TsError) as e:
            call(layout)
        assert e.value.status == BAD_PATTERN


@pytest.mark.gpu
def test_taken():
    for call in _calls("cuda:0")[:1]:
        for layout in pkg.SFLayout:
            assert tuple(call(layout)[1].shape) == pkg.sf_shape(4, 64, layout)
