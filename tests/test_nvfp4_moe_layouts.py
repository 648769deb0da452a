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


class _Library:
    """Keeps the layout that a fused call hands over."""

    def __init__(self):
        self.layouts = []

    def _call(self, outs):
        self.layouts.append(outs._obj.sf_layout)
        return 0

    def ts_fused_reduce_norm(self, *args):
        return self._call(args[9])

    def ts_reducescatter_fused_norm(self, *args):
        return self._call(args[11])


def test_fused_calls_hand_over_no_other_layout(monkeypatch):
    from reduce_residual_rmsnorm_gb300 import _binding

    fake = _Library()
    monkeypatch.setattr(_binding, "library", lambda path=None: fake)
    monkeypatch.setattr(_binding, "_dev", lambda t, name, dtype=None: t)
    x, g = torch.zeros(2, 32, dtype=torch.bfloat16), torch.ones(1)
    for layout in (0, 1, 2, 3, -1, *LAYOUTS):
        want = layout if layout in (0, 1, 2, 3) else -1
        pkg.ts_fused_reduce_norm(3, [x], x, x[0], 1e-6, g, residual_out=x.clone(), quant_out=x, scale_out=x, sf_layout=layout, stream=0)
        pkg.ts_reducescatter_fused_norm(3, [x], 0, residual=x, gamma=x[0], scale_factor=g, residual_out=x.clone(), quant_out=x,
                                        scale_out=x, sf_layout=layout, stream=0)
        assert fake.layouts[-2:] == [want, want], layout


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
