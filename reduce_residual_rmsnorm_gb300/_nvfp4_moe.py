"""The NVFP4 and expert-routing entry points on tensors (include/ts_nvfp4_moe.h).

Shapes, types and places are checked in csrc/python_calls.cpp, everything else
by the library, whose statuses become ``TsError``.  A call runs on the tensors'
device, on that device's current stream unless ``stream`` is given (a
``torch.cuda.Stream`` or a raw handle), and allocates the outputs it is not
given.  ``launch_with_pdl``: programmatic dependent launch (TS_FLAG_PDL).
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

from ._binding import SFLayout, _check, library
from .build import CALLS_PATH, calls_match

_calls = None


def _native():
    """The compiled calls (built by ``__graft_entry__.build()``), loaded on the first one."""
    global _calls
    if _calls is None:
        library()
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError(f"{CALLS_PATH} is missing: build the CUDA library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        if not calls_match():
            raise RuntimeError(f"{CALLS_PATH} was built for another PyTorch or Python: build the CUDA library again "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        from . import _python_calls
        _calls = _python_calls
    return _calls


class MoERows(NamedTuple):
    """Where ``ts_moe_sort`` put the (token, slot) entries."""
    row_of: torch.Tensor        # int32 [T, k]: the entry's row, -1 without one
    row_src: torch.Tensor       # int32 [rows]: the row's entry t*k + slot, -1 without one
    expert_start: torch.Tensor  # int32 [E + 1]: an expert's first row
    expert_count: torch.Tensor  # int32 [E]: an expert's entries


def ts_nvfp4_quantize(x: torch.Tensor, scale_factor: torch.Tensor, *, row_src: torch.Tensor | None = None,
                      quant_out: torch.Tensor | None = None, scale_out: torch.Tensor | None = None,
                      sf_layout: int = SFLayout.LINEAR, launch_with_pdl: bool = False, stream=None):
    """bf16 rows ``x`` [T, K] to NVFP4 with the global scale ``scale_factor`` (fp32, one value).

    Returns (codes uint8 [T, K/2], scale factors uint8 of ``sf_shape(T, K, sf_layout)``).  With ``row_src`` (of
    ``ts_moe_sort``) the rows without an entry are left out.
    """
    return _native().quantize(x, scale_factor, row_src, quant_out, scale_out, sf_layout, launch_with_pdl, stream)


def ts_nvfp4_dequantize(quant: torch.Tensor, scale: torch.Tensor, scale_factor: torch.Tensor, *,
                        sf_layout: int = SFLayout.LINEAR, row_src: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None) -> torch.Tensor:
    """The bf16 values [T, K] that codes [T, K/2], their scale factors and the global scale stand for."""
    return _native().dequantize(quant, scale, scale_factor, sf_layout, row_src, out, launch_with_pdl, stream)


def ts_nvfp4_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                  alpha: torch.Tensor, *, out: torch.Tensor | None = None, launch_with_pdl: bool = False,
                  stream=None) -> torch.Tensor:
    """``out`` [M, N] = bf16(alpha A B^T) of NVFP4 codes ``a`` [M, K/2] and ``b`` [N, K/2] with SWIZZLED_128x4
    scale factors; ``alpha`` (fp32, one value) is 1 / (g_A g_B)."""
    return _native().gemm(a, a_scale, b, b_scale, alpha, out, launch_with_pdl, stream)


def ts_moe_rows(T: int, k: int, num_experts: int, row_align: int = 1) -> int:
    """Rows that hold the sorted entries of any routing of T tokens to k of ``num_experts`` experts each."""
    n = int(library().ts_moe_rows(int(T), int(k), int(num_experts), int(row_align)))
    if n < 0:
        raise ValueError(f"ts_moe_rows: T={T}, k={k}, num_experts={num_experts}, row_align={row_align} out of range")
    return n


def ts_moe_sort(expert_ids: torch.Tensor, num_experts: int, *, row_align: int = 1, rows: MoERows | None = None,
                launch_with_pdl: bool = False, stream=None) -> MoERows:
    """The stable order by expert of int32 ``expert_ids`` [T, k]; ids outside 0..num_experts-1 get no row.

    ``row_align``: each expert's rows start at a multiple of it (128 for the NVFP4 products).  ``rows``: buffers of
    an earlier call to write into; ``row_src`` may be longer than ``ts_moe_rows``.
    """
    of, src, start, count = rows if rows is not None else (None, None, None, None)
    return MoERows._make(_native().sort(expert_ids, num_experts, row_align, of, src, start, count, launch_with_pdl, stream))


def ts_moe_dispatch(x: torch.Tensor, rows: MoERows, scale_factor: torch.Tensor | None = None, *,
                    out: torch.Tensor | None = None, quant_out: torch.Tensor | None = None,
                    scale_out: torch.Tensor | None = None, sf_layout: int = SFLayout.SWIZZLED_128x4,
                    launch_with_pdl: bool = False, stream=None):
    """Token rows ``x`` [T, H] in expert order: bf16 [rows, H], or with ``scale_factor`` NVFP4 codes and scale factors.

    Rows without an entry are left as they were.  Returns ``out`` or (quant_out, scale_out).
    """
    return _native().dispatch(x, rows.row_of, rows.row_src.numel(), scale_factor, out, quant_out, scale_out, sf_layout,
                              launch_with_pdl, stream)


def ts_nvfp4_grouped_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                          alpha: torch.Tensor, rows: MoERows, *, out: torch.Tensor | None = None,
                          launch_with_pdl: bool = False, stream=None) -> torch.Tensor:
    """Each expert's NVFP4 product with its own rows: ``a`` [rows, K/2] sorted with row_align 128, ``b`` [E, N, K/2],
    ``b_scale`` [E, ceil(N/128)*128, ceil(K/64)*4], ``alpha`` fp32 [E].  Returns ``out`` bf16 [rows, N], in which the
    rows without an entry are left as they were."""
    return _native().grouped_gemm(a, a_scale, b, b_scale, alpha, rows.expert_start, rows.expert_count, rows.row_of.numel(),
                                  out, launch_with_pdl, stream)


def ts_moe_combine(y: torch.Tensor, rows: MoERows, weights: torch.Tensor | None = None, *,
                   out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None) -> torch.Tensor:
    """The experts' rows ``y`` [rows, H] weighted (fp32 [T, k]; None: 1) and summed back into token order: bf16 [T, H].

    Without weights it is the gradient of ``ts_moe_dispatch``.
    """
    return _native().combine(y, rows.row_of, weights, out, launch_with_pdl, stream)


def ts_moe_combine_grad(dout: torch.Tensor, y: torch.Tensor, rows: MoERows, weights: torch.Tensor, *,
                        dy: torch.Tensor | None = None, dweights: torch.Tensor | None = None,
                        launch_with_pdl: bool = False, stream=None):
    """The gradient of ``ts_moe_combine`` for ``dout`` [T, H]: (dy bf16 like ``y``, dweights fp32 [T, k]).

    Rows of ``dy`` without an entry are left as they were.
    """
    return _native().combine_grad(dout, y, rows.row_of, weights, dy, dweights, launch_with_pdl, stream)


def ts_stalled_waits() -> int:
    """Waits inside the product kernels of the current device that ran into their limit (0 unless something is wrong)."""
    n = ctypes.c_uint32(0)
    _check(library().ts_stalled_waits(ctypes.byref(n)))
    return n.value
