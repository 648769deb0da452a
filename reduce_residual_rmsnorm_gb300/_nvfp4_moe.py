"""Binding of the NVFP4 and expert-routing entry points (include/ts_nvfp4_moe.h).

Argument marshalling only, as in ``_binding``: shapes, types and places are
checked here, everything else by the library, whose statuses become
``TsError``.  A call runs on the tensors' device, on that device's current
stream unless ``stream`` is given, and allocates the outputs it is not given.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

import torch

from ._binding import TS_FLAG_PDL, SFLayout, _check, _dev, _empty_like_place, _ptr, _stream, library, sf_shape

_I32, _F32, _U8, _BF16 = torch.int32, torch.float32, torch.uint8, torch.bfloat16


class MoERows(NamedTuple):
    """Where ``ts_moe_sort`` put the (token, slot) entries."""
    row_of: torch.Tensor        # int32 [T, k]: the entry's row, -1 without one
    row_src: torch.Tensor       # int32 [rows]: the row's entry t*k + slot, -1 without one
    expert_start: torch.Tensor  # int32 [E + 1]: an expert's first row
    expert_count: torch.Tensor  # int32 [E]: an expert's entries


@contextlib.contextmanager
def _on(stream, tensors):
    """The stream argument of a call on these tensors, with their device current."""
    devices = {t.device for t in tensors if t is not None and t.is_cuda}
    if len(devices) > 1:
        raise ValueError(f"tensors on different devices: {sorted(str(d) for d in devices)}")
    device = devices.pop() if devices else None
    if device is None or device.index == torch.cuda.current_device():
        yield _stream(stream)
    else:
        with torch.cuda.device(device):
            yield _stream(stream)


def _flat(t, name, dtype, shape=None):
    """A contiguous tensor of a type (and shape)."""
    _dev(t, name, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _on_gpu(t, name, dtype, shape=None):
    """As _flat, in device memory (the tensor copy engine reads it)."""
    _flat(t, name, dtype, shape)
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t


def _matrix(t, name, shape=None):
    """A bf16 matrix with unit column stride; its row stride."""
    _dev(t, name, _BF16)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    # (a single row has no stride that matters; torch may report any)
    return int(t.stride(0)) if t.shape[0] > 1 else max(int(t.stride(0)), -(-t.shape[1] // 8) * 8)


def _one(t, name):
    _dev(t, name, _F32)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one value")
    return t


def _flags(launch_with_pdl):
    return TS_FLAG_PDL if launch_with_pdl else 0


def ts_nvfp4_quantize(x: torch.Tensor, scale_factor: torch.Tensor, *, row_src: torch.Tensor | None = None,
                      quant_out: torch.Tensor | None = None, scale_out: torch.Tensor | None = None,
                      sf_layout: int = SFLayout.LINEAR, launch_with_pdl: bool = False, stream=None):
    """bf16 rows ``x`` [T, K] to NVFP4 with the global scale ``scale_factor`` (fp32, one value).

    Returns (codes uint8 [T, K/2], scale factors uint8 of ``sf_shape(T, K, sf_layout)``).  With ``row_src`` (of
    ``ts_moe_sort``) the rows without an entry are left out.
    """
    ldx = _matrix(x, "x")
    T, K = x.shape
    _one(scale_factor, "scale_factor")
    if row_src is not None:
        _flat(row_src, "row_src", _I32, (T,))
    if quant_out is None:
        quant_out = _empty_like_place((T, K // 2), _U8, x)
    if scale_out is None:
        scale_out = _empty_like_place(sf_shape(T, K, sf_layout), _U8, x)
    _flat(quant_out, "quant_out", _U8, (T, K // 2))
    _flat(scale_out, "scale_out", _U8, sf_shape(T, K, sf_layout))
    with _on(stream, (x, scale_factor, row_src, quant_out, scale_out)) as s:
        _check(library().ts_nvfp4_quantize(_ptr(x), T, K, ldx, _ptr(scale_factor), _ptr(row_src), _ptr(quant_out),
                                           _ptr(scale_out), int(sf_layout), _flags(launch_with_pdl), s))
    return quant_out, scale_out


def ts_nvfp4_dequantize(quant: torch.Tensor, scale: torch.Tensor, scale_factor: torch.Tensor, *,
                        sf_layout: int = SFLayout.LINEAR, row_src: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """The bf16 values [T, K] that codes [T, K/2], their scale factors and the global scale stand for."""
    _flat(quant, "quant", _U8)
    if quant.dim() != 2:
        raise ValueError("quant must be [T, K/2]")
    T, K = quant.shape[0], 2 * quant.shape[1]
    _flat(scale, "scale", _U8, sf_shape(T, K, sf_layout))
    _one(scale_factor, "scale_factor")
    if row_src is not None:
        _flat(row_src, "row_src", _I32, (T,))
    if out is None:
        out = _empty_like_place((T, K), _BF16, quant)
    ldo = _matrix(out, "out", (T, K))
    with _on(stream, (quant, scale, scale_factor, row_src, out)) as s:
        _check(library().ts_nvfp4_dequantize(_ptr(quant), _ptr(scale), int(sf_layout), T, K, _ptr(scale_factor),
                                             _ptr(row_src), _ptr(out), ldo, _flags(launch_with_pdl), s))
    return out


def ts_nvfp4_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                  alpha: torch.Tensor, *, out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """``out`` [M, N] = bf16(alpha A B^T) of NVFP4 codes ``a`` [M, K/2] and ``b`` [N, K/2] with SWIZZLED_128x4
    scale factors; ``alpha`` (fp32, one value) is 1 / (g_A g_B)."""
    _on_gpu(a, "a", _U8)
    _on_gpu(b, "b", _U8)
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError("a must be [M, K/2] and b [N, K/2]")
    M, N, K = a.shape[0], b.shape[0], 2 * a.shape[1]
    _on_gpu(a_scale, "a_scale", _U8, sf_shape(M, K, SFLayout.SWIZZLED_128x4))
    _on_gpu(b_scale, "b_scale", _U8, sf_shape(N, K, SFLayout.SWIZZLED_128x4))
    _one(alpha, "alpha")
    if out is None:
        out = torch.empty((M, N), dtype=_BF16, device=a.device)
    ldo = _matrix(out, "out", (M, N))
    with _on(stream, (a, a_scale, b, b_scale, alpha, out)) as s:
        _check(library().ts_nvfp4_gemm(_ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale), _ptr(alpha), M, N, K, _ptr(out),
                                       ldo, _flags(launch_with_pdl), s))
    return out


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
    _flat(expert_ids, "expert_ids", _I32)
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be [T, k]")
    T, k = expert_ids.shape
    if rows is None:
        cap = ts_moe_rows(T, k, num_experts, row_align)
        rows = MoERows(*(_empty_like_place(s, _I32, expert_ids)
                         for s in ((T, k), (cap,), (num_experts + 1,), (num_experts,))))
    _flat(rows.row_of, "rows.row_of", _I32, (T, k))
    _flat(rows.row_src, "rows.row_src", _I32)
    _flat(rows.expert_start, "rows.expert_start", _I32, (num_experts + 1,))
    _flat(rows.expert_count, "rows.expert_count", _I32, (num_experts,))
    with _on(stream, (expert_ids, *rows)) as s:
        _check(library().ts_moe_sort(_ptr(expert_ids), T, k, int(num_experts), int(row_align), rows.row_src.numel(),
                                     _ptr(rows.row_of), _ptr(rows.row_src), _ptr(rows.expert_start),
                                     _ptr(rows.expert_count), _flags(launch_with_pdl), s))
    return rows


def ts_moe_dispatch(x: torch.Tensor, rows: MoERows, scale_factor: torch.Tensor | None = None, *,
                    out: torch.Tensor | None = None, quant_out: torch.Tensor | None = None,
                    scale_out: torch.Tensor | None = None, sf_layout: int = SFLayout.SWIZZLED_128x4,
                    launch_with_pdl: bool = False, stream=None):
    """Token rows ``x`` [T, H] in expert order: bf16 [rows, H], or with ``scale_factor`` NVFP4 codes and scale factors.

    Rows without an entry are left as they were.  Returns ``out`` or (quant_out, scale_out).
    """
    ldx = _matrix(x, "x")
    T, H = x.shape
    _flat(rows.row_of, "rows.row_of", _I32)
    if rows.row_of.dim() != 2 or rows.row_of.shape[0] != T:
        raise ValueError("rows.row_of must be [T, k]")
    n, k = rows.row_src.numel(), rows.row_of.shape[1]
    if scale_factor is None:
        if quant_out is not None or scale_out is not None:
            raise ValueError("quant_out and scale_out need scale_factor")
        if out is None:
            out = _empty_like_place((n, H), _BF16, x)
        _flat(out, "out", _BF16, (n, H))
        bufs = (_ptr(out), None, None, None)
    else:
        if out is not None:
            raise ValueError("out and scale_factor exclude each other")
        _one(scale_factor, "scale_factor")
        if quant_out is None:
            quant_out = _empty_like_place((n, H // 2), _U8, x)
        if scale_out is None:
            scale_out = _empty_like_place(sf_shape(n, H, sf_layout), _U8, x)
        _flat(quant_out, "quant_out", _U8, (n, H // 2))
        _flat(scale_out, "scale_out", _U8, sf_shape(n, H, sf_layout))
        bufs = (None, _ptr(scale_factor), _ptr(quant_out), _ptr(scale_out))
    with _on(stream, (x, rows.row_of, out, scale_factor, quant_out, scale_out)) as s:
        _check(library().ts_moe_dispatch(_ptr(x), T, H, ldx, _ptr(rows.row_of), k, n, *bufs, int(sf_layout),
                                         _flags(launch_with_pdl), s))
    return out if scale_factor is None else (quant_out, scale_out)


def ts_nvfp4_grouped_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                          alpha: torch.Tensor, rows: MoERows, *, out: torch.Tensor | None = None,
                          launch_with_pdl: bool = False, stream=None):
    """Each expert's NVFP4 product with its own rows: ``a`` [rows, K/2] sorted with row_align 128, ``b`` [E, N, K/2],
    ``b_scale`` [E, ceil(N/128)*128, ceil(K/64)*4], ``alpha`` fp32 [E].  Returns ``out`` bf16 [rows, N], in which the
    rows without an entry are left as they were."""
    _on_gpu(a, "a", _U8)
    _on_gpu(b, "b", _U8)
    if a.dim() != 2 or b.dim() != 3 or a.shape[1] != b.shape[2]:
        raise ValueError("a must be [rows, K/2] and b [E, N, K/2]")
    n, K = a.shape[0], 2 * a.shape[1]
    E, N = b.shape[:2]
    _on_gpu(a_scale, "a_scale", _U8, sf_shape(n, K, SFLayout.SWIZZLED_128x4))
    _on_gpu(b_scale, "b_scale", _U8, (E, *sf_shape(N, K, SFLayout.SWIZZLED_128x4)))
    _flat(alpha, "alpha", _F32, (E,))
    _flat(rows.expert_start, "rows.expert_start", _I32, (E + 1,))
    _flat(rows.expert_count, "rows.expert_count", _I32, (E,))
    if out is None:
        out = torch.empty((n, N), dtype=_BF16, device=a.device)
    ldo = _matrix(out, "out", (n, N))
    with _on(stream, (a, a_scale, b, b_scale, alpha, rows.expert_start, rows.expert_count, out)) as s:
        _check(library().ts_nvfp4_grouped_gemm(_ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale), _ptr(alpha),
                                               _ptr(rows.expert_start), _ptr(rows.expert_count), E, n,
                                               rows.row_of.numel(), N, K, _ptr(out), ldo, _flags(launch_with_pdl), s))
    return out


def ts_moe_combine(y: torch.Tensor, rows: MoERows, weights: torch.Tensor | None = None, *,
                   out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """The experts' rows ``y`` [rows, H] weighted (fp32 [T, k]; None: 1) and summed back into token order: bf16 [T, H].

    Without weights it is the gradient of ``ts_moe_dispatch``.
    """
    ldy = _matrix(y, "y")
    n, H = y.shape
    _flat(rows.row_of, "rows.row_of", _I32)
    if rows.row_of.dim() != 2:
        raise ValueError("rows.row_of must be [T, k]")
    T, k = rows.row_of.shape
    if weights is not None:
        _flat(weights, "weights", _F32, (T, k))
    if out is None:
        out = _empty_like_place((T, H), _BF16, y)
    ldo = _matrix(out, "out", (T, H))
    with _on(stream, (y, rows.row_of, weights, out)) as s:
        _check(library().ts_moe_combine(_ptr(y), n, H, ldy, _ptr(rows.row_of), _ptr(weights), T, k, _ptr(out), ldo,
                                        _flags(launch_with_pdl), s))
    return out


def ts_moe_combine_grad(dout: torch.Tensor, y: torch.Tensor, rows: MoERows, weights: torch.Tensor, *,
                        dy: torch.Tensor | None = None, dweights: torch.Tensor | None = None,
                        launch_with_pdl: bool = False, stream=None):
    """The gradient of ``ts_moe_combine`` for ``dout`` [T, H]: (dy bf16 like ``y``, dweights fp32 [T, k]).

    Rows of ``dy`` without an entry are left as they were.
    """
    ldd, ldy = _matrix(dout, "dout"), _matrix(y, "y")
    n, H = y.shape
    _flat(rows.row_of, "rows.row_of", _I32)
    if rows.row_of.dim() != 2 or dout.shape != (rows.row_of.shape[0], H):
        raise ValueError("dout must be [T, H] for rows.row_of [T, k] and y [rows, H]")
    T, k = rows.row_of.shape
    _flat(weights, "weights", _F32, (T, k))
    if dy is None:
        dy = _empty_like_place((n, H), _BF16, y)
    lddy = _matrix(dy, "dy", (n, H))
    if dweights is None:
        dweights = _empty_like_place((T, k), _F32, y)
    _flat(dweights, "dweights", _F32, (T, k))
    with _on(stream, (dout, y, rows.row_of, weights, dy, dweights)) as s:
        _check(library().ts_moe_combine_grad(_ptr(dout), ldd, _ptr(y), ldy, n, H, _ptr(rows.row_of), _ptr(weights), T, k,
                                             _ptr(dy), lddy, _ptr(dweights), _flags(launch_with_pdl), s))
    return dy, dweights


def ts_stalled_waits() -> int:
    """Waits inside the product kernels of the current device that ran into their limit (0 unless something is wrong)."""
    n = ctypes.c_uint32(0)
    _check(library().ts_stalled_waits(ctypes.byref(n)))
    return n.value
