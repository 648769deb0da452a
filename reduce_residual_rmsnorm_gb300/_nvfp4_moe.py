"""Binding of the NVFP4 and expert-routing entry points (include/ts_nvfp4_moe.h).

Argument marshalling only, as in ``_binding``: shapes, types and places are
checked here, everything else by the library, whose statuses become
``TsError``.  A call runs on the tensors' device, on that device's current
stream unless ``stream`` is given, and allocates the outputs it is not given.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._binding import TS_FLAG_PDL, SFLayout, _check, _dev, _empty_like_place, library, sf_shape

_I32, _F32, _U8, _BF16 = torch.int32, torch.float32, torch.uint8, torch.bfloat16
_128x4 = int(SFLayout.SWIZZLED_128x4)


class MoERows(NamedTuple):
    """Where ``ts_moe_sort`` put the (token, slot) entries."""
    row_of: torch.Tensor        # int32 [T, k]: the entry's row, -1 without one
    row_src: torch.Tensor       # int32 [rows]: the row's entry t*k + slot, -1 without one
    expert_start: torch.Tensor  # int32 [E + 1]: an expert's first row
    expert_count: torch.Tensor  # int32 [E]: an expert's entries


def _new(shape, dtype, like):
    """A new contiguous tensor where `like` lives, and its address."""
    t = torch.empty(shape, dtype=dtype, device=like.device) if like.is_cuda else _empty_like_place(shape, dtype, like)
    return t, t.data_ptr()


# The checks below cost the calling thread a few attribute reads per tensor in
# the ordinary case and say what is wrong only in the other one: a decoded
# token's call is shorter on the GPU than its marshalling.

def _flat(t, name, dtype, shape=None):
    """A contiguous tensor of a type (and shape); its address."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        _dev(t, name, dtype)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _on_gpu(t, name, dtype, shape=None):
    """As _flat, in device memory (the tensor copy engine reads it)."""
    p = _flat(t, name, dtype, shape)
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return p


def _matrix(t, name, shape=None):
    """A bf16 matrix with unit column stride; its address and row stride."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is _BF16):
        _dev(t, name, _BF16)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, unit = t.stride()
    rows, cols = t.shape
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if rows <= 1:  # a single row has no stride that matters; torch may report any
        ld = max(ld, -(-cols // 8) * 8)
    return t.data_ptr(), ld


def _one(t, name):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is _F32):
        _dev(t, name, _F32)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one value")
    return t.data_ptr()


def _rows_of(rows, T=None):
    """row_of [T, k] of MoERows; its address, T and k."""
    p = _flat(rows.row_of, "rows.row_of", _I32)
    shape = rows.row_of.shape
    if len(shape) != 2 or (T is not None and shape[0] != T):
        raise ValueError("rows.row_of must be [T, k]")
    return p, shape[0], shape[1]


def _call(name, stream, launch_with_pdl, tensors, *args):
    """One library call: the tensors' device current, the flags and the stream behind the other arguments."""
    device = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != device and d >= 0:
                if device >= 0:
                    raise ValueError(f"tensors on different devices: cuda:{device}, cuda:{d}")
                device = d
    now = torch.cuda.current_device()
    if device < 0:
        device = now
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    else:
        stream = int(getattr(stream, "cuda_stream", stream))
    flags = TS_FLAG_PDL if launch_with_pdl else 0
    fn = getattr(library(), name)
    if device == now:
        status = fn(*args, flags, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, flags, stream)
    if status:
        _check(status)


def ts_nvfp4_quantize(x: torch.Tensor, scale_factor: torch.Tensor, *, row_src: torch.Tensor | None = None,
                      quant_out: torch.Tensor | None = None, scale_out: torch.Tensor | None = None,
                      sf_layout: int = SFLayout.LINEAR, launch_with_pdl: bool = False, stream=None):
    """bf16 rows ``x`` [T, K] to NVFP4 with the global scale ``scale_factor`` (fp32, one value).

    Returns (codes uint8 [T, K/2], scale factors uint8 of ``sf_shape(T, K, sf_layout)``).  With ``row_src`` (of
    ``ts_moe_sort``) the rows without an entry are left out.
    """
    xp, ldx = _matrix(x, "x")
    T, K = x.shape
    layout = int(sf_layout)
    gp = _one(scale_factor, "scale_factor")
    rp = None if row_src is None else _flat(row_src, "row_src", _I32, (T,))
    sf = sf_shape(T, K, layout)
    if quant_out is None:
        quant_out, qp = _new((T, K // 2), _U8, x)
    else:
        qp = _flat(quant_out, "quant_out", _U8, (T, K // 2))
    if scale_out is None:
        scale_out, sp = _new(sf, _U8, x)
    else:
        sp = _flat(scale_out, "scale_out", _U8, sf)
    _call("ts_nvfp4_quantize", stream, launch_with_pdl, (x, scale_factor, row_src, quant_out, scale_out),
          xp, T, K, ldx, gp, rp, qp, sp, layout)
    return quant_out, scale_out


def ts_nvfp4_dequantize(quant: torch.Tensor, scale: torch.Tensor, scale_factor: torch.Tensor, *,
                        sf_layout: int = SFLayout.LINEAR, row_src: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """The bf16 values [T, K] that codes [T, K/2], their scale factors and the global scale stand for."""
    qp = _flat(quant, "quant", _U8)
    if quant.dim() != 2:
        raise ValueError("quant must be [T, K/2]")
    T, K = quant.shape
    K *= 2
    layout = int(sf_layout)
    sp = _flat(scale, "scale", _U8, sf_shape(T, K, layout))
    gp = _one(scale_factor, "scale_factor")
    rp = None if row_src is None else _flat(row_src, "row_src", _I32, (T,))
    if out is None:
        (out, op), ldo = _new((T, K), _BF16, quant), K
    else:
        op, ldo = _matrix(out, "out", (T, K))
    _call("ts_nvfp4_dequantize", stream, launch_with_pdl, (quant, scale, scale_factor, row_src, out),
          qp, sp, layout, T, K, gp, rp, op, ldo)
    return out


def ts_nvfp4_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                  alpha: torch.Tensor, *, out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """``out`` [M, N] = bf16(alpha A B^T) of NVFP4 codes ``a`` [M, K/2] and ``b`` [N, K/2] with SWIZZLED_128x4
    scale factors; ``alpha`` (fp32, one value) is 1 / (g_A g_B)."""
    ap, bp = _on_gpu(a, "a", _U8), _on_gpu(b, "b", _U8)
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError("a must be [M, K/2] and b [N, K/2]")
    M, K = a.shape
    N, K = b.shape[0], 2 * K
    asp = _on_gpu(a_scale, "a_scale", _U8, sf_shape(M, K, _128x4))
    bsp = _on_gpu(b_scale, "b_scale", _U8, sf_shape(N, K, _128x4))
    alp = _one(alpha, "alpha")
    if out is None:
        (out, op), ldo = _new((M, N), _BF16, a), N
    else:
        op, ldo = _matrix(out, "out", (M, N))
    _call("ts_nvfp4_gemm", stream, launch_with_pdl, (a, a_scale, b, b_scale, alpha, out),
          ap, asp, bp, bsp, alp, M, N, K, op, ldo)
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
    ip = _flat(expert_ids, "expert_ids", _I32)
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be [T, k]")
    T, k = expert_ids.shape
    E = int(num_experts)
    if rows is None:
        n = ts_moe_rows(T, k, E, row_align)
        (row_of, of), (row_src, src) = _new((T, k), _I32, expert_ids), _new((n,), _I32, expert_ids)
        (starts, start), (counts, count) = _new((E + 1,), _I32, expert_ids), _new((E,), _I32, expert_ids)
        rows = MoERows(row_of, row_src, starts, counts)
    else:
        n = rows.row_src.numel()
        of = _flat(rows.row_of, "rows.row_of", _I32, (T, k))
        src = _flat(rows.row_src, "rows.row_src", _I32)
        start = _flat(rows.expert_start, "rows.expert_start", _I32, (E + 1,))
        count = _flat(rows.expert_count, "rows.expert_count", _I32, (E,))
    _call("ts_moe_sort", stream, launch_with_pdl, (expert_ids, *rows),
          ip, T, k, E, int(row_align), n, of, src, start, count)
    return rows


def ts_moe_dispatch(x: torch.Tensor, rows: MoERows, scale_factor: torch.Tensor | None = None, *,
                    out: torch.Tensor | None = None, quant_out: torch.Tensor | None = None,
                    scale_out: torch.Tensor | None = None, sf_layout: int = SFLayout.SWIZZLED_128x4,
                    launch_with_pdl: bool = False, stream=None):
    """Token rows ``x`` [T, H] in expert order: bf16 [rows, H], or with ``scale_factor`` NVFP4 codes and scale factors.

    Rows without an entry are left as they were.  Returns ``out`` or (quant_out, scale_out).
    """
    xp, ldx = _matrix(x, "x")
    T, H = x.shape
    of, _, k = _rows_of(rows, T)
    n = rows.row_src.numel()
    layout = int(sf_layout)
    if scale_factor is None:
        if quant_out is not None or scale_out is not None:
            raise ValueError("quant_out and scale_out need scale_factor")
        if out is None:
            out = _empty_like_place((n, H), _BF16, x)
        bufs = (_flat(out, "out", _BF16, (n, H)), None, None, None)
    else:
        if out is not None:
            raise ValueError("out and scale_factor exclude each other")
        gp = _one(scale_factor, "scale_factor")
        sf = sf_shape(n, H, layout)
        if quant_out is None:
            quant_out = _empty_like_place((n, H // 2), _U8, x)
        if scale_out is None:
            scale_out = _empty_like_place(sf, _U8, x)
        bufs = (None, gp, _flat(quant_out, "quant_out", _U8, (n, H // 2)), _flat(scale_out, "scale_out", _U8, sf))
    _call("ts_moe_dispatch", stream, launch_with_pdl, (x, rows.row_of, out, scale_factor, quant_out, scale_out),
          xp, T, H, ldx, of, k, n, *bufs, layout)
    return out if scale_factor is None else (quant_out, scale_out)


def ts_nvfp4_grouped_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                          alpha: torch.Tensor, rows: MoERows, *, out: torch.Tensor | None = None,
                          launch_with_pdl: bool = False, stream=None):
    """Each expert's NVFP4 product with its own rows: ``a`` [rows, K/2] sorted with row_align 128, ``b`` [E, N, K/2],
    ``b_scale`` [E, ceil(N/128)*128, ceil(K/64)*4], ``alpha`` fp32 [E].  Returns ``out`` bf16 [rows, N], in which the
    rows without an entry are left as they were."""
    ap, bp = _on_gpu(a, "a", _U8), _on_gpu(b, "b", _U8)
    if a.dim() != 2 or b.dim() != 3 or a.shape[1] != b.shape[2]:
        raise ValueError("a must be [rows, K/2] and b [E, N, K/2]")
    n, K = a.shape
    K *= 2
    E, N, _ = b.shape
    asp = _on_gpu(a_scale, "a_scale", _U8, sf_shape(n, K, _128x4))
    bsp = _on_gpu(b_scale, "b_scale", _U8, (E, *sf_shape(N, K, _128x4)))
    alp = _flat(alpha, "alpha", _F32, (E,))
    start = _flat(rows.expert_start, "rows.expert_start", _I32, (E + 1,))
    count = _flat(rows.expert_count, "rows.expert_count", _I32, (E,))
    if out is None:
        (out, op), ldo = _new((n, N), _BF16, a), N
    else:
        op, ldo = _matrix(out, "out", (n, N))
    _call("ts_nvfp4_grouped_gemm", stream, launch_with_pdl,
          (a, a_scale, b, b_scale, alpha, rows.expert_start, rows.expert_count, out),
          ap, asp, bp, bsp, alp, start, count, E, n, rows.row_of.numel(), N, K, op, ldo)
    return out


def ts_moe_combine(y: torch.Tensor, rows: MoERows, weights: torch.Tensor | None = None, *,
                   out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """The experts' rows ``y`` [rows, H] weighted (fp32 [T, k]; None: 1) and summed back into token order: bf16 [T, H].

    Without weights it is the gradient of ``ts_moe_dispatch``.
    """
    yp, ldy = _matrix(y, "y")
    n, H = y.shape
    of, T, k = _rows_of(rows)
    wp = None if weights is None else _flat(weights, "weights", _F32, (T, k))
    if out is None:
        (out, op), ldo = _new((T, H), _BF16, y), H
    else:
        op, ldo = _matrix(out, "out", (T, H))
    _call("ts_moe_combine", stream, launch_with_pdl, (y, rows.row_of, weights, out),
          yp, n, H, ldy, of, wp, T, k, op, ldo)
    return out


def ts_moe_combine_grad(dout: torch.Tensor, y: torch.Tensor, rows: MoERows, weights: torch.Tensor, *,
                        dy: torch.Tensor | None = None, dweights: torch.Tensor | None = None,
                        launch_with_pdl: bool = False, stream=None):
    """The gradient of ``ts_moe_combine`` for ``dout`` [T, H]: (dy bf16 like ``y``, dweights fp32 [T, k]).

    Rows of ``dy`` without an entry are left as they were.
    """
    yp, ldy = _matrix(y, "y")
    n, H = y.shape
    of, T, k = _rows_of(rows)
    dp, ldd = _matrix(dout, "dout", (T, H))
    wp = _flat(weights, "weights", _F32, (T, k))
    if dy is None:
        (dy, dyp), lddy = _new((n, H), _BF16, y), H
    else:
        dyp, lddy = _matrix(dy, "dy", (n, H))
    if dweights is None:
        dweights, dwp = _new((T, k), _F32, y)
    else:
        dwp = _flat(dweights, "dweights", _F32, (T, k))
    _call("ts_moe_combine_grad", stream, launch_with_pdl, (dout, y, rows.row_of, weights, dy, dweights),
          dp, ldd, yp, ldy, n, H, of, wp, T, k, dyp, lddy, dwp)
    return dy, dweights


def ts_stalled_waits() -> int:
    """Waits inside the product kernels of the current device that ran into their limit (0 unless something is wrong)."""
    n = ctypes.c_uint32(0)
    _check(library().ts_stalled_waits(ctypes.byref(n)))
    return n.value
