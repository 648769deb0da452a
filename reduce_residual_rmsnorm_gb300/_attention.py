"""The rotary, 4-bit cache and attention entry points on tensors (include/ts_attention.h).

As in ``_nvfp4_moe``: shapes, types and places are checked in csrc/python_calls.cpp, everything else by the library,
whose statuses become ``TsError``.  A call runs on the tensors' device, on that device's current stream unless
``stream`` is given, and allocates the outputs and the workspace it is not given.  Heads are bf16 [T, heads, D] whose
rows are contiguous within a token (columns of a wider projection, viewed as heads, are).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._nvfp4_moe import _native


class KVCache(NamedTuple):
    """A paged cache of keys and values in NVFP4 (``ts_kv_cache`` makes one).

    A slot, page * page_size + offset, holds one token; the bytes of a page are those of ``ts_kv_cache_t``."""
    pages: torch.Tensor    # uint8 [pages, heads, page_size / 16, 18 * head_dim]
    k_scale: torch.Tensor  # fp32, one value: the global scale of K
    v_scale: torch.Tensor  # fp32, one value: the global scale of V

    @property
    def page_size(self) -> int:
        return 16 * self.pages.shape[2]

    @property
    def heads(self) -> int:
        return self.pages.shape[1]

    @property
    def head_dim(self) -> int:
        return self.pages.shape[3] // 18


def ts_kv_cache(num_pages: int, heads: int, head_dim: int, k_scale: torch.Tensor, v_scale: torch.Tensor, *,
                page_size: int = 64, device="cuda") -> KVCache:
    """An empty cache: ``num_pages`` pages of ``page_size`` tokens (a multiple of 16), 9/8 byte an element of K and V.

    ``k_scale``, ``v_scale``: the global scales (448 * 6 / the largest |value|, as for ``ts_nvfp4_quantize``)."""
    if page_size < 16 or page_size % 16 != 0:
        raise ValueError(f"page_size = {page_size} must be a multiple of 16")
    if head_dim < 16 or head_dim > 256 or head_dim % 16 != 0:
        raise ValueError(f"head_dim = {head_dim} must be a multiple of 16 in 16..256")
    pages = torch.zeros((num_pages, heads, page_size // 16, 18 * head_dim), dtype=torch.uint8, device=device)
    return KVCache(pages, k_scale, v_scale)


def ts_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor | None, k_weight: torch.Tensor | None,
                    positions: torch.Tensor, cos_sin: torch.Tensor, eps: float = 1e-6, *, interleaved: bool = False,
                    v: torch.Tensor | None = None, cache: KVCache | None = None, slots: torch.Tensor | None = None,
                    q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                    launch_with_pdl: bool = False, stream=None):
    """Each head's RMSNorm of queries and keys and their rotation by position, in one pass.

    ``q`` [T, q_heads, D], ``k`` [T, k_heads, D]; ``q_weight``, ``k_weight`` bf16 [D], or both None to leave the norm
    out; ``positions`` int32 [T]; ``cos_sin`` fp32 [max_pos, rot], rot/2 cosines then rot/2 sines; ``interleaved``:
    the pairs are neighbours instead of halves.  ``q_out``, ``k_out`` may be ``q``, ``k``.  With a ``cache`` the keys
    and ``v`` go into its ``slots`` (int32 [T], negative: not kept), and ``k_out`` is written only if given.
    Returns (q_out, k_out or None).  A token whose position is outside the table is left out.
    """
    pages, ks, vs = cache if cache is not None else (None, None, None)
    return _native().qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, v, pages, ks, vs, slots,
                                  q_out, k_out, launch_with_pdl, stream)


def ts_qk_norm_rope_grad(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                         q_weight: torch.Tensor | None, k_weight: torch.Tensor | None, positions: torch.Tensor,
                         cos_sin: torch.Tensor, eps: float = 1e-6, *, interleaved: bool = False,
                         dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                         dq_weight: torch.Tensor | None = None, dk_weight: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """The gradient of ``ts_qk_norm_rope``: (dq, dk bf16, dq_weight, dk_weight fp32 [D] or None without weights).

    ``q``, ``k`` are the forward call's inputs, which it must not have written in place; ``dq``, ``dk`` may be ``dq_out``,
    ``dk_out``.
    """
    return _native().qk_norm_rope_grad(dq_out, dk_out, q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, dq, dk,
                                       dq_weight, dk_weight, workspace, launch_with_pdl, stream)


def ts_kv_cache_read(cache: KVCache, slots: torch.Tensor, *, k_out: torch.Tensor | None = None,
                     v_out: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """The bf16 keys and values [T, heads, D] that the cache's ``slots`` (int32 [T]) hold.

    New outputs are where the cache is.  Tokens with a slot outside the cache are left as they were (in a new output:
    undefined).
    """
    return _native().kv_cache_read(*cache, slots, k_out, v_out, launch_with_pdl, stream)


def ts_nvfp4_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                       cu_q: torch.Tensor | None = None, *, max_q: int | None = None, scale: float | None = None,
                       causal: bool = True, window: int = 0, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, return_lse: bool = False,
                       workspace: torch.Tensor | None = None, launch_with_pdl: bool = False, stream=None):
    """Attention of the last queries of each sequence over its keys and values in the cache.

    ``q`` [T, q_heads, D], D 64 or 128, q_heads a multiple of the cache's; ``block_table`` int32 [B, max_pages],
    ``kv_lens`` int32 [B] (with the new tokens'); ``cu_q`` int32 [B + 1]: where each sequence's queries begin, None
    for one each.  ``max_q``: a bound of a sequence's queries, which chooses the kernel (None: T).  ``scale``: None
    for 1 / sqrt(D).  ``window``: keys that a query sees at most, 0 for all.  Returns ``out`` like ``q``, with
    ``return_lse`` also the logarithm of the sums, fp32 [T, q_heads].  A query that sees no key gets zeros and -inf.
    """
    return _native().attention(q, *cache, block_table, kv_lens, cu_q, max_q, scale, causal, window, out, lse, return_lse,
                               workspace, launch_with_pdl, stream)
