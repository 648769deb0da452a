"""The attention entry points without a GPU: every refusal is made on the host before any launch (the pointers are
fake addresses that nothing dereferences), and calls without rows validate and return."""
import ctypes

import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from reduce_residual_rmsnorm_gb300 import _binding
from reduce_residual_rmsnorm_gb300 import build as libbuild

OK, BAD_PATTERN, NULL, SHAPE, ALIGN, UNSUPPORTED, ALIAS = 0, -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkg.library()


def _at(i):
    return 0x7F0000000000 + i * (1 << 36)


CACHE = dict(pages=_at(30), num_pages=12, page_size=32, heads=2, head_dim=64, k_scale=_at(31), v_scale=_at(32))
# name -> arguments in order, every one valid
CALLS = {
    "ts_qk_norm_rope": dict(q=_at(0), ldq=400, k=_at(1), ldk=136, T=9, q_heads=6, k_heads=2, head_dim=64, q_weight=_at(2),
                            k_weight=_at(3), eps=1e-6, positions=_at(4), cos_sin=_at(5), max_pos=100, rot=32, interleaved=0,
                            q_out=_at(6), ldqo=384, k_out=_at(7), ldko=128, v=_at(8), ldv=128, cache=CACHE, slots=_at(9),
                            flags=0, stream=None),
    "ts_qk_norm_rope_grad": dict(dq_out=_at(0), lddqo=384, dk_out=_at(1), lddko=128, q=_at(2), ldq=400, k=_at(3), ldk=136,
                                 T=9, q_heads=6, k_heads=2, head_dim=64, q_weight=_at(4), k_weight=_at(5), eps=1e-6,
                                 positions=_at(6), cos_sin=_at(7), max_pos=100, rot=32, interleaved=1, dq=_at(8), lddq=384,
                                 dk=_at(9), lddk=128, dq_weight=_at(10), dk_weight=_at(11), workspace=_at(12), flags=1,
                                 stream=None),
    "ts_kv_cache_read": dict(cache=CACHE, slots=_at(0), T=9, k_out=_at(1), ldk=128, v_out=_at(2), ldv=136, flags=0,
                             stream=None),
    "ts_nvfp4_attention": dict(q=_at(0), ldq=400, T=9, q_heads=6, cu_q=_at(1), B=4, max_q=3, cache=CACHE, block_table=_at(2),
                               max_pages=5000, kv_lens=_at(3), scale=0.125, causal=1, window=70000, out=_at(4), ldo=384,
                               lse=_at(5), workspace=_at(6), flags=0, stream=None),
}
R, G, V, A = CALLS
T_ALL = ((R, "T"), (G, "T"), (V, "T"), (A, "T"))


def _call(lib, name, **change):
    args = dict(CALLS[name])
    for key, v in change.items():
        if key.startswith("cache_"):
            args["cache"] = dict(args["cache"], **{key[6:]: v})
        else:
            assert key in args
            args[key] = v
    if isinstance(args.get("cache"), dict):
        args["cache"] = ctypes.byref(_binding.TsKvCache(*args["cache"].values()))
    return getattr(lib, name)(*args.values()), lib.ts_last_error_detail().decode()


REFUSED = [
    *[(n, dict(flags=f), UNSUPPORTED) for n in CALLS for f in (2, 8, 1 << 31)],
    *[(n, {r: v}, SHAPE) for n, r in T_ALL for v in (-1, 1 << 31)],
    *[(n, dict(T=1 << 30), SHAPE) for n in (R, G, V, A)],
    *[(n, {h: v}, SHAPE) for n in (R, G) for h in ("q_heads", "k_heads") for v in (0, -1, 1025)],
    *[(n, dict(head_dim=v), SHAPE) for n in (R, G) for v in (0, 8, 72, 272, -64)],
    *[(n, dict(rot=v), SHAPE) for n in (R, G) for v in (0, 8, 24, 80, -16)],
    *[(n, dict(max_pos=v), SHAPE) for n in (R, G) for v in (0, -1, 1 << 31)],
    *[(n, dict(interleaved=v), SHAPE) for n in (R, G) for v in (2, -1)],
    *[(n, dict(eps=v), UNSUPPORTED) for n in (R, G) for v in (-1.0, float("nan"), float("inf"))],
    *[(n, {ld: v}, SHAPE) for n, lds in ((R, ("ldq", "ldk", "ldqo", "ldko", "ldv")),
                                         (G, ("lddqo", "lddko", "ldq", "ldk", "lddq", "lddk")), (V, ("ldk", "ldv")),
                                         (A, ("ldq", "ldo"))) for ld in lds for v in (64, 1028, -400, (1 << 30) + 8)],
    *[(n, {"cache_" + f: v}, SHAPE) for n in (R, V, A) for f, v in (
        ("num_pages", -1), ("num_pages", 1 << 26), ("page_size", 0), ("page_size", 24), ("page_size", 65552), ("heads", 0),
        ("heads", 1025), ("head_dim", 0), ("head_dim", 40), ("head_dim", 272))],
    (R, dict(cache_heads=1), SHAPE), (R, dict(cache_head_dim=128), SHAPE),
    (R, dict(cache=None), UNSUPPORTED), (R, dict(cache=None, v=None), UNSUPPORTED), (R, dict(cache=None, slots=None), UNSUPPORTED),
    (R, dict(q_weight=None), UNSUPPORTED), (R, dict(k_weight=None), UNSUPPORTED), (G, dict(q_weight=None), UNSUPPORTED),
    (G, dict(q_weight=None, k_weight=None), UNSUPPORTED), (G, dict(q_weight=None, k_weight=None, dk_weight=None), UNSUPPORTED),
    (V, dict(cache=None), NULL), (A, dict(cache=None), NULL),
    (A, dict(q_heads=5), SHAPE), (A, dict(q_heads=0), SHAPE), (A, dict(q_heads=1026), SHAPE),
    (A, dict(cache_head_dim=80, ldq=480, ldo=480), UNSUPPORTED), (A, dict(cache_head_dim=256, ldq=2048, ldo=2048), UNSUPPORTED),
    (A, dict(max_q=0), SHAPE), (A, dict(max_q=-1), SHAPE), (A, dict(B=-1), SHAPE), (A, dict(B=65537), SHAPE),
    (A, dict(cu_q=None), SHAPE), (A, dict(max_pages=-1), SHAPE), (A, dict(max_pages=(1 << 25) + 1), SHAPE),
    *[(A, dict(scale=v), UNSUPPORTED) for v in (0.0, -1.0, float("nan"), float("inf"))],
    (A, dict(causal=2), SHAPE), (A, dict(window=-1), SHAPE), (A, dict(causal=0), UNSUPPORTED),
    *[(n, {b: None}, NULL) for n, bs in (
        (R, ("q", "k", "positions", "cos_sin", "q_out", "v", "slots", "cache_k_scale", "cache_v_scale", "cache_pages")),
        (G, ("dq_out", "dk_out", "q", "k", "positions", "cos_sin", "dq", "dk", "dq_weight", "dk_weight", "workspace")),
        (V, ("cache_pages", "cache_k_scale", "cache_v_scale", "slots")),
        (A, ("q", "block_table", "kv_lens", "out", "workspace", "cache_pages", "cache_k_scale", "cache_v_scale"))) for b in bs],
    (R, dict(cache=None, v=None, slots=None, k_out=None), NULL),
    *[(n, {b: (CALLS[n].get(b) or CACHE[b[6:]]) + off}, ALIGN) for n, bs, off in (
        (R, ("q", "k", "q_weight", "k_weight", "cos_sin", "q_out", "k_out", "v", "cache_pages"), 8),
        (R, ("positions", "slots", "cache_k_scale", "cache_v_scale"), 2),
        (G, ("dq_out", "dk_out", "q", "k", "q_weight", "k_weight", "cos_sin", "dq", "dk", "workspace"), 8),
        (G, ("positions", "dq_weight", "dk_weight"), 2), (V, ("k_out", "v_out", "cache_pages"), 8), (V, ("slots",), 2),
        (A, ("q", "out", "workspace", "cache_pages"), 8), (A, ("cu_q", "block_table", "kv_lens", "lse"), 2)) for b in bs],
    *[(n, {b: CALLS[n][over] + off}, ALIAS) for n, b, over, off in (
        (R, "q_out", "q", 0), (R, "q_out", "k", 0), (R, "k_out", "q_out", 16), (R, "k_out", "v", 0), (R, "q_out", "cos_sin", 0),
        (R, "k_out", "slots", 16), (G, "dq", "q", 0), (G, "dk", "dq", 0), (G, "dq", "dq_out", 16), (G, "dq_weight", "dk_weight", 0),
        (G, "workspace", "dk", 128), (V, "k_out", "v_out", 16), (V, "k_out", "slots", 0), (A, "out", "q", 0), (A, "lse", "out", 64),
        (A, "workspace", "out", 16), (A, "out", "kv_lens", 0))],
    (R, dict(cache_pages=_at(6)), ALIAS), (V, dict(k_out=CACHE["pages"] + 512), ALIAS), (A, dict(out=CACHE["pages"]), ALIAS),
]


@pytest.mark.parametrize("name,change,want", REFUSED, ids=lambda v: str(v)[:60])
def test_refused(lib, name, change, want):
    st, detail = _call(lib, name, **change)
    assert st == want, (name, change, st, detail)
    assert detail


def test_no_rows(lib):
    none = {R: ("q", "k", "positions", "q_out", "k_out", "v", "slots"), V: ("slots", "k_out", "v_out"),
            A: ("q", "out", "workspace", "lse")}
    for n, names in none.items():
        change = dict(T=0) if n != A else dict(T=0, B=0, cu_q=None)
        assert _call(lib, n, **change) == (OK, "")
        assert _call(lib, n, **change, **{b: None for b in names}) == (OK, "")
    assert _call(lib, A, B=0) == (OK, "")
    assert _call(lib, V, k_out=None, v_out=None) == (OK, "")
    no_norm = dict(q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, workspace=None)
    assert _call(lib, G, T=0, **no_norm, dq=None, dk=None) == (OK, "")


def test_columns_of_one_matrix_do_not_overlap(lib):
    """q, k and v as columns of one matrix of rows, in place; a column further and they do."""
    row, base = 640, _at(0)
    whole = dict(T=0, q=base, ldq=row, k=base + 384 * 2, ldk=row, v=base + 512 * 2, ldv=row, q_out=base, ldqo=row,
                 k_out=base + 384 * 2, ldko=row)
    assert _call(lib, R, **whole) == (OK, "")  # (without rows nothing overlaps)
    # with rows: refused only where columns meet (the position table is checked last, so a bad one shows the way)
    st, detail = _call(lib, R, **dict(whole, T=9, cos_sin=None))
    assert st == NULL and "cos_sin" in detail
    for bad in (dict(q_out=base + 16), dict(k_out=base + 376 * 2), dict(k_out=base + 392 * 2), dict(q_out=base + 272 * 2),
                dict(ldqo=row + 8), dict(k_out=base + row * 2 - 64 * 2)):
        st, detail = _call(lib, R, **dict(whole, T=9), **{k: v for k, v in bad.items()}) if not set(bad) & set(whole) else \
            _call(lib, R, **{**whole, "T": 9, **bad})
        assert st == ALIAS, (bad, st, detail)


def test_workspaces(lib):
    assert lib.ts_qk_norm_rope_grad_workspace(128) > 0
    for bad in (0, 8, 24, 272, -16):
        assert lib.ts_qk_norm_rope_grad_workspace(bad) == -1
    size = lib.ts_nvfp4_attention_workspace
    assert size(1, 8, 1, 128, 1, 4096, 0) == 0 and size(0, 8, 1, 128, 1, 0, 0) == 0  # one launch
    assert size(100, 8, 1, 128, 1, 1 << 20, 64) == 0 < size(100, 8, 1, 128, 1, 1 << 20, 0)  # a window bounds the keys
    last = 0
    for args in ((1, 8, 1, 128, 1, 4096, 0), (500, 8, 1, 128, 1, 4096, 0), (500, 8, 1, 128, 2, 4096, 0), (500, 8, 1, 128, 40, 1 << 30, 0)):
        assert size(*args) >= last and size(*args) % 16 == 0
        last = size(*args)
    assert last > 0
    for bad in ((1, 0, 1, 128, 1, 16, 0), (1, 6, 4, 128, 1, 16, 0), (1, 8, 1, 96, 1, 16, 0), (1, 8, 1, 128, 0, 16, 0), (1, 8, 0, 128, 1, 16, 0),
                (1, 8, -1, 128, 1, 16, 0), (-1, 8, 1, 128, 1, 16, 0), (65537, 8, 1, 128, 1, 16, 0), (1, 8, 1, 128, 1, -1, 0),
                (1, 8, 1, 128, 1, (1 << 30) + 1, 0), (1, 8, 1, 128, 1, 16, -1)):
        assert size(*bad) == -1


def test_python_refusals():
    """Tensors in pageable host memory never reach the library; nor does a cache of a wrong form."""
    x, w, i, f = torch.zeros(4, 2, 64).bfloat16(), torch.ones(64).bfloat16(), torch.zeros(4, dtype=torch.int32), torch.ones(1)
    table = torch.zeros(8, 64)
    cache = pkg.KVCache(torch.zeros(2, 2, 4, 18 * 64, dtype=torch.uint8), f, f)
    assert (cache.page_size, cache.heads, cache.head_dim) == (64, 2, 64)
    for call in (lambda: pkg.ts_qk_norm_rope(x, x, w, w, i, table), lambda: pkg.ts_qk_norm_rope_grad(x, x, x, x, w, w, i, table),
                 lambda: pkg.ts_kv_cache_read(cache, i), lambda: pkg.ts_nvfp4_attention(x, cache, i.view(4, 1), i)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    for bad in (dict(page_size=24), dict(page_size=0), dict(head_dim=40), dict(head_dim=272)):
        with pytest.raises(ValueError):
            pkg.ts_kv_cache(**{**dict(num_pages=2, heads=2, head_dim=64, k_scale=f, v_scale=f, device="cpu"), **bad})


def test_ctypes_signatures(lib):
    for name, args in CALLS.items():
        assert len(getattr(lib, name).argtypes) == len(args), name
