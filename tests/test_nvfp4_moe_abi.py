"""The NVFP4 and expert-routing entry points without a GPU: every refusal is made
on the host before any launch (the pointers are fake addresses that nothing
dereferences), and calls without rows validate and return."""
import ctypes

import numpy as np
import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from reduce_residual_rmsnorm_gb300 import build as libbuild
from tests import nvfp4_ref as ref

OK, BAD_PATTERN, NULL, SHAPE, ALIGN, UNSUPPORTED, ALIAS = 0, -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkg.library()


def _at(i):
    return 0x7F0000000000 + i * (1 << 36)


# name -> arguments in order, every one valid
CALLS = {
    "ts_nvfp4_quantize": dict(x=_at(0), T=9, K=96, ldx=104, scale_factor=_at(1), row_src=None, quant_out=_at(2),
                              scale_out=_at(3), sf_layout=0, flags=0, stream=None),
    "ts_nvfp4_dequantize": dict(quant=_at(0), scale=_at(1), sf_layout=2, T=9, K=96, scale_factor=_at(2), row_src=_at(3),
                                out=_at(4), ldo=96, flags=1, stream=None),
    "ts_nvfp4_gemm": dict(a=_at(0), a_scale=_at(1), b=_at(2), b_scale=_at(3), alpha=_at(4), M=9, N=72, K=96, out=_at(5),
                          ldo=80, flags=0, stream=None),
    "ts_moe_sort": dict(expert_ids=_at(0), T=9, k=4, E=6, row_align=128, rows=1024, row_of=_at(1), row_src=_at(2),
                        expert_start=_at(3), expert_count=_at(4), flags=0, stream=None),
    "ts_moe_dispatch": dict(x=_at(0), T=9, H=96, ldx=96, row_of=_at(1), k=4, rows=1024, out=_at(2), scale_factor=None,
                            quant_out=None, scale_out=None, sf_layout=0, flags=0, stream=None),
    "ts_nvfp4_grouped_gemm": dict(a=_at(0), a_scale=_at(1), b=_at(2), b_scale=_at(3), alpha=_at(4), expert_start=_at(5),
                                  expert_count=_at(6), E=6, rows=1024, entries=36, N=72, K=96, out=_at(7), ldo=72,
                                  flags=0, stream=None),
    "ts_moe_combine": dict(y=_at(0), rows=40, H=96, ldy=96, row_of=_at(1), weights=_at(2), T=9, k=4, out=_at(3), ldo=96,
                           flags=0, stream=None),
    "ts_moe_combine_grad": dict(dout=_at(0), ldd=96, y=_at(1), ldy=96, rows=40, H=96, row_of=_at(2), weights=_at(3), T=9,
                                k=4, dy=_at(4), lddy=96, dweights=_at(5), flags=0, stream=None),
}
Q, D, G, S, P, X, C, R = CALLS


def _call(lib, name, **change):
    args = dict(CALLS[name])
    assert set(change) <= set(args)
    args.update(change)
    return getattr(lib, name)(*args.values()), lib.ts_last_error_detail().decode()


REFUSED = [
    *[(n, dict(flags=f), UNSUPPORTED) for n in CALLS for f in (2, 8, 1 << 31)],
    *[(n, {r: v}, SHAPE) for n, r in ((Q, "T"), (D, "T"), (G, "M"), (S, "T"), (P, "T"), (X, "rows"), (C, "T"), (R, "T"),
                                      (S, "rows"), (P, "rows"), (C, "rows")) for v in (-1, 1 << 31)],
    *[(n, {c: v}, SHAPE) for n, c in ((Q, "K"), (D, "K"), (G, "K"), (X, "K"), (P, "H"), (C, "H"), (R, "H"), (G, "N"),
                                      (X, "N")) for v in (0, -16, 4)],
    (Q, dict(K=24), SHAPE), (D, dict(K=24), SHAPE), (G, dict(K=48), SHAPE), (X, dict(K=80), SHAPE), (G, dict(N=20), SHAPE),
    (X, dict(N=(1 << 24) + 8, ldo=1 << 25), SHAPE), (P, dict(H=100, ldx=104), SHAPE),
    *[(n, {c: 65568, ld: 65600}, UNSUPPORTED) for n, c, ld in ((Q, "K", "ldx"), (D, "K", "ldo"), (P, "H", "ldx"),
                                                               (C, "H", "ldy"))],
    (G, dict(K=65568), UNSUPPORTED), (X, dict(K=65568), UNSUPPORTED),
    *[(n, {ld: v}, SHAPE) for n, ld in ((Q, "ldx"), (D, "ldo"), (G, "ldo"), (P, "ldx"), (X, "ldo"), (C, "ldy"), (C, "ldo"),
                                        (R, "ldd"), (R, "ldy"), (R, "lddy")) for v in (64, 100, -104, (1 << 30) + 8)],
    (Q, dict(sf_layout=3), BAD_PATTERN), (D, dict(sf_layout=-1), BAD_PATTERN),
    (P, dict(out=None, scale_factor=_at(3), quant_out=_at(4), scale_out=_at(5), sf_layout=7), BAD_PATTERN),
    *[(n, dict(k=v), SHAPE) for n in (S, P, C, R) for v in (0, 65, -1)],
    *[(n, dict(T=1 << 28), SHAPE) for n in (S, P, C, R)],
    *[(n, dict(E=v), SHAPE) for n in (S, X) for v in (0, 1025, -2)],
    (S, dict(row_align=0), SHAPE), (S, dict(row_align=257), SHAPE), (S, dict(rows=895), SHAPE),
    (X, dict(rows=1000), SHAPE), (X, dict(entries=-1), SHAPE), (X, dict(E=1024, N=1 << 22, ldo=1 << 22), SHAPE),
    # NVFP4 rows: a multiple of 16 columns, all buffers or none
    (P, dict(out=None, H=104, ldx=104, scale_factor=_at(3), quant_out=_at(4), scale_out=_at(5)), SHAPE),
    (P, dict(scale_factor=_at(3)), UNSUPPORTED), (P, dict(quant_out=_at(4), scale_out=_at(5)), UNSUPPORTED),
    (P, dict(out=None), NULL), (P, dict(out=None, scale_factor=_at(3), quant_out=_at(4)), NULL),
    (P, dict(out=None, quant_out=_at(3), scale_out=_at(4)), NULL),
    *[(n, {b: None}, NULL) for n, bs in (
        (Q, ("x", "scale_factor", "quant_out", "scale_out")), (D, ("quant", "scale", "scale_factor", "out")),
        (G, ("a", "a_scale", "b", "b_scale", "alpha", "out")),
        (S, ("expert_ids", "row_of", "row_src", "expert_start", "expert_count")), (P, ("x", "row_of")),
        (X, ("a", "a_scale", "b", "b_scale", "alpha", "expert_start", "expert_count", "out")), (C, ("y", "row_of", "out")),
        (R, ("dout", "y", "row_of", "weights", "dy", "dweights"))) for b in bs],
    *[(n, {b: CALLS[n][b] + off}, ALIGN) for n, bs, off in (
        (Q, ("x", "quant_out"), 8), (Q, ("scale_factor", "scale_out"), 2), (D, ("quant", "out"), 8),
        (D, ("scale", "scale_factor", "row_src"), 2), (G, ("a", "a_scale", "b", "b_scale", "out"), 8), (G, ("alpha",), 2),
        (S, ("expert_ids", "row_of", "row_src", "expert_start", "expert_count"), 2), (P, ("x", "out"), 8), (P, ("row_of",), 2),
        (X, ("a", "a_scale", "b", "b_scale", "out"), 8), (X, ("alpha", "expert_start", "expert_count"), 2),
        (C, ("y", "out"), 8), (C, ("row_of", "weights"), 2), (R, ("dout", "y", "dy"), 8),
        (R, ("row_of", "weights", "dweights"), 2)) for b in bs],
    *[(n, {b: CALLS[n][over] + off}, ALIAS) for n, b, over, off in (
        (Q, "quant_out", "x", 16), (Q, "scale_out", "quant_out", 4), (Q, "scale_out", "scale_factor", 0),
        (D, "out", "quant", 0), (D, "out", "row_src", 32), (G, "out", "a", 0), (G, "out", "b_scale", 512), (G, "out", "alpha", 0),
        (S, "row_of", "expert_ids", 0), (S, "row_src", "row_of", 4), (S, "expert_count", "expert_start", 24),
        (P, "out", "x", 0), (P, "out", "row_of", 16), (X, "out", "b", 6 * 72 * 48 - 16), (X, "out", "expert_start", 16),
        (C, "out", "y", 160), (C, "out", "weights", 0), (R, "dy", "y", 0), (R, "dy", "dout", 0), (R, "dweights", "weights", 0),
        (R, "dweights", "dy", 40 * 96 * 2 - 4))],
]


@pytest.mark.parametrize("name,change,want", REFUSED, ids=lambda v: str(v)[:60])
def test_refused(lib, name, change, want):
    st, detail = _call(lib, name, **change)
    assert st == want, (name, change, st, detail)
    assert detail


def test_no_rows(lib):
    for n, r in ((Q, "T"), (D, "T"), (G, "M"), (P, "T"), (P, "rows"), (X, "rows"), (C, "T"), (R, "T")):
        st, detail = _call(lib, n, **{r: 0})
        assert st == OK and detail == "", (n, detail)
    assert _call(lib, Q, T=0, x=None, quant_out=None, scale_out=None)[0] == OK
    assert _call(lib, G, M=0, a=None, out=None)[0] == OK
    assert _call(lib, C, T=0, row_of=None, weights=None, out=None)[0] == OK


def test_overlap_counts_to_the_last_byte(lib):
    assert _call(lib, S, expert_count=_at(3) + 4 * 6)[0] == ALIAS  # expert_start has E + 1 entries
    last = CALLS[Q]["x"] + (8 * 104 + 96) * 2  # the end of the last strided row
    assert _call(lib, Q, quant_out=last - 16)[0] == ALIAS


def test_moe_rows(lib):
    for T, k, E, align in ((0, 1, 1, 1), (1, 8, 64, 128), (16, 8, 64, 128), (4096, 8, 64, 128), (5, 3, 7, 1), (9, 64, 1024, 256)):
        n = T * k
        assert pkg.ts_moe_rows(T, k, E, align) == ref.up(n + min(n, E) * (align - 1), align)
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 65, 1, 1), (1 << 30, 1, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                (1, 1, 1, 257)):
        assert lib.ts_moe_rows(*bad) == -1
        with pytest.raises(ValueError):
            pkg.ts_moe_rows(*bad)


def test_moe_rows_hold_every_routing():
    """The rows that any routing needs: the bound is reached when every expert holds one entry more than a multiple."""
    r = np.random.RandomState(0)
    for _ in range(200):
        T, k, E, align = r.randint(0, 20), r.randint(1, 9), r.randint(1, 30), r.choice([1, 2, 8, 128])
        ids = r.randint(-1, E + 1, (T, k))
        cap = pkg.ts_moe_rows(T, k, E, align)
        _, _, start, count = ref.sort_rows(ids, E, align, cap)
        assert start[-1] <= cap and cap % align == 0 and (start[:-1] % align == 0).all() and count.sum() <= T * k


def test_stalled_waits_needs_a_place(lib):
    assert lib.ts_stalled_waits(None) == NULL


def test_python_refusals():
    """Tensors in pageable host memory, of another type or shape, never reach the library."""
    f, u, b = torch.ones(1), torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4, 16).bfloat16()
    rows = pkg.MoERows(*(torch.zeros(2, 2, dtype=torch.int32) for _ in range(4)))
    for call in (lambda: pkg.ts_nvfp4_quantize(b, f), lambda: pkg.ts_nvfp4_dequantize(u, u, f),
                 lambda: pkg.ts_nvfp4_gemm(u, u, u, u, f), lambda: pkg.ts_moe_sort(rows.row_of, 4),
                 lambda: pkg.ts_moe_dispatch(b, rows), lambda: pkg.ts_moe_combine(b, rows),
                 lambda: pkg.ts_moe_combine_grad(b, b, rows, f), lambda: pkg.ts_nvfp4_grouped_gemm(u, u, u, u, f, rows)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_reference_round_trip():
    """The plain reference itself: known codes, ties to even, both swizzled layouts invertible."""
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]])
    code, sf = ref.quantize(x, 1.0)
    assert sf.tolist() == [[7 << 3]]  # amax 6 -> scale 1
    assert code.tolist() == [[0, 2, 2, 4, 4, 6, 6, 7, 8, 10, 10, 12, 12, 14, 14, 15]]
    assert np.array_equal(ref.unpack(ref.pack(code)), code)
    r = np.random.RandomState(0)
    for layout in (0, 1, 2):
        s = r.randint(0, 127, (300, 9)).astype(np.uint8)
        assert np.array_equal(ref.pick(ref.lay_out(s, layout), 300, 9, layout), s)


def test_ctypes_signatures(lib):
    for name, args in CALLS.items():
        assert len(getattr(lib, name).argtypes) == len(args), name
    assert lib.ts_moe_rows.restype is ctypes.c_int64
