"""The attention example of README.md, run as it stands: its outputs and gradients are those of the definitions."""
import os
import re

import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu


def test_attention_example():
    import __graft_entry__

    __graft_entry__.build()
    dev = torch.device("cuda:0")
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md"), encoding="utf-8") as f:
        code = next(c for c in re.findall(r"```python\n(.*?)```", f.read(), flags=re.S) if "ts_kv_cache(" in c)
    T, hq, hk, D = 40, 8, 2, 128
    g = torch.Generator(device=dev).manual_seed(0)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev).bfloat16()

    q, k, v, qw, kw = rand(T, hq, D), rand(T, hk, D), rand(T, hk, D), rand(D), rand(D)
    # (a sequence of 39 tokens and one of 1: "a token each" takes the first two queries)
    pos = torch.cat((torch.arange(39), torch.zeros(1))).int().to(dev)
    slots = torch.cat((torch.arange(39), torch.tensor([64]))).int().to(dev)
    names = dict(ts=pkg, q=q.clone(), k=k.clone(), v=v, q_weight=qw, k_weight=kw, positions=pos, angles=ref.angles(64, D).to(dev),
                 slots=slots, num_pages=2, k_heads=hk, k_scale=torch.tensor([100.0], device=dev), v_scale=torch.tensor([100.0], device=dev),
                 block_table=torch.tensor([[0], [1]], dtype=torch.int32, device=dev), most=39,
                 kv_lens=torch.tensor([39, 1], dtype=torch.int32, device=dev), cu_q=torch.tensor([0, 39, 40], dtype=torch.int32, device=dev))
    dqr, dkr = rand(T, hq, D), rand(T, hk, D)
    names.update(dqr=dqr, dkr=dkr, dq=dqr, dk=dkr)
    # the line for a token each wants as many queries as sequences
    code = re.sub(r"^(out = ts\.ts_nvfp4_attention\()(\w+)(, cache, block_table, kv_lens\)).*$", r"\1\2[:2]\3", code, flags=re.M)
    exec(code, names)
    c = names["cache"]
    qr = pkg.ts_qk_norm_rope(q, k, qw, kw, pos, names["angles"], 1e-6)[0]
    want, _, slack, _ = ref.attention(qr, c.pages, c.k_scale.double(), c.v_scale.double(), names["block_table"], [39, 1], [0, 39, 40], D ** -0.5)
    assert bool(((names["out"].double() - want).abs() <= 2.0 ** -8 * want.abs() + slack).all())
    for dy, x, w, dx, dw in ((dqr, q, qw, names["dq"], names["dqw"]), (dkr, k, kw, names["dk"], names["dkw"])):
        want, want_w = ref.rope_grad(dy, x, w, pos, names["angles"], 1e-6, False)
        # fp32 sums of D and of T * heads terms, of magnitudes r |g| (1 + |x r|^2) and |d x r|
        r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
        xr = (x.double() * r).abs()
        big = r * 2 * dy.double().abs().amax(-1, keepdim=True) * w.double().abs().max() * (1 + xr.amax(-1, keepdim=True) ** 2)
        assert bool(((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + (D + 16) * 2.0 ** -23 * big).all())
        mag = (2 * dy.double().abs().amax(-1, keepdim=True) * xr).sum((0, 1))
        assert bool(((dw.double() - want_w).abs() <= (D + 64) * 2.0 ** -24 * mag).all())
