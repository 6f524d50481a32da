"""Attention over FP8 caches whose scores are so large that FP32 numbers near them are
far apart: the weights' factor of 2^15 must not be lost in, or added to, the largest score.

With a scale of ln 2 a score is its own logarithm to the base 2. Every token scores
+-16384 448 n, n channels of the largest code, and some one FP32 step of that more, both exactly,
so that the weights are exact powers of two.

Tolerances: outputs as in test_gpu_attn; lse has two roundings of FP32 and one of its logarithm,
each half of a step: 2^-22 of the value covers four."""
import math

import pytest
import torch

from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[40], [31, 64, 200, 1000]])
@pytest.mark.parametrize("dim,q_heads,T", [(64, 2, 1), (128, 2, 1), (128, 32, 1), (128, 16, 4), (256, 2, 1), (256, 64, 1)])
@pytest.mark.parametrize("n", [2, 4, 8, 16, 32])
def test_steps_of_large_scores(cuda_lib, n, dim, q_heads, T, lens):
    c = Case(lens, T=T, q_heads=q_heads, kv_heads=2, dim=dim, kv="fp8", seed=n + dim)
    score = 16384.0 * 448 * n
    step = 2.0 ** (math.floor(math.log2(score)) - 23)
    c.ks, c.vs = torch.ones(2), torch.ones(2)
    raw = c.k_cache.view(torch.uint8).cpu().view(torch.float8_e4m3fn)
    for b, m in enumerate(lens):
        k = torch.zeros((m, 2, dim))
        k[:, 0, :n], k[:, 1, :n] = 448.0, -448.0                # one cache head of either sign
        k[[i for i in (5, 20, 60, 130, 555) if i < m], :, dim - 1] = 1.0
        v = torch.randn((m, 2, dim)).to(torch.float8_e4m3fn)
        c.tokens[b] = (k.double(), v.double())
        for i in range(m):
            page, at = int(c.table[b, i // c.ps]), i % c.ps
            raw[page, :, at] = k[i].to(torch.float8_e4m3fn)
            c.v_cache[page, :, at] = v[i].cuda()
    c.k_cache = raw.cuda()
    c.q = torch.zeros(c.q.shape, dtype=torch.bfloat16)
    c.q[..., :n], c.q[..., dim - 1] = 16384.0, step
    out, lse = (x.cpu().double() for x in c.run(c.layer(scale=math.log(2.0))))
    w_out, w_lse = c.want(math.log(2.0))
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    lim = max(float(v.abs().max()) for _, v in c.tokens) * (2.0 ** -13 + 2.0 ** -12)
    lo, hi = (w_out - lim).bfloat16().double(), (w_out + lim).bfloat16().double()
    assert bool(((out >= lo) & (out <= hi)).all()), float((out - w_out).abs().max())
    assert bool(((lse - w_lse).abs() <= 2.0 ** -22 * w_lse.abs()).all())
