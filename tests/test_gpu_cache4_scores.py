"""Attention over 4-bit caches whose scores are so large that neighbouring FP32 numbers are several
powers of two apart in weight: a weight must not leave FP16's range where the allowance under
which nothing is rescaled falls between two scores.

Every token scores +-16384 2688 = +-44040192 (neighbours are 4 apart), some 4 more, both exactly.
With a scale of ln 2 a score is its own logarithm to the base 2, so that every sum, product and join on
the way is exact, and the ratio of the two weights is 16; with a scale of 1 it is e^4.

Tolerances: outputs as in test_gpu_cache4; lse, near 3e7 or 4.4e7, has two roundings of FP32 and one of
its logarithm, each half of a step: 2^-22 of the value covers four."""
import math

import pytest
import torch

import test_gpu_cache4
from test_gpu_cache4 import Case

pytestmark = pytest.mark.gpu


def case(monkeypatch, lens, T, q_heads, dim, scale, more):
    """Two cache heads, one of either sign; the tokens in `more` score 4 more."""
    monkeypatch.setattr(test_gpu_cache4, "scales", lambda heads, seed=0: (torch.ones(heads), torch.ones(heads)))

    def spoil(b, k, v):
        k[:] = 0.0
        k[:, 0, 0], k[:, 1, 0] = 2688.0, -2688.0
        at = [i for i in more if i < len(k)]
        k[at, :, dim - 16], k[at, :, dim - 15] = 1.5, 1.0       # block scale 1/4: codes 6 and 4
    c = Case(lens, T=T, q_heads=q_heads, kv_heads=2, dim=dim, scale=scale, spoil=spoil, seed=dim + T)
    c.q[:] = 0.0
    c.q[..., 0], c.q[..., dim - 15] = 16384.0, 4.0
    assert torch.equal(c.tokens[0][0][:, 0, 0], torch.full((lens[0],), 2688.0, dtype=torch.float64))
    return c


def check(c):
    out, lse = (x.double() for x in c.run())
    w_out, w_lse = c.want()
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    lim = max(float(v.abs().max()) for _, v in c.tokens) * (2.0 ** -13 + 2.0 ** -12)
    lo, hi = (w_out - lim).bfloat16().double(), (w_out + lim).bfloat16().double()
    assert bool(((out >= lo) & (out <= hi)).all()), float((out - w_out).abs().max())
    assert bool(((lse - w_lse).abs() <= 2.0 ** -22 * w_lse.abs()).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_heads,T", [(2, 1), (16, 2), (32, 1), (16, 4), (128, 1)])
def test_next_score_is_past_the_allowance(cuda_lib, monkeypatch, dim, q_heads, T):
    """The larger score in the second group that a warp takes, with 1 to 64 query rows a cache head."""
    check(case(monkeypatch, [31, 31, 63, 200], T, q_heads, dim, math.log(2.0), [20, 30, 60, 130]))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_next_score_is_past_the_allowance_in_a_later_slot(cuda_lib, monkeypatch, dim):
    """Shares of several units a block: whole slots, the larger score in one that the same warp takes later."""
    check(case(monkeypatch, [1000] * 80, 1, 4, dim, math.log(2.0), [200, 201, 550, 999]))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_ratio_of_e4(cuda_lib, monkeypatch, dim):
    check(case(monkeypatch, [31], 1, 2, dim, 1.0, [20]))
