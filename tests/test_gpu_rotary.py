"""Rotary positions against the definition in 64 bits.

Tolerances, for a pair (u, v). The angle's fraction of a turn is exact to 2^-32
turns: 2^-29.3 radians; what is left of it after the quarters is below 0.8 and rounded
to 24 bits: 2^-24.3; sincospif is off by at most 2^-23 (CUDA's table: 1 and 2 units in
the last place of values up to 1); gain, two products and a sum: 2^-24 each, of u and v
or of their turned values: in all below 2^-21 (|u| + |v|) |gain|. An output is rounded
once: FP32 within that, BF16 between the roundings of the two ends."""
import math

import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
FAR = [0, 1, -1, 7, 4095, 131071, 1048579, 2 ** 31 - 1, -2 ** 31, -12345, 2 ** 24 + 1]


def positions(n, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    p = torch.randint(0, 200000, (n,), generator=g)
    p[:min(n, len(FAR))] = torch.tensor(FAR[:n])
    return p.to(torch.int32)


def turned(x, pos, rope):
    """x [tokens][heads][dim] in 64 bits, its rotated channels turned, and the tolerance of each value."""
    R = rope.rotary_dim
    # whole turns drop out in whole numbers, from the 64-bit fractions (which have their own test)
    t = [[(int(p) * (int(w) % 2 ** 64)) % 2 ** 64 / 2 ** 64 for w in rope.turns.cpu()] for p in pos]
    a = torch.tensor(t, dtype=torch.float64).reshape(len(pos), 1, R // 2) * (2 * math.pi)
    cos, sin = a.cos() * rope.gain, a.sin() * rope.gain
    out, lim = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    at = (slice(0, R, 2), slice(1, R, 2)) if rope.interleaved else (slice(0, R // 2), slice(R // 2, R))
    u, v = (x[..., i].double() for i in at)
    out[..., at[0]], out[..., at[1]] = u * cos - v * sin, v * cos + u * sin
    for i in at:
        lim[..., i] = (u.abs() + v.abs()) * abs(rope.gain) * 2.0 ** -21
    return out, lim


def check(got, x, pos, rope):
    want, lim = turned(x.cpu(), pos, rope)
    lo, hi = (want - lim).to(got.dtype).double(), (want + lim).to(got.dtype).double()
    if got.dtype == torch.float32:                             # the ends' own rounding
        lo, hi = lo - lim * 2.0 ** -2, hi + lim * 2.0 ** -2
    g = got.cpu().double()
    bad = ~((g >= lo) & (g <= hi))
    assert not bool(bad.any()), f"{int(bad.sum())} off, worst {float(((g - want).abs() / lim.clamp(min=1e-300))[bad].max()):.2f}x"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads,dim,R", [(1, 2, 2), (3, 64, 64), (5, 80, 24), (40, 128, 128), (2, 64, 36), (7, 128, 32), (1, 256, 64),
                                         (2, 130, 66), (3, 7, 6), (1, 1024, 1024), (4, 128, 12), (4, 48, 40)])
def test_shapes(cuda_lib, io, inter, heads, dim, R):
    """Every width of access: even and odd numbers of pairs, of channels beside them, and of tokens."""
    rope = rssm.Rope(R, interleaved=inter, base=500000.0 if R > 2 else 10.0)
    for n in (1, 2, 13):
        torch.manual_seed(dim + n)
        x = torch.randn((n, heads, dim)).to(IO[io])
        pos = positions(n, n)
        out = torch.full_like(x, float("nan"), device="cuda")
        rssm.rotary(out, x.cuda(), pos.cuda(), rope)
        check(out, x, pos, rope)
        same = x.cuda()
        rssm.rotary(same, same, pos.cuda(), rope)              # in place: the same bits
        assert torch.equal(same, out)


@pytest.mark.parametrize("n", [607, 2431, 2432, 2433, 5003])
def test_many_tokens(cuda_lib, n):
    """On both sides of the size at which a block takes four tokens."""
    rope = rssm.Rope(32, scaling="yarn", factor=8.0, original=4096)
    torch.manual_seed(n)
    x = torch.randn((n, 3, 64)).bfloat16()
    pos = positions(n)
    out = torch.empty_like(x, device="cuda")
    rssm.rotary(out, x.cuda(), pos.cuda(), rope)
    check(out, x, pos, rope)


@pytest.mark.parametrize("scaling", sorted(rssm.ROPE))
def test_scalings_turn_by_their_frequencies(cuda_lib, scaling):
    rope = rssm.Rope(64, scaling=scaling, factor=4.0, original=2048)
    w = torch.tensor(rope.frequencies, dtype=torch.float64)
    x = torch.zeros((9, 1, 64))
    x[..., :32] = 1.0
    pos = torch.arange(9, dtype=torch.int32)
    out = torch.empty_like(x, device="cuda")
    rssm.rotary(out, x.cuda(), pos.cuda(), rope)
    a = pos.double()[:, None] * w
    want = torch.cat([a.cos(), a.sin()], -1)[:, None] * rope.gain
    assert float((out.cpu().double() - want).abs().max()) < 2.0 ** -20 * rope.gain


def test_given_frequencies_and_gain(cuda_lib):
    rope = rssm.Rope(8, inv_freq=[1.0, -0.25, 0.0, 3.5], gain=-2.0)
    x, pos = torch.randn((11, 2, 10)), positions(11)
    out = torch.empty_like(x, device="cuda")
    rssm.rotary(out, x.cuda(), pos.cuda(), rope)
    check(out, x, pos, rope)


@pytest.mark.parametrize("off,step", [(0, 640), (8, 648), (4, 644), (2, 642), (1, 641), (3, 700)])
def test_slices_and_alignments(cuda_lib, off, step):
    """Heads that are a slice of a wider projection, wherever it begins; what lies beside the output stays."""
    n, heads, dim = 21, 4, 64
    rope = rssm.Rope(64)
    wide = torch.randn(off + n * step).bfloat16().cuda()
    x = wide.as_strided((n, heads, dim), (step, dim, 1), off)
    to = torch.full((off + n * step,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = to.as_strided((n, heads, dim), (step, dim, 1), off)
    pos = positions(n)
    rssm.rotary(out, x, pos.cuda(), rope)
    check(out, x, pos, rope)
    out.fill_(7.0)
    assert bool((to == 7.0).all())


def test_not_finite_stays_where_it_is(cuda_lib):
    """A NaN or an infinity reaches its own pair, and nothing else."""
    rope = rssm.Rope(64)
    x = torch.randn((6, 3, 96)).bfloat16()
    clean = torch.empty_like(x, device="cuda")
    pos = positions(6)
    rssm.rotary(clean, x.cuda(), pos.cuda(), rope)
    x[2, 1, 5], x[3, 0, 40], x[4, 2, 80] = float("nan"), float("inf"), float("inf")
    out = torch.empty_like(x, device="cuda")
    rssm.rotary(out, x.cuda(), pos.cuda(), rope)
    same = (out == clean).cpu()
    for t, h, d in ((2, 1, 5), (2, 1, 37), (3, 0, 40), (3, 0, 8), (4, 2, 80)):
        assert not bool(same[t, h, d])
        same[t, h, d] = True
    assert bool(same.all()) and float(out[4, 2, 80]) == float("inf")


def test_back_again(cuda_lib):
    rope = rssm.Rope(128, base=1e6)
    x, pos = torch.randn((50, 2, 128)), positions(50)
    pos[pos == -2 ** 31] = 5                                   # has no opposite
    a, b = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    rssm.rotary(a, x.cuda(), pos.cuda(), rope)
    rssm.rotary(b, a, -pos.cuda(), rope)
    pair = x[..., :64].abs() + x[..., 64:].abs()
    assert bool(((b.cpu() - x).abs() <= 2 * 2.0 ** -20 * torch.cat([pair, pair], -1)).all())


def test_captured_and_on_another_stream(cuda_lib):
    rope = rssm.Rope(64)
    x, pos = torch.randn((5, 2, 64), device="cuda"), positions(5).cuda()
    out, want = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rssm.rotary(want, x, pos, rope)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rssm.rotary(out, x, pos, rope)
    x += 1
    pos += 3
    g.replay()
    torch.cuda.synchronize()
    check(out, x, pos.cpu(), rope)
    rssm.rotary(want, x, pos, rope)
    assert torch.equal(out, want)


def test_nothing_to_do(cuda_lib):
    rope = rssm.Rope(64)
    x = torch.empty((0, 2, 64), device="cuda")
    rssm.rotary(x, x, torch.empty(0, dtype=torch.int32, device="cuda"), rope)


def test_refusals(cuda_lib):
    rope = rssm.Rope(64)
    x = torch.zeros((4, 2, 64), device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for a, what in (((x, x, pos.long(), rope), "positions"), ((x, x, pos[:3], rope), "positions"), ((x, x, pos.cpu(), rope), "positions"),
                    ((x.bfloat16(), x, pos, rope), "out"), ((x[:3], x, pos, rope), "out"), ((x, x.half(), pos, rope), "x"),
                    ((x, x[:, 0], pos, rope), "x"), ((x, x.transpose(0, 1), pos, rope), "positions"),
                    ((x[..., :32], x[..., :32], pos, rope), "rope"), ((x, x[:1].expand(4, 2, 64), pos, rope), "x: tokens overlap"),
                    ((x[:1].expand(4, 2, 64), x, pos, rope), "out: tokens overlap"), ((x.cpu(), x, pos, rope), "out")):
        with pytest.raises(ValueError, match=what):
            rssm.rotary(*a)
    both = torch.zeros((4, 4, 64), device="cuda")
    with pytest.raises(rssm.RssmError):                        # out begins where x does, with another stride
        rssm.rotary(both.view(-1)[:8 * 64].view(4, 2, 64), both[:, :2], pos, rope)
