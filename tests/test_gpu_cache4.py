"""The 4-bit (NVFP4) cache: what append writes and read gives back, rotary positions
on the way, and the attention over it, against their definitions.

Written values are compared bit by bit: the definition is a sequence of FP32 operations,
each rounded once, and read rounds its product once more. Rotated keys are compared
with those that `rotary` makes of the same values in FP32.

Tolerances of the attention, for values of size vmax = max |v|: as over FP8 caches, the
weights carry 11 bits (2^-12), the rest is below 2^-13; block scales and codes multiply
exactly. lse: 2^-14 absolute."""
import math

import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2      # a rounding: half of a step of 2^-7 of the power of two below the value
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
KV = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def quantised(x, s):
    """x [tokens][heads][dim], s [heads] -> the values that the cache holds for it, FP32."""
    b16 = x.float().unflatten(-1, (-1, 16))
    m = torch.where(b16.isnan(), 0.0, b16.abs()).amax(-1)
    b = (m * (1 / (6 * s))[:, None]).clamp(max=448).to(torch.float8_e4m3fn).float()
    inv = torch.where(b > 0, 1 / (b * s[:, None]), 0.0)
    y = b16 * inv[..., None]
    # nearest, and on a border the code that is even
    a = y.abs()
    code = sum((a > t if even else a >= t).int() for t, even in
               ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)))
    v = E2M1[code] * y.sign() * (b * s[:, None])[..., None]
    return torch.where(b16.isnan().any(-1, keepdim=True), float("nan"), v).flatten(-2)


def scales(heads, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.rand(heads, generator=g) * 0.004 + 0.002, torch.rand(heads, generator=g) * 0.002 + 0.001


def caches(num, heads, ps, dim, kv, fill=0xFF, beside=False):
    """Caches whose every byte is `fill` (0xFF: NaN scales); beside: K and V of a page in one array."""
    row, dt = (dim // 2 + dim // 16, torch.uint8) if kv == "nvfp4" else (dim, KV[kv])
    n = row * dt.itemsize
    both = torch.full((num, 2, heads, ps, n) if beside else (2, num, heads, ps, n), fill, dtype=torch.uint8, device="cuda").view(dt)
    return (both[:, 0], both[:, 1]) if beside else (both[0], both[1])


def layer(k_cache, v_cache, kv, ks, vs, q_heads, batch=1, max_pages=4, **kw):
    s = kv in ("fp8", "nvfp4")
    return rssm.Attention(k_cache, v_cache, batch=batch, q_heads=q_heads, max_pages=max_pages, k_scale=ks.cuda() if s else None,
                          v_scale=vs.cuda() if s else None, **kw)


def stored(x, s, kv):
    """The values that a cache holds for x (already in the layer's type, or rotated in FP32), as read gives them."""
    if kv == "f32":
        return x.float()
    if kv == "bf16":
        return x.bfloat16()
    if kv == "fp8":
        return ((x.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float() * s[:, None]).bfloat16()
    return quantised(x, s).bfloat16()


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=12345.0, posinf=None, neginf=None), torch.nan_to_num(b, nan=12345.0, posinf=None, neginf=None)) \
        and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("kv", ["nvfp4", "fp8", "bf16", "f32"])
@pytest.mark.parametrize("dim,heads,ps,n,beside", [(64, 1, 16, 1, False), (64, 3, 48, 37, True), (128, 8, 16, 64, False), (128, 2, 32, 2500, True),
                                                   (256, 2, 64, 130, False), (256, 5, 16, 17, True)])
def test_written_and_read_back(cuda_lib, kv, dim, heads, ps, n, beside):
    """Shuffled slots, some negative: what is written comes back, the rest of the cache and of the outputs stays."""
    torch.manual_seed(dim + n)
    num = n // ps + 5
    ks, vs = scales(heads, n)
    k_cache, v_cache = caches(num, heads, ps, dim, kv, beside=beside)
    a = layer(k_cache, v_cache, kv, ks, vs, heads)
    qkv = torch.randn((n, 3 * heads, dim)).to(a.dtype)
    qkv[:, :, 3] *= 30
    qkv[: n // 3, :, 16:32] = 0                                # blocks of zeros
    slots = torch.randperm(num * ps)[:n].to(torch.int32)
    slots[5::7] = -1
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    dq = qkv.cuda()
    a.append(dq[:, heads:2 * heads], dq[:, 2 * heads:], slots.cuda())
    out = torch.full((n, 2 * heads, dim), 7.0, dtype=a.dtype, device="cuda")
    a.read(out[:, :heads], out[:, heads:], slots.cuda())
    live = slots >= 0
    assert bool((out.cpu()[~live] == 7.0).all())
    assert same(out[:, :heads].cpu()[live], stored(k, ks, kv)[live])
    assert same(out[:, heads:].cpu()[live], stored(v, vs, kv)[live])
    assert a.get_error() == (0, 0, 0, 0)
    # every slot that was not written still reads as the fill
    rest = torch.ones(num * ps, dtype=torch.bool)
    rest[slots[live].long()] = False
    at = rest.nonzero().flatten().to(torch.int32).cuda()
    r = torch.zeros((2, len(at), heads, dim), dtype=a.dtype, device="cuda")
    a.read(r[0], r[1], at)
    assert bool(r.isnan().all())


@pytest.mark.parametrize("kv", ["nvfp4", "bf16"])
@pytest.mark.parametrize("off,step", [(0, 384), (8, 392), (4, 388), (2, 386), (1, 385)])
def test_alignments(cuda_lib, kv, off, step):
    """Rows wherever they begin, in and out."""
    n, heads, dim, ps = 19, 2, 64, 16
    ks, vs = scales(heads)
    a = layer(*caches(3, heads, ps, dim, kv), kv, ks, vs, heads)
    flat = torch.randn(off + n * step).bfloat16().cuda()
    k, v = (flat.as_strided((n, heads, dim), (step, dim, 1), off + i * heads * dim) for i in (0, 1))
    slots = torch.randperm(3 * ps)[:n].to(torch.int32).cuda()
    a.append(k, v, slots)
    to = torch.full((off + n * step,), 7.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = (to.as_strided((n, heads, dim), (step, dim, 1), off + i * heads * dim) for i in (0, 1))
    a.read(ko, vo, slots)
    assert same(ko.cpu(), stored(k.cpu(), ks, kv)) and same(vo.cpu(), stored(v.cpu(), vs, kv))
    ko.fill_(7.0), vo.fill_(7.0)
    assert bool((to == 7.0).all())


def test_borders_and_extremes(cuda_lib):
    """Values on the borders between codes, blocks whose scale is the smallest, zero, or the largest, infinities and NaN."""
    ks = torch.tensor([2.0 ** -8])
    vs = torch.tensor([0.003])
    a = layer(*caches(1, 1, 16, 64, "nvfp4"), "nvfp4", ks, vs, 1)
    x = torch.zeros((16, 1, 64))
    unit = 2.0 ** -8                                           # block scale 1: codes stand for multiples of this
    x[0, 0, :16] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6]) * unit
    x[1, 0, :16] = torch.linspace(-1, 1, 16) * 6 * unit * 2.0 ** -9           # the smallest scale
    x[2, 0, :16] = torch.linspace(-1, 1, 16) * 6 * unit * 2.0 ** -10          # half of it: on the border to zero
    x[3, 0, :16] = torch.linspace(-1, 1, 16) * 6 * unit * 2.0 ** -10 * 1.01
    x[4, 0, :16] = torch.linspace(-1, 1, 16) * 6 * unit * 448
    x[5, 0, :16] = torch.linspace(-1, 1, 16) * 1e30                           # beyond the largest
    x[6, 0, :16] = torch.linspace(-1, 1, 16)
    x[6, 0, 3] = float("inf")
    x[7, 0, 3] = float("-inf")
    x[8, 0, :16] = torch.linspace(-1, 1, 16)
    x[8, 0, 7] = float("nan")
    x[8, 0, 16:32] = 1.0
    x[9, 0, :16] = 1e-40                                       # subnormal
    x[10] = 2.0 ** -20
    x = x.bfloat16()
    slots = torch.arange(16, dtype=torch.int32, device="cuda")
    a.append(x.cuda(), x.cuda(), slots)
    k, v = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    a.read(k, v, slots)
    want = stored(x, ks, "nvfp4"), stored(x, vs, "nvfp4")
    # an infinity is held as the largest value, and the block's others under that scale
    for w, s in zip(want, (ks, vs)):
        for t in (6, 7):
            big = x[t, 0].isinf()
            w[t, 0][big] = (6 * 448 * s * x[t, 0][big].float().sign()).bfloat16()
    assert same(k.cpu(), want[0]) and same(v.cpu(), want[1])
    assert [float(t) for t in k[0, 0, :16].float() / unit] == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6]
    assert bool(k[8, 0, :16].isnan().all()) and not bool(k[8, 0, 16:].isnan().any())


@pytest.mark.parametrize("kv", ["nvfp4", "fp8", "bf16", "f32"])
@pytest.mark.parametrize("dim,R,inter", [(64, 64, False), (64, 36, False), (128, 128, True), (128, 24, False), (128, 66, True), (256, 64, False),
                                         (256, 2, True), (64, 62, True)])
@pytest.mark.parametrize("n", [1, 33, 2434])
def test_rotated_on_the_way(cuda_lib, kv, dim, R, inter, n):
    """Keys rotated in FP32 and rounded once into the cache, queries beside them; the keys themselves stay."""
    torch.manual_seed(dim + R + n)
    heads, q_heads, ps = 2, 6, 16
    rope = rssm.Rope(R, interleaved=inter, base=1000.0 if R > 2 else 10.0, gain=1.25)
    num = n // ps + 3
    ks, vs = scales(heads, n)
    a = layer(*caches(num, heads, ps, dim, kv), kv, ks, vs, q_heads)
    qkv = torch.randn((n, q_heads + 2 * heads, dim)).to(a.dtype).cuda()
    before = qkv.clone()
    q, k, v = qkv.split([q_heads, heads, heads], 1)
    pos = torch.randint(-5, 100000, (n,), dtype=torch.int32).cuda()
    slots = torch.randperm(num * ps)[:n].to(torch.int32)
    slots[3::9] = -1
    live, slots = (slots >= 0), slots.cuda()
    q_out = torch.full((n, q_heads, dim), float("nan"), dtype=a.dtype, device="cuda")
    a.append(k, v, slots, rope=rope, positions=pos, q=q, q_out=q_out)
    assert torch.equal(qkv, before)
    ko, vo = torch.empty((2, n, heads, dim), dtype=a.dtype, device="cuda")
    a.read(ko, vo, slots)
    turned = torch.empty((n, heads, dim), device="cuda")
    rssm.rotary(turned, k.float(), pos, rope)
    assert same(ko.cpu()[live], stored(turned.cpu(), ks, kv)[live])
    assert same(vo.cpu()[live], stored(v.cpu(), vs, kv)[live])
    want = torch.empty_like(q_out)
    rssm.rotary(want, q, pos, rope)
    assert torch.equal(q_out, want)
    a.append(k, v, slots, rope=rope, positions=pos, q=q, q_out=q)              # in place
    assert torch.equal(q, want) and torch.equal(qkv[:, q_heads:], before[:, q_heads:])
    fresh = layer(*caches(num, heads, ps, dim, kv), kv, ks, vs, q_heads)
    fresh.append(k, v, slots, rope=rope, positions=pos)                        # keys alone
    k2, v2 = torch.empty_like(ko), torch.empty_like(vo)
    fresh.read(k2, v2, slots)
    assert same(k2.cpu()[live], ko.cpu()[live]) and same(v2.cpu()[live], vo.cpu()[live])
    assert a.get_error() == (0, 0, 0, 0) and fresh.get_error() == (0, 0, 0, 0)


@pytest.mark.parametrize("kv", ["nvfp4", "bf16"])
def test_slots_past_the_cache_are_reported(cuda_lib, kv):
    heads, dim, ps = 2, 64, 16
    ks, vs = scales(heads)
    rope = rssm.Rope(64)
    x = torch.randn((3, heads, dim), device="cuda").bfloat16()
    slots = torch.tensor([5, 32, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    a = layer(*caches(2, heads, ps, dim, kv), kv, ks, vs, heads)
    for call in (lambda: a.append(x, x, slots, rope=rope, positions=pos), lambda: a.append(x, x, slots),
                 lambda: a.read(x.clone(), x.clone(), slots)):
        call()
        err = a.get_error()
        assert err[0] == rssm.RSSM_DEV_ATTN_SLOT and err[1] == 2 and err[2] in (1, 2) and err[3] in (32, 2 ** 31 - 1)
    y = torch.full_like(x, 7.0)
    a.read(y, torch.empty_like(y), slots)
    assert bool((y[1:] == 7.0).all()) and bool((y[0] != 7.0).any())


class Case:
    """A 4-bit cache with `lens` tokens (the T new ones included) on shuffled pages, written by append. Every byte that
    holds no token is 0xFF: NaN."""

    def __init__(self, lens, T=1, q_heads=8, kv_heads=2, dim=128, ps=16, window=0, seed=0, beside=False, spoil=None, scale=0.0):
        self.__dict__.update(lens=lens, T=T, q_heads=q_heads, kv_heads=kv_heads, dim=dim, window=window, scale=scale)
        g = torch.Generator()
        g.manual_seed(seed)
        B = len(lens)
        held = [-(-n // ps) for n in lens]
        self.max_pages = max(held + [1]) + 1
        num = sum(held) + 3
        order = torch.randperm(num, generator=g)
        table = torch.full((B, self.max_pages), 2 ** 31 - 1, dtype=torch.int32)
        ks, vs = scales(kv_heads, seed)
        self.k_cache, self.v_cache = caches(num, kv_heads, ps, dim, "nvfp4", beside=beside)
        self.kw = dict(k_scale=ks.cuda(), v_scale=vs.cuda())
        write = rssm.Attention(self.k_cache, self.v_cache, batch=1, q_heads=q_heads, max_pages=1, **self.kw)
        self.tokens, at = [], 0
        for b, n in enumerate(lens):
            table[b, :held[b]] = order[at:at + held[b]].int()
            at += held[b]
            k, v = (torch.randn((n, kv_heads, dim), generator=g).bfloat16() for _ in "kv")
            if spoil:
                spoil(b, k, v)
            i = torch.arange(n)
            slots = (table[b, i // ps].long() * ps + i % ps).int()
            write.append(k.cuda(), v.cuda(), slots.cuda())
            self.tokens.append((quantised(k, ks).double(), quantised(v, vs).double()))
        self.q = torch.randn((B, T, q_heads, dim), generator=g).bfloat16()
        self.table, self.lens_d = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def layer(self, **kw):
        a = dict(batch=len(self.lens), q_heads=self.q_heads, max_pages=self.max_pages, max_draft=self.T, window=self.window,
                 scale=self.scale, **self.kw)
        a.update(kw)
        return rssm.Attention(self.k_cache, self.v_cache, **a)

    def run(self, layer=None, q=None):
        layer = layer or self.layer()
        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:3], float("nan"), device="cuda")
        layer.decode(out, self.q.cuda() if q is None else q, self.lens_d, self.table, T=self.T, lse=lse)
        assert layer.get_error() == (0, 0, 0, 0)
        return out.cpu(), lse.cpu()

    def seen(self, b, t):
        p = self.lens[b] - self.T + t
        return slice(max(0, p - self.window + 1) if self.window else 0, max(0, p + 1))

    def want(self):
        Hk, D = self.kv_heads, self.dim
        out = torch.zeros(self.q.shape, dtype=torch.float64)
        lse = torch.full(self.q.shape[:3], -math.inf, dtype=torch.float64)
        for b in range(len(self.lens)):
            for t in range(self.T):
                k, v = (x[self.seen(b, t)] for x in self.tokens[b])
                if len(k):
                    q = self.q[b, t].double().reshape(Hk, self.q_heads // Hk, D)
                    s = torch.einsum("hgd,nhd->hgn", q, k) * (self.scale or 1 / math.sqrt(D))
                    l = torch.logsumexp(s, -1)
                    out[b, t] = torch.einsum("hgn,nhd->hgd", torch.exp(s - l[..., None]), v).reshape(self.q_heads, D)
                    lse[b, t] = l.reshape(self.q_heads)
        return out, lse

    def check(self, got):
        out, lse = got[0].double(), got[1].double()
        w_out, w_lse = self.want()
        vmax = max([float(v.nan_to_num().abs().max()) for _, v in self.tokens if v.numel()] + [0.0])
        lim = vmax * (2.0 ** -13 + 2.0 ** -12)
        nan = w_out.isnan()
        assert torch.equal(out.isnan(), nan)
        lo, hi = (w_out - lim).bfloat16().double(), (w_out + lim).bfloat16().double()
        bad = ~((out >= lo) & (out <= hi)) & ~nan
        assert not bool(bad.any()), f"out: {int(bad.sum())} off, worst {float((out - w_out).abs()[~nan].max() / lim):.2f}x the tolerance"
        empty = w_lse == -math.inf
        assert torch.equal(lse == -math.inf, empty) and torch.equal(lse.isnan(), w_lse.isnan())
        rest = ~empty & ~w_lse.isnan()
        assert bool((lse - w_lse)[rest].abs().le(2.0 ** -14).all()), float((lse - w_lse)[rest].abs().max())


EDGES = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 100, 129, 257]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads,T", [(4, 4, 1), (8, 2, 1), (8, 1, 1), (16, 1, 1), (10, 2, 3), (16, 2, 4), (24, 1, 2), (40, 1, 3), (3, 3, 8)])
def test_lengths_at_the_edges(cuda_lib, dim, q_heads, kv_heads, T):
    """Every way that a request can end in a page, a group and a unit, with no token, fewer tokens than drafts, and 1
    to 120 query rows a cache head."""
    Case_ = Case(EDGES, T=T, q_heads=q_heads, kv_heads=kv_heads, dim=dim, seed=dim + T)
    Case_.check(Case_.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,T", [(1, 1), (5, 1), (16, 4), (17, 3), (100, 2), (1000, 8)])
def test_windows(cuda_lib, dim, window, T):
    c = Case(EDGES + [700], T=T, q_heads=6, kv_heads=2, dim=dim, window=window, seed=window)
    c.check(c.run())


@pytest.mark.parametrize("dim,lens,ps,q_heads,kv_heads,T,beside", [
    (128, [5000], 64, 8, 2, 1, True), (64, [3000, 17, 2100], 32, 16, 1, 1, False), (256, [2600, 900], 48, 8, 1, 4, True),
    (128, [777 + 61 * i for i in range(37)], 16, 4, 4, 1, False), (128, [12000], 128, 16, 1, 2, False), (256, [4000, 1], 16, 40, 1, 3, False)])
def test_long_requests_split_over_blocks(cuda_lib, dim, lens, ps, q_heads, kv_heads, T, beside):
    c = Case(lens, T=T, q_heads=q_heads, kv_heads=kv_heads, dim=dim, ps=ps, seed=len(lens), beside=beside)
    first = c.run()
    c.check(first)
    again = c.run()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dim,T,window", [(64, 3, 0), (128, 4, 0), (256, 2, 0), (128, 3, 40)])
def test_nan_reaches_those_who_see_it(cuda_lib, dim, T, window):
    """A NaN among the drafts' own values, and one at the window's start, spoils the drafts that see it and no other."""
    lens = [70, 33, 16, 5]

    def spoil(b, k, v):
        n = len(v)
        if b != 1:
            v[n - 1, 0, 3] = float("nan")                      # the last draft's own
        if b == 1:
            k[n - 2, 1, 20] = float("nan")
        if window and b == 0:
            v[n - T - window + 1, 1, 40] = float("nan")        # only the first draft still sees it
    c = Case(lens, T=T, q_heads=8, kv_heads=2, dim=dim, window=window, spoil=spoil, seed=dim)
    out, lse = c.run()
    for b in range(len(lens)):
        for t in range(T):
            k, v = (x[c.seen(b, t)] for x in c.tokens[b])
            for h in range(8):
                bad_k = bool(k[:, h // 4].isnan().any())
                # a NaN value spoils its own block of channels
                bad_v = v[:, h // 4].isnan().any(0) | bad_k if len(v) else torch.zeros(dim, dtype=torch.bool)
                assert torch.equal(out[b, t, h].isnan(), bad_v), (b, t, h)
                assert bool(lse[b, t, h].isnan()) == bad_k
    w_out, w_lse = c.want()
    ok = ~out.isnan()
    lim = float(max(v.nan_to_num().abs().max() for _, v in c.tokens)) * (2.0 ** -13 + 2.0 ** -12) + BF16 * w_out.nan_to_num().abs()
    assert bool(((out.double() - w_out).abs() <= lim)[ok & ~w_out.isnan()].all())


@pytest.mark.parametrize("scale", [0.5, -0.3, 1e-30])
def test_scales_of_the_scores(cuda_lib, scale):
    c = Case([40, 300], q_heads=4, kv_heads=2, dim=64, scale=scale, seed=3)
    c.check(c.run())


def test_queries_of_every_size(cuda_lib):
    """Rows of queries from the smallest to near the largest BF16 numbers, zeros, and rows that hold an infinity or a NaN."""
    c = Case([200], q_heads=8, kv_heads=1, dim=128, scale=1.0, seed=5)
    size = [1e-38, 1e-20, 1e-3, 0.0, 0.3, 1e-39]
    for h, s in enumerate(size):
        c.q[0, 0, h] = (c.q[0, 0, h].float() * s).bfloat16()
    c.q[0, 0, 6] = 0
    c.q[0, 0, 6, 5] = float("nan")
    c.q[0, 0, 7] = 0
    c.q[0, 0, 7, 17] = 3.0e38                                  # scores of either sign, far beyond each other
    out, lse = c.run()
    w_out, w_lse = c.want()
    lim = float(c.tokens[0][1].abs().max()) * (2.0 ** -13 + 2.0 ** -12) + BF16 * w_out.nan_to_num().abs()
    assert bool(((out.double() - w_out).abs() <= lim)[0, 0, :6].all()) and bool((lse.double() - w_lse)[0, 0, :6].abs().le(2.0 ** -14).all())
    assert bool(out[0, 0, 6].isnan().all()) and bool(lse[0, 0, 6].isnan())
    # scores of 9e38 are beyond FP32 and count as infinite
    assert bool(out[0, 0, 7].isnan().all())
    c.q[0, 0, 7, 17] = 3.0e37
    out, lse = c.run()
    top = c.tokens[0][0][:, 0, 17].argmax()                    # all weight on the largest
    ties = c.tokens[0][0][:, 0, 17] == c.tokens[0][0][top, 0, 17]
    want = c.tokens[0][1][ties, 0].mean(0)
    assert float((out[0, 0, 7].double() - want).abs().max()) <= float(want.abs().max()) * 2.0 ** -8 + 2.0 ** -10


def test_only_scores_of_minus_infinity(cuda_lib):
    """A row whose every score is -inf weighs nothing."""
    def spoil(b, k, v):
        k[:] = 1.0
    c = Case([20, 3], q_heads=4, kv_heads=1, dim=64, spoil=spoil)
    c.q[0, 0, 1] = 0.0
    c.q[0, 0, 1, 7] = float("-inf")
    out, lse = c.run()
    assert bool((out[0, 0, 1] == 0).all()) and float(lse[0, 0, 1]) == -math.inf
    assert not bool(out[0, 0, 0].isnan().any())


def test_drafts_after_append_equal_single_steps(cuda_lib):
    """Rows are independent of each other: a draft's outputs are within the tolerance of the one-token step's."""
    c = Case([130, 64], T=4, q_heads=8, kv_heads=2, dim=128, seed=9)
    out, lse = c.run()
    one = c.layer(max_draft=1)
    for t in range(4):
        o = torch.empty((2, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
        l = torch.empty((2, 1, 8), device="cuda")
        one.decode(o, c.q[:, t:t + 1].cuda().contiguous(), c.lens_d - 3 + t, c.table, T=1, lse=l)
        assert float((o.cpu().double() - out[:, t:t + 1].double()).abs().max()) < 2.0 ** -7
        assert float((l.cpu() - lse[:, t:t + 1]).abs().max()) < 2.0 ** -14


def test_bad_lengths_and_pages_are_reported(cuda_lib):
    c = Case([40, 40], q_heads=4, kv_heads=2, dim=64, seed=2)
    a = c.layer()
    out, lse = torch.empty((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 1, 4), device="cuda")
    lens = torch.tensor([40, 10 ** 6], dtype=torch.int32, device="cuda")
    table = c.table.clone()
    table[1] = 0
    a.decode(out, c.q.cuda(), lens, table, lse=lse)
    assert a.get_error()[:3] == (rssm.RSSM_DEV_ATTN_LEN, 1, 1)
    table = c.table.clone()
    table[0, 1] = 2 ** 31 - 1                                  # its 16 tokens read as zeros
    a.decode(out, c.q.cuda(), c.lens_d, table, lse=lse)
    err = a.get_error()
    assert err[0] == rssm.RSSM_DEV_ATTN_PAGE and err[2] == 0
    c.tokens[0][0][16:32] = 0
    c.tokens[0][1][16:32] = 0
    c.check((out.cpu(), lse.cpu()))


def test_captured_steps_share_a_workspace(cuda_lib):
    """Two layers of one workspace in two captured graphs, replayed in turn with new inputs."""
    cs = [Case([300, 7], q_heads=8, kv_heads=2, dim=128, seed=1), Case([900], T=3, q_heads=4, kv_heads=1, dim=64, seed=2)]
    big = max(cs, key=lambda c: c.layer().workspace.numel()).layer().workspace
    made = []
    for c in cs:
        a = c.layer(workspace=big)
        q = c.q.cuda()
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:3], device="cuda")
        a.decode(out, q, c.lens_d, c.table, T=c.T, lse=lse)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.decode(out, q, c.lens_d, c.table, T=c.T, lse=lse)
        made.append((c, a, q, out, lse, g))
    for turn in range(3):
        for c, a, q, out, lse, g in made:
            c.q = torch.randn(c.q.shape).bfloat16()
            q.copy_(c.q)
            g.replay()
        torch.cuda.synchronize()
        for c, a, q, out, lse, g in made:
            c.check((out.cpu(), lse.cpu()))
            assert a.get_error() == (0, 0, 0, 0)


def test_refusals(cuda_lib):
    ks, vs = scales(2)
    kc, vc = caches(2, 2, 16, 64, "nvfp4")
    with pytest.raises(ValueError, match="k_scale"):
        rssm.Attention(kc, vc, batch=1, q_heads=4, max_pages=2)
    with pytest.raises(rssm.RssmError):
        rssm.Attention(kc, vc, batch=1, q_heads=4, max_pages=2, in_dtype="f32", k_scale=ks.cuda(), v_scale=vs.cuda())
    a = layer(kc, vc, "nvfp4", ks, vs, 4)
    rope = rssm.Rope(64)
    x, q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    pos = slots.clone()
    for kw, what in ((dict(positions=pos), "go with rope"), (dict(q=q, q_out=q), "go with rope"), (dict(rope=rope), "positions"),
                     (dict(rope=rope, positions=pos.long()), "positions"), (dict(rope=rope, positions=pos[:2]), "positions"),
                     (dict(rope=rope, positions=pos, q=q), "q and q_out"), (dict(rope=rope, positions=pos, q_out=q), "q and q_out"),
                     (dict(rope=rope, positions=pos, q=q[:, :3], q_out=q), "q: shape"),
                     (dict(rope=rope, positions=pos, q=q, q_out=q.float()), "q_out: dtype"),
                     (dict(rope=rssm.Rope(128), positions=pos), "rope: 128")):
        with pytest.raises(ValueError, match=what):
            a.append(x, x, slots, **kw)
    for args, what in (((x.float(), x, slots), "k: dtype"), ((x, x[:2], slots), "v: shape"), ((x, x, slots.long()), "slots"),
                       ((x, x.cpu(), slots), "v: on cpu")):
        with pytest.raises(ValueError, match=what):
            a.read(*args)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    a.read(none, none, slots[:0])
    a.append(none, none, slots[:0], rope=rope, positions=pos[:0])


@pytest.mark.parametrize("kv", ["nvfp4", "fp8", "bf16"])
@pytest.mark.parametrize("off,step", [(4, 772), (2, 770), (1, 769)])
def test_rotated_from_rows_wherever_they_begin(cuda_lib, kv, off, step):
    n, heads, q_heads, dim, ps = 21, 2, 4, 64, 16
    ks, vs = scales(heads)
    rope = rssm.Rope(64)
    a = layer(*caches(3, heads, ps, dim, kv), kv, ks, vs, q_heads)
    flat = torch.randn(off + n * step).bfloat16().cuda()
    q, k, v = (flat.as_strided((n, h, dim), (step, dim, 1), off + at * dim) for h, at in ((q_heads, 0), (heads, q_heads), (heads, q_heads + heads)))
    slots, pos = torch.randperm(3 * ps)[:n].to(torch.int32).cuda(), torch.arange(n, dtype=torch.int32, device="cuda") * 1000
    out, want, turned = torch.empty((n, q_heads, dim), dtype=torch.bfloat16, device="cuda"), torch.empty((n, q_heads, dim), dtype=torch.bfloat16, device="cuda"), torch.empty((n, heads, dim), device="cuda")
    a.append(k, v, slots, rope=rope, positions=pos, q=q, q_out=out)
    rssm.rotary(want, q.contiguous(), pos, rope)
    rssm.rotary(turned, k.float().contiguous(), pos, rope)
    ko, vo = torch.empty((2, n, heads, dim), dtype=torch.bfloat16, device="cuda")
    a.read(ko, vo, slots)
    assert torch.equal(out, want)
    assert same(ko.cpu(), stored(turned.cpu(), ks, kv)) and same(vo.cpu(), stored(v.cpu(), vs, kv))


def test_a_cache_beyond_4_gb(cuda_lib):
    """Pages whose bytes lie past 2^32, in the writer, the reader and the attention."""
    heads, dim, ps, num = 8, 128, 16, 520_000                  # 9216 bytes a page: 4.8 GB each
    ks, vs = scales(heads)
    k_cache, v_cache = (torch.empty((num, heads, ps, dim // 16 * 9), dtype=torch.uint8, device="cuda") for _ in "kv")
    lens, table = [50, 33], torch.tensor([[num - 1, 5, num - 7, num - 300], [num - 2, 470_000, num - 3, 0]], dtype=torch.int32)
    a = layer(k_cache, v_cache, "nvfp4", ks, vs, 16, batch=2, max_pages=4)
    q = torch.randn((2, 1, 16, dim)).bfloat16()
    out, lse = torch.empty_like(q, device="cuda"), torch.empty((2, 1, 16), device="cuda")
    held = []
    for b, n in enumerate(lens):
        k, v = (torch.randn((n, heads, dim)).bfloat16() for _ in "kv")
        i = torch.arange(n)
        slots = (table[b, i // ps].long() * ps + i % ps).int().cuda()
        a.append(k.cuda(), v.cuda(), slots)
        ko, vo = torch.empty((2, n, heads, dim), dtype=torch.bfloat16, device="cuda")
        a.read(ko, vo, slots)
        held.append((quantised(k, ks), quantised(v, vs)))
        assert same(ko.cpu(), held[b][0].bfloat16()) and same(vo.cpu(), held[b][1].bfloat16())
    a.decode(out, q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda(), lse=lse)
    assert a.get_error() == (0, 0, 0, 0)
    for b in range(2):
        k, v = (x.double() for x in held[b])
        s = torch.einsum("hgd,nhd->hgn", q[b, 0].double().view(heads, 2, dim), k) / math.sqrt(dim)
        l = torch.logsumexp(s, -1)
        w = torch.einsum("hgn,nhd->hgd", torch.exp(s - l[..., None]), v).reshape(16, dim)
        lim = float(v.abs().max()) * (2.0 ** -13 + 2.0 ** -12) + BF16 * w.abs()
        assert bool(((out[b, 0].cpu().double() - w).abs() <= lim).all())
        assert float((lse[b, 0].cpu().double() - l.reshape(16)).abs().max()) <= 2.0 ** -14


def test_a_long_tail_under_one_large_score(cuda_lib):
    """Weights of 2^-22 of the largest, 20,000 of them, add up as they should, although each is far below the output's rounding."""
    n, dim = 20001, 64

    def spoil(b, k, v):
        k[:] = 0.0
        k[:, :, :16] = 1.0                                     # every tail token's score: q.k of the first block
        k[0, :, :16] = 0.0
        k[0, :, 16:32] = 1.0
        v[:] = 1.0
        v[0] = 0.0
    c = Case([n], q_heads=1, kv_heads=1, dim=dim, scale=1.0, spoil=spoil)
    held = float(c.tokens[0][0][1, 0, 0])
    gap = 22 * math.log(2.0)                                   # the first token's score over the others'
    c.q[:] = 0.0
    c.q[0, 0, 0, 16] = gap / held
    c.check(c.run())
    w_out, _ = c.want()
    assert float(w_out[0, 0, 0, 0]) > 0.003                     # the tail is what the output is made of
    out, _ = c.run()
    assert abs(float(out[0, 0, 0, 0]) / float(w_out[0, 0, 0, 0]) - 1) < 2.0 ** -7


@pytest.mark.parametrize("scale", [1.0, 0.0123, 0.3333333, 2.0 ** -7, 7.77, 3e-39, 1e-31, 1e31])
def test_fp8_codes_of_every_bf16_number(cuda_lib, scale):
    """The writer with rotary positions, at position 0, stores what the writer without them does: the rounded quotient's code."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits.view(1024, 1, 64)
    k = torch.where(x.isfinite(), x, torch.zeros_like(x))      # a pair's infinity would reach its other half
    s = torch.tensor([scale])
    slots, pos = torch.randperm(1024).to(torch.int32).cuda(), torch.zeros(1024, dtype=torch.int32, device="cuda")
    made = []
    for kw in ({}, dict(rope=rssm.Rope(64), positions=pos)):
        c = caches(64, 1, 16, 64, "fp8", fill=0)
        layer(*c, "fp8", s, s, 1).append(k.cuda(), x.cuda(), slots, **kw)
        made.append([t.view(torch.uint8).cpu() for t in c])
    assert torch.equal(made[0][1], made[1][1])
    # a key's zero may change its sign: -0 cos 0 - u sin 0
    differ = made[0][0] != made[1][0]
    assert bool(((made[0][0][differ] | made[1][0][differ]) == 0x80).all())
