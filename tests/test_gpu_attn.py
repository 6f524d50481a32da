"""The attention over a paged cache, and the cache's writer, against the
definition in 64 bits, request by request over the tokens that each sees.

Tolerances, for values of size vmax = max |v| and n tokens. The weights w sum
to 1, so an error of x in every weight gives at most x vmax.
  all      FP32 sums of scores (|s| < 40 in units of 1): 2^-18 relative in a
           weight; sums over tokens in FP32, in parts of at most a few thousand
           terms of one sign each: below 2^-13 vmax with all of the above
  BF16     weights carry 16 bits: 2^-16
  FP8      weights carry 11 bits: 2^-12
  FP32     two-term products: 2^-20 relative in a score, 2^-16 vmax in all
An output is rounded once, so it lies between the roundings of the two ends.
lse: 2^-14 absolute."""
import math

import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm

pytestmark = pytest.mark.gpu

KV = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


class Case:
    """A cache with `lens` tokens (the T new ones included) on shuffled pages. Every slot that
    holds no token, and every page that no request holds, is poison."""

    def __init__(self, lens, T=1, q_heads=8, kv_heads=2, dim=128, ps=16, window=0, kv="bf16", seed=0, poison=True,
                 interleave=False, extra_pages=3):
        self.__dict__.update(locals())
        g = torch.Generator()
        g.manual_seed(seed)
        B = len(lens)
        held = [-(-n // ps) for n in lens]
        self.max_pages = max(held + [1]) + 1
        num = sum(held) + extra_pages
        order = torch.randperm(num, generator=g)
        table = torch.full((B, self.max_pages), 2 ** 31 - 1, dtype=torch.int32)    # never read past a request
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h].int()
            at += h
        self.io = torch.float32 if kv == "f32" else torch.bfloat16
        self.ks = torch.rand(kv_heads, generator=g) * 0.01 + 0.01 if kv == "fp8" else None
        self.vs = torch.rand(kv_heads, generator=g) * 0.01 + 0.01 if kv == "fp8" else None
        self.tokens = []                                       # per request: stored k, v [len][Hk][D] in 64 bits
        caches = torch.full((2, num, kv_heads, ps, dim), float("nan") if poison else 0.0).to(KV[kv])
        if poison and kv != "fp8":
            caches[:, ::2] = float("inf")
        raw = caches.view(torch.uint8) if kv == "fp8" else caches
        for b, n in enumerate(lens):
            pair = []
            for i, s in ((0, self.ks), (1, self.vs)):
                x = torch.randn((n, kv_heads, dim), generator=g)
                x = (x / s[:, None]).clamp(-448, 448).to(KV[kv]) if kv == "fp8" else x.to(KV[kv])
                for j in range(held[b]):
                    part = x[j * ps:(j + 1) * ps].transpose(0, 1)
                    raw[i, table[b, j], :, :part.shape[1]] = part.contiguous().view(raw.dtype)
                pair.append(x.double() * s.double()[:, None] if kv == "fp8" else x.double())
            self.tokens.append(pair)
        self.q = torch.randn((B, T, q_heads, dim), generator=g).to(self.io)
        if interleave:                                         # K and V of a page side by side in one array
            both = caches.view(torch.uint8) if kv == "fp8" else caches
            both = both.transpose(0, 1).contiguous().cuda()
            both = both.view(KV[kv])
            self.k_cache, self.v_cache = both[:, 0], both[:, 1]
        else:
            self.k_cache, self.v_cache = caches[0].cuda(), caches[1].cuda()
        self.table, self.lens_d = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def layer(self, **kw):
        fp8 = self.kv == "fp8"
        a = dict(batch=len(self.lens), q_heads=self.q_heads, max_pages=self.max_pages, max_draft=self.T, window=self.window,
                 k_scale=self.ks.cuda() if fp8 else None, v_scale=self.vs.cuda() if fp8 else None)
        a.update(kw)
        return rssm.Attention(self.k_cache, self.v_cache, **a)

    def run(self, layer=None, q=None, **kw):
        layer = layer or self.layer()
        q = self.q.cuda() if q is None else q
        out = torch.full(self.q.shape, float("nan"), dtype=self.io, device="cuda")
        lse = torch.full(self.q.shape[:3], float("nan"), device="cuda")
        layer.decode(out, q, self.lens_d, self.table, T=self.T, lse=lse, **kw)
        return out, lse

    def want(self, scale=None):
        """out, lse in 64 bits."""
        T, Hq, Hk, D, W = self.T, self.q_heads, self.kv_heads, self.dim, self.window
        scale = scale or 1 / math.sqrt(D)
        out = torch.zeros(self.q.shape, dtype=torch.float64)
        lse = torch.full(self.q.shape[:3], -math.inf, dtype=torch.float64)
        for b, n in enumerate(self.lens):
            k, v = self.tokens[b]
            for t in range(T):
                p = n - T + t
                if p < 0:
                    continue
                lo = max(0, p - W + 1) if W else 0
                q = self.q[b, t].double().reshape(Hk, Hq // Hk, D)
                s = torch.einsum("hgd,nhd->hgn", q, k[lo:p + 1]) * scale
                l = torch.logsumexp(s, -1)
                out[b, t] = torch.einsum("hgn,nhd->hgd", torch.exp(s - l[..., None]), v[lo:p + 1]).reshape(Hq, D)
                lse[b, t] = l.reshape(Hq)
        return out, lse

    def check(self, got, scale=None):
        out, lse = (x.cpu().double() for x in got)
        w_out, w_lse = self.want(scale)
        vmax = max([float(v.abs().max()) for _, v in self.tokens if v.numel()] + [0.0])
        lim = vmax * {"f32": 2.0 ** -16, "bf16": 2.0 ** -13, "fp8": 2.0 ** -13 + 2.0 ** -12}[self.kv]
        lo, hi = (w_out - lim).to(self.io).double(), (w_out + lim).to(self.io).double()
        bad = ~((out >= lo) & (out <= hi))
        assert not bool(bad.any()), f"out: {int(bad.sum())} off, worst {float((out - w_out).abs().max() / lim):.2f}x the tolerance"
        empty = w_lse == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        assert bool((lse - w_lse)[~empty].abs().le(2.0 ** -14).all()), float((lse - w_lse)[~empty].abs().max())


EDGES = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 100, 129, 257]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads,T", [(4, 4, 1), (8, 2, 1), (16, 1, 1), (10, 2, 3), (16, 2, 4), (24, 1, 2), (40, 1, 3)])
def test_lengths_at_the_edges(cuda_lib, kv, dim, q_heads, kv_heads, T):
    """Every way that a request can end in a page, a group and a unit, with no
    token, fewer tokens than drafts, and up to 120 query rows a cache head."""
    c = Case(EDGES, T=T, q_heads=q_heads, kv_heads=kv_heads, dim=dim, kv=kv, seed=dim + T)
    layer = c.layer()
    c.check(c.run(layer))
    assert layer.get_error() == (0, 0, 0, 0)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window,T", [(1, 1), (5, 1), (16, 4), (17, 3), (100, 2), (1000, 8)])
def test_windows(cuda_lib, kv, window, T):
    c = Case(EDGES + [700], T=T, q_heads=6, kv_heads=2, dim=64, window=window, kv=kv, seed=window)
    c.check(c.run())


def test_a_window_longer_than_any_request(cuda_lib):
    c = Case([1, 40, 300], T=3, q_heads=4, kv_heads=2, dim=64, seed=12)
    for window in (300, 2 ** 31 - 1):
        c.check(c.run(c.layer(window=window)))


@pytest.mark.parametrize("lens,kv_heads,ps,kv", [
    ([20000], 1, 16, "bf16"), ([30001, 3], 2, 64, "fp8"), ([1], 1, 16, "bf16"), ([5000, 1, 0, 7777], 3, 48, "bf16"),
    ([3000] * 5, 2, 128, "f32"), ([(i * 37) % 200 for i in range(700)], 2, 16, "bf16"), ([0] * 40, 2, 16, "fp8")])
def test_split_and_join(cuda_lib, lens, kv_heads, ps, kv):
    """Long requests split over many blocks, and many short ones in one block."""
    c = Case(lens, q_heads=4 * kv_heads, kv_heads=kv_heads, dim=64, ps=ps, kv=kv, seed=len(lens))
    layer = c.layer()
    got = c.run(layer)
    c.check(got)
    again = c.run(layer)                                       # the counters are back at zero; same bits
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert layer.get_error()[0] == 0


@pytest.mark.parametrize("kv,dim,T", [("bf16", 64, 1), ("bf16", 128, 8), ("bf16", 256, 4), ("fp8", 64, 1), ("fp8", 256, 8),
                                      ("f32", 128, 4), ("f32", 256, 8)])
def test_long_shares(cuda_lib, kv, dim, T):
    """Blocks whose share is many times their ring of slots: the small cache is
    read by many requests through tables that repeat its pages."""
    c = Case([1500], T=T, q_heads=8, kv_heads=2, dim=dim, kv=kv, seed=dim)
    one, one_lse = c.run()
    c.check((one, one_lse))
    n = 300
    c.table, c.lens_d, c.lens = c.table.repeat(n, 1), c.lens_d.repeat(n), c.lens * n
    c.q = c.q.repeat(n, 1, 1, 1)
    out, lse = c.run()
    vmax = float(c.tokens[0][1].abs().max())
    # the same sums in other parts: 2^-12 vmax (FP8 weights) and a rounding of the output
    lim = 2.0 ** -11 * vmax + (one.float().abs() * 2.0 ** -7 if kv != "f32" else 0)
    assert bool(((out.float() - one.float()).abs() <= lim).all())
    assert float((lse - one_lse).abs().max()) < 2.0 ** -13


def test_large_scores_and_scale(cuda_lib):
    """Scores whose exponentials pass FP32 either way, and a given scale."""
    c = Case([300, 40], q_heads=4, kv_heads=2, dim=64, seed=2)
    c.q *= 100
    for s in (1.0, -0.5):
        layer = c.layer(scale=s)
        out, lse = c.run(layer)
        want, w_lse = c.want(s)
        assert float((out.cpu().double() - want).abs().max()) < 0.05      # scores of thousands: 2^-12 absolute each
        assert float(((lse.cpu().double() - w_lse) / w_lse.abs().clamp(min=1)).abs().max()) < 2.0 ** -18


@pytest.mark.parametrize("mag", [1e-30, 1e30])
def test_fp8_query_range(cuda_lib, mag):
    """Queries far outside FP16's range over an FP8 cache: small ones give the
    plain mean, large ones the value of the best token."""
    c = Case([50], q_heads=2, kv_heads=1, dim=64, kv="fp8", seed=4)
    c.q = (c.q.float() * mag).to(torch.bfloat16)
    out, _ = c.run()
    want, _ = c.want()
    lim = float(c.tokens[0][1].abs().max()) * 2.0 ** -11
    out = out.cpu()
    assert bool(((out >= (want - lim).to(out.dtype)) & (out <= (want + lim).to(out.dtype))).all())


@pytest.mark.parametrize("mag", [1.0, 1e6, 1e30])
def test_fp8_infinite_query(cuda_lib, mag):
    """Beside an infinite query element the others, whatever their size, stay
    finite: a row whose scores are all -inf is empty."""
    c = Case([50], q_heads=4, kv_heads=2, dim=64, kv="fp8", seed=4)
    raw = c.k_cache.view(torch.uint8)
    raw[c.table[0, :4].long()] |= 0x80                         # keys below zero, one dimension apart from it
    raw[..., 5].clamp_(min=0x88)
    c.q = (c.q.float().abs() * mag).neg().to(torch.bfloat16)   # finite terms above zero
    c.q[..., 5] = math.inf
    out, lse = c.run()
    assert not bool(out.any()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dim,T,lens", [(64, 1, [5000, 64]), (128, 1, [20000]), (256, 4, [3000, 100])])
def test_fp8_small_weights(cuda_lib, dim, T, lens):
    """A long tail under a few large scores: every 16th token scores 18 above the
    others and has value 0, so the output is made of weights of e^-18 = 2^-26 of
    the largest alone. Each is within 2^-12 of itself, and so is their sum, as
    all values are positive; the division adds less than as much again."""
    B, ps = len(lens), 16
    held = [-(-n // ps) for n in lens]
    k, v = torch.zeros((sum(held), 1, ps, dim)), torch.ones((sum(held), 1, ps, dim))
    k[:, :, 0, 0] = 18
    v[:, :, 0] = 0
    table = torch.full((B, max(held)), -1, dtype=torch.int32)
    for b, h in enumerate(held):
        table[b, :h] = torch.arange(h) + sum(held[:b])
    one = torch.ones(1, device="cuda")
    kc, vc = (x.cuda().to(torch.float8_e4m3fn) for x in (k, v))
    layer = rssm.Attention(kc, vc, batch=B, q_heads=1, max_pages=max(held), max_draft=T, scale=1.0, k_scale=one, v_scale=one)
    q = torch.zeros((B, T, 1, dim), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    layer.decode(out, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda(), T=T, lse=lse)
    out, lse = out.cpu(), lse.cpu()
    for b, n in enumerate(lens):
        for t in range(T):
            seen = n - T + t + 1
            large = -(-seen // ps)
            tail = (seen - large) * math.exp(-18.0)
            want = torch.tensor(tail / (large + tail), dtype=torch.float64)
            lo, hi = ((want * (1 + e)).to(out.dtype) for e in (-2.0 ** -11, 2.0 ** -11))
            assert bool(((out[b, t] >= lo) & (out[b, t] <= hi)).all()), (float(out[b, t, 0, 0]), float(want))
            assert abs(float(lse[b, t, 0]) - (18 + math.log(large + tail))) < 2.0 ** -14


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("what", ["one", "all", "query", "lowest"])
def test_scores_of_minus_infinity(cuda_lib, kv, dim, what):
    """Keys that a row sees with a score of -inf, or of the type's lowest value,
    weigh nothing; a row that sees no others is empty."""
    c = Case([41, 16], q_heads=4, kv_heads=2, dim=dim, kv=kv, poison=False, seed=dim)
    c.q[..., 5] = c.q[..., 5].abs() + 0.5
    low = {"lowest": torch.finfo(c.io).min}.get(what, -math.inf)
    at = {"one": [7, 20], "lowest": [7, 20], "all": range(41), "query": range(41)}[what]
    for b, n in enumerate(c.lens):
        k = c.tokens[b][0]
        for i in at:
            if i < n:
                new = -k[i, :, 5].abs() - 0.25 if what == "query" else torch.full((2,), low, dtype=torch.float64)
                k[i, :, 5] = new
                c.k_cache[c.table[b, i // 16], :, i % 16, 5] = new.to(c.io).cuda()
    if what == "query":
        c.q[..., 5] = math.inf
    out, lse = c.run()
    if what in ("all", "query"):
        assert not bool(out.any()) and bool((lse == -math.inf).all())
    else:
        c.check((out, lse))


@pytest.mark.parametrize("kv", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("what", [float("inf"), float("nan")])
def test_unseen_values_that_are_not_finite(cuda_lib, kv, what):
    """A draft's key and value of infinity or NaN reach only the drafts that
    see it, at the end of the request and at the window's start."""
    if kv == "fp8" and what == float("inf"):
        what = float("nan")                                    # E4M3 has no infinity
    for window, at in ((0, 1), (0, 2), (20, -1)):
        c = Case([45, 100, 17], T=3, q_heads=6, kv_heads=2, dim=64, window=window, kv=kv, seed=9)
        layer = c.layer()
        clean, clean_lse = c.run(layer)
        b, n = 1, 100
        tok = n - 3 + at if at >= 0 else n - 3 - window + 1    # draft `at`'s own token; the first that draft 0 sees
        slot = (int(c.table[b, tok // 16]), tok % 16)
        for cache in (c.k_cache, c.v_cache):
            cache[slot[0], 1, slot[1]] = torch.full((64,), what, device="cuda").to(cache.dtype)
        got, lse = c.run(layer)
        seen = list(range(at, 3)) if at >= 0 else [0]
        for bb in range(3):
            for t in range(3):
                hit = bb == b and t in seen
                assert torch.equal(got[bb, t, :3], clean[bb, t, :3]) and torch.equal(lse[bb, t, :3], clean_lse[bb, t, :3])
                if hit:
                    assert bool(torch.isnan(got[bb, t, 3:]).all())
                else:
                    assert torch.equal(got[bb, t, 3:], clean[bb, t, 3:])


def test_interleaved_caches_and_query_slices(cuda_lib):
    """K and V of a page in one array, and q as a slice of a wider projection."""
    for kv in ("bf16", "fp8", "f32"):
        c = Case([70, 16, 500], T=2, q_heads=4, kv_heads=2, dim=128, kv=kv, interleave=True, seed=6)
        assert not c.k_cache.is_contiguous()
        wide = torch.full((3 * 2, 8, 128), float("nan"), dtype=c.io, device="cuda")
        wide[:, 2:6] = c.q.reshape(6, 4, 128).cuda()
        c.check(c.run(q=wide[:, 2:6]))


def test_offsets_past_32_bits(cuda_lib):
    """Pages beyond 2^31 elements (and bytes) of a large cache."""
    c = Case([100, 33], q_heads=4, kv_heads=8 // 4, dim=128, ps=64, kv="fp8", seed=8, poison=False)
    pages = 150_000                                            # 150,000 * 2 * 64 * 128 = 2.46e9
    small = (c.k_cache, c.v_cache)
    big = []
    for s in small:
        x = torch.zeros((pages, 2, 64, 128), dtype=torch.uint8, device="cuda")
        x[pages - s.shape[0]:] = s.view(torch.uint8)
        big.append(x.view(torch.float8_e4m3fn))
    c.k_cache, c.v_cache = big
    t = c.table.clone()
    t[t < 1000] += pages - small[0].shape[0]
    c.table = t
    layer = c.layer()
    c.check(c.run(layer))
    # and the writer: the last slot of the last page
    k = torch.randn(1, 2, 128, device="cuda").to(torch.bfloat16)
    layer.append(k, k, torch.tensor([pages * 64 - 1], dtype=torch.int32, device="cuda"))
    want = (k.float() / c.ks.cuda()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(big[0][-1, :, -1].view(torch.uint8), want[0].view(torch.uint8))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("dim,offset", [(64, 0), (256, 0), (128, 1)])
def test_append(cuda_lib, kv, dim, offset):
    """The writer puts each token where its slot says and touches nothing else;
    negative slots are skipped, slots past the cache skipped and reported."""
    c = Case([0, 0], kv_heads=3, q_heads=3, dim=dim, kv=kv, extra_pages=9, poison=False, seed=1)
    layer = c.layer()
    n = 37
    g = torch.Generator(device="cuda")
    g.manual_seed(dim)
    wide = (torch.randn((n, 3 * dim * 2 + 8), generator=g, device="cuda") * 3).to(c.io)
    wide[3, 5:9] = torch.tensor([float("nan"), 1e9, -1e9, 0.0], device="cuda").to(c.io)
    k, v = wide[:, offset:offset + 3 * dim], wide[:, offset + 3 * dim:offset + 6 * dim]
    slots = torch.randperm(9 * 16, generator=torch.Generator().manual_seed(2))[:n].int()
    slots[7], slots[20] = -1, 9 * 16 + 3
    want = []
    for x, cache, s in ((k, c.k_cache, c.ks), (v, c.v_cache, c.vs)):
        y = x.reshape(n, 3, dim)
        if kv == "fp8":
            y = (y.float() / s.cuda()[:, None]).clamp(-448, 448)
        y = y.to(KV[kv])
        e = cache.clone()
        for i, sl in enumerate(slots.tolist()):
            if 0 <= sl < 9 * 16:
                e.view(torch.uint8)[sl // 16, :, sl % 16] = y[i].contiguous().view(torch.uint8)
        want.append(e)
    layer.append(k, v, slots.cuda())
    for e, cache in zip(want, (c.k_cache, c.v_cache)):
        a, b = cache.float(), e.float()
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    assert layer.get_error() == (rssm.RSSM_DEV_ATTN_SLOT, 1, 20, 9 * 16 + 3)


def test_reported_lengths_and_pages(cuda_lib):
    """A negative length and one past the table are cut to the range, a page
    past the cache is read as zeros; each is reported, and the other requests
    are not touched."""
    c = Case([40, 50, 60], q_heads=4, kv_heads=2, dim=64, seed=5)
    layer = c.layer()
    good = c.run(layer)
    c.lens_d[1] = -4
    out, lse = c.run(layer)
    assert layer.get_error() == (rssm.RSSM_DEV_ATTN_LEN, 1, 1, -4)
    assert not bool(out[1].any()) and bool((lse[1] == -math.inf).all())
    assert torch.equal(out[[0, 2]], good[0][[0, 2]])
    c.lens_d[1] = 50
    c.table[1, 1] = c.k_cache.shape[0]
    out, lse = c.run(layer)
    assert layer.get_error()[0] == rssm.RSSM_DEV_ATTN_PAGE
    assert torch.equal(out[[0, 2]], good[0][[0, 2]]) and bool(torch.isfinite(out).all())


def test_shared_workspace_streams_and_graphs(cuda_lib):
    """Two layers on one workspace, a call on another stream, and a captured
    call that is replayed with other lengths."""
    a = Case([3000, 10], q_heads=8, kv_heads=2, dim=64, seed=1)
    b = Case([100, 2000, 5], q_heads=4, kv_heads=4, dim=128, T=2, kv="fp8", seed=2)
    ws = torch.empty(max(rssm.rssm_attn_workspace_size(x.layer().cfg) for x in (a, b)), dtype=torch.uint8, device="cuda")
    la, lb = a.layer(workspace=ws), b.layer(workspace=ws)
    for _ in range(2):
        a.check(a.run(la))
        b.check(b.run(lb))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = a.run(la, stream=s)
    s.synchronize()
    a.check(got)
    q = a.q.cuda()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.decode(out, q, a.lens_d, a.table, lse=lse)
    for lens in ([3000, 10], [17, 0], [2999, 3]):
        a.lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        full = a.tokens
        a.lens, a.tokens = lens, [[x[:n] for x in pair] for pair, n in zip(full, lens)]
        graph.replay()
        a.check((out, lse))
        a.tokens = full


@pytest.mark.parametrize("one,two", [
    (dict(q_heads=32, kv_heads=2), dict(q_heads=32, kv_heads=8)),
    (dict(lens=64), dict(lens=256)),
    (dict(q_heads=16, kv_heads=1, T=4), dict(q_heads=8, kv_heads=8)),
    (dict(lens=3, long=9000), dict(lens=300, kv_heads=4))])
def test_layers_of_other_shapes_on_one_workspace(cuda_lib, one, two):
    """Layers that differ in cache heads, batch or drafts, with requests split over
    blocks, called in turn on one workspace: each as on its own."""
    def case(seed, lens=256, long=90, **kw):
        n = [(i * 37 + seed) % long + 1 for i in range(lens - 1)] + [long * 3]
        return Case(n, **{**dict(q_heads=4, kv_heads=2, dim=64, seed=seed), **kw})

    a, b = case(1, **one), case(2, **two)
    alone = [c.run() for c in (a, b)]
    for c, got in zip((a, b), alone):
        c.check(got)
    ws = torch.empty(max(rssm.rssm_attn_workspace_size(c.layer().cfg) for c in (a, b)), dtype=torch.uint8, device="cuda")
    layers = [c.layer(workspace=ws) for c in (a, b)]
    for _ in range(3):
        for c, layer, want in zip((a, b), layers, alone):
            out, lse = c.run(layer)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            assert layer.get_error() == (0, 0, 0, 0)


@pytest.mark.parametrize("first", [rssm.RSSM_DEV_TIMEOUT, rssm.RSSM_DEV_ATTN_LEN])
def test_workspace_after_a_wait_ran_out(cuda_lib, first):
    """What a call that gave up leaves (its mark beside the error word, whatever
    code came first, and counters between zero and their last value) is cleared
    by get_error; the state is written by the host, no wait runs out here."""
    c = Case([3000, 200, 77], q_heads=4, kv_heads=2, dim=64, seed=7)
    layer = c.layer()
    want = c.run(layer)
    words = layer.workspace.view(torch.int32)
    counters = slice(64, 64 + 3 * 304)             # behind the error word's 256 bytes: a count per block, two per round
    torch.cuda.synchronize()
    assert not bool(words[counters].any())
    words[:5] = torch.tensor([first, 3, -1, 0, 1], dtype=torch.int32)
    words[counters] = 1
    assert layer.get_error() == (first, 3, -1, 0)
    torch.cuda.synchronize()
    assert not bool(words[:64 + 3 * 304].any())
    got = c.run(layer)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert layer.get_error() == (0, 0, 0, 0)


def test_fewer_drafts_than_the_most(cuda_lib):
    c = Case([90, 33], T=1, q_heads=16, kv_heads=2, dim=128, seed=3)
    c.check(c.run(c.layer(max_draft=8)))


def test_binding_refuses(cuda_lib):
    c = Case([40, 50], q_heads=4, kv_heads=2, dim=64, seed=5)
    layer = c.layer()
    q, out = c.q.cuda(), torch.empty(c.q.shape, dtype=c.io, device="cuda")
    good = dict(out=out, q=q, lens=c.lens_d, table=c.table)
    for kw in (dict(q=q.float()), dict(q=q[:1]), dict(q=q.transpose(2, 3)), dict(lens=c.lens_d.long()), dict(table=c.table[:, :1]),
               dict(out=out.float()), dict(lse=torch.empty(3, device="cuda")), dict(q=q.cpu()), dict(q=q[:1].expand(2, 1, 4, 64))):
        a = dict(good)
        a.update(kw)
        with pytest.raises(ValueError):
            layer.decode(**a)
    with pytest.raises(rssm.RssmError) as e:
        two = torch.empty((2, 2, 4, 64), dtype=c.io, device="cuda")
        layer.decode(two, two, c.lens_d, c.table, T=2)
    assert e.value.status == rssm.RSSM_ERR_CAPACITY
    with pytest.raises(rssm.RssmError):
        odd = torch.empty(2 * 4 * 64 + 1, dtype=c.io, device="cuda")[1:].view(2, 1, 4, 64)   # not on 16 bytes
        layer.decode(out, odd, c.lens_d, c.table)
    for kw in (dict(q_heads=3), dict(window=-1), dict(max_draft=0), dict(max_draft=9), dict(scale=float("nan"))):
        with pytest.raises(rssm.RssmError):
            c.layer(**kw)
    with pytest.raises(rssm.RssmError):
        c.layer(workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        c.layer(k_scale=torch.ones(2, device="cuda"))
    k8 = torch.zeros((4, 2, 16, 64), device="cuda").to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        rssm.Attention(k8, k8, batch=1, q_heads=2, max_pages=2)
    for shape in ((4, 2, 8, 64), (4, 2, 16, 96)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(rssm.RssmError):
            rssm.Attention(x, x, batch=1, q_heads=2, max_pages=2)
    with pytest.raises(ValueError):
        layer.append(q, q, torch.zeros(2, dtype=torch.int32, device="cuda"))
