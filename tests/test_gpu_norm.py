"""add_norm and gated_norm against their formulas in 64 bits.

Tolerances. With e = 2^-24 (half an ulp in FP32): a sum of squares of n terms,
held in at most 32 terms a thread and then in a tree, is within (32 + 20) e of
itself; rsqrt, the means and the products add less than 12 e, expf and the
divisions of the gate less than 8 e; so a norm is within 80 e = 2^-17.6 of
itself. The residual sum is within 80 e of |scale gate a| and e of itself. An
output is rounded once, so it lies between the roundings of the two ends."""
import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm

pytestmark = pytest.mark.gpu

E = 80 * 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _close(got, want, span, what):
    """got is a rounding of a value within E span of want."""
    lo, hi = (want - E * span - 1e-37).to(got.dtype), (want + E * span + 1e-37).to(got.dtype)
    bad = ~((got >= lo) & (got <= hi))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off"


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ref_add(u, x, w, w_post, gate, scale, eps, off):
    u, n = u.double(), u.shape[-1]
    a = torch.zeros_like(u)
    if x is not None:
        a = x.double()
        if w_post is not None:
            a = a / ((a * a).sum(-1, keepdim=True) / n + eps).sqrt() * (off + w_post.double())
        if gate is not None:
            a = a * gate.double()
        a = a * scale
    s = u + a
    r = 1 / ((s * s).sum(-1, keepdim=True) / n + eps).sqrt()
    return s, s * r * (off + w.double()), a, r * (off + w.double()).abs()


@pytest.mark.parametrize("rows,dim,res,io,post,gate", [
    (1, 4096, BF16, BF16, False, None), (1, 1, F32, F32, True, "row"), (5, 7, F32, BF16, True, "row"),
    (3, 64, BF16, F32, False, "channel"), (33, 200, BF16, BF16, True, "channel"), (2, 8200, F32, BF16, True, None),
    (1000, 1024, F32, BF16, True, "row"), (700, 5003, BF16, BF16, False, "row"), (3, 16392, F32, F32, True, "row"),
    (2, 32768, F32, F32, True, "channel"), (1, 32767, BF16, BF16, True, "row"), (257, 8192, F32, F32, False, None),
    (64, 100, F32, F32, True, None), (12, 248, BF16, BF16, False, None)])
def test_add_norm(cuda_lib, rows, dim, res, io, post, gate):
    g = _gen(rows * 7919 + dim)
    u, x = (_randn(g, rows, dim) * 3).to(res), _randn(g, rows, dim).to(io)
    w = 1 + 0.3 * _randn(g, dim)
    w_post = 1 + 0.3 * _randn(g, dim) if post else None
    gt = None if gate is None else _randn(g, *((dim,) if gate == "channel" else (rows, dim))).to(io)
    u_out, n_out = torch.full_like(u, float("nan")), torch.full_like(x, float("nan"))
    rssm.add_norm(n_out, u, w, x=x, u_out=u_out, w_post=w_post, gate=gt, scale=0.7, eps=1e-5)
    s, n, a, r = _ref_add(u, x, w, w_post, gt, float(torch.tensor(0.7)), 1e-5, 0.0)
    _close(u_out, s, a.abs() + s.abs(), "u_out")
    _close(n_out, n, n.abs() + (a.abs() + s.abs()) * r, "n_out")
    # in place gives the same bits, and so do slices of wider arrays
    u2, x2 = u.clone(), x.clone()
    rssm.add_norm(x2, u2, w, x=x2, u_out=u2, w_post=w_post, gate=gt, scale=0.7, eps=1e-5)
    assert torch.equal(u2, u_out) and torch.equal(x2, n_out)
    for pad in (8, 3):                               # 16-byte rows and others
        wide = torch.full((rows, dim + pad), float("nan"), device="cuda")
        us, xs = wide.to(res, copy=True)[:, pad:], wide.to(io, copy=True)[:, pad:]
        us.copy_(u)
        xs.copy_(x)
        no, uo = torch.empty_like(wide, dtype=io)[:, :dim], torch.empty_like(wide, dtype=res)[:, :dim]
        rssm.add_norm(no, us, w, x=xs, u_out=uo, w_post=w_post, gate=gt, scale=0.7, eps=1e-5)
        _close(uo, s, a.abs() + s.abs(), "u_out, wide rows")
        _close(no, n, n.abs() + (a.abs() + s.abs()) * r, "n_out, wide rows")


def test_add_norm_parts(cuda_lib):
    """Without x (a plain norm), without u_out, without n_out, with offset
    weights, and a row of zeros."""
    g = _gen(3)
    u, x, w = _randn(g, 6, 320), _randn(g, 6, 320).to(BF16), 0.2 * _randn(g, 320)
    u[2] = 0
    n_out = torch.empty_like(x)
    rssm.add_norm(n_out, u, w, w_offset=1.0)
    s, n, a, r = _ref_add(u, None, w, None, None, 1.0, 1e-6, 1.0)
    _close(n_out, n, n.abs() + (a.abs() + s.abs()) * r, "norm alone")
    assert not bool(n_out[2].any())
    u_out = torch.empty_like(u)
    rssm.add_norm(None, u, None, x=x, u_out=u_out, scale=-1.5)
    _close(u_out, u.double() - 1.5 * x.double(), 1.5 * x.double().abs() + u_out.double().abs(), "sum alone")
    rssm.add_norm(n_out, u, w, x=x, w_post=w, w_offset=1.0)
    s, n, a, r = _ref_add(u, x, w, w, None, 1.0, 1e-6, 1.0)
    _close(n_out, n, n.abs() + (a.abs() + s.abs()) * r, "no u_out")
    rssm.add_norm(torch.empty(0, 320, device="cuda"), u[:0], w)


def test_rows_do_not_mix(cuda_lib):
    """A row of NaN and infinities reaches no other row, in every row layout."""
    for dim in (24, 100, 256, 2000, 4096):
        g = _gen(dim)
        u, w = _randn(g, 9, dim), 1 + 0 * _randn(g, dim)
        a, b = torch.empty_like(u), torch.empty_like(u)
        rssm.add_norm(a, u, w)
        u[4, ::2], u[4, 1::2] = float("nan"), float("inf")
        rssm.add_norm(b, u, w)
        keep = [i for i in range(9) if i != 4]
        assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(b[4]).all())


@pytest.mark.parametrize("rows,dim,group,first,io,act", [
    (1, 8192, 1024, False, BF16, "silu"), (256, 8192, 1024, False, BF16, "silu"), (300, 4096, 128, True, BF16, "silu"),
    (7, 640, 128, True, F32, "sigmoid"), (5, 192, 64, True, BF16, "sigmoid"), (11, 3 * 784, 784, False, F32, "silu"),
    (3, 35, 7, True, F32, "silu"), (2, 33, 33, False, BF16, "silu"), (2, 2 * 16392, 16392, False, F32, "sigmoid"),
    (129, 768, 256, True, BF16, "silu"), (1, 8, 1, True, F32, "silu"), (40, 24, 8, False, BF16, "silu")])
def test_gated_norm(cuda_lib, rows, dim, group, first, io, act):
    g = _gen(rows * 31 + dim)
    y, z = _randn(g, rows, dim).to(io), (2 * _randn(g, rows, dim + 16)).to(io)[:, 16:]
    for wn in sorted({dim, group}):
        w = 1 + 0.3 * _randn(g, wn)
        out = torch.full_like(y, float("nan"))
        rssm.gated_norm(out, y, z, w, group=group, norm_first=first, act=act, eps=1e-5)
        yd, zd, wd = y.double(), z.double(), w.double()
        gate = torch.sigmoid(zd) * (zd if act == "silu" else 1.0)
        v = (yd if first else yd * gate).reshape(rows, -1, group)
        v = (v / ((v * v).sum(-1, keepdim=True) / group + 1e-5).sqrt()).reshape(rows, dim)
        v = v * (wd if wn == dim else wd.repeat(dim // group))
        want = v * gate if first else v
        _close(out, want, want.abs(), "gated_norm")
        y2 = y.clone()
        rssm.gated_norm(y2, y2, z, w, group=group, norm_first=first, act=act, eps=1e-5)
        assert torch.equal(y2, out)


def test_norms_on_another_stream_and_in_a_graph(cuda_lib):
    g = _gen(11)
    u, x, w = _randn(g, 64, 4096), _randn(g, 64, 4096), 1 + 0.1 * _randn(g, 4096)
    n1, n2, uo = torch.empty_like(x), torch.zeros_like(x), torch.empty_like(u)
    rssm.add_norm(n1, u, w, x=x, u_out=uo)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    rssm.add_norm(n2, u, w, x=x, u_out=uo, stream=s)
    s.synchronize()
    assert torch.equal(n1, n2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rssm.add_norm(n2, u, w, x=x, u_out=uo)
        rssm.gated_norm(n2, n2, x, w)
    n2.zero_()
    graph.replay()
    rssm.gated_norm(n1, n1, x, w)
    torch.cuda.synchronize()
    assert torch.equal(n1, n2)


def test_weights_written_by_the_call_in_front(cuda_lib):
    """A norm whose weights, and an attention whose scales, an overlapped call has
    just written, again and again over the same addresses, in and out of a graph."""
    g = _gen(5)
    dim, n = 4096, 40
    src = [_randn(g, 1, dim).abs() + 0.1 for _ in range(n)]
    ones, u = torch.ones(dim, device="cuda"), _randn(g, 300, dim).to(BF16)
    w, outs = torch.zeros(1, dim, device="cuda"), [torch.empty_like(u) for _ in range(n)]
    k8 = _randn(g, 4, 8, 16, 64).to(torch.float8_e4m3fn)
    scale, heads = torch.ones(1, 8, device="cuda"), [(s[:, :8] * 0.01).contiguous() for s in src]
    layer = rssm.Attention(k8, k8, batch=4, q_heads=8, max_pages=1, k_scale=scale.view(8), v_scale=scale.view(8))
    q = _randn(g, 4, 1, 8, 64).to(BF16)
    lens, table = (torch.full((4,), 16, dtype=torch.int32, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda"))
    att = [torch.empty_like(q) for _ in range(n)]

    def chain(sync):
        for s, h, o, a in zip(src, heads, outs, att):
            rssm.add_norm(w, s, ones)
            sync()
            rssm.add_norm(o, u, w.view(dim))
            rssm.gated_norm(o, o, u, w.view(dim), group=1024)
            rssm.add_norm(None, h, None, x=h, u_out=scale)
            sync()
            layer.decode(a, q, lens, table)
            sync()

    chain(torch.cuda.synchronize)
    want = [[t.clone() for t in ts] for ts in (outs, att)]
    assert not torch.equal(want[0][0], want[0][1]) and not torch.equal(want[1][0], want[1][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for go in (lambda: chain(lambda: None), graph.replay):
        for _ in range(3):
            for t in outs + att + [w, scale]:
                t.fill_(1)
            go()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs + att, want[0] + want[1]))


def test_binding_refuses(cuda_lib):
    u = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    n = torch.empty_like(u)
    for kw in (dict(u=u.half()), dict(u=u.t()), dict(w=w[:32]), dict(w=w.double()), dict(x=u.to(BF16)), dict(n_out=n.cpu()),
               dict(x=u[:2]), dict(u_out=n.to(BF16)), dict(x=u, gate=w.to(BF16)), dict(x=u, gate=w[:10]), dict(u=u[:1].expand(4, 64))):
        a = dict(n_out=n, u=u, w=w)
        a.update(kw)
        with pytest.raises(ValueError):
            rssm.add_norm(**a)
    for kw in (dict(w=None), dict(gate=w), dict(eps=-1.0), dict(eps=float("nan"))):
        a = dict(n_out=n, u=u, w=w)
        a.update(kw)
        with pytest.raises(rssm.RssmError):
            rssm.add_norm(**a)
    with pytest.raises(rssm.RssmError):
        rssm.add_norm(torch.empty(1, 40000, device="cuda"), torch.empty(1, 40000, device="cuda"), torch.empty(40000, device="cuda"))
    for kw in (dict(z=u.to(BF16)), dict(act="tanh"), dict(w=w[:3])):
        a = dict(out=n, y=u, z=u, w=w)
        a.update(kw)
        with pytest.raises(ValueError):
            rssm.gated_norm(**a)
    with pytest.raises(rssm.RssmError):
        rssm.gated_norm(n, u, u, w, group=48)
