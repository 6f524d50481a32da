"""Rotary positions and the 4-bit cache in the hybrid stack, as a serving loop runs
them: page table, norms, SSM layers, the writer with its rotation and the attention,
against the same steps in float64 with the same storage points, and draft rounds
against token-by-token steps. The tolerances are the hybrid stack's own.

They do not cover a 4-bit code that comes out as its neighbour because a key or value
before it came out as a neighbouring bf16 number: with one token in the cache such a
code moves one of 512 channels by up to a third of its block's largest value, about
0.8, and the projection behind it by 3 x 0.8 / sqrt(512) = 0.1 of vectors of 4. So 4-bit
stacks are compared where both sides hold the same codes."""
import math

import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm
from _gpu import TOL_LOW, vec_err
from hybrid_ssm_decode_gb300.stack import HybridShape, HybridStack
from test_gpu_cache4 import quantised
from test_gpu_hybrid_stack import SHAPE, Reference, _bf, _inputs

pytestmark = pytest.mark.gpu


class Attended(Reference):
    """The reference stack for a pattern of attention layers alone, with rotary positions."""

    def __init__(self, stack, seed, rope):
        super().__init__(stack, seed)
        self.rope, self.at = rope, 0

    def turn(self, x):
        R = self.rope.rotary_dim
        a = self.at * torch.tensor(self.rope.frequencies, dtype=torch.float64)
        cos, sin = a.cos() * self.rope.gain, a.sin() * self.rope.gain
        i, j = (slice(0, R, 2), slice(1, R, 2)) if self.rope.interleaved else (slice(0, R // 2), slice(R // 2, R))
        y = x.clone()
        y[..., i], y[..., j] = x[..., i] * cos - x[..., j] * sin, x[..., j] * cos + x[..., i] * sin
        return y

    def step(self, u):
        s, B, out = self.s, self.s.batch, None
        for li in range(len(s.pattern)):
            w = self.w[li]
            u = u if out is None else u + out
            qkv = _bf(_bf(self.norm(u, w["norm"])) @ w["qkv"]).view(B, -1, s.attn_dim)
            q, k, v = qkv.split([s.q_heads, s.kv_heads, s.kv_heads], dim=1)
            self.kv[li][0].append(_bf(self.turn(k)))
            self.kv[li][1].append(v)
            K, V = (torch.stack(c, 1) for c in self.kv[li])
            qg = _bf(self.turn(q)).view(B, s.kv_heads, -1, s.attn_dim)
            p = torch.softmax(torch.einsum("bhgd,bnhd->bhgn", qg, K) / math.sqrt(s.attn_dim), -1)
            out = _bf(_bf(torch.einsum("bhgn,bnhd->bhgd", p, V).reshape(B, -1)) @ w["out"])
        self.at += 1
        return self.norm(u + out, self.final)


@pytest.mark.parametrize("inter", [False, True])
def test_steps_match_reference(cuda_lib, inter):
    rope = rssm.Rope(48, interleaved=inter, scaling="yarn", factor=4.0, original=64)
    stack = HybridStack(HybridShape(**{**SHAPE.__dict__, "pattern": "AA"}), seed=3, rope=rope)
    ref = Attended(stack, 3, rope)
    for u in _inputs(20, 7):
        got = stack.step(u)
        want = ref.step(u.double().cpu())
        assert vec_err(got.double().cpu().numpy(), want.numpy()) < TOL_LOW
    assert all(e[0] == 0 for e in stack.errors())
    stack.close()


def test_4bit_steps_over_their_own_codes(cuda_lib):
    """Each step's keys and values are in the cache with the codes of their definition, and its output is that of the
    attention in float64 over what the cache holds."""
    rope = rssm.Rope(64, base=300.0)
    s = HybridShape(**{**SHAPE.__dict__, "pattern": "A"})
    stack = HybridStack(s, kv="nvfp4", seed=6, rope=rope)
    w, layer = stack.weights[0], stack.layers[0]
    ref = Reference(stack, 6)
    n, slots, ones = torch.empty((s.batch, s.d_model), dtype=torch.bfloat16, device="cuda"), [], torch.ones(s.kv_heads)
    for at, u in enumerate(_inputs(20, 29)):
        got = stack.step(u)
        slots.append(stack.buffers[1]["slots"].clone())
        rssm.add_norm(n, u, w["norm"])
        qkv = (n @ w["qkv"]).view(s.batch, -1, s.attn_dim)
        q, k, v = qkv.split([s.q_heads, s.kv_heads, s.kv_heads], dim=1)
        pos = torch.full((s.batch,), at, dtype=torch.int32, device="cuda")
        kf, qr = torch.empty(k.shape, device="cuda"), torch.empty_like(q.contiguous())
        rssm.rotary(kf, k.float(), pos, rope)
        rssm.rotary(qr, q, pos, rope)
        K, V = torch.empty((2, len(slots) * s.batch, s.kv_heads, s.attn_dim), dtype=torch.bfloat16, device="cuda")
        layer.read(K, V, torch.cat(slots))
        K, V = (x.view(-1, s.batch, s.kv_heads, s.attn_dim).transpose(0, 1).cpu() for x in (K, V))
        assert torch.equal(K[:, -1], quantised(kf.cpu(), ones).bfloat16())
        assert torch.equal(V[:, -1], quantised(v.cpu(), ones).bfloat16())
        qg = qr.double().cpu().view(s.batch, s.kv_heads, -1, s.attn_dim)
        p = torch.softmax(torch.einsum("bhgd,bnhd->bhgn", qg, K.double()) / math.sqrt(s.attn_dim), -1)
        o = _bf(torch.einsum("bhgn,bnhd->bhgd", p, V.double()).reshape(s.batch, -1))
        want = ref.norm(u.double().cpu() + _bf(o @ ref.w[0]["out"]), ref.final)
        assert vec_err(got.double().cpu().numpy(), want.numpy()) < TOL_LOW
    stack.close()


def test_4bit_drafts_turned_down_leave_no_trace(cuda_lib):
    """Rounds whose rejected drafts are others, with the same drafts kept: the kept ones' outputs are the same bits."""
    T = 3
    shape = HybridShape(**{**SHAPE.__dict__, "max_draft": T})
    rope = rssm.Rope(64, base=500.0)
    a, b = (HybridStack(shape, kv="nvfp4", seed=5, rope=rope) for _ in "ab")
    for u, other, n in zip(_inputs(8, 11, T), _inputs(8, 12, T), [3, 0, 2, 1, 3, 3, 0, 2]):
        mixed = torch.cat([u[:, :n], other[:, n:]], 1).contiguous()
        x, y = a.step(u), b.step(mixed)
        assert torch.equal(x[:, :n], y[:, :n])
        for s in (a, b):
            s.verify(T, torch.full((shape.batch,), n, dtype=torch.int32, device="cuda"))
        assert a.pages.lens.tolist() == b.pages.lens.tolist()
    assert all(e[0] == 0 for s in (a, b) for e in s.errors())
    a.close()
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_draft_rounds_match_single_steps(cuda_lib, kv):
    """Rounds of 3 drafts of which 0 to 3 stay: positions go back with them."""
    T = 3
    shape = HybridShape(**{**SHAPE.__dict__, "max_draft": T})
    rope = rssm.Rope(64, base=500.0)
    a, b = (HybridStack(shape, kv=kv, seed=5, rope=rope) for _ in "ab")
    for u, n in zip(_inputs(8, 11, T), [3, 0, 2, 1, 3, 3, 0, 2]):
        drafts = a.step(u)
        a.verify(T, torch.full((shape.batch,), n, dtype=torch.int32, device="cuda"))
        for t in range(n):
            one = b.step(u[:, t].contiguous())
            assert vec_err(drafts[:, t].double().cpu().numpy(), one.double().cpu().numpy()) < TOL_LOW
    assert all(e[0] == 0 for s in (a, b) for e in s.errors())
    a.close()
    b.close()


def test_a_captured_step(cuda_lib):
    """A whole step in a CUDA graph, replayed on a second stack's inputs, gives the bits of the uncaptured steps."""
    rope = rssm.Rope(64)
    shape = HybridShape(**{**SHAPE.__dict__, "pattern": "A"})
    a, b = (HybridStack(shape, kv="nvfp4", seed=8, rope=rope) for _ in "ab")
    us = _inputs(6, 19)
    for s in (a, b):
        s.step(us[0])
    u = us[1].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = a.step(u)
    for x in us[1:]:
        u.copy_(x)
        g.replay()
        assert torch.equal(out, b.step(x))
    assert a.pages.lens.tolist() == b.pages.lens.tolist() == [6] * shape.batch
    a.close()
    b.close()


def test_a_request_moves_to_a_new_cache(cuda_lib):
    """Tokens read back from a 4-bit cache and written to another, on other pages: the same codes, so the same attention."""
    heads, dim, ps, n = 2, 128, 16, 77
    scale = torch.full((heads,), 0.01, device="cuda")
    pages = [rssm.PageTable(1, ps, 9, 9, free=torch.randperm(9).to(torch.int32).cuda()) for _ in "ab"]
    x = torch.randn((n, 2, heads, dim), device="cuda").bfloat16()
    q = torch.randn((1, 1, 8, dim), device="cuda").bfloat16()
    outs, held = [], x
    for p in pages:
        cache = torch.full((9, 2, heads, ps, dim // 16 * 9), 0xFF, dtype=torch.uint8, device="cuda")
        layer = rssm.Attention(cache[:, 0], cache[:, 1], batch=1, q_heads=8, max_pages=9, k_scale=scale, v_scale=scale)
        slots = torch.empty(n, dtype=torch.int32, device="cuda")
        p.extend(slots, new=torch.tensor([n], dtype=torch.int32, device="cuda"))
        layer.append(held[:, 0], held[:, 1], slots)
        out = torch.empty_like(q)
        layer.decode(out, q, p.lens, p.table)
        outs.append(out)
        back = torch.empty_like(x)
        layer.read(back[:, 0], back[:, 1], slots)
        if held is not x:
            assert torch.equal(back, held)
        held = back
        assert layer.get_error() == (0, 0, 0, 0)
    assert float((outs[0] - outs[1]).abs().max()) <= 2.0 ** -7 * float(outs[0].abs().max())


def test_new_calls_refuse_a_device_that_is_not_current(cuda_lib, monkeypatch):
    bf16 = torch.bfloat16
    cache = torch.zeros((8, 2, 16, 36), dtype=torch.uint8, device="cuda")
    scale, one = torch.ones(2, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    attn = rssm.Attention(cache, cache.clone(), batch=2, q_heads=2, max_pages=2, k_scale=scale, v_scale=scale)
    x = torch.ones((2, 2, 64), dtype=bf16, device="cuda")
    rope = rssm.Rope(64)
    calls = [lambda: attn.append(x, x, one), lambda: attn.append(x, x, one, rope=rope, positions=one, q=x, q_out=x.clone()),
             lambda: attn.read(x.clone(), x.clone(), one), lambda: rssm.rotary(x.clone(), x, one, rope)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(rssm.hybrid, "_current_device", lambda: torch.cuda.current_device() + 1, raising=False)
    for call in calls:
        with pytest.raises(ValueError):
            call()
