"""The hybrid stack on the GPU (page table, cache writer, paged attention, norms
and the SSM layers together) against the same stack in float64 with the same bf16
storage points, and its draft rounds against token-by-token steps. As for the
SSM stack, an element whose float32 and float64 values round to neighbouring bf16
values moves a layer's output by one bf16 ulp, which keeps the per-vector error
below 2e-2."""
import math

import numpy as np
import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm
import synth
from _gpu import TOL_LOW, vec_err
from hybrid_ssm_decode_gb300.stack import HybridShape, HybridStack

pytestmark = pytest.mark.gpu

SHAPE = HybridShape(pattern="MAMA", batch=3, heads=8, head_dim=64, state_dim=64, groups=2, k=4, q_heads=8, kv_heads=2,
                    attn_dim=64, num_pages=40, max_pages=8)


def _bf(x):
    return x.to(torch.float32).to(torch.bfloat16).double()


class Reference:
    def __init__(self, stack, seed):
        self.s, self.w = stack.shape, [{k: v.double().cpu() for k, v in w.items()} for w in stack.weights]
        self.final = stack.final_norm.double().cpu()
        self.params, self.state, self.kv = [], [], []
        s = self.s
        for li, kind in enumerate(s.pattern):
            lw = synth.Mamba2Workload(f"stack_layer{li}", batch=s.batch, heads=s.heads, head_dim=s.head_dim,
                                      state_dim=s.state_dim, groups=s.groups, k=s.k, dtype="bf16", seed=seed * 1009 + li)
            self.params.append([torch.from_numpy(np.asarray(p, np.float64)) for p in synth.mamba2_params(lw)])
            self.state.append(torch.zeros(s.batch, s.heads, s.head_dim, s.state_dim, dtype=torch.float64))
            self.kv.append([[], []])

    @staticmethod
    def norm(x, w):
        return x / ((x * x).mean(-1, keepdim=True) + 1e-6).sqrt() * w

    def step(self, u):
        s, B = self.s, self.s.batch
        out = None
        for li, kind in enumerate(s.pattern):
            w = self.w[li]
            exact = u if out is None else u + out
            n = _bf(self.norm(exact, w["norm"]))
            u = exact
            if kind == "M":
                A, D = self.params[li]
                x, z, Bt, Ct = (_bf(n @ w[k]) for k in ("x", "z", "B", "C"))
                dt = _bf(torch.log1p(torch.exp(_bf(n @ w["dt"]) + w["dt_bias"])))
                x = x.view(B, s.heads, s.head_dim)
                grp = torch.arange(s.heads) // (s.heads // s.groups)
                Bh, Ch = (t.view(B, s.groups, s.state_dim)[:, grp] for t in (Bt, Ct))
                h = self.state[li]
                h = torch.exp(dt * A)[..., None, None] * h + (dt[..., None] * x)[..., None] * Bh[:, :, None, :]
                self.state[li] = h
                y = _bf((h * Ch[:, :, None, :]).sum(-1) + D[None, :, None] * x).view(B, -1)
                g = (y * z * torch.sigmoid(z)).view(B, s.groups, -1)
                g = (g / ((g * g).mean(-1, keepdim=True) + 1e-6).sqrt()).view(B, -1) * w["gate"]
                out = _bf(_bf(g) @ w["out"])
            else:
                qkv = _bf(n @ w["qkv"]).view(B, -1, s.attn_dim)
                q, k, v = qkv.split([s.q_heads, s.kv_heads, s.kv_heads], dim=1)
                self.kv[li][0].append(k)
                self.kv[li][1].append(v)
                K, V = (torch.stack(c, 1) for c in self.kv[li])          # [B][n][Hk][D]
                qg = q.view(B, s.kv_heads, -1, s.attn_dim)
                p = torch.softmax(torch.einsum("bhgd,bnhd->bhgn", qg, K) / math.sqrt(s.attn_dim), -1)
                out = _bf(_bf(torch.einsum("bhgn,bnhd->bhgd", p, V).reshape(B, -1)) @ w["out"])
        return self.norm(u + out, self.final)


def _inputs(n, seed, T=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = (SHAPE.batch, SHAPE.d_model) if T is None else (SHAPE.batch, T, SHAPE.d_model)
    return [torch.randn(shape, generator=g, device="cuda") for _ in range(n)]


def test_stack_matches_reference(cuda_lib):
    stack = HybridStack(SHAPE, seed=3)
    ref = Reference(stack, 3)
    for u in _inputs(20, 7):                       # crosses a page (16) and several flushes (k = 4)
        got = stack.step(u)
        want = ref.step(u.double().cpu())
        assert vec_err(got.double().cpu().numpy(), want.numpy()) < TOL_LOW
    assert all(e[0] == 0 for e in stack.errors())
    assert stack.pages.lens.tolist() == [20] * SHAPE.batch
    stack.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_draft_rounds_match_single_steps(cuda_lib, kv):
    """Rounds of 3 drafts of which 0 to 3 stay, against a stack that steps through the tokens that stayed."""
    T = 3
    shape = HybridShape(**{**SHAPE.__dict__, "max_draft": T})
    a, b = HybridStack(shape, kv=kv, seed=5), HybridStack(shape, kv=kv, seed=5)
    rounds = _inputs(8, 11, T)
    acc = [3, 0, 2, 1, 3, 3, 0, 2]                 # the same for every request, so that b can follow
    for u, n in zip(rounds, acc):
        drafts = a.step(u)
        a.verify(T, torch.full((shape.batch,), n, dtype=torch.int32, device="cuda"))
        for t in range(n):
            one = b.step(u[:, t].contiguous())
            assert vec_err(drafts[:, t].double().cpu().numpy(), one.double().cpu().numpy()) < TOL_LOW
        assert a.pages.lens.tolist() == b.pages.lens.tolist()
        assert int(a.pages.free_count) == int(b.pages.free_count)
    assert all(e[0] == 0 for s in (a, b) for e in s.errors())
    a.close()
    b.close()


def test_a_refused_round_leaves_no_trace(cuda_lib):
    """A request that finds the pool empty in one round, beside others that do
    not, goes on as one whose drafts of that round were all turned down."""
    T = 3
    tight, wide = (HybridStack(HybridShape(**{**SHAPE.__dict__, "max_draft": T, "num_pages": n}), seed=4) for n in (5, 40))

    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    for i, u in enumerate(_inputs(9, 17, T)):
        if i == 6:                                 # the first request ends: there is room again
            for s in (tight, wide):
                s.pages.truncate(i32(0, 99, 99))
        a, b = tight.step(u), wide.step(u)
        refused = i == 5                           # from 15 to 18 tokens: three pages more, two left
        assert tight.pages.refused.tolist() == [0, 0, int(refused)]
        assert torch.equal(a[:2], b[:2]) and (refused or torch.equal(a[2], b[2]))
        tight.verify(T, i32(3, 3, 3))
        wide.verify(T, i32(3, 3, 0 if refused else 3))
        assert tight.pages.lens.tolist() == wide.pages.lens.tolist()
    assert [e[:2] for e in tight.errors()][0] == (rssm.RSSM_DEV_PAGES_EMPTY, 1)
    tight.close()
    wide.close()


def test_requests_come_and_go(cuda_lib):
    """A request that ends gives its pages back, and a new one in its place does not see its tokens."""
    shape = HybridShape(**{**SHAPE.__dict__, "pattern": "A"})
    stack, fresh = HybridStack(shape, seed=9), HybridStack(shape, seed=9)
    us = _inputs(25, 13)
    for u in us[:18]:
        stack.step(u)
    stack.pages.truncate(torch.tensor([18, 0, 18], dtype=torch.int32, device="cuda"))
    for u in us[18:]:
        got, want = stack.step(u), fresh.step(u)
        assert torch.equal(got[1], want[1])
    assert stack.pages.lens.tolist() == [25, 7, 25]
    assert int(stack.pages.free_count) == shape.num_pages - 5
    stack.close()
    fresh.close()


def test_calls_refuse_a_device_that_is_not_current(cuda_lib, monkeypatch):
    """Every call, with signatures seen before and new ones; nothing is launched."""
    bf16 = torch.bfloat16
    pages = rssm.PageTable(2, 16, 8, 2)
    cache = torch.zeros((8, 2, 16, 64), dtype=bf16, device="cuda")
    attn = rssm.Attention(cache, cache, batch=2, q_heads=2, max_pages=2)
    one, x, w = torch.ones(2, dtype=torch.int32, device="cuda"), torch.ones((2, 2, 64), dtype=bf16, device="cuda"), torch.ones(64, device="cuda")
    row = x[:, 0].contiguous()
    calls = [lambda: pages.extend(one.clone(), T=1), lambda: pages.rollback(1, one), lambda: pages.truncate(one), lambda: pages.get_error(),
             lambda: attn.append(x, x, one), lambda: attn.decode(torch.empty_like(x).view(2, 1, 2, 64), x, one, pages.table),
             lambda: attn.get_error(), lambda: rssm.add_norm(row.clone(), row, w), lambda: rssm.gated_norm(row.clone(), row, row, w),
             lambda: rssm.PageTable(2, 16, 8, 2), lambda: rssm.Attention(cache, cache, batch=2, q_heads=2, max_pages=2)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    before = pages.workspace.clone()
    monkeypatch.setattr(rssm.hybrid, "_current_device", lambda: torch.cuda.current_device() + 1, raising=False)
    for call in calls:
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(before, pages.workspace)


def test_refuses_a_bad_shape(cuda_lib):
    with pytest.raises(ValueError):
        HybridStack(HybridShape(pattern="MX", batch=1))
    with pytest.raises(ValueError):
        HybridStack(HybridShape(pattern="", batch=1))
    with pytest.raises(ValueError):
        HybridStack(SHAPE, kv="fp4")
