"""The attention side by the C names (rssm_pages_*, rssm_attn_*, rssm_add_norm,
rssm_gated_norm) on handles and buffers of the caller's own, beside the classes
and functions on tensors: the same bits."""
import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32


def _randn(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def test_page_table_and_attention_by_the_c_names(cuda_lib):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    batch, ps, num, most, T = 3, 16, 12, 4, 2
    pages = rssm.PageTable(batch, ps, num, most)
    kc, vc = _randn(g, num, 2, ps, 64), _randn(g, num, 2, ps, 64)
    attn = rssm.Attention(kc, vc, batch=batch, q_heads=4, max_pages=most, max_draft=T)

    cfg = rssm.PagesConfig(batch, ps, num, most)
    lay = rssm.rssm_pages_layout_for(cfg)
    ws = torch.empty(lay.total_bytes, dtype=torch.uint8, device="cuda")
    ph = rssm.rssm_pages_create(cfg, ws, lay.total_bytes)
    lens, table = ws[lay.lens:lay.lens + 4 * batch].view(I32), ws[lay.table:lay.table + 4 * batch * most].view(I32)
    kc2, vc2 = kc.clone(), vc.clone()
    acfg = rssm.AttnConfig(batch=batch, q_heads=4, kv_heads=2, head_dim=64, page_size=ps, num_pages=num, max_pages=most,
                           max_draft=T, in_dtype=rssm.RSSM_BF16, kv_dtype=rssm.RSSM_BF16)
    size = rssm.rssm_attn_workspace_size(acfg)
    aws = torch.empty(size, dtype=torch.uint8, device="cuda")
    ah = rssm.rssm_attn_create(acfg, kc2, vc2, None, None, aws, size)

    new = torch.tensor([20, 1, 33], dtype=I32, device="cuda")
    accepted = torch.tensor([0, 2, 1], dtype=I32, device="cuda")
    slots, slots2, pos, pos2 = (torch.full((54,), -7, dtype=I32, device="cuda") for _ in range(4))
    pages.extend(slots, new=new, positions=pos)
    rssm.rssm_pages_extend(ph, 0, new, slots2, pos2, 54)
    assert torch.equal(slots, slots2) and torch.equal(pos, pos2)
    pages.extend(slots[:6], T=T)
    rssm.rssm_pages_extend(ph, T, None, slots2, None, 6)
    assert torch.equal(slots, slots2)
    k, v, q = _randn(g, 6, 2, 64), _randn(g, 6, 2, 64), _randn(g, batch, T, 4, 64)
    out, out2, lse, lse2 = torch.empty_like(q), torch.zeros_like(q), torch.empty(batch, T, 4, device="cuda"), torch.zeros(batch, T, 4, device="cuda")
    attn.append(k, v, slots[:6])
    rssm.rssm_attn_append(ah, 6, k, 0, v, 0, slots2)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    attn.decode(out, q, pages.lens, pages.table, T=T, lse=lse)
    rssm.rssm_attn_decode(ah, T, q, 0, lens, table, out2, lse2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    pages.rollback(T, accepted)
    rssm.rssm_pages_rollback(ph, T, accepted)
    pages.truncate(new)
    rssm.rssm_pages_truncate(ph, new)
    assert torch.equal(lens, pages.lens) and torch.equal(table, pages.table.view(-1))
    assert rssm.rssm_pages_get_error(ph) == rssm.rssm_attn_get_error(ah) == (0, 0, 0, 0)
    rssm.rssm_pages_destroy(ph)
    rssm.rssm_attn_destroy(ah)


def test_norms_by_the_c_names(cuda_lib):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    u, x, z, w = _randn(g, 5, 96, dtype=torch.float32), _randn(g, 5, 96), _randn(g, 5, 96), _randn(g, 96, dtype=torch.float32)
    n, n2, s, s2 = torch.empty_like(x), torch.zeros_like(x), torch.empty_like(u), torch.zeros_like(u)
    rssm.add_norm(n, u, w, x=x, u_out=s, w_post=w, gate=z, scale=0.5, w_offset=1.0)
    cfg = rssm.AddNormConfig(rows=5, dim=96, res_dtype=rssm.RSSM_F32, dtype=rssm.RSSM_BF16, eps=1e-6, scale=0.5, w_offset=1.0, gate_stride=96)
    rssm.rssm_add_norm(cfg, u, x, w, z, w, s2, n2)
    assert torch.equal(n, n2) and torch.equal(s, s2)
    rssm.gated_norm(n, x, z, w, group=32, act="sigmoid")
    cfg = rssm.GatedNormConfig(rows=5, dim=96, group=32, w_dim=96, dtype=rssm.RSSM_BF16, act=rssm.RSSM_GATE_SIGMOID, eps=1e-6)
    rssm.rssm_gated_norm(cfg, x, z, w, n2)
    assert torch.equal(n, n2)
