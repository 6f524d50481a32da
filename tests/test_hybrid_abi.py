"""The page table, attention and norm entry points without a GPU: structs match
the Python mirror, layouts and sizes, and host-checkable errors come back as
status codes before any CUDA call."""
import ctypes
import os
import subprocess

import pytest

import hybrid_ssm_decode_gb300 as rssm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, CAPACITY = rssm.RSSM_OK, rssm.RSSM_ERR_INVALID_ARG, rssm.RSSM_ERR_UNSUPPORTED, rssm.RSSM_ERR_CAPACITY


@pytest.fixture(scope="module")
def lib():
    rssm.build()
    return rssm.load()


def test_struct_layouts_match_header(tmp_path):
    structs = {"rssm_pages_config": rssm.PagesConfig, "rssm_pages_layout": rssm.PagesLayout,
               "rssm_attn_config": rssm.AttnConfig, "rssm_add_norm_config": rssm.AddNormConfig,
               "rssm_gated_norm_config": rssm.GatedNormConfig}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "rssm.h"', "int main(void){"]
    for s, cls in structs.items():
        lines.append(f'printf("{s} size %zu\\n", sizeof({s}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{s} {f} %zu\\n", offsetof({s}, {f}));')
    consts = ("RSSM_DEV_PAGES_EMPTY RSSM_DEV_PAGES_ROW RSSM_DEV_PAGES_COUNT RSSM_DEV_PAGES_SLOTS RSSM_DEV_ATTN_LEN "
              "RSSM_DEV_ATTN_PAGE RSSM_DEV_ATTN_SLOT RSSM_KV_FP8 RSSM_GATE_SILU RSSM_GATE_SIGMOID").split()
    lines += [f'printf("const {c} %zu\\n", (size_t){c});' for c in consts] + ["return 0;}"]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in out if x}
    for s, cls in structs.items():
        assert got[(s, "size")] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[(s, f)] == getattr(cls, f).offset, (s, f)
    for c in consts:
        assert got[("const", c)] == getattr(rssm, c), c


def test_overlapped_kernels_read_coherently():
    """A kernel that takes its place beside the one in front of it may find data
    that is not written yet in the read-only path: its sources use none."""
    csrc = os.path.join(ROOT, "hybrid_ssm_decode_gb300", "csrc")
    for name in ("norm.cu", "attn.cu", "attn_decode.cuh", "pages.cu", "overlap.cuh"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for word in ("__ldg(", "ld.global.nc", "__restrict__"):
            assert word not in text, f"{name}: {word}"


def test_pages_layout(lib):
    lay = rssm.rssm_pages_layout_for(rssm.PagesConfig(100, 16, 5000, 70))
    assert lay.lens == 0 and lay.table >= 400 and lay.free >= lay.table + 4 * 7000
    assert lay.free_count >= lay.free + 4 * 5000 and lay.err > lay.free_count and lay.total_bytes >= lay.err + 16
    assert all(getattr(lay, f) % 256 == 0 for f in ("lens", "table", "free", "free_count", "err", "total_bytes"))


@pytest.mark.parametrize("cfg", [(0, 16, 5, 5), (1, 0, 5, 5), (1, 16, 0, 5), (1, 16, 5, 0), (1, 16, 2 ** 27, 1),
                                 (2 ** 16, 1, 5, 2 ** 15), (1, 2 ** 20, 5, 2 ** 11)])
def test_pages_refusals(lib, cfg):
    lay = rssm.PagesLayout()
    assert lib.rssm_pages_layout_for(ctypes.byref(rssm.PagesConfig(*cfg)), ctypes.byref(lay)) == INVALID


def test_pages_host_errors(lib):
    cfg, h = rssm.PagesConfig(4, 16, 8, 2), ctypes.c_void_p(0)
    need = rssm.rssm_pages_layout_for(cfg).total_bytes
    c = ctypes.byref(cfg)
    assert lib.rssm_pages_create(c, None, need, None, None, ctypes.byref(h)) == INVALID
    assert lib.rssm_pages_create(c, 4096 + 64, need, None, None, ctypes.byref(h)) == INVALID
    assert lib.rssm_pages_create(c, 4096, need, 4098, None, ctypes.byref(h)) == INVALID
    assert lib.rssm_pages_create(c, 4096, need - 1, None, None, ctypes.byref(h)) == CAPACITY
    assert lib.rssm_pages_create(c, 4096, need, None, None, None) == INVALID
    assert lib.rssm_pages_extend(None, 1, None, 4096, None, 4, None) == INVALID
    assert lib.rssm_pages_rollback(None, 1, 4096, None) == INVALID
    assert lib.rssm_pages_truncate(None, 4096, None) == INVALID
    assert lib.rssm_pages_get_error(None, (ctypes.c_int32 * 4)(), None) == INVALID
    assert lib.rssm_pages_destroy(None) == INVALID
    assert h.value is None


def _attn(**kw):
    a = dict(batch=4, q_heads=8, kv_heads=2, head_dim=128, page_size=16, num_pages=100, max_pages=10, max_draft=1,
             in_dtype=rssm.RSSM_BF16, kv_dtype=rssm.RSSM_BF16, window=0, scale=0.0, page_stride=0)
    a.update(kw)
    return rssm.AttnConfig(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(kv_dtype=rssm.RSSM_KV_FP8), OK), (dict(in_dtype=rssm.RSSM_F32, kv_dtype=rssm.RSSM_F32), OK),
    (dict(head_dim=64), OK), (dict(head_dim=256, max_draft=8), OK), (dict(page_size=48), OK), (dict(scale=-2.0), OK),
    (dict(page_stride=2 * 2 * 16 * 128), OK), (dict(q_heads=7), INVALID), (dict(batch=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(window=-1), INVALID), (dict(max_draft=0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(in_dtype=rssm.RSSM_F16), INVALID), (dict(kv_dtype=9), INVALID),
    (dict(page_stride=100), INVALID), (dict(page_stride=2 * 16 * 128 + 4), INVALID), (dict(num_pages=2 ** 27), INVALID),
    (dict(max_pages=2 ** 27), INVALID), (dict(batch=2 ** 20, max_pages=2 ** 11), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(max_draft=9), UNSUPPORTED),
    (dict(in_dtype=rssm.RSSM_F32), UNSUPPORTED), (dict(kv_dtype=rssm.RSSM_F32), UNSUPPORTED)])
def test_attention_config(lib, kw, status):
    n = ctypes.c_size_t(0)
    assert lib.rssm_attn_workspace_size(ctypes.byref(_attn(**kw)), ctypes.byref(n)) == status
    assert (n.value > 0) == (status == OK)


def test_attention_workspaces_are_laid_out_alike(lib):
    """What a call must leave at zero lies at the same place for every layer, so
    that layers can share a workspace: no region before the parts, whose size
    goes by the rows that a block takes, grows with the batch, heads or drafts."""
    def size(**kw):
        return rssm.rssm_attn_workspace_size(_attn(**kw))

    for shapes in ((dict(), dict(batch=4096), dict(q_heads=64, kv_heads=64), dict(q_heads=16, kv_heads=1), dict(max_draft=4)),
                   (dict(q_heads=32, kv_heads=1, max_draft=8), dict(batch=500, q_heads=64, kv_heads=1))):
        assert len({size(**kw) for kw in shapes}) == 1, shapes


def test_attention_host_errors(lib):
    cfg, h = _attn(), ctypes.c_void_p(0)
    need = rssm.rssm_attn_workspace_size(cfg)
    c, out = ctypes.byref(cfg), ctypes.byref(h)
    create = lib.rssm_attn_create
    assert create(c, None, 4096, None, None, 4096, need, None, out) == INVALID
    assert create(c, 4104, 4096, None, None, 4096, need, None, out) == INVALID
    assert create(c, 4096, 4096, None, None, None, need, None, out) == INVALID
    assert create(c, 4096, 4096, None, None, 4096 + 16, need, None, out) == INVALID
    assert create(c, 4096, 4096, 4096, 4096, 4096, need, None, out) == INVALID          # scales without FP8
    assert create(ctypes.byref(_attn(kv_dtype=rssm.RSSM_KV_FP8)), 4096, 4096, 4096, None, 4096, need, None, out) == INVALID
    assert create(c, 4096, 4096, None, None, 4096, need - 1, None, out) == CAPACITY
    assert create(c, 4096, 4096, None, None, 4096, need, None, None) == INVALID
    assert lib.rssm_attn_append(None, 1, 4096, 0, 4096, 0, 4096, None) == INVALID
    assert lib.rssm_attn_decode(None, 1, 4096, 0, 4096, 4096, 4096, None, None) == INVALID
    assert lib.rssm_attn_get_error(None, (ctypes.c_int32 * 4)(), None) == INVALID
    assert lib.rssm_attn_destroy(None) == INVALID
    assert h.value is None


def _add(**kw):
    a = dict(rows=4, dim=64, res_dtype=rssm.RSSM_F32, dtype=rssm.RSSM_BF16, eps=1e-6, scale=1.0, w_offset=0.0)
    a.update(kw)
    return rssm.AddNormConfig(**a)


def test_norm_host_errors(lib):
    def add(cfg, u=4096, x=4096, wp=None, g=None, w=4096, uo=4096, no=4096):
        return lib.rssm_add_norm(ctypes.byref(cfg), u, x, wp, g, w, uo, no, None)

    assert lib.rssm_add_norm(None, 4096, 4096, None, None, 4096, 4096, 4096, None) == INVALID
    for kw in (dict(rows=-1), dict(dim=0), dict(res_dtype=rssm.RSSM_F16), dict(dtype=7), dict(eps=-1.0), dict(eps=float("nan")),
               dict(u_stride=63), dict(x_stride=1), dict(gate_stride=5), dict(u_out_stride=-64), dict(n_out_stride=2)):
        assert add(_add(**kw)) == INVALID, kw
    assert add(_add(dim=32769)) == UNSUPPORTED
    assert add(_add(), u=None) == INVALID and add(_add(), uo=None, no=None) == INVALID and add(_add(), w=None) == INVALID
    assert add(_add(), x=None, g=4096) == INVALID and add(_add(), x=None, wp=4096) == INVALID
    assert add(_add(rows=0), u=None, x=None, w=None, uo=None, no=None) == OK

    def gated(y=4096, z=4096, w=4096, o=4096, **kw):
        a = dict(rows=4, dim=64, group=32, w_dim=32, dtype=rssm.RSSM_BF16, norm_first=1, act=1, eps=1e-6, w_offset=0.0)
        a.update(kw)
        return lib.rssm_gated_norm(ctypes.byref(rssm.GatedNormConfig(**a)), y, z, w, o, None)

    for kw in (dict(rows=-1), dict(dim=0), dict(group=0), dict(group=48), dict(w_dim=16), dict(dtype=0), dict(norm_first=2),
               dict(act=0), dict(eps=-1.0), dict(y_stride=3), dict(z_stride=3), dict(out_stride=3), dict(rows=2 ** 31)):
        assert gated(**kw) == INVALID, kw
    assert gated(dim=65536, group=65536, w_dim=65536) == UNSUPPORTED
    for k in ("y", "z", "w", "o"):
        assert gated(**{k: None}) == INVALID
    assert gated(rows=0, y=None, z=None, w=None, o=None) == OK


def _any_device(monkeypatch):
    """Lets CPU tensors past the device check: what comes next is tested."""
    monkeypatch.setattr(rssm.hybrid, "_cuda", lambda device, name: None)


def test_binding_refuses_pages_that_overlap(lib, monkeypatch):
    """A cache expanded over its pages has stride 0, which the library takes for
    a dense cache of that many pages; so do pages closer than their size."""
    import torch
    _any_device(monkeypatch)
    one = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    close = torch.zeros(20000, dtype=torch.bfloat16).as_strided((4, 2, 16, 64), (1024, 1024, 64, 1))
    dense = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for k, v in ((one.expand(4, 2, 16, 64),) * 2, (close, close), (dense, one.expand(4, 2, 16, 64))):
        with pytest.raises(ValueError):
            rssm.Attention(k, v, batch=1, q_heads=2, max_pages=2)


def test_binding_refuses_a_workspace_that_is_not_dense(lib, monkeypatch):
    """Its size is taken for the bytes behind its address."""
    import torch
    _any_device(monkeypatch)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    need = rssm.rssm_attn_workspace_size(_attn(batch=1, q_heads=2, head_dim=64, num_pages=4, max_pages=2))
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            rssm.Attention(cache, cache, batch=1, q_heads=2, max_pages=2, workspace=ws)


def test_binding_refuses_a_device_that_is_not_current(monkeypatch):
    """A launch goes to the current device, whatever the tensors' own: the check
    that every call makes as it takes its stream."""
    monkeypatch.setattr(rssm.hybrid, "_current_device", lambda: 1, raising=False)
    for stream in (None, 64):
        with pytest.raises(ValueError):
            rssm.hybrid._stream_of(stream, 0)
    assert rssm.hybrid._stream_of(64, 1) == 64


def test_binding_refuses_cpu_tensors(lib):
    """The checks come before any call of the library."""
    import torch
    x, w = torch.zeros(2, 64), torch.ones(64)
    with pytest.raises(ValueError):
        rssm.add_norm(x, x, w)
    with pytest.raises(ValueError):
        rssm.gated_norm(x, x, x, w)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rssm.Attention(cache, cache, batch=1, q_heads=2, max_pages=2)
    with pytest.raises(ValueError):
        rssm.PageTable(2, 16, 8, 2, device="cpu")
