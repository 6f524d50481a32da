"""Rotary positions and the 4-bit cache without a GPU: structs match the Python
mirror, the frequencies are those of their formulas, and host-checkable errors come
back as status codes or ValueErrors before any CUDA call."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, CAPACITY = rssm.RSSM_OK, rssm.RSSM_ERR_INVALID_ARG, rssm.RSSM_ERR_UNSUPPORTED, rssm.RSSM_ERR_CAPACITY


@pytest.fixture(scope="module")
def lib():
    rssm.build()
    return rssm.load()


def test_struct_layouts_match_header(tmp_path):
    structs = {"rssm_attn_rotary": rssm.AttnRotary, "rssm_rope_config": rssm.RopeConfig, "rssm_rotary_config": rssm.RotaryConfig}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "rssm.h"', "int main(void){"]
    for s, cls in structs.items():
        lines.append(f'printf("{s} size %zu\\n", sizeof({s}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{s} {f} %zu\\n", offsetof({s}, {f}));')
    consts = "RSSM_KV_NVFP4 RSSM_ROPE_PLAIN RSSM_ROPE_LINEAR RSSM_ROPE_NTK RSSM_ROPE_YARN RSSM_ROPE_WAVELENGTH".split()
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
    csrc = os.path.join(ROOT, "hybrid_ssm_decode_gb300", "csrc")
    for name in ("place.cu", "attn_nvfp4.cuh", "attn_nvfp4.cu"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for word in ("__ldg(", "ld.global.nc", "__restrict__"):
            assert word not in text, f"{name}: {word}"


def _freq(R, scaling, base, f, original, fast=0.0, slow=0.0):
    """The formulas of the header, pair by pair."""
    if scaling == "ntk":
        base *= f ** (R / (R - 2))
    fast, slow = fast or (32.0 if scaling == "yarn" else 4.0), slow or 1.0
    if scaling == "yarn":
        ch = [R * math.log(original / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow)]
        lo, hi = max(math.floor(ch[0]), 0), min(math.ceil(ch[1]), R - 1)
    out = []
    for i in range(R // 2):
        w = base ** (-2 * i / R)
        r = 0.0
        if scaling == "linear":
            r = 1.0
        if scaling == "yarn":
            r = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
        if scaling == "wavelength":
            r = 1 - min(max((original * w / (2 * math.pi) - slow) / (fast - slow), 0), 1)
        out.append(r * w / f + (1 - r) * w)
    return out


@pytest.mark.parametrize("scaling", sorted(rssm.ROPE))
@pytest.mark.parametrize("R,base,f,original", [(128, 10000.0, 4.0, 4096), (64, 500000.0, 8.0, 8192), (24, 10000.0, 32.0, 2048),
                                               (4, 100.0, 2.0, 16), (1024, 1e6, 16.0, 32768)])
def test_frequencies(lib, scaling, R, base, f, original):
    got, gain = rssm.rssm_rope_frequencies(rssm.RopeConfig(R, rssm.ROPE[scaling], base, f, original, 0, 0, 0))
    want = _freq(R, scaling, base, f, original)
    assert all(abs(g / w - 1) < 1e-13 for g, w in zip(got, want)) and len(got) == len(want)
    assert abs(gain - (0.1 * math.log(f) + 1 if scaling == "yarn" else 1)) < 1e-6
    got, gain = rssm.rssm_rope_frequencies(rssm.RopeConfig(R, rssm.ROPE[scaling], base, f, original, 16.0, 2.0, 0.5))
    want = _freq(R, scaling, base, f, original, 16.0, 2.0)
    assert all(abs(g / w - 1) < 1e-13 for g, w in zip(got, want)) and gain == 0.5


def test_turns(lib):
    """To the last of 64 bits but three, for frequencies of either sign and of many turns."""
    # 1 / 2 pi to 80 digits
    inv = Fraction(15915494309189533576888376337251436203445964574045644874766734405889679763422653, 10 ** 80)
    freq = [1.0, -1.0, 0.1, 1e-3, 7.5e-12, -7.5e-12, 2.0 ** -60, 0.0, 3.0, 2 * math.pi, 12345.678, -1e9 / 3, 1 / 3]
    for w, t in zip(freq, rssm.rssm_rope_turns(freq)):
        want = Fraction(w) * inv * 2 ** 64
        off = (Fraction(t) - want) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        # below 2^-61 turns, or the 2^-106 of the turns that a product of doubles and its remainder keep
        assert off <= max(8, abs(want) / 2 ** 104), (w, float(off))


@pytest.mark.parametrize("bad", [dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=1026), dict(rotary_dim=-2), dict(scaling=5), dict(scaling=-1),
                                 dict(base=1.0), dict(base=math.inf), dict(base=math.nan), dict(factor=0.0), dict(factor=math.nan),
                                 dict(original=0.0), dict(original=math.inf), dict(fast=1.0, slow=1.0), dict(fast=math.inf), dict(slow=-1.0),
                                 dict(gain=math.inf), dict(gain=math.nan), dict(scaling=rssm.RSSM_ROPE_NTK, rotary_dim=2)])
def test_frequency_refusals(lib, bad):
    a = dict(rotary_dim=64, scaling=rssm.RSSM_ROPE_YARN, base=10000.0, factor=4.0, original=4096.0, fast=0.0, slow=0.0, gain=0.0)
    freq, gain = (ctypes.c_double * 512)(), ctypes.c_float(0)
    assert lib.rssm_rope_frequencies(ctypes.byref(rssm.RopeConfig(**a)), freq, ctypes.byref(gain)) == OK
    assert lib.rssm_rope_frequencies(ctypes.byref(rssm.RopeConfig(**{**a, **bad})), freq, ctypes.byref(gain)) == INVALID
    c = ctypes.byref(rssm.RopeConfig(**a))
    assert lib.rssm_rope_frequencies(None, freq, ctypes.byref(gain)) == INVALID
    assert lib.rssm_rope_frequencies(c, None, ctypes.byref(gain)) == INVALID
    assert lib.rssm_rope_frequencies(c, freq, None) == INVALID


def test_turns_refusals(lib):
    f, t = (ctypes.c_double * 2)(1.0, math.inf), (ctypes.c_uint64 * 2)()
    assert lib.rssm_rope_turns(2, f, t) == INVALID and lib.rssm_rope_turns(1, f, t) == OK
    assert lib.rssm_rope_turns(0, f, t) == INVALID and lib.rssm_rope_turns(1, None, t) == INVALID and lib.rssm_rope_turns(1, f, None) == INVALID


@pytest.mark.parametrize("bad,status", [
    (dict(tokens=-1), INVALID), (dict(tokens=2 ** 31), INVALID), (dict(heads=0), INVALID), (dict(dim=0), INVALID), (dict(dtype=9), INVALID),
    (dict(rotary_dim=0), INVALID), (dict(rotary_dim=33), INVALID), (dict(rotary_dim=66), INVALID), (dict(interleaved=2), INVALID),
    (dict(gain=math.nan), INVALID), (dict(x_stride=255), INVALID), (dict(out_stride=255), INVALID), (dict(heads=2 ** 19), INVALID),
    (dict(dim=2048, rotary_dim=1026), UNSUPPORTED), (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(positions=0), INVALID), (dict(turns=0), INVALID),
    (dict(x=4097), INVALID), (dict(out=4097), INVALID), (dict(positions=4098), INVALID), (dict(turns=4100), INVALID),
    (dict(out=4096, out_stride=512), INVALID)])
def test_rotary_host_errors(lib, bad, status):
    ptr = dict(x=4096, out=8192, positions=16384, turns=32768)
    a = dict(tokens=3, heads=4, dim=64, rotary_dim=64, interleaved=0, dtype=rssm.RSSM_BF16, gain=1.0, x_stride=0, out_stride=0)
    for k, v in bad.items():
        (ptr if k in ptr else a)[k] = v
    assert lib.rssm_rotary(ctypes.byref(rssm.RotaryConfig(**a)), ptr["x"], ptr["positions"], ptr["turns"], ptr["out"], None) == status
    if status == INVALID and not set(bad) & set(ptr) and "tokens" not in bad:
        a["tokens"] = 0                                        # sizes are looked at all the same
        assert lib.rssm_rotary(ctypes.byref(rssm.RotaryConfig(**a)), None, None, None, None, None) == INVALID
    assert lib.rssm_rotary(None, 4096, 16384, 32768, 8192, None) == INVALID


def test_no_tokens(lib):
    c = rssm.RotaryConfig(tokens=0, heads=4, dim=64, rotary_dim=64, dtype=rssm.RSSM_F32, gain=1.0)
    assert lib.rssm_rotary(ctypes.byref(c), None, None, None, None, None) == OK


def test_cache4_configurations(lib):
    """A page stride counts bytes, and needs room for 9/16 of the elements."""
    n = ctypes.c_size_t(0)

    def size(**kw):
        a = dict(batch=2, q_heads=8, kv_heads=2, head_dim=128, page_size=16, num_pages=4, max_pages=4, max_draft=1,
                 in_dtype=rssm.RSSM_BF16, kv_dtype=rssm.RSSM_KV_NVFP4, window=0, scale=0.0, page_stride=0)
        a.update(kw)
        return lib.rssm_attn_workspace_size(ctypes.byref(rssm.AttnConfig(**a)), ctypes.byref(n))

    page = 2 * 16 * 72
    assert size() == OK and size(page_stride=page) == OK and size(page_stride=2 * page) == OK
    assert size(page_stride=page - 16) == INVALID and size(page_stride=page + 8) == INVALID
    assert size(in_dtype=rssm.RSSM_F32) == UNSUPPORTED and size(head_dim=96) == UNSUPPORTED and size(page_size=24) == UNSUPPORTED
    assert size(kv_dtype=6) == INVALID


def test_python_refusals(lib):
    for kw, what in ((dict(rotary_dim=63), "rotary_dim"), (dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=2000), "rotary_dim"),
                     (dict(rotary_dim=64, scaling="other"), "scaling"), (dict(rotary_dim=64, gain=math.inf), "gain"),
                     (dict(rotary_dim=64, inv_freq=[1.0] * 31), "inv_freq"),
                     (dict(rotary_dim=64, inv_freq=[1.0] * 32, scaling="ntk", factor=2.0), "inv_freq"),
                     (dict(rotary_dim=64, device="cpu"), "device")):
        with pytest.raises(ValueError, match=what):
            rssm.Rope(**kw)
    for kw in (dict(scaling="yarn", factor=4.0), dict(scaling="linear", factor=0.0), dict(base=0.5), dict(inv_freq=[math.nan] * 32)):
        with pytest.raises(rssm.RssmError):
            rssm.Rope(64, **kw)
    x = torch.zeros((2, 3, 64))
    with pytest.raises(ValueError, match="x: on cpu"):
        rssm.rotary(x, x, torch.zeros(2, dtype=torch.int32), type("R", (), dict(rotary_dim=64, interleaved=False, gain=1.0, turns=x, signature=()))())
    cache = torch.zeros((2, 1, 16, 72), dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_cache: on cpu"):
        rssm.Attention(cache, cache, batch=1, q_heads=1, max_pages=1)
    with pytest.raises(ValueError, match="rows of 70 bytes"):
        rssm.Attention(cache[..., :70], cache[..., :70], batch=1, q_heads=1, max_pages=1)
