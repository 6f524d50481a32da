"""Rotary positions, the cache's writer and its reader at the sizes of prompts, where a block takes
several tokens: 2 from 16 tokens a multiprocessor on, 4 from 32, 8 from 64 and 16 from 128. Bit by bit
against the same tokens in calls of at most 1000, where a block takes one, which the other tests hold against
the definitions."""
import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm
from test_gpu_cache4 import caches, layer, scales

pytestmark = pytest.mark.gpu

CHUNK = 1000


def tokens(per_sm, beyond):
    return per_sm * torch.cuda.get_device_properties(0).multi_processor_count + beyond


def chunks(n):
    assert CHUNK < tokens(16, 0)
    return [slice(i, i + CHUNK) for i in range(0, n, CHUNK)]


def bits(t):
    return t.view(torch.uint8)


# vectors of 8 and 4; 32 threads a head, so that a block of 8 has no group for every token of a tile of 16;
# half a head of 27 pairs, one at a time; heads of more pairs than a block has threads (tiles of 8 at most)
SHAPES = [(2, 64, 64, False, torch.bfloat16), (1, 256, 256, False, torch.float32), (3, 128, 54, True, torch.float32),
          (2, 80, 80, False, torch.bfloat16), (1, 1024, 1022, False, torch.float32)]


@pytest.mark.parametrize("heads,dim,rot,inter,dtype", SHAPES)
@pytest.mark.parametrize("per_sm,beyond", [(16, -1), (16, 1), (32, 3), (64, -1), (64, 0), (64, 1), (128, -1), (128, 0), (128, 1), (128, 15)])
def test_rotary(cuda_lib, per_sm, beyond, heads, dim, rot, inter, dtype):
    n = tokens(per_sm, beyond)
    g = torch.Generator(device="cuda")
    g.manual_seed(n + dim)
    x = torch.randn((n, heads + 1, dim), generator=g, device="cuda").to(dtype)[:, :heads]
    pos = torch.randint(-1000, 1 << 30, (n,), generator=g, device="cuda", dtype=torch.int32)
    rope = rssm.Rope(rot, interleaved=inter, gain=1.1)
    room = torch.full((n + 1, heads, dim), 7.0, dtype=dtype, device="cuda")
    out, want = room[:n], torch.empty((n, heads, dim), dtype=dtype, device="cuda")
    rssm.rotary(out, x, pos, rope)
    for s in chunks(n):
        rssm.rotary(want[s], x[s], pos[s], rope)
    assert torch.equal(bits(out), bits(want)) and bool((room[n] == 7.0).all())
    beside = x.clone()
    rssm.rotary(x, x, pos, rope)                                # in place: what is beside stays where it is
    assert torch.equal(x, want) and torch.equal(x[..., rot:], beside[..., rot:])


@pytest.mark.parametrize("kv", ["nvfp4", "fp8", "bf16", "f32"])
@pytest.mark.parametrize("dim,rot,inter", [(64, 64, False), (128, 54, True), (256, 64, False)])
@pytest.mark.parametrize("per_sm,beyond", [(32, 1), (64, -1), (64, 1), (128, 0), (128, 15)])
def test_append_and_read(cuda_lib, per_sm, beyond, dim, rot, inter, kv):
    n, heads, q_heads, ps = tokens(per_sm, beyond), 2, 4, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(n + dim)
    num = n // ps + 2
    ks, vs = scales(heads)
    made, at_once = (caches(num, heads, ps, dim, kv) for _ in range(2))
    one, many = (layer(*c, kv, ks, vs, q_heads) for c in (at_once, made))
    qkv = torch.randn((n, q_heads + 2 * heads, dim), generator=g, device="cuda").to(one.dtype)
    q, k, v = qkv.split([q_heads, heads, heads], 1)
    slots = torch.randperm(num * ps, generator=g, device="cuda")[:n].to(torch.int32)
    slots[7::11] = -1
    pos = torch.randint(0, 100000, (n,), generator=g, device="cuda", dtype=torch.int32)
    rope = rssm.Rope(rot, interleaved=inter)
    qo = torch.full((2, n, q_heads, dim), 7.0, dtype=one.dtype, device="cuda")
    for kw in (dict(rope=rope), {}):
        def call(a, s, to):
            more = dict(kw, positions=pos[s], q=q[s], q_out=to[s]) if kw else {}
            a.append(k[s], v[s], slots[s], **more)
        call(one, slice(None), qo[0])
        for s in chunks(n):
            call(many, s, qo[1])
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(at_once, made))
        assert torch.equal(qo[0], qo[1])
    got, want = (torch.full((2, n, heads, dim), 7.0, dtype=one.dtype, device="cuda") for _ in range(2))
    one.read(got[0], got[1], slots)
    for s in chunks(n):
        many.read(want[0, s], want[1, s], slots[s])
    assert torch.equal(bits(got), bits(want)) and bool((got[:, 7::11] == 7.0).all())
    assert one.get_error() == (0, 0, 0, 0) and many.get_error() == (0, 0, 0, 0)
