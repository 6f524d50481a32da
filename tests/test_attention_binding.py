"""The attention binding's calls on the host: what they pass on, and what they refuse."""
import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm

BF16 = torch.bfloat16


class Calls:
    """In the place of the library: keeps the arguments of the last call."""

    def __getattr__(self, name):
        def call(*args):
            self.last = (name, args)
            return 0
        return call


def attention(monkeypatch):
    """A layer of 2 cache heads of 64 and 4 query heads, on CPU tensors and without a handle."""
    monkeypatch.setattr(rssm.hybrid, "_stream_of", lambda stream, device: stream)
    a = object.__new__(rssm.Attention)
    a.handle, a.device, a.dtype, a._seen, a._fn = 0, torch.device("cpu"), BF16, {}, Calls()
    a.cfg = rssm.AttnConfig(batch=1, q_heads=4, kv_heads=2, head_dim=64)
    return a


def test_append_takes_the_stream_behind_the_slots(monkeypatch):
    """Its fourth argument is the stream, with or without a name; what goes with rope has to be named."""
    a = attention(monkeypatch)
    x, slots = torch.zeros((3, 2, 64), dtype=BF16), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: a.append(x, x, slots, 64), lambda: a.append(x, x, slots, stream=64)):
        call()
        name, args = a._fn.last
        assert name == "rssm_attn_append" and args[-1] == 64
    with pytest.raises(TypeError):
        a.append(x, x, slots, None, slots)


@pytest.fixture(scope="module")
def lib():
    rssm.build()
    return rssm.load()


def test_a_rope_stays_as_it_is_made(lib, monkeypatch):
    """Calls keep what they concluded about a Rope by its signature: a later gain would reach new shapes alone."""
    monkeypatch.setattr(rssm.hybrid, "_cuda", lambda device, name: None)
    rope = rssm.Rope(64, base=500.0, gain=1.5, device="cpu")
    freq = list(rope.frequencies)
    for name, value in (("gain", 0.5), ("interleaved", True), ("rotary_dim", 32), ("frequencies", freq[:1]),
                        ("turns", rope.turns.clone()), ("signature", ())):
        with pytest.raises(AttributeError, match="stays as it is made"):
            setattr(rope, name, value)
        with pytest.raises(AttributeError, match="stays as it is made"):
            delattr(rope, name)
    with pytest.raises(TypeError):
        rope.frequencies[0] = 0.0
    assert (rope.gain, rope.interleaved, rope.rotary_dim, list(rope.frequencies)) == (1.5, False, 64, freq)
    assert rope.signature[:3] == (64, False, 1.5)


@pytest.mark.parametrize("rot,device,what", [(128, "cpu", "rope: 128 rotated channels"), (64, "meta", "rope: on cpu")])
def test_a_stack_refuses_a_rope_that_its_layers_would(lib, monkeypatch, rot, device, what):
    """Before its first step: there the page table and the layers in front have already moved on."""
    from hybrid_ssm_decode_gb300.stack import HybridShape, HybridStack
    monkeypatch.setattr(rssm.hybrid, "_cuda", lambda device, name: None)
    rope = rssm.Rope(rot, device="cpu")
    with pytest.raises(ValueError, match=what):
        HybridStack(HybridShape("MA", 1, q_heads=2, kv_heads=1, attn_dim=64), device=device, rope=rope)
