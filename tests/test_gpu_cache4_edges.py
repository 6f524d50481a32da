"""4-bit caches at the ends of what their scales may be."""
import pytest
import torch

from test_gpu_cache4 import caches, layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1e-45, 1e-40, 4e-40, 1e-38, 1e30])
def test_zeros_stay_zeros_under_every_scale(cuda_lib, scale):
    """Below 2^-128 / 6 the reciprocal of 6 scale is infinite: a block of zeros beside one that is not stays zero all the same,
    and one that is not is held at the largest value, 6 448 scale, with its sign."""
    s = torch.tensor([scale])
    a = layer(*caches(1, 1, 16, 64, "nvfp4"), "nvfp4", s, s, 1)
    x = torch.zeros((16, 1, 64))
    x[3, 0, 16:32] = 1.0
    x[4, 0, 32:48] = -1.0
    x = x.bfloat16().cuda()
    slots = torch.arange(16, dtype=torch.int32, device="cuda")
    a.append(x, x, slots)
    k, v = torch.empty_like(x), torch.empty_like(x)
    a.read(k, v, slots)
    want = (x.double().cpu() * (6 * 448 * s.double()) if scale < 1 else torch.zeros(x.shape)).bfloat16()
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
