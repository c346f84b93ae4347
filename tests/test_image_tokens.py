"""The example that runs the token-row operators together, against the same
network in binary32 on unquantised rows."""
import importlib.util
import os

import pytest
import torch

import image_preprocessing_gb300 as trfn
from image_preprocessing_gb300 import synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("image_tokens", os.path.join(ROOT, "examples", "image_tokens.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
@pytest.mark.parametrize("images,width", [(1, 128), (6, 320)])
def test_example_follows_the_network_in_binary32(images, width):
    """Every 8-bit value is within 1/254 of its row's largest, about 1.1 %
    of a near-normal row's rms; weights and rows give 1.6 % in each of three
    products, which add to 2.8 %, and bfloat16 rounding is small beside it."""
    e = _example()
    mean, std, _ = trfn.tr_norm_preset("IMAGENET")
    src = torch.from_numpy(synth.pixels_uniform(3, images, 224, 224, 3)).cuda()
    net = e.build(width, seed=4)
    rows = e.patches(src, mean, std, None)
    assert rows.shape == (images * 196, 768)
    positions = 0.02 * torch.randn((rows.size(0), width), device="cuda", dtype=torch.bfloat16)
    y, h = e.forward(net, rows, positions)

    g = torch.Generator(device="cuda").manual_seed(4)
    w = [torch.randn((n, k), generator=g, device="cuda") / k ** 0.5 for n, k in ((width, 768), (2 * width, width), (width, 2 * width))]

    def norm(v):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)

    h1 = rows.float() @ w[0].t() + positions.float()
    x = torch.nn.functional.gelu(norm(h1) @ w[1].t()) @ w[2].t()
    want = norm(x + h1)
    assert float((y.float() - want).norm() / want.norm()) < 0.04
    dx, dweight = e.norm_gradients(torch.ones_like(y), h, net["norm2"])
    hd = h.double()
    s = torch.rsqrt(hd.square().mean(1, keepdim=True) + 1e-6)
    assert torch.allclose(dweight.double(), (hd * s).sum(0), rtol=0, atol=1e-5 * rows.size(0))
    exact = s * (1 - hd * s * s * hd.mean(1, keepdim=True))
    assert float((dx.double() - exact).norm() / exact.norm()) < 2.0 ** -8
    assert trfn.tr_device_status() == 0
