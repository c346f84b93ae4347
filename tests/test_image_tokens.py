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


@pytest.mark.gpu
def test_token_rows_after_overlapping_batches():
    """Batches that overlap each other, then a token-row call on the output
    before the last: it waits for all of them."""
    mean, std, _ = trfn.tr_norm_preset("IMAGENET")
    N, C = 64, 3
    srcs = [torch.from_numpy(synth.pixels_uniform(20 + k, N, 224, 224, C)).cuda() for k in range(3)]
    ws = [torch.zeros(trfn.tr_workspace_bytes(), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = torch.empty((N, 224, 224, C), dtype=torch.float16, device="cuda")
    trfn.tr_fused_norm(srcs[1], want, mean, std, out_dtype=trfn.OUT_F16)
    rows = want.view(N * 224, 224 * C)
    q0, s0 = torch.empty(rows.shape, dtype=torch.int8, device="cuda"), torch.empty(rows.size(0), device="cuda")
    trfn.tr_quantize_rows(rows, q0, s0)
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [torch.zeros_like(want) for _ in range(3)]
        q, s = torch.zeros_like(q0), torch.zeros_like(s0)
        for k in range(3):
            trfn.tr_fused_norm(srcs[k], outs[k], mean, std, out_dtype=trfn.OUT_F16, workspace=ws[k % 2], overlap_previous=True)
        trfn.tr_quantize_rows(outs[1].view(N * 224, 224 * C), q, s)
        assert torch.equal(q, q0) and torch.equal(s, s0)
