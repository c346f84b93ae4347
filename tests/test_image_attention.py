"""The example's attention block, which runs layer norm, the 8-bit product,
rotary positions and attention together, against the same block in binary32 on
unquantised rows; and its pieces once more through a captured graph."""
import importlib.util
import os

import pytest
import torch

import image_preprocessing_gb300 as trfn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("image_tokens", os.path.join(ROOT, "examples", "image_tokens.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _block(x, wqkv, wout, images, head):
    """y and h of the block, plainly."""
    rows, width = x.shape
    n, heads = rows // images, width // head

    def norm(v):
        v = v - v.mean(1, keepdim=True)
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-5)

    qkv = (norm(x) @ wqkv.t()).view(images, n, 3, heads, head)
    k = torch.arange(head // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2 * k / head)
    c, s = angle.cos().to(x.dtype)[None, :, None], angle.sin().to(x.dtype)[None, :, None]

    def turn(v):
        a, b = v[..., :head // 2], v[..., head // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k, v = turn(qkv[:, :, 0]), turn(qkv[:, :, 1]), qkv[:, :, 2]
    p = torch.softmax(torch.einsum("bihd,bjhd->bhij", q, k) / head ** 0.5, -1)
    h = torch.einsum("bhij,bjhd->bihd", p, v).reshape(rows, width) @ wout.t() + x
    return norm(h), h


@pytest.mark.gpu
@pytest.mark.parametrize("images,width", [(1, 128), (6, 320)])
def test_attention_block_follows_the_network_in_binary32(images, width):
    """The 8-bit rows and weights of two products are off by 1.1 % each of a near-normal row's rms, 1.6 % a
    product.  The scores (near normal, of rms 1 by the products' scaling) carry 1.6 % of noise as well, which
    moves a mean of values about as much again; the second product adds its own 1.6 %: 2.8 % of the part that
    joins the stream, whose rms is below the stream's."""
    e = _example()
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((images * 196, width), generator=g, device="cuda").bfloat16()
    net = e.build_attention(width, seed=4)
    y, h = e.attend(net, x, images)
    g = torch.Generator(device="cuda").manual_seed(4)
    wqkv = torch.randn((3 * width, width), generator=g, device="cuda") / width ** 0.5
    wout = torch.randn((width, width), generator=g, device="cuda") / width ** 0.5
    want, want_h = _block(x.float(), wqkv, wout, images, e.HEAD)
    assert float((h.float() - want_h).norm() / want_h.norm()) < 0.04
    assert float((y.float() - want).norm() / want.norm()) < 0.04
    dx, dweight, dbias = e.layer_norm_gradients(torch.ones_like(y), h, net["weight2"])
    hd = h.double()
    u = hd - hd.mean(1, keepdim=True)
    u = u * torch.rsqrt(u.square().mean(1, keepdim=True) + 1e-5)
    assert torch.allclose(dweight.double(), u.sum(0), rtol=0, atol=1e-5 * images * 196)
    assert torch.equal(dbias, torch.full_like(dbias, images * 196))
    # the gradient of a sum over normalised values is that of nothing but the last bits
    assert float(dx.abs().max()) < 1e-3
    assert trfn.tr_device_status() == 0


@pytest.mark.gpu
def test_attention_block_captured_in_a_graph():
    e = _example()
    images, width = 3, 256
    x = torch.randn((images * 196, width), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    net = e.build_attention(width)
    want, want_h = e.attend(net, x, images)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        e.attend(net, x, images)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            y, h = e.attend(net, x, images)
    for _ in range(3):
        y.zero_()
        h.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(h, want_h)
