"""From a uint8 image batch to a network's hidden rows, on the GPU: the fused
normalisation, its patches in 8 bits, the patch embedding as an 8-bit integer
product, and one pre-norm block (RMS norm with the residual's addition, 8-bit
output; two products), then a training step's gradients of a norm.

    python examples/image_tokens.py [images] [width]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import image_preprocessing_gb300 as trfn  # noqa: E402
from image_preprocessing_gb300 import synth  # noqa: E402

SIDE, PATCH = 224, 16


class Linear8:
    """A layer's weights in 8 bits with a scale for each channel, laid out once."""

    def __init__(self, weight, bias=None):
        self.w = torch.empty(weight.shape, dtype=torch.int8, device="cuda")
        self.scale = torch.empty(weight.size(0), device="cuda")
        self.bias = bias
        self.workspace = None
        trfn.tr_quantize_rows(weight, self.w, self.scale)

    def __call__(self, q, scale):
        M, K = q.shape
        N = self.w.size(0)
        need = trfn.tr_int8_matmul_workspace_bytes(M, N, K)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        trfn.tr_int8_matmul(q, scale, self.w, self.scale, y, bias=self.bias, workspace=self.workspace)
        return y


def patches(images, mean, std, records):
    """The normalised FP16 batch as rows of 16 x 16 x 3 values."""
    N = images.size(0)
    dst = torch.empty((N, SIDE, SIDE, 3), dtype=torch.float16, device="cuda")
    trfn.tr_fused_norm(images, dst, mean, std, records, out_dtype=trfn.OUT_F16)
    n = SIDE // PATCH
    return dst.view(N, n, PATCH, n, PATCH, 3).transpose(2, 3).reshape(N * n * n, PATCH * PATCH * 3)


def quantised(rows):
    q = torch.empty(rows.shape, dtype=torch.int8, device="cuda")
    scale = torch.empty(rows.size(0), device="cuda")
    trfn.tr_quantize_rows(rows, q, scale)
    return q, scale


def forward(net, rows, positions):
    """Hidden rows after one block, and what the gradient step below needs."""
    x = net["embed"](*quantised(rows))
    # positions are the residual that joins the embedding; the norm's 8-bit rows feed the next product
    q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    scale, h = torch.empty(x.size(0), device="cuda"), torch.empty_like(x)
    trfn.tr_rms_norm(x, q, weight=net["norm1"], residual=positions, residual_out=h, scale=scale)
    x = net["up"](q, scale)
    x = net["down"](*quantised(torch.nn.functional.gelu(x)))
    y, h2 = torch.empty_like(x), torch.empty_like(x)
    trfn.tr_rms_norm(x, y, weight=net["norm2"], residual=h, residual_out=h2)
    return y, h2


def norm_gradients(dy, h, weight):
    rows, cols = h.shape
    dx, dweight = torch.empty_like(h), torch.empty(cols, device="cuda")
    workspace = torch.empty(trfn.tr_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    trfn.tr_rms_norm_backward(dy, h, dx, weight=weight, dweight=dweight, workspace=workspace)
    return dx, dweight


def build(width, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def matrix(n, k):
        return torch.randn((n, k), generator=g, device="cuda") / k ** 0.5

    return {"embed": Linear8(matrix(width, PATCH * PATCH * 3), bias=torch.zeros(width, device="cuda")),
            "up": Linear8(matrix(2 * width, width)), "down": Linear8(matrix(width, 2 * width)),
            "norm1": torch.ones(width, device="cuda"), "norm2": torch.ones(width, device="cuda")}


def main(images=8, width=512):
    torch.cuda.set_device(0)
    mean, std, _ = trfn.tr_norm_preset("IMAGENET")
    src = torch.from_numpy(synth.pixels_uniform(11, images, SIDE, SIDE, 3)).cuda()
    records, _ = trfn.tr_sample_aug_params(12, 0, images, SIDE, SIDE)
    net = build(width)
    rows = patches(src, mean, std, torch.from_numpy(records).cuda())
    positions = 0.02 * torch.randn((rows.size(0), width), device="cuda", dtype=torch.bfloat16)
    y, h = forward(net, rows, positions)
    dx, dweight = norm_gradients(torch.ones_like(y), h, net["norm2"])
    torch.cuda.synchronize()
    print("%d images -> %d tokens of %d; hidden rms %.4f, |dx| %.4g, |dweight| %.4g" % (
        images, rows.size(0), width, y.float().square().mean().sqrt().item(), dx.float().norm().item(), dweight.norm().item()))
    return y


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:]))
