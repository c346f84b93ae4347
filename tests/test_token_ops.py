"""Token-row operators (include/tr_token_ops.h) against their definitions in
64 bits, and their refusals.

Tolerances.  u is the output type's half unit (2^-24, 2^-11, 2^-8).  A row's
sums are taken in binary32 by at most 32 additions in a thread, 5 in a warp
and 32 across warps, so a sum of n positive terms is within 80 * 2^-24 of
itself, its inverse root within 40 * 2^-24 and a few roundings more: ROW =
2^-18 covers the norm.  Sums of signed terms are held to 2^-17 of the sum of
magnitudes.  An 8-bit value is within a half of its unrounded value, plus 127
times the relative error of what it is rounded from.  The integer product is
exact up to its conversion, two scalings and the bias: 4 * 2^-24 of the sum of
the magnitudes.  Every bound adds the rounding to the output's type."""
import ctypes
import os
import subprocess
import sys
import time

import pytest
import torch

import image_preprocessing_gb300 as trfn
from image_preprocessing_gb300 import TrError, _native, build

OK, INVALID, NOT_SUPPORTED = 0, 1, 2
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
ROW = 2.0 ** -18
TYPES = [torch.float32, torch.float16, torch.bfloat16]
NAMES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
gpu = pytest.mark.gpu


def name_of(v):
    return NAMES.get(v, str(v))


class Buffers:
    """Matrices inside larger buffers whose bytes around them must not change."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.kept = []

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda")

    def put(self, values, dtype, pad=0, shift=0):
        t = self.empty(values.shape[0], values.shape[1], dtype, pad, shift)
        t.copy_(values)
        return t

    def empty(self, rows, cols, dtype, pad=0, shift=0):
        whole = torch.zeros(rows * (cols + pad) + shift + 64, dtype=dtype, device="cuda")
        whole.view(torch.uint8).fill_(0x5A)
        t = whole[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        self.kept.append((whole, t))
        return t

    def check_around(self):
        for whole, t in self.kept:
            off = t.storage_offset()
            inside = torch.zeros(whole.numel(), dtype=torch.bool, device="cuda")
            inside[off:off + t.size(0) * t.stride(0)].view(t.size(0), t.stride(0))[:, :t.size(1)] = True
            size = whole.element_size()
            got = whole.view(torch.uint8).view(-1, size)[~inside]
            assert bool((got == 0x5A).all()), "bytes outside the matrix changed"


def near(got, want, slack, dtype):
    """|got - want| <= slack + the rounding of want to dtype."""
    bound = slack + UNIT[dtype] * (want.abs() + slack) + LEAST[dtype]
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


def norm_exact(x, r, w, eps):
    h = x.double() if r is None else x.double() + r.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, y if w is None else y * w.double()


def check_q8(q, scale, y, rel):
    """8-bit rows and scales against unrounded 64-bit rows."""
    a = y.abs().amax(1)
    zero = a < 2.0 ** -119
    assert bool((scale[zero] == 0).all()) and bool((q[zero] == 0).all())
    q, scale, y, a = q[~zero], scale[~zero], y[~zero], a[~zero]
    assert bool(((scale.double() - a / 127).abs() <= (rel + 2.0 ** -23) * a / 127).all())
    at = y / a[:, None] * 127
    assert bool(((q.double() - at).abs() <= 0.5 + 127 * (2 * rel + 2.0 ** -22)).all())
    assert q.numel() == 0 or int(q.int().abs().max()) <= 127


# sizes around each change of threads a row, odd ones, and the longest
COLS = [1, 2, 7, 31, 96, 255, 256, 257, 511, 768, 999, 1024, 1025, 2047, 2056, 4096, 4100, 8191, 8200, 16384, 16385, 32768]


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("cols", COLS)
def test_rms_norm_sizes(cols, dtype):
    b = Buffers(cols)
    rows = 5 if cols > 2048 else 19
    for pad, shift in ((0, 0), (16, 0), (3, 1)):
        x = b.put(b.randn(rows, cols), dtype, pad, shift)
        r = b.put(b.randn(rows, cols) * 3, dtype, pad, shift)
        w = 1 + 0.2 * b.randn(cols)
        out, ho = b.empty(rows, cols, dtype, pad, shift), b.empty(rows, cols, dtype, pad, shift)
        trfn.tr_rms_norm(x, out, weight=w, residual=r, residual_out=ho, eps=1e-5)
        h, y = norm_exact(x, r, w, 1e-5)
        near(ho, h, 2.0 ** -24 * h.abs(), dtype)
        near(out, y, ROW * y.abs(), dtype)
        b.check_around()
        b.kept.clear()
        x = b.put(b.randn(rows, cols), dtype, pad, shift)
        out = b.empty(rows, cols, dtype, pad, shift)
        trfn.tr_rms_norm(x, out)
        h, y = norm_exact(x, None, None, 1e-6)
        near(out, y, ROW * y.abs(), dtype)
        b.check_around()
        b.kept.clear()


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("cols", COLS)
def test_rms_norm_q8_and_quantize_sizes(cols, dtype):
    b = Buffers(cols + 1)
    rows = 5 if cols > 2048 else 19
    for pad, shift in ((0, 0), (16, 0), (3, 1)):
        x = b.put(b.randn(rows, cols), dtype, pad, shift)
        r = b.put(b.randn(rows, cols), dtype, pad, shift)
        w = 1 + 0.2 * b.randn(cols)
        ho, q = b.empty(rows, cols, dtype, pad, shift), b.empty(rows, cols, torch.int8, pad, shift)
        scale = torch.empty(rows, device="cuda")
        trfn.tr_rms_norm(x, q, weight=w, residual=r, residual_out=ho, scale=scale, eps=1e-5)
        h, y = norm_exact(x, r, w, 1e-5)
        near(ho, h, 2.0 ** -24 * h.abs(), dtype)
        check_q8(q, scale, y, ROW)
        b.check_around()
        b.kept.clear()
        x = b.put(b.randn(rows, cols) * 40, dtype, pad, shift)
        q = b.empty(rows, cols, torch.int8, pad, shift)
        trfn.tr_quantize_rows(x, q, scale)
        check_q8(q, scale, x.double(), 2.0 ** -23)
        for back_type in TYPES:
            back = b.empty(rows, cols, back_type, pad, shift)
            trfn.tr_dequantize_rows(q, scale, back)
            assert torch.equal(back, (q.float() * scale[:, None]).to(back_type))
        b.check_around()
        b.kept.clear()


@gpu
def test_q8_ties_go_to_even_and_the_largest_is_127():
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -127.0, 126.5, 3.0]], device="cuda")
    q, scale = torch.empty(1, 10, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    trfn.tr_quantize_rows(x, q, scale)
    assert scale.item() == 1.0
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, -2, -127, 126, 3]


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("cols", [8, 100, 1024, 5000])
def test_q8_rows_that_hold_nothing_or_no_numbers(cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(7, cols, generator=g, device="cuda").to(dtype)
    x[1] = 0
    x[2] = -0.0
    x[3, cols // 2] = float("inf")
    x[4, cols - 1] = float("nan")
    x[5, 0] = float("-inf")
    q, scale = torch.empty(7, cols, dtype=torch.int8, device="cuda"), torch.empty(7, device="cuda")
    w = torch.ones(cols, device="cuda")
    for norm in (False, True):
        q.fill_(55)
        if norm:
            trfn.tr_rms_norm(x, q, weight=w, scale=scale, eps=1e-6)
        else:
            trfn.tr_quantize_rows(x, q, scale)
        assert q[1:6].count_nonzero().item() == 0
        assert scale[1:3].tolist() == [0.0, 0.0]
        assert bool(scale[3:6].isnan().all())
        check_q8(q[[0, 6]], scale[[0, 6]], norm_exact(x[[0, 6]], None, None, 1e-6)[1] if norm else x[[0, 6]].double(), ROW)
    # the float output: zeros of zero rows, NaN where the definition has it
    out = torch.empty_like(x)
    trfn.tr_rms_norm(x, out, weight=w, eps=1e-6)
    assert out[1:3].count_nonzero().item() == 0
    for row in (3, 4, 5):
        assert bool(out[row].isnan().any())


@gpu
def test_q8_of_rows_near_the_smallest_numbers():
    x = torch.zeros(4, 64, device="cuda")
    x[0, 3] = 2.0 ** -119
    x[1, 3] = 2.0 ** -120
    x[2, 3] = 2.0 ** -149
    x[3, 3], x[3, 4] = -(2.0 ** -118), 2.0 ** -119
    q, scale = torch.empty(4, 64, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    trfn.tr_quantize_rows(x, q, scale)
    assert q[:, 3].tolist() == [127, 0, 0, -127] and q[3, 4].item() in (63, 64)
    assert scale[1:3].tolist() == [0.0, 0.0] and scale[0].item() > 0


@gpu
@pytest.mark.parametrize("rows", [0, 1, 2, 8, 9, 1000])
def test_rms_norm_row_counts(rows):
    b = Buffers(rows)
    x, r = b.put(b.randn(rows, 320), torch.float16), b.put(b.randn(rows, 320), torch.float16)
    out = b.empty(rows, 320, torch.float16)
    before = trfn.tr_launch_count()
    trfn.tr_rms_norm(x, out, residual=r)
    assert trfn.tr_launch_count() - before == (1 if rows else 0)
    near(out, norm_exact(x, r, None, 1e-6)[1], ROW * 8, torch.float16)
    b.check_around()


@gpu
@pytest.mark.parametrize("cols", [100, 1024, 4096])
def test_rms_norm_in_place_and_repeated_rows(cols):
    b = Buffers(cols)
    base = b.randn(33, cols).half()
    row = b.randn(1, cols).half()
    h, y = norm_exact(base, row.expand(33, cols), None, 1e-6)
    x, r = base.clone(), row.expand(33, cols)   # stride 0
    out = torch.empty_like(x)
    trfn.tr_rms_norm(x, out, residual=r, residual_out=x)
    near(x, h, 2.0 ** -24 * h.abs(), torch.float16)
    near(out, y, ROW * y.abs(), torch.float16)
    x, r = base.clone(), row.expand(33, cols).contiguous()
    trfn.tr_rms_norm(x, x, residual=r, residual_out=r)
    near(r, h, 2.0 ** -24 * h.abs(), torch.float16)
    near(x, y, ROW * y.abs(), torch.float16)
    # column blocks of one buffer
    both = torch.empty(33, 2 * cols, dtype=torch.float16, device="cuda")
    both[:, :cols] = base
    trfn.tr_rms_norm(both[:, :cols], both[:, cols:])
    assert torch.equal(both[:, :cols], base)
    near(both[:, cols:], norm_exact(base, None, None, 1e-6)[1], ROW * 8, torch.float16)


def grad_exact(dy, h, w, dres, eps):
    dy, h = dy.double(), h.double()
    s = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    g = dy if w is None else dy * w.double()
    dx = s * (g - h * s * s * (g * h).mean(1, keepdim=True))
    size = s * (g.abs() + h.abs() * s * s * (g * h).abs().mean(1, keepdim=True))
    if dres is not None:
        dx, size = dx + dres.double(), size + dres.double().abs()
    return dx, size, (dy * h * s).sum(0), (dy * h * s).abs().sum(0)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("cols", COLS)
def test_rms_norm_backward_sizes(cols, dtype):
    b = Buffers(cols + 2)
    for rows, pad, shift in ((19, 0, 0), (1, 16, 0), (23, 3, 1)):
        h = b.put(b.randn(rows, cols) * 2, dtype, pad, shift)
        dy = b.put(b.randn(rows, cols), dtype, pad, shift)
        dres = b.put(b.randn(rows, cols), dtype, pad, shift)
        w = 1 + 0.2 * b.randn(cols)
        dx = b.empty(rows, cols, dtype, pad, shift)
        dw = torch.full((cols,), 7.0, device="cuda")
        ws = torch.empty(trfn.tr_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        ws.fill_(0xFF)
        trfn.tr_rms_norm_backward(dy, h, dx, weight=w, dweight=dw, dresidual=dres, eps=1e-5, workspace=ws)
        want, size, want_w, size_w = grad_exact(dy, h, w, dres, 1e-5)
        near(dx, want, 2.0 ** -17 * size, dtype)
        near(dw, want_w, (rows + 200) * 2.0 ** -24 * size_w, torch.float32)
        b.check_around()
        b.kept.clear()


@gpu
@pytest.mark.parametrize("rows,cols", [(0, 64), (1, 64), (2, 1000), (1216, 48), (1217, 48), (5000, 264), (3001, 2049)])
def test_rms_norm_backward_row_counts_and_options(rows, cols):
    b = Buffers(rows)
    h, dy = b.randn(rows, cols), b.randn(rows, cols)
    dx, dw = torch.empty_like(h), torch.full((cols,), 7.0, device="cuda")
    ws = torch.empty(trfn.tr_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    trfn.tr_rms_norm_backward(dy, h, dx, dweight=dw, workspace=ws)
    want, size, want_w, size_w = grad_exact(dy, h, None, None, 1e-6)
    near(dx, want, 2.0 ** -17 * size, torch.float32)
    near(dw, want_w, (rows + 200) * 2.0 ** -24 * size_w, torch.float32)
    again = torch.empty_like(dw)
    trfn.tr_rms_norm_backward(dy, h, dx, dweight=again, workspace=ws)
    assert torch.equal(dw, again)
    only = torch.empty_like(h)
    trfn.tr_rms_norm_backward(dy, h, only)   # no dweight, no workspace
    assert torch.equal(only, dx)
    trfn.tr_rms_norm_backward(dy, h, dy)     # over dy
    assert torch.equal(dy, dx)


@gpu
def test_rms_norm_backward_against_differences():
    """dx and dweight along random directions against central differences of
    the 64-bit forward (step 1e-5: truncation about 1e-10, rounding 1e-11)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, cols, eps, step = 12, 333, 1e-3, 1e-5
    h, dy, v = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(3))
    w, vw = (torch.randn(cols, generator=g, device="cuda") for _ in range(2))
    dx, dw = torch.empty_like(h), torch.empty_like(w)
    ws = torch.empty(trfn.tr_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    trfn.tr_rms_norm_backward(dy, h, dx, weight=w, dweight=dw, eps=eps, workspace=ws)

    def loss(h_, w_):
        return float((norm_exact(h_, None, w_, eps)[1] * dy.double()).sum())

    hd, wd, vd, vwd = h.double(), w.double(), v.double(), vw.double()
    along = (loss(hd + step * vd, wd) - loss(hd - step * vd, wd)) / (2 * step)
    size = grad_exact(dy, h, w, None, eps)[1]
    assert abs(float((dx.double() * vd).sum()) - along) <= 2.0 ** -16 * float((size * vd.abs()).sum()) + 1e-6
    along = (loss(hd, wd + step * vwd) - loss(hd, wd - step * vwd)) / (2 * step)
    size_w = grad_exact(dy, h, w, None, eps)[3]
    assert abs(float((dw.double() * vwd).sum()) - along) <= 2.0 ** -16 * float((size_w * vwd.abs()).sum()) + 1e-6


def product_exact(x, w):
    return x.double() @ w.double().t()   # exact: below 2^53


def check_product(x, w, dtype, bias, pad=0, shift=0, seed=0, xs=None, ws_=None):
    """One product with random scales against the exact sums."""
    b = Buffers(seed)
    M, K, N = x.size(0), x.size(1), w.size(0)
    sx = 0.01 + 0.02 * b.randn(M).abs() if xs is None else xs
    sw = 0.01 + 0.02 * b.randn(N).abs() if ws_ is None else ws_
    bv = b.randn(N) * 5 if bias else None
    y = b.empty(M, N, dtype, pad, shift)
    work = torch.full((trfn.tr_int8_matmul_workspace_bytes(M, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
    trfn.tr_int8_matmul(x, sx, w, sw, y, bias=bv, workspace=work)
    part = product_exact(x, w) * sx.double()[:, None] * sw.double()
    want = part if bv is None else part + bv.double()
    size = part.abs() if bv is None else part.abs() + bv.double().abs()
    near(y, want, 4 * 2.0 ** -24 * size, dtype)
    b.check_around()


def any_int8(g, rows, cols, pad=0, shift=0):
    whole = torch.randint(-128, 128, (rows * (cols + pad) + shift + 16,), generator=g, device="cuda", dtype=torch.int8)
    return whole[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


M_SIZES = [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 196, 257, 515]


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("M", M_SIZES)
def test_int8_matmul_tokens(M, dtype):
    g = torch.Generator(device="cuda").manual_seed(M)
    for N, K, pad, shift in ((256, 512, 0, 0), (130, 96, 0, 0), (77, 333, 0, 0), (640, 1040, 16, 0), (65, 1111, 5, 3),
                             (1, 64, 0, 0), (300, 1, 0, 0), (513, 15, 1, 0)):
        check_product(any_int8(g, M, K, pad, shift), any_int8(g, N, K, pad, shift), dtype, N % 2 == 0, pad, shift, seed=N)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (3, 5000, 2048), (48, 1000, 8192), (300, 384, 20000), (1024, 1024, 768),
                                   (2049, 515, 640), (4000, 1536, 1023), (12544, 256, 128), (2049, 1539, 640), (1100, 4097, 333), (515, 4096, 1040), (20000, 1000, 65),
                                   (8192, 300, 2100), (700, 9000, 4096), (30001, 1000, 200), (21000, 2050, 130)])
def test_int8_matmul_larger(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    check_product(any_int8(g, M, K), any_int8(g, N, K), torch.float32, True)
    check_product(any_int8(g, M, K), any_int8(g, N, K), torch.float16, False, xs=torch.full((M,), 2.0 ** -12, device="cuda"))


@gpu
@pytest.mark.parametrize("M", [1, 5, 40, 200, 600])
@pytest.mark.parametrize("K", [1024, 1040, 4097, 131071])
def test_int8_matmul_sums_are_exact_at_their_largest(M, K):
    """All products at their largest, of one sign: every partial sum is as
    large as it gets.  With scales of one and a cancelling channel the
    binary32 output shows the integer itself below 2^24."""
    N = 140
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    x[:, 0] = torch.arange(M, device="cuda") % 100
    w[1, :] = 127
    w[2, K // 2:] = 127          # near cancellation: the sums meet again near zero
    w[3, ::2] = 127
    w[4, :] = 1
    one = torch.ones(max(M, N), device="cuda")
    y = torch.empty(M, N, device="cuda")
    work = torch.empty(trfn.tr_int8_matmul_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    trfn.tr_int8_matmul(x, one[:M], w, one[:N], y, workspace=work)
    want = product_exact(x, w)
    assert torch.equal(y, want.float())   # the exact sum, rounded to binary32 once
    small = want.abs() < 2 ** 24
    assert bool((y.double()[small] == want[small]).all())


@gpu
def test_int8_matmul_empty_sizes_and_scales_without_numbers():
    g = torch.Generator(device="cuda").manual_seed(1)
    bias = torch.randn(70, generator=g, device="cuda")
    y = torch.full((9, 70), 3.0, device="cuda")
    sx, sw = torch.ones(9, device="cuda"), torch.ones(70, device="cuda")
    nothing = torch.empty(9, 0, dtype=torch.int8, device="cuda"), torch.empty(70, 0, dtype=torch.int8, device="cuda")
    trfn.tr_int8_matmul(nothing[0], sx, nothing[1], sw, y, bias=bias)
    assert torch.equal(y, bias.expand(9, 70))
    trfn.tr_int8_matmul(nothing[0], sx, nothing[1], sw, y)
    assert y.count_nonzero().item() == 0
    before = trfn.tr_launch_count()
    trfn.tr_int8_matmul(nothing[0][:0], sx[:0], nothing[1], sw, y[:0], bias=bias)
    assert trfn.tr_launch_count() == before
    for M in (9, 200, 700):
        x, w = any_int8(g, M, 80), any_int8(g, 70, 80)
        sx = torch.ones(M, device="cuda")
        sx[3], sx[4] = float("nan"), 0.0
        y = torch.empty(M, 70, device="cuda")
        work = torch.empty(trfn.tr_int8_matmul_workspace_bytes(M, 70, 80), dtype=torch.uint8, device="cuda")
        trfn.tr_int8_matmul(x, sx, w, sw, y, workspace=work)
        assert bool(y[3].isnan().all()) and y[4].count_nonzero().item() == 0
        keep = [i for i in range(M) if i != 3]
        assert torch.equal(y[keep], (product_exact(x, w).float() * sx[:, None])[keep])


@gpu
def test_rows_far_apart():
    """Row offsets beyond 2^31 elements."""
    far = 2 ** 31 + 48
    whole = torch.zeros(2 * far + 4096, dtype=torch.float16, device="cuda")
    x = torch.as_strided(whole, (3, 640), (far, 1))
    g = torch.Generator(device="cuda").manual_seed(2)
    values = torch.randn(3, 640, generator=g, device="cuda").half()
    x.copy_(values)
    out = torch.empty(3, 640, dtype=torch.float16, device="cuda")
    trfn.tr_rms_norm(x, out)
    near(out, norm_exact(values, None, None, 1e-6)[1], ROW * 8, torch.float16)
    dx = torch.as_strided(whole, (3, 640), (far, 1), 1024)
    trfn.tr_rms_norm_backward(out, x, dx)
    want, size, _, _ = grad_exact(out, values, None, None, 1e-6)
    near(dx, want, 2.0 ** -17 * size, torch.float16)
    small = torch.empty(3, 640, dtype=torch.int8, device="cuda")
    scale = torch.empty(3, device="cuda")
    trfn.tr_quantize_rows(x, small, scale)
    check_q8(small, scale, values.double(), 2.0 ** -23)
    eight = whole.view(torch.int8)
    q = torch.as_strided(eight, (3, 640), (far, 1))
    trfn.tr_quantize_rows(values, q, scale)
    assert torch.equal(q, small)
    back = torch.empty_like(values)
    trfn.tr_dequantize_rows(q, scale, back)
    assert torch.equal(back, (small.float() * scale[:, None]).half())
    for M in (3, 200):
        xm = any_int8(g, M, 640)
        y, near_y = torch.empty(M, 3, device="cuda"), torch.empty(M, 3, device="cuda")
        work = torch.empty(trfn.tr_int8_matmul_workspace_bytes(M, 3, 640), dtype=torch.uint8, device="cuda")
        ones = torch.ones(M, device="cuda")
        trfn.tr_int8_matmul(xm, ones, q, scale, y, workspace=work)
        trfn.tr_int8_matmul(xm, ones, small, scale, near_y, workspace=work)
        assert torch.equal(y, near_y)


@gpu
def test_no_wait_ran_out():
    """The product's pipelines report a wait that ran out in the status word."""
    g = torch.Generator(device="cuda").manual_seed(8)
    for _ in range(20):
        check_product(any_int8(g, 3000, 1024), any_int8(g, 2048, 1024), torch.bfloat16, True)
    assert trfn.tr_device_status() == 0


@gpu
def test_other_stream_and_graph():
    """The calls run on the stream they are given, and can be captured."""
    g = torch.Generator(device="cuda").manual_seed(3)
    side = torch.cuda.Stream()
    for M in (4, 150, 9000):
        x = torch.randn(M, 512, generator=g, device="cuda").half()
        w = any_int8(g, 384, 512)
        sw = torch.rand(384, generator=g, device="cuda")
        q, scale = torch.empty(M, 512, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        y, first = torch.empty(M, 384, device="cuda"), torch.empty(M, 384, device="cuda")
        work = torch.empty(trfn.tr_int8_matmul_workspace_bytes(M, 384, 512), dtype=torch.uint8, device="cuda")

        def both(out, stream=None):
            trfn.tr_rms_norm(x, q, scale=scale, stream=stream)
            trfn.tr_int8_matmul(q, scale, w, sw, out, workspace=work, stream=stream)

        both(first)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            both(y)
        side.synchronize()
        assert torch.equal(y, first)
        y.fill_(0)
        torch.cuda.synchronize()
        both(y, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(y, first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            both(y)
        y.fill_(0)
        x.mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, -first)


def test_refusals_of_the_norm():
    L = _native.lib()
    X, R, W, O, H, S = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000

    def call(x=X, r=R, w=W, o=O, h=H, s=S, rows=4, cols=64, sx=64, sr=64, so=64, sh=64, dt=1, odt=1, eps=1e-6):
        return L.tr_rms_norm(x, r, w, o, h, s, rows, cols, sx, sr, so, sh, dt, odt, eps, None)

    assert call(rows=0) == OK
    bad = [dict(x=None), dict(o=None), dict(rows=-1), dict(cols=0), dict(sx=-1), dict(so=63), dict(sh=63), dict(dt=3, odt=3),
           dict(dt=7), dict(odt=0), dict(odt=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
           dict(x=X + 1), dict(r=R + 1), dict(w=W + 2), dict(o=O + 1), dict(h=H + 1), dict(r=None),   # h without a residual
           dict(odt=3, s=None), dict(odt=3, s=S + 2), dict(o=X + 2), dict(o=X + 128), dict(h=O), dict(o=W), dict(h=W),
           dict(odt=3, s=O), dict(odt=3, s=X + 64), dict(o=X, so=128), dict(odt=3, o=X), dict(so=2 ** 41)]
    for kw in bad:
        assert call(**kw) == INVALID, kw
    assert call(cols=trfn.tokens.MAX_ROW + 1, sx=1 << 20, sr=1 << 20, so=1 << 20, sh=1 << 20) == NOT_SUPPORTED
    assert call(rows=2 ** 31) == NOT_SUPPORTED


def test_refusals_of_the_gradient():
    L = _native.lib()
    Y, H, W, R, X, D, T = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000, 0x700000

    def call(dy=Y, h=H, w=W, r=R, x=X, d=D, rows=4, cols=64, sy=64, sh=64, sr=64, sx=64, dt=1, eps=1e-6, ws=T):
        return L.tr_rms_norm_backward(dy, h, w, r, x, d, rows, cols, sy, sh, sr, sx, dt, eps, ws, None)

    assert call(rows=0, d=None) == OK
    for kw in [dict(dy=None), dict(h=None), dict(x=None), dict(rows=-1), dict(cols=0), dict(sy=-1), dict(sx=63), dict(dt=3),
               dict(eps=-1.0), dict(ws=None), dict(ws=T + 8), dict(d=D + 1), dict(w=W + 1), dict(x=Y + 2), dict(x=W),
               dict(d=X), dict(d=W), dict(ws=Y), dict(ws=D), dict(r=R + 1), dict(x=R, sx=128)]:
        assert call(**kw) == INVALID, kw
    assert call(cols=40000) == NOT_SUPPORTED
    assert L.tr_rms_norm_backward_workspace_bytes(4, 64) >= 4 * 64
    assert L.tr_rms_norm_backward_workspace_bytes(-1, 64) == 0


def test_refusals_of_quantisation_and_product():
    L = _native.lib()
    X, Q, S, Y, W, T, B = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x10000000, 0x700000
    assert L.tr_quantize_rows(X, Q, S, 0, 64, 64, 64, 1, None) == OK
    for args in [(None, Q, S, 4, 64, 64, 64, 1), (X, None, S, 4, 64, 64, 64, 1), (X, Q, None, 4, 64, 64, 64, 1),
                 (X, Q, S, 4, 64, 64, 63, 1), (X, Q, S, 4, 64, -1, 64, 1), (X, Q, S, 4, 64, 64, 64, 3),
                 (X + 1, Q, S, 4, 64, 64, 64, 1), (X, X, S, 4, 64, 64, 64, 1), (X, Q, Q, 4, 64, 64, 64, 1),
                 (X, Q, S + 2, 4, 64, 64, 64, 1), (X, Q, S, -1, 64, 64, 64, 1), (X, Q, S, 4, 0, 64, 64, 1)]:
        assert L.tr_quantize_rows(*args, None) == INVALID, args
    for args in [(None, S, Y, 4, 64, 64, 64, 1), (Q, None, Y, 4, 64, 64, 64, 1), (Q, S, None, 4, 64, 64, 64, 1),
                 (Q, S, Y, 4, 64, 64, 63, 1), (Q, S, Y + 1, 4, 64, 64, 64, 1), (Q, S, Q, 4, 64, 64, 64, 1),
                 (Q, S, Y, 4, 64, 64, 64, 3), (Q, S, S, 4, 64, 64, 64, 0)]:
        assert L.tr_dequantize_rows(*args, None) == INVALID, args

    def call(x=X, sx=S, w=W, sw=S + 0x1000, b=B, y=Y, M=4, N=8, K=64, lx=64, lw=64, ly=8, dt=1, ws=T):
        return L.tr_int8_matmul(x, sx, w, sw, b, y, M, N, K, lx, lw, ly, dt, ws, None)

    assert call(M=0) == OK and call(N=0, ly=0) == OK
    for kw in [dict(x=None), dict(sx=None), dict(w=None), dict(sw=None), dict(y=None), dict(M=-1), dict(N=-1), dict(K=-1),
               dict(lx=-1), dict(ly=7), dict(dt=3), dict(dt=-1), dict(sx=S + 1), dict(b=B + 2), dict(y=Y + 1), dict(y=X),
               dict(y=W), dict(y=S), dict(y=B)]:
        assert call(**kw) == INVALID, kw
    assert call(K=131072, lx=131072, lw=131072) == NOT_SUPPORTED
    assert call(M=2 ** 31) == NOT_SUPPORTED and call(N=2 ** 31, ly=2 ** 31) == NOT_SUPPORTED
    need = L.tr_int8_matmul_workspace_bytes(5000, 4096, 4096)
    if need:   # a size that needs a workspace: none, and one off its alignment
        big = dict(M=5000, N=4096, K=4096, lx=4096, lw=4096, ly=4096, x=1 << 32, w=2 << 32, y=3 << 32)
        assert call(ws=None, **big) == INVALID and call(ws=(4 << 32) + 8, **big) == INVALID


def test_python_refusals():
    m = torch.zeros(4, 64, dtype=torch.float16)
    v = torch.zeros(64)
    with pytest.raises(TrError, match="CUDA"):
        trfn.tr_rms_norm(m, m)
    with pytest.raises(TrError, match="matrix"):
        trfn.tr_rms_norm(m[0], m[0])
    with pytest.raises(TrError, match="another type"):
        trfn.tr_rms_norm(m, m, residual=m.float())
    with pytest.raises(TrError, match="another type"):
        trfn.tr_quantize_rows(m, m, v[:4])
    with pytest.raises(TrError, match="another type"):
        trfn.tr_int8_matmul(m, v[:4], m, v[:4], m)
    with pytest.raises(TrError):
        trfn.tr_rms_norm_backward(m, m, m, dweight=v)


@gpu
def test_python_refusals_on_the_gpu():
    m = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    v = torch.zeros(64, device="cuda")
    for call in (lambda: trfn.tr_rms_norm(m, m[:3]),
                 lambda: trfn.tr_rms_norm(m, m.t().contiguous().t()),
                 lambda: trfn.tr_rms_norm(m, torch.empty_like(m), weight=v[:63]),
                 lambda: trfn.tr_rms_norm(m, q),
                 lambda: trfn.tr_rms_norm(m, q, scale=v),
                 lambda: trfn.tr_rms_norm(m, m.float()),
                 lambda: trfn.tr_rms_norm(m, m[:, :63]),
                 lambda: trfn.tr_rms_norm_backward(m, m, torch.empty_like(m), dweight=v),
                 lambda: trfn.tr_rms_norm_backward(m, m, torch.empty_like(m), dweight=v, workspace=v[:1]),
                 lambda: trfn.tr_dequantize_rows(q, v[:4], q),
                 lambda: trfn.tr_int8_matmul(q, v[:4], q, v[:4], m),
                 lambda: trfn.tr_int8_matmul(q, v[:3], q, v[:4], m[:, :4])):
        with pytest.raises(TrError):
            call()


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("cols", [3, 257, 999, 1021, 2049, 8191])
def test_odd_rows_in_place_and_repeated(cols, dtype):
    """Rows off 16-byte boundaries whose ends share 16 bytes with their
    neighbours: outputs over inputs, a repeated row, no weights."""
    b = Buffers(cols + 7)
    rows = 37
    base, row = b.randn(rows, cols).to(dtype), b.randn(1, cols).to(dtype)
    w = 1 + 0.2 * b.randn(cols)
    h, y = norm_exact(base, row.expand(rows, cols), w, 1e-5)
    x, r = base.clone(), row.expand(rows, cols).contiguous()
    trfn.tr_rms_norm(x, x, weight=w, residual=r, residual_out=r, eps=1e-5)
    near(r, h, 2.0 ** -24 * h.abs(), dtype)
    near(x, y, ROW * y.abs(), dtype)
    x, out = base.clone(), torch.empty_like(base)
    trfn.tr_rms_norm(x, out, weight=w, residual=row.expand(rows, cols), residual_out=x, eps=1e-5)   # stride 0
    near(x, h, 2.0 ** -24 * h.abs(), dtype)
    near(out, y, ROW * y.abs(), dtype)
    q, scale = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    trfn.tr_rms_norm(base, q, scale=scale, eps=1e-5)
    check_q8(q, scale, norm_exact(base, None, None, 1e-5)[1], ROW)
    dy, stored = b.randn(rows, cols).to(dtype), base.clone()
    want, size, _, _ = grad_exact(dy, stored, None, None, 1e-6)
    trfn.tr_rms_norm_backward(dy, stored, stored)   # over h
    near(stored, want, 2.0 ** -17 * size, dtype)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("M,N", [(1, 4096), (2, 20000), (3, 7), (2048, 2048), (4096, 1024), (50176, 129)])
def test_int8_matmul_of_nothing_gives_the_bias(M, N, dtype):
    """K = 0 at every size, those among them that would take the copies of
    many tokens."""
    b = Buffers(M)
    x, w = torch.empty(M, 0, dtype=torch.int8, device="cuda"), torch.empty(N, 0, dtype=torch.int8, device="cuda")
    sx, sw, bias = b.randn(M), b.randn(N), b.randn(N)
    assert trfn.tr_int8_matmul_workspace_bytes(M, N, 0) == 0
    y = b.empty(M, N, dtype, 3, 1)
    trfn.tr_int8_matmul(x, sx, w, sw, y, bias=bias)
    assert torch.equal(y, bias.to(dtype).expand(M, N))
    trfn.tr_int8_matmul(x, sx, w, sw, y)
    assert y.count_nonzero().item() == 0
    b.check_around()
    assert trfn.tr_device_status() == 0


@gpu
def test_errors_of_earlier_calls_are_not_reported():
    """A transfer station for a device that does not exist leaves the
    runtime's last error set; no token-row call takes it for its own."""
    slots = [torch.empty(4096, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((9, 64), generator=g, device="cuda")
    q, scale = torch.empty(9, 64, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")
    y, out, dx = torch.empty(9, 9, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    dw = torch.empty(64, device="cuda")
    ws = torch.empty(trfn.tr_rms_norm_backward_workspace_bytes(9, 64), dtype=torch.uint8, device="cuda")
    big, big_scale = any_int8(g, 9000, 768), torch.ones(9000, device="cuda")
    big_y = torch.empty(9000, 300, device="cuda")
    big_ws = torch.empty(trfn.tr_int8_matmul_workspace_bytes(9000, 300, 768), dtype=torch.uint8, device="cuda")
    for call, launches in ((lambda: trfn.tr_quantize_rows(x, q, scale), 1),
                           (lambda: trfn.tr_dequantize_rows(q, scale, out), 1),
                           (lambda: trfn.tr_rms_norm(x, out), 1),
                           (lambda: trfn.tr_rms_norm_backward(x, x, dx, dweight=dw, workspace=ws), 2),
                           (lambda: trfn.tr_int8_matmul(q[:1], scale[:1], q, scale, y[:1]), 1),
                           (lambda: trfn.tr_int8_matmul(q, scale, q, scale, y), 1),
                           (lambda: trfn.tr_int8_matmul(big, big_scale, big[:300], big_scale[:300], big_y, workspace=big_ws), 2)):
        trfn.TransferStation(4096, slots, *streams).close()
        before = trfn.tr_launch_count()
        call()
        assert trfn.tr_launch_count() - before == launches
    torch.cuda.synchronize()


def test_matrices_beyond_the_address_space_are_refused():
    """Rows whose distances add up to 2^64 elements: their ends must not wrap
    round to where they look harmless."""
    L = _native.lib()
    X, Q, S, R, W, H = 1 << 40, 1 << 41, 1 << 42, 1 << 43, 1 << 44, 1 << 45
    near_by = 64
    for rows, far in ((2 ** 24 + 1, 2 ** 40), (2 ** 30 + 1, 2 ** 40), (2 ** 30 + 1, 2 ** 34)):
        assert L.tr_quantize_rows(X, Q, S, rows, 64, far, near_by, 1, None) == INVALID
        assert L.tr_quantize_rows(X, Q, S, rows, 64, near_by, far, 1, None) == INVALID
        assert L.tr_dequantize_rows(Q, S, X, rows, 64, far, near_by, 0, None) == INVALID
        assert L.tr_rms_norm(X, R, None, Q, H, None, rows, 64, near_by, far, near_by, near_by, 1, 1, 1e-6, None) == INVALID
        assert L.tr_rms_norm(X, R, None, Q, H, None, rows, 64, near_by, near_by, near_by, far, 1, 1, 1e-6, None) == INVALID
        assert L.tr_rms_norm_backward(X, R, None, None, Q, None, rows, 64, near_by, far, 0, near_by, 1, 1e-6, None, None) == INVALID
        assert L.tr_int8_matmul(X, S, W, S + (1 << 40), None, Q, rows, 8, 64, far, 64, 8, 0, H, None) == INVALID
        assert L.tr_int8_matmul(X, S, W, S + (1 << 40), None, Q, 8, rows, 64, 64, far, 2 ** 32, 0, H, None) == INVALID


class Elsewhere:
    """Stands in for a contiguous tensor on a GPU of any number."""

    is_cuda = True

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), device

    def get_device(self):
        return self.device

    def stride(self):
        return self.shape[1], 1

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000


def test_tensors_on_other_devices_are_refused(monkeypatch):
    """Nothing reaches the library unless every tensor is on the current device."""
    t = trfn.tokens
    t._elem(torch.zeros(1))   # fills the module's tables
    calls = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 4096
            return lambda *a: calls.append(name) or 0

    current = [0]
    monkeypatch.setattr(t, "lib", Library)
    monkeypatch.setattr(t, "_current_stream", lambda device: 0)
    monkeypatch.setattr(t, "_current_device", lambda: current[0], raising=False)

    def f(n=None, device=0):
        return Elsewhere(torch.float32, *((4, 64) if n is None else (n,)), device=device)

    def i8(device=0):
        return Elsewhere(torch.int8, 4, 64, device=device)

    def space(device=0):
        return Elsewhere(torch.uint8, 4096, device=device)

    entries = {
        "tr_rms_norm": lambda a: t.tr_rms_norm(f(device=a[0]), i8(a[1]), weight=f(64, a[2]), residual=f(device=a[3]),
                                               residual_out=f(device=a[4]), scale=f(4, a[5])),
        "tr_rms_norm_backward": lambda a: t.tr_rms_norm_backward(f(device=a[0]), f(device=a[1]), f(device=a[2]), weight=f(64, a[3]),
                                                                 dweight=f(64, a[4]), dresidual=f(device=a[5]), workspace=space(a[6])),
        "tr_quantize_rows": lambda a: t.tr_quantize_rows(f(device=a[0]), i8(a[1]), f(4, a[2])),
        "tr_dequantize_rows": lambda a: t.tr_dequantize_rows(i8(a[0]), f(4, a[1]), f(device=a[2])),
        "tr_int8_matmul": lambda a: t.tr_int8_matmul(i8(a[0]), f(4, a[1]), i8(a[2]), f(4, a[3]),
                                                     Elsewhere(torch.float32, 4, 4, device=a[4]), bias=f(4, a[5]), workspace=space(a[6])),
    }
    count = {"tr_rms_norm": 6, "tr_rms_norm_backward": 7, "tr_quantize_rows": 3, "tr_dequantize_rows": 3, "tr_int8_matmul": 7}
    for name, call in entries.items():
        n = count[name]
        for device in (0, 1):
            current[0] = device
            calls.clear()
            call([device] * n)   # all on the current device
            assert calls == [name]
            for at in range(n):   # one of them elsewhere, or on the CPU
                for other in (1 - device, -1):
                    with pytest.raises(TrError):
                        call([other if i == at else device for i in range(n)])
            with pytest.raises(TrError, match="current device"):
                call([1 - device] * n)   # all of them elsewhere
            assert calls == [name]


@pytest.fixture(scope="module")
def early_release(tmp_path_factory):
    """early_release(out, ns): fills an int8 tensor ns after it has let the next kernel start."""
    path = str(tmp_path_factory.mktemp("early") / "early_release.so")
    source = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "early_release.cu")
    subprocess.run([build._nvcc(), "-shared", *build.ARCH, "-O2", "-Xcompiler", "-fPIC", "-o", path, source], check=True)
    fn = ctypes.CDLL(path).early_release
    fn.argtypes = [ctypes.c_void_p, ctypes.c_longlong, ctypes.c_ulonglong, ctypes.c_void_p]
    return lambda out, ns: fn(out.data_ptr(), out.numel(), ns, torch.cuda.current_stream().cuda_stream)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (16, 256, 256), (40, 300, 4096), (196, 512, 1000), (9000, 300, 768)])
def test_a_long_kernel_before_the_product_does_not_count_as_its_wait(early_release, M, N, K):
    """The kernel before lets the product start, then runs longer than the
    limit of the product's waits (1 s) and writes x last of all."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    w = any_int8(g, N, K)
    ones = torch.ones(max(M, N), device="cuda")
    y = torch.zeros(M, N, device="cuda")
    work = torch.empty(trfn.tr_int8_matmul_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert early_release(x, 1_500_000_000) == 0
    trfn.tr_int8_matmul(x, ones[:M], w, ones[:N], y, workspace=work)
    torch.cuda.synchronize()
    filled = (torch.arange(M * K, device="cuda") * 7 % 251 - 125).to(torch.int8).view(M, K)
    assert torch.equal(x, filled)
    assert torch.equal(y, product_exact(filled, w).float())
    assert trfn.tr_device_status() == 0


@gpu
@pytest.mark.parametrize("M,N,K", [(16, 256, 256), (40, 300, 4096), (128, 16384, 640), (600, 384, 20000), (196, 300, 333), (9000, 300, 768),
                                   (9000, 600, 2100)])
def test_a_product_whose_wait_runs_out_stores_no_unfinished_sums(M, N, K):
    """The first stage of the first CTA waits for an arrival that never comes
    (tr_tune_tiled's test hook): the launch ends by itself and reports it, and
    what it has written is right."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, w = any_int8(g, M, K), any_int8(g, N, K)
    ones = torch.ones(max(M, N), device="cuda")
    y = torch.full((M, N), 0.5, device="cuda")   # no sum of integers
    work = torch.empty(trfn.tr_int8_matmul_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    want = product_exact(x, w).float()
    assert trfn.tr_device_status(clear=True) == 0
    try:
        trfn.tr_tune_tiled(0, 0, 0, 64)
        t0 = time.perf_counter()
        trfn.tr_int8_matmul(x, ones[:M], w, ones[:N], y, workspace=work)
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        trfn.tr_tune_tiled(0, 0, 0, 0)
    assert 0.5 < elapsed < 30
    assert trfn.tr_device_status(clear=True) == 1
    written = y != 0.5
    assert not bool(written[0, 0])
    assert torch.equal(y[written], want[written])
    trfn.tr_int8_matmul(x, ones[:M], w, ones[:N], y, workspace=work)
    assert torch.equal(y, want)
    assert trfn.tr_device_status() == 0


@gpu
def test_reading_the_device_status_costs_what_it_did():
    """In a process without products it is two small copies (the word, and the
    site of a failed check), no dearer than two elements of a tensor read one
    by one; products add one copy."""
    script = """
import time, torch
import image_preprocessing_gb300 as trfn
value = torch.zeros(1, device="cuda")
def best(call):
    times = []
    for _ in range(300):
        t0 = time.perf_counter()
        call()
        times.append(time.perf_counter() - t0)
    return min(times)
mean, std, _ = trfn.tr_norm_preset("IMAGENET")
src = torch.zeros((1, 32, 32, 3), dtype=torch.uint8, device="cuda")
trfn.tr_fused_norm(src, torch.empty((1, 32, 32, 3), dtype=torch.float16, device="cuda"), mean, std)
before = best(trfn.tr_device_status) / best(value.item)
q, one, y = torch.ones(16, 64, dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda"), torch.empty(16, 16, device="cuda")
trfn.tr_int8_matmul(q, one, q, one, y)
assert trfn.tr_device_status() == 0 and bool((y == 64).all())
print(before, best(trfn.tr_device_status) / best(value.item))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    before, after = map(float, r.stdout.split())
    assert before <= 2 and after <= 3


def test_int8_matmul_workspace_of_the_largest_batch_serves_all():
    sizes = trfn.tr_int8_matmul_workspace_bytes
    for N, K in ((1024, 768), (300, 640), (64, 64), (4096, 4096), (515, 515), (16384, 100), (2048, 131071)):
        last = 0
        for M in list(range(1, 5200)) + [50176, 50177, 10 ** 6]:
            now = sizes(M, N, K)
            assert now >= last, (M, N, K)
            last = now
    assert sizes(1, 16384, 8192) == sizes(2, 16384, 8192) == 0


def test_gradient_workspace_of_the_most_rows_serves_all():
    sizes = trfn.tr_rms_norm_backward_workspace_bytes
    for cols in (1, 64, 511, 512, 513, 1024, 1025, 4096, 8193, 32768):
        of_rows = [sizes(rows, cols) for rows in list(range(1, 3000)) + [50176, 2 ** 31 - 1]]
        assert of_rows == sorted(of_rows) and of_rows[0] >= 4 * cols, cols


@gpu
@pytest.mark.parametrize("N,K,largest", [(1024, 768, 2305), (300, 640, 4338), (1024, 1024, 5000)])
def test_int8_matmul_in_the_workspace_of_the_largest_batch(N, K, largest):
    """Smaller batches stay inside it, whichever kernels they take."""
    g = torch.Generator(device="cuda").manual_seed(N)
    size = trfn.tr_int8_matmul_workspace_bytes(largest, N, K)
    whole = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    w, ones = any_int8(g, N, K), torch.ones(max(N, largest), device="cuda")
    for M in (3, 200, 1000, 2048, 2304, 2305, 4096, 4337, largest):
        if M > largest:
            continue
        x, y = any_int8(g, M, K), torch.zeros(M, N, device="cuda")
        trfn.tr_int8_matmul(x, ones[:M], w, ones[:N], y, workspace=whole[:size])
        assert torch.equal(y, product_exact(x, w).float()), M
        assert bool((whole[size:] == 0x5A).all())


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("rows,cols", [(12501, 64), (12501, 257), (15001, 504), (12501, 506), (9003, 511), (12501, 512), (5003, 999),
                                       (5003, 1024), (3501, 2041), (2001, 4096), (1777, 4095), (901, 8191), (901, 8192), (801, 9001),
                                       (701, 16384), (501, 20000)])
def test_rms_norm_backward_through_many_rows(rows, cols, dtype):
    """Each CTA goes through several rows, past the ones copied ahead at its
    start: aligned rows, dense rows off 16-byte boundaries, and rows that do
    not lie alike.  The bounds are those of the sizes above."""
    b = Buffers(cols + 3)
    w = 1 + 0.2 * b.randn(cols)
    ws = torch.empty(trfn.tr_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    h0, dy0, dres0 = b.randn(rows, cols) * 2, b.randn(rows, cols), b.randn(rows, cols)
    for pads, shift in (((0, 0, 0, 0), 0), ((3, 0, 8, 1), 1)):
        h, dy, dres = (b.put(v, dtype, pad, shift) for v, pad in zip((h0, dy0, dres0), pads))
        dx, dw = b.empty(rows, cols, dtype, pads[3], shift), torch.full((cols,), 7.0, device="cuda")
        trfn.tr_rms_norm_backward(dy, h, dx, weight=w, dweight=dw, dresidual=dres, eps=1e-5, workspace=ws)
        want, size, want_w, size_w = grad_exact(dy, h, w, dres, 1e-5)
        near(dx, want, 2.0 ** -17 * size, dtype)
        near(dw, want_w, (rows + 200) * 2.0 ** -24 * size_w, torch.float32)
        b.check_around()
        dense = dx.clone()
        trfn.tr_rms_norm_backward(dy, h, dres, weight=w, dresidual=dres, eps=1e-5)   # over the residual's gradient
        assert torch.equal(dres, dense)
        b.kept.clear()
