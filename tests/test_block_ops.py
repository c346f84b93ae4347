"""Layer norm and its gradients, rotary positions and attention
(include/tr_token_ops.h) against their definitions in 64 bits, and their
refusals.

Tolerances.  u is the output type's half unit (2^-24, 2^-11, 2^-8).
Norms: a row's sums are taken in binary32 by at most 32 additions in a thread,
5 in a warp and 32 across warps, so a sum of n terms is within 2^-17 of the sum
of their magnitudes; a mean within 2^-17 of mean |h| = the row's DM.  A value
less the mean is off by DM and a rounding, the variance by DM^2 and 2^-17 of
itself.
Rotary: a phase is rounded to 2^-25 half turns (2^-23 radians), sine and cosine
to 2 units: 2^-21 of |a| + |b| covers both with the products.
Attention: a score is off by 2^-18 of sum |q_d k_d| (128 products, summed 16 at a
time by the tensor cores; up to 256 one by one in the plain kernel), a weight by
that and its own exponent's rounding, relative to itself, and by half a unit of
the type where it is rounded (2^-25 at least in binary16, of weights whose largest
is 1 or more); sums over n keys by n/16 steps of 2^-22.  All of it relative to
sum p |v| / sum p.  Every bound adds the rounding to the output's type."""
import ctypes
import math
import os
import subprocess
import time

import pytest
import torch

import image_preprocessing_gb300 as trfn
from image_preprocessing_gb300 import TrError, _native, build

OK, INVALID, NOT_SUPPORTED = 0, 1, 2
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
TYPES = [torch.float32, torch.float16, torch.bfloat16]
SHORT = [torch.float16, torch.bfloat16]
NAMES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
SUM = 2.0 ** -17
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
        whole.view(torch.uint8).fill_(0xFF)   # NaN in the float types: bytes around a matrix must not reach a result
        t = whole[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        self.kept.append((whole, t))
        return t

    def check_around(self):
        for whole, t in self.kept:
            off = t.storage_offset()
            inside = torch.zeros(whole.numel(), dtype=torch.bool, device="cuda")
            inside[off:off + t.size(0) * t.stride(0)].view(t.size(0), t.stride(0))[:, :t.size(1)] = True
            got = whole.view(torch.uint8).view(-1, whole.element_size())[~inside]
            assert bool((got == 0xFF).all()), "bytes outside the matrix changed"
        self.kept.clear()


def near(got, want, slack, dtype):
    """|got - want| <= slack + the rounding of want to dtype."""
    bound = slack + UNIT[dtype] * (want.abs() + slack) + LEAST[dtype]
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).nan_to_num(nan=float("inf")).max())


# ------------------------------------------------------------------ layer norm ---

def layer_exact(x, r, w, b, eps):
    """h, y and what y may be off by."""
    h = x.double() if r is None else x.double() + r.double()
    d = h - h.mean(1, keepdim=True)
    s = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    w = torch.ones(x.size(1), device="cuda", dtype=torch.float64) if w is None else w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    dm = SUM * h.abs().mean(1, keepdim=True)
    slack = s * w.abs() * dm + (w * d * s).abs() * (SUM + (dm * s) ** 2) + 2.0 ** -22 * ((w * d * s).abs() + b.abs())
    return h, d * s * w + b, slack


# around each change of threads a row, odd ones, and the longest
COLS = [1, 2, 7, 31, 64, 96, 128, 255, 257, 505, 508, 511, 512, 768, 999, 1024, 1025, 2047, 2056, 4096, 4100, 8191, 8200, 16385,
        32768]


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("cols", COLS)
def test_layer_norm_sizes(cols, dtype):
    buf = Buffers(cols)
    rows = 5 if cols > 2048 else 19
    for pad, shift in ((0, 0), (16, 0), (3, 1)):
        x = buf.put(buf.randn(rows, cols) + 2, dtype, pad, shift)
        r = buf.put(buf.randn(rows, cols) * 3, dtype, pad, shift)
        w, b = 1 + 0.2 * buf.randn(cols), 0.3 * buf.randn(cols)
        h, y, slack = layer_exact(x, r, w, b, 1e-5)
        out, ho = buf.empty(rows, cols, dtype, pad, shift), buf.empty(rows, cols, dtype, pad, shift)
        trfn.tr_layer_norm(x, out, weight=w, bias=b, residual=r, residual_out=ho)
        near(ho, h, 2.0 ** -24 * h.abs(), dtype)
        near(out, y, slack, dtype)
        # 8 bits: within a half of the unrounded value, and what the row's largest is off by
        q, scale = buf.empty(rows, cols, torch.int8, pad, shift), torch.empty(rows, device="cuda")
        trfn.tr_layer_norm(x, q, weight=w, bias=b, residual=r, residual_out=ho, scale=scale)
        near(ho, h, 2.0 ** -24 * h.abs(), dtype)
        a, off = y.abs().amax(1, keepdim=True), slack.amax(1, keepdim=True)
        assert bool(((scale.double()[:, None] - a / 127).abs() <= (off + 2.0 ** -22 * a) / 127).all())
        some = a > 1e-30
        at = torch.where(some, y * 127 / a, torch.zeros_like(a))
        rel = torch.where(some, off / a, torch.zeros_like(a))
        assert bool(((q.double() - at).abs() <= 0.5 + 127 * (2 * rel + 2.0 ** -21)).all())
        # neither residual, weight nor bias; one of them
        for w1, b1 in ((None, None), (w, None), (None, b)):
            out = buf.empty(rows, cols, dtype, pad, shift)
            trfn.tr_layer_norm(x, out, weight=w1, bias=b1, eps=1e-3)
            _, y1, slack1 = layer_exact(x, None, w1, b1, 1e-3)
            near(out, y1, slack1, dtype)
        buf.check_around()


def layer_grad_exact(dy, h, w, dres, eps):
    dy, h = dy.double(), h.double()
    d = h - h.mean(1, keepdim=True)
    s = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    u = d * s
    g = dy if w is None else dy * w.double()
    dx = s * (g - g.mean(1, keepdim=True) - u * (g * u).mean(1, keepdim=True))
    du = SUM * h.abs().mean(1, keepdim=True) * s
    size = s * (g.abs() + g.abs().mean(1, keepdim=True) + u.abs() * (g * u).abs().mean(1, keepdim=True))
    slack = size * (2 * SUM + 3 * du * du) + s * du * ((g * u).abs().mean(1, keepdim=True) + u.abs() * g.abs().mean(1, keepdim=True))
    if dres is not None:
        dx, slack = dx + dres.double(), slack + 2.0 ** -22 * dres.double().abs()
    dw, db = (dy * u).sum(0), dy.sum(0)
    dw_slack = (dy * u).abs().sum(0) * 2 * SUM + (dy.abs() * (du + u.abs() * du * du)).sum(0)
    return dx, slack, dw, dw_slack, db, SUM * dy.abs().sum(0)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("cols", COLS)
def test_layer_norm_backward_sizes(cols, dtype):
    buf = Buffers(cols + 1)
    rows = 9 if cols > 2048 else 77
    for pad, shift in ((0, 0), (16, 0), (3, 1)):
        h = buf.put(buf.randn(rows, cols) * 2 + 1, dtype, pad, shift)
        dy = buf.put(buf.randn(rows, cols), dtype, pad, shift)
        dres = buf.put(buf.randn(rows, cols), dtype, pad, shift)
        w = 1 + 0.2 * buf.randn(cols)
        ws = torch.empty(trfn.tr_layer_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        for weight, residual, sums in ((w, dres, (1, 1)), (None, None, (1, 1)), (w, None, (0, 1)), (w, dres, (1, 0)), (w, dres, (0, 0))):
            dx = buf.empty(rows, cols, dtype, pad, shift)
            dw = torch.full((cols,), 7.0, device="cuda") if sums[0] else None
            db = torch.full((cols,), 7.0, device="cuda") if sums[1] else None
            ws.fill_(0xFF)
            trfn.tr_layer_norm_backward(dy, h, dx, weight=weight, dweight=dw, dbias=db, dresidual=residual,
                                        workspace=ws if any(sums) else None)
            want, slack, want_w, slack_w, want_b, slack_b = layer_grad_exact(dy, h, weight, residual, 1e-5)
            near(dx, want, slack, dtype)
            if sums[0]:
                near(dw, want_w, slack_w, torch.float32)
            if sums[1]:
                near(db, want_b, slack_b, torch.float32)
        buf.check_around()


@gpu
@pytest.mark.parametrize("rows,cols", [(5000, 1024), (4001, 511), (20000, 60), (700, 4096), (3000, 100)])
def test_layer_norm_backward_many_rows(rows, cols):
    """Rows beyond one for each row group of the grid."""
    buf = Buffers(rows)
    h, dy = buf.put(buf.randn(rows, cols), torch.float16), buf.put(buf.randn(rows, cols), torch.float16)
    dx, dw, db = torch.empty_like(h), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(trfn.tr_layer_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    trfn.tr_layer_norm_backward(dy, h, dx, dweight=dw, dbias=db, workspace=ws)
    want, slack, want_w, slack_w, want_b, slack_b = layer_grad_exact(dy, h, None, None, 1e-5)
    near(dx, want, slack, torch.float16)
    near(dw, want_w, slack_w, torch.float32)
    near(db, want_b, slack_b, torch.float32)
    again = [torch.empty_like(t) for t in (dx, dw, db)]
    trfn.tr_layer_norm_backward(dy, h, again[0], dweight=again[1], dbias=again[2], workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))


@gpu
def test_layer_norm_gradients_against_differences():
    """dx, dweight and dbias of sum(y * dy) by central differences in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, cols = 4, 37
    x = torch.randn(rows, cols, generator=g, device="cuda")
    dy = torch.randn(rows, cols, generator=g, device="cuda")
    w, b = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda"), torch.randn(cols, generator=g, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(trfn.tr_layer_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    trfn.tr_layer_norm_backward(dy, x, dx, weight=w, dweight=dw, dbias=db, workspace=ws)
    wide = [t.double() for t in (x, w, b)]

    def loss():
        return (layer_exact(wide[0], None, wide[1], wide[2], 1e-5)[1] * dy.double()).sum().item()

    step = 1e-5
    for which, grad in ((0, dx), (1, dw), (2, db)):
        flat, got = wide[which].view(-1), grad.view(-1)
        for i in range(0, flat.numel(), 5):
            keep = flat[i].item()
            flat[i] = keep + step
            up = loss()
            flat[i] = keep - step
            down = loss()
            flat[i] = keep
            # the difference's own error: step^2 and 2^-52 / step of sums near 100
            assert abs((up - down) / (2 * step) - got[i].item()) < 1e-6 * 100 + 2.0 ** -17 * 10


@gpu
def test_layer_norm_far_means_and_equal_rows():
    cols = 1024
    g = torch.Generator(device="cuda").manual_seed(1)
    x = 1000 + torch.randn(3, cols, generator=g, device="cuda")
    out = torch.empty_like(x)
    trfn.tr_layer_norm(x, out)
    _, y, slack = layer_exact(x, None, None, None, 1e-5)
    near(out, y, slack, torch.float32)
    x = torch.full((2, cols), 3.0, device="cuda")   # no variance: the bias
    b = torch.randn(cols, generator=g, device="cuda")
    trfn.tr_layer_norm(x, out[:2], bias=b)
    assert torch.equal(out[:2], b.expand(2, cols))
    q, scale = torch.empty(2, cols, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    trfn.tr_layer_norm(x, q, scale=scale)
    assert q.count_nonzero().item() == 0 and scale.tolist() == [0.0, 0.0]


@gpu
@pytest.mark.parametrize("cols", [8, 100, 1001, 1024, 5000])
def test_layer_norm_rows_without_numbers(cols):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(5, cols, generator=g, device="cuda").half()
    x[1, cols // 2], x[3, cols - 1] = float("inf"), float("nan")
    q, scale, out = torch.empty(5, cols, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda"), torch.empty_like(x)
    trfn.tr_layer_norm(x, q, scale=scale)
    trfn.tr_layer_norm(x, out)
    for row in range(5):
        bad = row in (1, 3)
        assert bool(scale[row].isnan()) == bad and bool(out[row].isnan().any()) == bad
        assert not bad or q[row].count_nonzero().item() == 0
    _, y, slack = layer_exact(x[[0, 2, 4]], None, None, None, 1e-5)
    near(out[[0, 2, 4]], y, slack, torch.float16)


@gpu
@pytest.mark.parametrize("cols", [100, 1024, 4096])
def test_layer_norm_in_place_and_repeated_rows(cols):
    buf = Buffers(cols)
    base, row = buf.randn(33, cols).half(), buf.randn(1, cols).half()
    h, y, slack = layer_exact(base, row.expand(33, cols), None, None, 1e-5)
    x, out = base.clone(), torch.empty_like(base)
    trfn.tr_layer_norm(x, out, residual=row.expand(33, cols), residual_out=x)   # stride 0
    near(x, h, 2.0 ** -24 * h.abs(), torch.float16)
    near(out, y, slack, torch.float16)
    x, r = base.clone(), row.expand(33, cols).contiguous()
    trfn.tr_layer_norm(x, x, residual=r, residual_out=r)
    near(r, h, 2.0 ** -24 * h.abs(), torch.float16)
    near(x, y, slack, torch.float16)
    for target in ("dy", "h", "dres"):
        t = {"dy": base.clone(), "h": base.flip(0).contiguous(), "dres": base.flip(1).contiguous()}
        want, slack, _, _, _, _ = layer_grad_exact(t["dy"], t["h"], None, t["dres"], 1e-5)
        trfn.tr_layer_norm_backward(t["dy"], t["h"], t[target], dresidual=t["dres"])
        near(t[target], want, slack, torch.float16)


@gpu
@pytest.mark.parametrize("rows", [0, 1, 8, 9])
def test_layer_norm_few_rows(rows):
    buf = Buffers(rows)
    x = buf.put(buf.randn(rows, 320), torch.float16)
    out = buf.empty(rows, 320, torch.float16)
    before = trfn.tr_launch_count()
    trfn.tr_layer_norm(x, out)
    assert trfn.tr_launch_count() - before == (1 if rows else 0)
    _, y, slack = layer_exact(x, None, None, None, 1e-5)
    near(out, y, slack, torch.float16)
    dw, db = torch.full((320,), 9.0, device="cuda"), torch.full((320,), 9.0, device="cuda")
    ws = torch.empty(trfn.tr_layer_norm_backward_workspace_bytes(max(rows, 1), 320), dtype=torch.uint8, device="cuda")
    trfn.tr_layer_norm_backward(x, x, out, dweight=dw, dbias=db, workspace=ws)
    if rows == 0:
        assert dw.count_nonzero().item() == 0 and db.count_nonzero().item() == 0


def test_layer_norm_workspace_never_shrinks():
    L = _native.lib()
    for cols in (1, 60, 500, 505, 506, 511, 512, 513, 1017, 1024, 2047, 4096, 4097, 32768):
        last = 0
        for rows in (1, 2, 7, 8, 9, 100, 303, 304, 305, 900, 912, 913, 5000, 10 ** 6):
            now = L.tr_layer_norm_backward_workspace_bytes(rows, cols)
            assert now >= last and now > 0
            last = now
    assert L.tr_layer_norm_backward_workspace_bytes(5, 32769) == 0


X, R, O, H, W, B, S, Z = (0x10000000 * (i + 1) for i in range(8))


@pytest.mark.parametrize("change,status", [
    ({}, None),
    ({"x": None}, INVALID), ({"out": None}, INVALID), ({"x": X + 1}, INVALID), ({"dtype": 3}, INVALID), ({"dtype": 9}, INVALID),
    ({"out_dtype": 0}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"rows": -1}, INVALID),
    ({"cols": 0}, INVALID), ({"cols": 32769}, NOT_SUPPORTED), ({"rows": 1 << 31}, NOT_SUPPORTED), ({"weight": W + 2}, INVALID),
    ({"bias": B + 1}, INVALID), ({"out": X + 2}, INVALID), ({"out": W}, INVALID), ({"out": B}, INVALID), ({"out_stride": 60}, INVALID),
    ({"x_stride": -1}, INVALID), ({"residual": None}, INVALID), ({"residual_out": O}, INVALID), ({"residual_out": B}, INVALID),
    ({"out_dtype": 3, "scale": None}, INVALID), ({"out_dtype": 3, "scale": B}, INVALID), ({"out_dtype": 3, "scale": X}, INVALID),
    ({"rows": 0}, OK),
])
def test_layer_norm_refusals(change, status):
    a = dict(x=X, residual=R, weight=W, bias=B, out=O, residual_out=H, scale=S, rows=8, cols=64, x_stride=64, residual_stride=64,
             out_stride=64, residual_out_stride=64, dtype=1, out_dtype=1, eps=1e-5, stream=None)
    a.update(change)
    if status is not None:
        assert _native.lib().tr_layer_norm(*a.values()) == status


@pytest.mark.parametrize("change,status", [
    ({"dy": None}, INVALID), ({"h": None}, INVALID), ({"dx": None}, INVALID), ({"dtype": 3}, INVALID), ({"eps": float("inf")}, INVALID),
    ({"workspace": None}, INVALID), ({"workspace": Z + 8}, INVALID), ({"dweight": None, "workspace": None}, INVALID),
    ({"dbias": W + 0x100}, INVALID), ({"dbias": S + 128}, INVALID), ({"dweight": Z}, INVALID), ({"dbias": Z + 256}, INVALID),
    ({"dbias": X}, INVALID), ({"dx": X + 2}, INVALID), ({"dx": W}, INVALID), ({"cols": 40000}, NOT_SUPPORTED),
    ({"rows": 0, "dweight": None, "dbias": None}, OK), ({"rows": 0, "dbias": S + 64}, INVALID),
])
def test_layer_norm_backward_refusals(change, status):
    a = dict(dy=X, h=H, weight=W, dresidual=R, dx=O, dweight=S, dbias=B, rows=8, cols=96, dy_stride=96, h_stride=96,
             dresidual_stride=96, dx_stride=96, dtype=1, eps=1e-5, workspace=Z, stream=None)
    a.update(change)
    if change.get("dbias") == W + 0x100:
        a["weight"] = W
    assert _native.lib().tr_layer_norm_backward(*a.values()) == status


# ---------------------------------------------------------------------- rotary ---

def frequencies(rot, base, scaling, factor, trained):
    if scaling == trfn.ROTARY_BASE:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * k / rot) for k in range(rot // 2)]
    if scaling == trfn.ROTARY_LINEAR:
        return [v / factor for v in f], 1.0
    if scaling != trfn.ROTARY_PARTS:
        return f, 1.0
    keep = [min(max((trained * v / (2 * math.pi) - 1) / 31, 0), 1) for v in f]
    return [v * (k + (1 - k) / factor) for v, k in zip(f, keep)], 0.1 * math.log(factor) + 1


@pytest.mark.parametrize("scaling", [trfn.ROTARY_UNSCALED, trfn.ROTARY_LINEAR, trfn.ROTARY_BASE, trfn.ROTARY_PARTS])
@pytest.mark.parametrize("rot", [4, 34, 64, 128, 512])
def test_rotary_frequencies(rot, scaling):
    f, m = trfn.tr_rotary_frequencies(rot, base=500000.0, scaling=scaling, factor=7.5, trained=8192)
    want, want_m = frequencies(rot, 500000.0, scaling, 7.5, 8192)
    assert len(f) == rot // 2 and m == pytest.approx(want_m, rel=2e-7)
    assert list(f) == pytest.approx(want, rel=1e-13)


def test_rotary_frequencies_at_their_ends():
    plain = list(trfn.tr_rotary_frequencies(64)[0])
    assert plain[0] == 1.0
    far = list(trfn.tr_rotary_frequencies(64, scaling=trfn.ROTARY_BASE, factor=16.0)[0])
    assert far[0] == 1.0 and far[-1] == pytest.approx(plain[-1] / 16, rel=1e-12)
    parts = list(trfn.tr_rotary_frequencies(64, scaling=trfn.ROTARY_PARTS, factor=16.0, trained=2048)[0])
    assert parts[0] == 1.0 and parts[-1] == pytest.approx(plain[-1] / 16, rel=1e-12)
    assert list(trfn.tr_rotary_frequencies(64, scaling=trfn.ROTARY_PARTS, factor=1.0, trained=2048)[0]) == pytest.approx(plain, rel=1e-15)


@pytest.mark.parametrize("args,status", [
    ((0, 1e4, 0, 1.0, 0), INVALID), ((3, 1e4, 0, 1.0, 0), INVALID), ((64, 1.0, 0, 1.0, 0), INVALID), ((64, float("nan"), 0, 1.0, 0), INVALID),
    ((64, 1e4, 4, 1.0, 0), INVALID), ((64, 1e4, -1, 1.0, 0), INVALID), ((64, 1e4, 1, 0.5, 0), INVALID), ((64, 1e4, 1, float("inf"), 0), INVALID),
    ((2, 1e4, 2, 2.0, 0), INVALID), ((64, 1e4, 3, 2.0, 0), INVALID), ((64, 1e308, 2, 1e300, 0), INVALID), ((514, 1e4, 0, 1.0, 0), NOT_SUPPORTED),
    ((64, 1e4, 0, 0.0, 0), OK),
])
def test_rotary_frequency_refusals(args, status):
    f, m = (ctypes.c_double * 600)(), ctypes.c_float()
    assert _native.lib().tr_rotary_frequencies(*args, f, ctypes.byref(m)) == status
    assert _native.lib().tr_rotary_frequencies(*args, None, ctypes.byref(m)) == INVALID
    assert _native.lib().tr_rotary_frequencies(*args, f, None) == INVALID


def rotary_exact(x, heads, freqs, positions, layout, magnitude, inverse):
    """The turned values, and |a| + |b| of their pairs."""
    tokens, cols = x.shape
    half = len(freqs)
    angle = positions.double()[:, None] * torch.tensor(list(freqs), dtype=torch.float64, device="cuda")
    c, s = angle.cos()[:, None] * magnitude, angle.sin()[:, None] * magnitude * (-1 if inverse else 1)
    v = x.double().reshape(tokens, heads, cols // heads).clone()
    size = torch.zeros_like(v)
    at = torch.arange(half, device="cuda")
    lo, hi = (at, at + half) if layout == trfn.ROTARY_HALVES else (2 * at, 2 * at + 1)
    a, b = v[:, :, lo].clone(), v[:, :, hi].clone()
    v[:, :, lo], v[:, :, hi] = a * c - b * s, b * c + a * s
    size[:, :, lo] = size[:, :, hi] = (a.abs() + b.abs()) * abs(magnitude)
    return v.reshape(tokens, cols), size.reshape(tokens, cols)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("heads,dim,rot", [(1, 2, 2), (3, 64, 64), (2, 128, 128), (5, 128, 32), (7, 80, 40), (2, 33, 30), (40, 96, 64),
                                           (3, 70, 62), (1, 256, 256), (2, 600, 512), (17, 16, 16), (2, 24, 8)])
def test_rotary_sizes(heads, dim, rot, dtype):
    buf = Buffers(dim + rot)
    freqs, _ = trfn.tr_rotary_frequencies(rot)
    for tokens, pad, shift in ((1, 0, 0), (29, 0, 0), (13, 16, 0), (11, 3, 1), (10, 6, 2)):
        x = buf.put(buf.randn(tokens, heads * dim), dtype, pad, shift)
        positions = torch.randint(0, 5000, (tokens,), generator=buf.g, device="cuda").to(torch.int32)
        for layout in (trfn.ROTARY_HALVES, trfn.ROTARY_PAIRS):
            for inverse in (False, True):
                out = buf.empty(tokens, heads * dim, dtype, pad, shift)
                trfn.tr_rotary(x, out, heads, freqs, positions=positions, layout=layout, magnitude=1.25, inverse=inverse)
                want, size = rotary_exact(x, heads, freqs, positions, layout, 1.25, inverse)
                near(out, want, 2.0 ** -21 * size, dtype)
                rest = x.reshape(tokens, heads, dim)[:, :, rot:]
                assert torch.equal(out.reshape(tokens, heads, dim)[:, :, rot:], rest)   # copied, not computed
                same = buf.put(x, dtype, pad, shift)
                trfn.tr_rotary(same, same, heads, freqs, positions=positions, layout=layout, magnitude=1.25, inverse=inverse)
                assert torch.equal(same, out)
        buf.check_around()


@gpu
@pytest.mark.parametrize("scaling", [trfn.ROTARY_UNSCALED, trfn.ROTARY_LINEAR, trfn.ROTARY_BASE, trfn.ROTARY_PARTS])
def test_rotary_far_positions(scaling):
    """Any 32-bit position: steps of a binary32 angle there would be 128 radians."""
    buf = Buffers(3)
    at = [0, 1, 2, 4095, 70001, 999999, 16777217, 123456789, 2 ** 31 - 1, -1, -77, -2 ** 31]
    positions = torch.tensor(at, dtype=torch.int32, device="cuda")
    x = buf.randn(len(at), 4 * 64)
    freqs, magnitude = trfn.tr_rotary_frequencies(64, scaling=scaling, factor=9.0, trained=4096)
    out = torch.empty_like(x)
    trfn.tr_rotary(x, out, 4, freqs, positions=positions, magnitude=magnitude)
    want, size = rotary_exact(x, 4, freqs, positions, trfn.ROTARY_HALVES, magnitude, False)
    # (the 64-bit angle, and 2^-53 of a frequency's turns, at positions of 2^31: 2^31 * 2^-52 radians)
    near(out, want, (2.0 ** -21 + 2.0 ** -20) * size, torch.float32)


@gpu
def test_rotary_without_positions_and_back():
    buf = Buffers(4)
    x = buf.randn(300, 6 * 128)
    freqs, _ = trfn.tr_rotary_frequencies(96)
    a, b, c = (torch.empty_like(x) for _ in range(3))
    trfn.tr_rotary(x, a, 6, freqs)
    trfn.tr_rotary(x, b, 6, list(freqs), positions=torch.arange(300, dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b)
    trfn.tr_rotary(a, c, 6, freqs, inverse=True)
    assert float((c - x).abs().max()) < 2.0 ** -18
    # the gradient is the transpose: <R x, y> = <x, R^T y>
    y = buf.randn(300, 6 * 128)
    trfn.tr_rotary(y, c, 6, freqs, magnitude=1.5, inverse=True)
    trfn.tr_rotary(x, b, 6, freqs, magnitude=1.5)
    left, right = (b.double() * y.double()).sum(1), (x.double() * c.double()).sum(1)
    assert float((left - right).abs().max()) < 2.0 ** -20 * 1.5 * float((x.double().abs() * y.double().abs()).sum(1).max()) * 2


@gpu
def test_rotary_rows_without_tokens_and_values_without_numbers():
    freqs, _ = trfn.tr_rotary_frequencies(8)
    x = torch.randn(4, 16, device="cuda").half()
    before = trfn.tr_launch_count()
    trfn.tr_rotary(x[:0], x[:0], 1, freqs)
    assert trfn.tr_launch_count() == before
    x[1, 12:] = float("nan")
    x[2, 0] = float("inf")
    out = torch.empty_like(x)
    trfn.tr_rotary(x, out, 1, freqs)
    assert bool(out[1, 12:].isnan().all()) and not bool(out[1, :12].isnan().any())
    bad = ~out[2].isfinite()
    assert bool(bad[[0, 4]].all()) and int(bad.sum()) == 2


F8 = (ctypes.c_double * 256)(*[0.5] * 256)
F_NAN = (ctypes.c_double * 256)(*[float("nan")] * 256)


@pytest.mark.parametrize("change,status", [
    ({"x": None}, INVALID), ({"out": None}, INVALID), ({"freqs": None}, INVALID), ({"freqs": F_NAN}, INVALID), ({"positions": W + 2}, INVALID),
    ({"tokens": -1}, INVALID), ({"heads": 0}, INVALID), ({"rot": 3}, INVALID), ({"rot": 0}, INVALID), ({"rot": 66}, INVALID),
    ({"dtype": 3}, INVALID), ({"layout": 2}, INVALID), ({"magnitude": float("inf")}, INVALID), ({"out": X + 2}, INVALID),
    ({"out": X, "out_stride": 130}, INVALID), ({"out_stride": 100}, INVALID), ({"positions": O}, INVALID), ({"x": X + 1}, INVALID),
    ({"heads": 65536}, NOT_SUPPORTED), ({"tokens": 1 << 31}, NOT_SUPPORTED), ({"dim": 1024, "rot": 514}, NOT_SUPPORTED), ({"tokens": 0}, OK),
])
def test_rotary_refusals(change, status):
    a = dict(x=X, out=O, positions=W, freqs=F8, tokens=8, heads=2, dim=64, rot=64, x_stride=128, out_stride=128, dtype=1, layout=0,
             magnitude=1.0, inverse=0, stream=None)
    a.update(change)
    assert _native.lib().tr_rotary(*a.values()) == status


# ------------------------------------------------------------------- attention ---

class Problem:
    """q, k, v of packed sequences inside buffers full of NaN, and the answer in 64 bits."""

    def __init__(self, seed, lq, lk, heads, kv_heads, dim, dtype, pad=0, shift=0, gap=0, slot=0, sharp=1.0):
        self.buf = b = Buffers(seed)
        self.lq, self.lk, self.heads, self.kv_heads, self.dim, self.dtype = lq, lk, heads, kv_heads, dim, dtype
        self.q_at, self.k_at = self.places(lq, gap, 0), self.places(lk, gap, slot)
        self.q = b.empty(self.q_at[-1], heads * dim, dtype, pad, shift)
        self.k = b.empty(self.k_at[-1], kv_heads * dim, dtype, pad, shift)
        self.v = b.empty(self.k_at[-1], kv_heads * dim, dtype, pad, shift)
        self.out = b.empty(self.q_at[-1], heads * dim, dtype, pad, shift)
        for s, n in enumerate(lq):
            self.q[self.q_at[s]:self.q_at[s] + n] = (b.randn(n, heads * dim) * sharp).to(dtype)
        for s, n in enumerate(lk):
            self.k[self.k_at[s]:self.k_at[s] + n] = b.randn(n, kv_heads * dim).to(dtype)
            self.v[self.k_at[s]:self.k_at[s] + n] = b.randn(n, kv_heads * dim).to(dtype)
        self.gaps = gap or slot

    @staticmethod
    def places(lengths, gap, slot):
        at = [0]
        for n in lengths:
            at.append(at[-1] + (slot if slot else n + gap))
        return at

    def arrays(self):
        def dev(v):
            return torch.tensor(v, dtype=torch.int32, device="cuda")
        q = {"q_starts": dev(self.q_at), "k_starts": dev(self.k_at)}
        if self.gaps:
            q.update(q_lengths=dev(self.lq), k_lengths=dev(self.lk))
        return q

    def run(self, causal, out=None, **more):
        n = trfn.tr_attention_workspace_bytes(self.q.size(0), len(self.lq), self.heads, self.kv_heads, self.dim)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        out = self.out if out is None else out
        trfn.tr_attention(self.q, self.k, self.v, out, self.heads, self.kv_heads, causal=causal, workspace=ws, **{**self.arrays(), **more})
        return out

    def check(self, out, causal, scale=None):
        group, d = self.heads // self.kv_heads, self.dim
        scale = d ** -0.5 if scale is None else scale
        unit = UNIT[self.dtype] if self.dtype != torch.float32 else 0.0
        for s, (nq, nk) in enumerate(zip(self.lq, self.lk)):
            if nq == 0:
                continue
            got = out[self.q_at[s]:self.q_at[s] + nq].double().reshape(nq, self.heads, d)
            q = self.q[self.q_at[s]:self.q_at[s] + nq].double().reshape(nq, self.heads, d)
            k = self.k[self.k_at[s]:self.k_at[s] + nk].double().reshape(nk, self.kv_heads, d)
            v = self.v[self.k_at[s]:self.k_at[s] + nk].double().reshape(nk, self.kv_heads, d)
            sees = torch.ones(nq, nk, dtype=torch.bool, device="cuda")
            if causal:
                sees = sees.tril(nk - nq)
            some = sees.any(1)
            assert bool((got[~some] == 0).all()), "a query that sees nothing gets zeros"
            if not bool(some.any()):
                continue
            for h in range(self.heads):
                x = q[some, h] @ k[:, h // group].t() * scale
                size = (q[some, h].abs() @ k[:, h // group].abs().t() * abs(scale)).masked_fill(~sees[some], 0).amax(1, keepdim=True)
                x = x.masked_fill(~sees[some], -math.inf)
                p = torch.softmax(x, 1)
                vh = v[:, h // group]
                want = p @ vh
                a = p @ vh.abs()
                delta = 2.0 ** -18 * size + 2.0 ** -21 * (size + 1)
                slack = a * (2 * delta + unit + (nk / 16 + 64) * 2.0 ** -22)
                if self.dtype == torch.float16:
                    slack = slack + 2.0 ** -25 * p.amax(1, keepdim=True) * (sees[some].double() @ vh.abs())
                near(got[some, h], want, slack, self.dtype)


# queries and keys of each sequence
LENGTHS = {
    "one": ([1], [1]),
    "tile": ([128], [128]),
    "odd": ([37], [37]),
    "long": ([300], [300]),
    "packed": ([3, 0, 130, 1, 257, 64], [3, 0, 130, 1, 257, 64]),
    "longer_keys": ([5, 129, 40], [300, 129, 513]),
    "fewer_keys": ([300, 7, 40, 2], [200, 0, 1, 1]),
    "step": ([1, 1, 1, 1], [1000, 1, 0, 385]),
    "few_new": ([4, 2], [700, 2]),
}


@gpu
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("lengths", LENGTHS)
def test_attention_lengths(lengths, dtype, causal):
    lq, lk = LENGTHS[lengths]
    for heads, kv_heads, dim in ((4, 2, 64), (3, 3, 128), (6, 1, 32)):
        p = Problem(len(lengths), lq, lk, heads, kv_heads, dim, dtype, gap=2, pad=8)
        p.check(p.run(causal), causal)
        kept = torch.full_like(p.out, 5.0)
        p.run(causal, out=kept)
        for s, n in enumerate(lq):
            assert bool((kept[p.q_at[s] + n:p.q_at[s + 1]] == 5.0).all()), "rows of no sequence are left as they were"
        p.buf.check_around()


@gpu
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("dim", [1, 3, 8, 16, 24, 40, 64, 72, 80, 96, 104, 120, 128, 129, 136, 200, 256])
def test_attention_head_lengths(dim, dtype, causal):
    for lq, lk, pad, shift in (([140, 9], [140, 9], 0, 0), ([1], [333], 8, 8), ([20], [150], 3, 1)):
        p = Problem(dim, lq, lk, 2, 1, dim, dtype, pad=pad, shift=shift)
        p.check(p.run(causal), causal)
        p.buf.check_around()


@gpu
@pytest.mark.parametrize("dtype", SHORT, ids=name_of)
@pytest.mark.parametrize("group", [1, 2, 3, 5, 6, 7, 8, 12, 16, 31, 64, 65, 100])
def test_attention_groups(group, dtype):
    for lq, lk in (([1, 1], [200, 3]), ([70], [70]), ([3, 150], [300, 150])):
        p = Problem(group, lq, lk, 2 * group, 2, 64, dtype)
        p.check(p.run(True), True)
        p.buf.check_around()


@gpu
@pytest.mark.parametrize("dtype", SHORT, ids=name_of)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("keys", [1, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 383, 385, 640])
def test_attention_key_counts(keys, dim, dtype):
    p = Problem(keys, [keys, 2], [keys, keys], 2, 2, dim, dtype)
    for causal in (False, True):
        p.check(p.run(causal), causal)
    p.buf.check_around()


@gpu
@pytest.mark.parametrize("dtype", SHORT, ids=name_of)
@pytest.mark.parametrize("dim,heads,kv_heads,lq,lk,causal", [
    (128, 8, 2, [2048], [2048], True),
    (128, 4, 4, [1500, 700], [1500, 700], False),
    (64, 12, 12, [196] * 30, [196] * 30, False),
    (64, 8, 1, [1000, 1, 30], [4000, 3000, 2500], True),
    (80, 10, 5, [911], [1822], True),
    (128, 32, 8, [1] * 5, [9000, 100, 0, 1, 5000], True),
    (128, 8, 1, [1], [20000], True),
    (64, 2, 2, [1], [33333], False),
])
def test_attention_large(dim, heads, kv_heads, lq, lk, causal, dtype):
    p = Problem(dim, lq, lk, heads, kv_heads, dim, dtype, slot=0)
    first = p.run(causal).clone()
    p.check(first, causal)
    assert torch.equal(p.run(causal), first), "the same call gives the same bits"
    p.buf.check_around()


@gpu
def test_attention_many_sequences():
    g = torch.Generator().manual_seed(3)
    for n, top in ((700, 40), (3000, 5)):
        lq = torch.randint(0, top, (n,), generator=g).tolist()
        p = Problem(n, lq, lq, 2, 1, 64, torch.float16)
        p.check(p.run(True), True)
        lk = torch.randint(0, 300, (n,), generator=g).tolist()
        p = Problem(n, [1] * n, lk, 2, 1, 64, torch.float16)
        p.check(p.run(True), True)


@gpu
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_of_empty_sequences_between_long_ones(dim):
    """Many items in a row that have no keys, or few, between items that have: more than there are places for
    what a part of the kernel tells the others."""
    p = Problem(dim, [1] * 24, [2000] * 12 + [0] + [2000] * 11, 32, 16, dim, torch.bfloat16)
    p.check(p.run(True), True)
    p = Problem(dim, [300] + [40] * 20 + [2] * 9, [700] + [0] * 20 + [500] * 9, 12, 12, dim, torch.float16)
    p.check(p.run(False), False)
    p = Problem(dim, [500, 90, 700, 3, 800], [100, 0, 900, 1, 300], 24, 24, dim, torch.float16)
    p.check(p.run(True), True)
    p.buf.check_around()
    assert trfn.tr_device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("sharp", [0.0, 8.0, 100.0])
def test_attention_of_even_and_sharp_scores(sharp, dtype):
    """From equal weights to one key that takes all, growing maxima included."""
    p = Problem(int(sharp), [200], [900], 2, 1, 64, dtype, sharp=sharp)
    p.check(p.run(False), False)
    # scores that grow along the keys: the maximum moves with every block
    p = Problem(7, [130], [900], 1, 1, 64, dtype)
    p.k[:] = 0
    p.k[:, 0] = torch.arange(900, device="cuda").to(dtype) / 8
    p.q[:, 0] = 8.0
    p.check(p.run(False), False)
    p.q[:, 0] = -8.0
    p.check(p.run(True), True)


@gpu
@pytest.mark.parametrize("dtype", SHORT, ids=name_of)
def test_attention_of_one_key_that_has_all_the_weight(dtype):
    """A maximum that grows by less than what makes the kernel start over (2^8) leaves the largest weight above 1 and
    rounded; the sum takes the same rounded weight, so the output is nearly that key's value within the output's
    own rounding: the rounding of its weight reaches it only through the other key's share, e^-gap."""
    p = Problem(6, [64], [256], 1, 1, 64, dtype)
    p.q[:] = 0
    p.k[:] = 0
    p.q[:, 0] = 8.0           # scores are the keys' first values
    p.k[:, 0] = -60.0
    p.k[0, 0] = -20.0         # the first block's maximum
    for top in (-15.9, -15.1, -14.9, -14.7):
        p.k[200, 0] = top
        p.check(p.run(False), False)
        gap = math.exp(float(p.k[200, 0].double() + 20))
        v = p.v.double()
        want = (v[200] * gap + v[0]) / (gap + 1)
        near(p.out, want.expand(64, 64), v.abs().max() * (4 * UNIT[dtype] / gap + 2.0 ** -18), dtype)


@gpu
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.5, 1e-30])
def test_attention_scales(scale):
    for dtype in TYPES:
        p = Problem(5, [60, 3], [200, 5], 2, 2, 64, dtype)
        p.check(p.run(True, scale=scale), True, scale=scale)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attention_of_what_is_not_seen(value, dim, dtype):
    """Keys and values that a query does not see do not reach it; those that it sees do."""
    for n, at in ((300, 170), (40, 39), (257, 256), (128, 64)):
        p = Problem(n, [n], [n], 2, 2, dim, dtype)
        p.v[at, 5] = value
        p.k[at] = 3.0
        out = p.run(True).clone()
        q, k, v = p.q[:at].clone(), p.k[:at].clone(), p.v[:at].clone()
        small = Problem(n, [at], [at], 2, 2, dim, dtype)
        small.q, small.k, small.v = q, k, v
        small.check(out[:at], True)
        got = out[at:, 5]
        assert bool((got.isnan() if math.isnan(value) else got == value).all()), "values that are seen count"
        others = [c for c in range(2 * dim) if c != 5]
        assert bool(out[:, others].isfinite().all())
        p.v[at, 5] = 1.0
        p.k[at, 3] = value
        out = p.run(True)
        small.check(out[:at], True)
        assert bool(out[at:, :dim].isnan().any(1).all()) or not math.isnan(value)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
def test_attention_of_scores_without_numbers(dtype):
    p = Problem(2, [70], [150], 2, 1, 64, dtype)
    p.q[3] = float("nan")
    p.q[5, :64] = float("inf")
    out = p.run(False)
    assert bool(out[3].isnan().all()) and bool(out[5, :64].isnan().all())
    keep = [i for i in range(70) if i not in (3, 5)]
    assert bool(out[keep].isfinite().all())


@gpu
@pytest.mark.parametrize("dtype", SHORT, ids=name_of)
def test_attention_keys_shared_by_sequences(dtype):
    p = Problem(8, [50, 1, 130], [300], 4, 2, 64, dtype)
    dev = {"q_starts": torch.tensor([0, 50, 51, 181], dtype=torch.int32, device="cuda"),
           "k_starts": torch.tensor([0, 0, 100, 0], dtype=torch.int32, device="cuda"),
           "k_lengths": torch.tensor([300, 300, 200], dtype=torch.int32, device="cuda")}
    p.gaps = 0
    p.q_at = [0, 50, 51, 181]
    p.k_at, p.lk = [0, 0, 100, 300], [300, 300, 200]
    out = torch.empty_like(p.out)
    n = trfn.tr_attention_workspace_bytes(181, 3, 4, 2, 64)
    trfn.tr_attention(p.q, p.k, p.v, out, 4, 2, causal=True, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"), **dev)
    p.check(out, True)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=name_of)
def test_attention_of_arrays_that_leave_the_matrices(dtype):
    """Starts and lengths are cut to the matrices on the GPU: nothing outside them is read or written."""
    p = Problem(9, [100], [100], 2, 2, 64, dtype)
    n = trfn.tr_attention_workspace_bytes(100, 3, 2, 2, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for starts, lengths, want in (
            ([-5, 40, 400, 7], None, ([40, 60, 0], [0, 40, 100])),
            ([0, 90, 100, 2 ** 31 - 1], [2 ** 31 - 1, -3, 5], ([100, 0, 0], [0, 90, 100])),
            ([60, 10, 5, 3], None, ([0, 0, 0], [60, 10, 5])),
            ([-2 ** 31, 2 ** 31 - 1, -1, 0], [50, 2 ** 31 - 1, 20], ([50, 0, 20], [0, 100, 0]))):
        p.lq = p.lk = want[0]
        p.q_at = p.k_at = want[1]
        t = torch.tensor(starts, dtype=torch.int32, device="cuda")
        ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        p.out.fill_(3.0)
        trfn.tr_attention(p.q, p.k, p.v, p.out, 2, 2, t, q_lengths=ln, workspace=ws)
        if starts[0] == -2 ** 31:   # two sequences of one start: the rows get either's output
            p.lq, p.lk = [0, 0, 0], [0, 0, 0]
        p.check(p.out, False)
        covered = torch.zeros(100, dtype=torch.bool, device="cuda")
        for a, m in zip(*[want[1], want[0]]):
            covered[a:a + m] = True
        assert bool((p.out[~covered] == 3.0).all())
        p.buf.check_around()


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=name_of)
def test_attention_of_repeated_and_interleaved_rows(dtype):
    """One key row that is repeated (stride 0), and queries, keys, values and outputs as column blocks of one buffer."""
    p = Problem(4, [70, 9], [70, 9], 2, 2, 64, dtype)
    row = p.buf.randn(1, 128).to(dtype)
    p.k = row.expand(79, 128)
    p.check(p.run(True), True)
    p.v = row.expand(79, 128)
    p.check(p.run(False), False)
    whole = torch.zeros(79, 4 * 128, dtype=dtype, device="cuda")
    whole[:, :384] = p.buf.randn(79, 384).to(dtype)
    p.q, p.k, p.v, out = (whole[:, i * 128:(i + 1) * 128] for i in range(4))
    kept = whole[:, :384].clone()
    p.check(p.run(True, out=out), True)
    assert torch.equal(whole[:, :384], kept)


@gpu
def test_attention_of_no_rows_and_no_sequences():
    e = torch.empty(0, 128, device="cuda", dtype=torch.float16)
    before = trfn.tr_launch_count()
    trfn.tr_attention(e, e, e, e, 2, 2, torch.zeros(2, dtype=torch.int32, device="cuda"))
    q = torch.ones(4, 128, device="cuda", dtype=torch.float16)
    out = torch.full_like(q, 2.0)
    trfn.tr_attention(q, q, q, out, 2, 2, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert trfn.tr_launch_count() == before and bool((out == 2.0).all())
    # queries without any key row
    for dtype in TYPES:
        q, out, e = q.to(dtype), torch.full((4, 128), 2.0, device="cuda", dtype=dtype), torch.empty(0, 128, device="cuda", dtype=dtype)
        ws = torch.empty(trfn.tr_attention_workspace_bytes(4, 1, 2, 2, 64), dtype=torch.uint8, device="cuda")
        trfn.tr_attention(q, e, e, out, 2, 2, torch.tensor([0, 4], dtype=torch.int32, device="cuda"),
                          torch.tensor([0, 0], dtype=torch.int32, device="cuda"), workspace=ws)
        assert bool((out == 0).all())


@gpu
def test_attention_offsets_beyond_32_bits():
    """Rows of a cache whose bytes and values are beyond 2^32 from its start."""
    rows, stride = 600000, 8192
    cache = torch.zeros(rows, stride, dtype=torch.bfloat16, device="cuda")   # 9.8 GB
    g = torch.Generator(device="cuda").manual_seed(1)
    n = 700
    k, v = cache[:, :64], cache[:, 4096:4160]
    k[-n:] = torch.randn(n, 64, generator=g, device="cuda").bfloat16()
    v[-n:] = torch.randn(n, 64, generator=g, device="cuda").bfloat16()
    p = Problem(3, [3], [n], 4, 1, 64, torch.bfloat16)
    p.k, p.v = k[-n:], v[-n:]
    ws = torch.empty(trfn.tr_attention_workspace_bytes(3, 1, 4, 1, 64), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    trfn.tr_attention(p.q, k, v, p.out, 4, 1, torch.tensor([0, 3], **i32), torch.tensor([rows - n, rows], **i32), causal=True, workspace=ws)
    p.check(p.out, True)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16], ids=name_of)
def test_attention_captured_with_other_lengths(dtype):
    """A captured step reads the lengths of the moment; two graphs with workspaces of their own run at once."""
    cap, heads, dim = 2000, 4, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(cap, 2 * dim, generator=g, device="cuda").to(dtype) for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    graphs = []
    for _ in range(2):
        q = torch.randn(1, heads * dim, generator=g, device="cuda").to(dtype)
        out, lengths = torch.empty_like(q), torch.tensor([1], **i32)
        ws = torch.empty(trfn.tr_attention_workspace_bytes(1, 1, heads, 2, dim), dtype=torch.uint8, device="cuda")
        starts_q, starts_k = torch.tensor([0, 1], **i32), torch.tensor([0, cap], **i32)
        args = (q, k, v, out, heads, 2, starts_q, starts_k, None, lengths, True, None, ws)
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            trfn.tr_attention(*args)
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                trfn.tr_attention(*args)
        graphs.append((graph, stream, q, out, lengths, args))
    torch.cuda.synchronize()
    for n in (1, 128, 1999, 777, 0):
        for graph, stream, q, out, lengths, args in graphs:
            lengths.fill_(n)
            out.fill_(9.0)
        torch.cuda.synchronize()
        for graph, stream, *_ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, q, out, lengths, args in graphs:
            p = Problem(1, [1], [n], heads, 2, dim, dtype)
            p.q, p.k, p.v = q, k[:n], v[:n]
            p.check(out, True)


def test_attention_workspace_never_shrinks():
    L = _native.lib()
    for heads, kv, dim in ((1, 1, 64), (32, 8, 128), (12, 12, 40), (64, 1, 128)):
        last = 0
        for rows in (1, 2, 100, 128, 129, 5000, 10 ** 6):
            now = L.tr_attention_workspace_bytes(rows, 4, heads, kv, dim)
            assert now >= last
            last = now
    assert L.tr_attention_workspace_bytes(0, 4, 8, 8, 64) == 0
    assert L.tr_attention_workspace_bytes(4, 4, 8, 3, 64) == 0


KV = 0x90000000


@pytest.mark.parametrize("change,status", [
    ({"q": None}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID), ({"out": None}, INVALID), ({"q_starts": None}, INVALID),
    ({"k_starts": None}, INVALID), ({"q_starts": W + 1}, INVALID), ({"q_lengths": W + 2}, INVALID), ({"dtype": 3}, INVALID),
    ({"heads": 3}, INVALID), ({"heads": 0}, INVALID), ({"kv_heads": 0}, INVALID), ({"dim": 0}, INVALID), ({"scale": float("nan")}, INVALID),
    ({"sequences": -1}, INVALID), ({"out": X}, INVALID), ({"out": R}, INVALID), ({"out": W}, INVALID), ({"out": S}, INVALID),
    ({"out_stride": 255}, INVALID), ({"q_stride": -1}, INVALID), ({"q": X + 1}, INVALID), ({"dim": 257}, NOT_SUPPORTED),
    ({"heads": 65536}, NOT_SUPPORTED), ({"sequences": 1 << 21}, NOT_SUPPORTED), ({"q_rows": 1 << 31}, NOT_SUPPORTED),
    ({"k_rows": 1 << 31}, NOT_SUPPORTED), ({"q_rows": 0}, OK), ({"sequences": 0}, OK),
])
def test_attention_refusals(change, status):
    a = dict(q=X, k=R, v=H, out=O, q_starts=W, k_starts=B, q_lengths=None, k_lengths=S, q_rows=8, k_rows=100, sequences=3, heads=4,
             kv_heads=2, dim=64, q_stride=256, k_stride=128, v_stride=128, out_stride=256, dtype=1, scale=0.1, causal=1, workspace=Z,
             stream=None)
    a.update(change)
    assert _native.lib().tr_attention(*a.values()) == status


@gpu
def test_binding_refusals():
    q = torch.ones(4, 128, device="cuda", dtype=torch.float16)
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, trfn.tr_attention_workspace_bytes(4, 1, 2, 2, 64)), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    trfn.tr_attention(q, q, q, out, 2, 2, starts, workspace=ws)
    for bad in ({"q": q.float()}, {"heads": 3}, {"kv_heads": 4}, {"q_starts": starts.long()}, {"q_starts": starts.cpu()}, {"k": q.cpu()},
                {"k_starts": starts[:1]}, {"k_lengths": starts[:1]}, {"v": q[:2]}, {"out": q}):
        a = dict(q=q, k=q, v=q, out=out, heads=2, kv_heads=2, q_starts=starts, workspace=ws)
        a.update(bad)
        with pytest.raises(TrError):
            trfn.tr_attention(**a)
    freqs, _ = trfn.tr_rotary_frequencies(64)
    for bad in ({"heads": 3}, {"freqs": freqs, "heads": 4}, {"positions": starts}, {"positions": torch.arange(4, device="cuda")},
                {"out": out.float()}, {"layout": 7}, {"magnitude": float("nan")}):
        a = dict(x=q, out=out, heads=2, freqs=freqs)
        a.update(bad)
        with pytest.raises(TrError):
            trfn.tr_rotary(**a)
    with pytest.raises(TrError):
        trfn.tr_rotary_frequencies(7)
    with pytest.raises(TrError):
        trfn.tr_layer_norm(q, out, bias=torch.ones(64, device="cuda"))
    with pytest.raises(TrError):
        trfn.tr_layer_norm_backward(q, q, out, dbias=torch.ones(128, device="cuda"))


# ------------------------------------------------- waits, streams and kernels before ---

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
@pytest.mark.parametrize("what", ["layer_norm", "layer_norm_backward", "rotary", "attention", "plain_attention"])
def test_a_kernel_that_releases_early_is_waited_for(early_release, what):
    """The kernel before lets the operator start and writes its input last of all, after longer than the limit of
    the operator's own waits."""
    rows, cols = 300, 256
    raw = torch.zeros(rows * cols * 2, dtype=torch.int8, device="cuda")
    x, out = raw.view(torch.bfloat16).view(rows, cols), torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    ws = torch.empty(trfn.tr_attention_workspace_bytes(rows, 2, 4, 4, 64), dtype=torch.uint8, device="cuda")
    freqs, _ = trfn.tr_rotary_frequencies(64)

    def run():
        if what == "layer_norm":
            trfn.tr_layer_norm(x, out)
        elif what == "layer_norm_backward":
            trfn.tr_layer_norm_backward(x, x, out)
        elif what == "rotary":
            trfn.tr_rotary(x, out, 4, freqs)
        elif what == "attention":
            trfn.tr_attention(x, x, x, out, 4, 4, starts, workspace=ws, scale=1e-3)
        else:
            trfn.tr_attention(x, x, x, out, 4, 4, starts, workspace=ws, scale=-1e-3)

    torch.cuda.synchronize()
    assert early_release(raw, 1_500_000_000) == 0
    run()
    torch.cuda.synchronize()
    got = out.clone()
    filled = (torch.arange(raw.numel(), device="cuda") * 7 % 251 - 125).to(torch.int8)
    assert torch.equal(raw, filled)
    out.zero_()
    run()
    assert torch.equal(got.view(torch.int16), out.view(torch.int16)) and trfn.tr_device_status() == 0


@gpu
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_whose_wait_runs_out(dim):
    """The first stage of the first CTA waits for an arrival that never comes (tr_tune_tiled's test hook): the
    launch ends by itself and reports it, and what it has written is right."""
    p = Problem(dim, [1500, 40, 900], [1500, 40, 900], 8, 4, dim, torch.bfloat16)
    want = p.run(False).clone()
    out = torch.full_like(want, float("nan"))
    assert trfn.tr_device_status(clear=True) == 0
    try:
        trfn.tr_tune_tiled(0, 0, 0, 64)
        t0 = time.perf_counter()
        p.run(False, out=out)
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        trfn.tr_tune_tiled(0, 0, 0, 0)
    assert 0.5 < elapsed < 30
    assert trfn.tr_device_status(clear=True) == 1
    written = ~out.isnan()
    assert not bool(written[0, 0]) and bool(written.any())
    assert torch.equal(out[written], want[written])
    assert torch.equal(p.run(False), want) and trfn.tr_device_status() == 0


@gpu
def test_two_streams_with_workspaces_of_their_own():
    problems = [Problem(s, [900, 3, 200], [900, 3, 200], 8, 2, 128, torch.bfloat16) for s in (1, 2)]
    want = [p.run(True).clone() for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    args = []
    for p in problems:
        n = trfn.tr_attention_workspace_bytes(p.q.size(0), 3, 8, 2, 128)
        args.append((p, p.arrays(), torch.empty(n, dtype=torch.uint8, device="cuda"), torch.zeros_like(p.out)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (p, arrays, ws, out) in zip(streams, args):
            trfn.tr_attention(p.q, p.k, p.v, out, 8, 2, causal=True, workspace=ws, stream=s, **arrays)
    torch.cuda.synchronize()
    for (p, _, _, out), w in zip(args, want):
        assert torch.equal(out, w)
    assert trfn.tr_device_status() == 0


@gpu
def test_attention_again_and_again_is_the_same():
    """Many launches one after the other, over sequences of every kind, with one workspace."""
    g = torch.Generator().manual_seed(11)
    for _ in range(12):
        n = int(torch.randint(1, 40, (1,), generator=g))
        kv, group, dim = [(1, 8, 128), (8, 1, 64), (4, 3, 96), (2, 5, 64)][int(torch.randint(0, 4, (1,), generator=g))]
        top = int(torch.randint(1, 1200, (1,), generator=g))
        lk = (torch.randint(0, top, (n,), generator=g) * (torch.rand(n, generator=g) < 0.8)).tolist()
        lq = lk if torch.rand(1, generator=g) < 0.5 else [1 + i % 3 for i in range(n)]
        p = Problem(n, lq, lk, kv * group, kv, dim, torch.float16)
        if sum(lq) == 0:
            continue
        first = p.run(True).clone()
        p.check(first, True)
        for _ in range(25):
            assert torch.equal(p.run(True), first)
    assert trfn.tr_device_status() == 0
