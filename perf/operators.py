"""Timed cases of the token-row operators: root-mean-square norm with the residual's addition (with an 8-bit output,
and its gradient), 8-bit quantisation of rows and reading them back, and the 8-bit integer matrix product with a
scale for each token and channel.

Tokens here are the 16x16 patches of normalised image batches (196 to a 224x224x3 image, 768 values each, 256 images
to a batch) and the hidden rows a network makes of them; serving takes one token at a time, training whole batches.
"""
import math

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -119   # rows whose largest magnitude is below this hold zeros in 8 bits
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token of a serving step: residual stream and norm, latency alone counts
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "residual": True, "q8": False, "pad": 0},
        # hidden rows of a training batch: 256 images x 196 patches
        {"name": "norm_batch", "op": "norm", "rows": 50176, "cols": 1024, "type": "f16", "residual": True, "q8": False, "pad": 0},
        # norm in front of an 8-bit product, 64 images; the 8-bit rows are read back as binary16
        {"name": "norm_q8_batch", "op": "norm", "rows": 12544, "cols": 4096, "type": "bf16", "residual": True, "q8": True, "pad": 0},
        # training: the norm's gradients over the batch, with the gradient that arrives along the residual stream
        {"name": "norm_grad_batch", "op": "grad", "rows": 50176, "cols": 1024, "type": "f16", "residual": True, "pad": 0},
        # training: an odd width inside a wider buffer, binary32
        {"name": "norm_grad_odd", "op": "grad", "rows": 1777, "cols": 999, "type": "f32", "residual": False, "pad": 5},
        # the batch's patches in 8 bits and back
        {"name": "quant_patches", "op": "quant", "rows": 50176, "cols": 768, "type": "f16", "pad": 0},
        # a small odd block inside a wider buffer
        {"name": "quant_odd", "op": "quant", "rows": 333, "cols": 1001, "type": "f32", "pad": 7},
        # one token through one layer: the weights are read once
        {"name": "product_token", "op": "product", "m": 1, "n": 4096, "k": 4096, "type": "bf16", "bias": False, "pad": 0},
        # a few sequences decoding together through a wide layer
        {"name": "product_few", "op": "product", "m": 16, "n": 16384, "k": 4096, "type": "f16", "bias": True, "pad": 0},
        # one image's patches through one layer
        {"name": "product_image", "op": "product", "m": 196, "n": 4096, "k": 1024, "type": "f16", "bias": True, "pad": 0},
        # patch embedding of the batch
        {"name": "product_patches", "op": "product", "m": 50176, "n": 1024, "k": 768, "type": "f16", "bias": True, "pad": 0},
        # a square layer over 64 images
        {"name": "product_large", "op": "product", "m": 12544, "n": 4096, "k": 4096, "type": "bf16", "bias": False, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    # about half the sizes as they fall (odd ones among them), half on a multiple of 16 where there is room
    if v > 64 and rng.random() < 0.5:
        v = v // 16 * 16
    return max(lo, min(hi, v))


def draw(rng):
    top = [work(c) for c in listed()]
    most_bytes, most_flops = max(w["bytes"] for w in top), max(w["flops"] for w in top)
    while True:
        op = rng.choice(["norm", "grad", "quant", "product", "product"])
        case = {"op": op}
        if op == "product":
            case.update(m=_log_int(rng, 1, 50176), n=_log_int(rng, 64, 16384), k=_log_int(rng, 64, 8192),
                        type=rng.choice(["f32", "f16", "bf16"]), bias=rng.random() < 0.5)
        else:
            case.update(rows=_log_int(rng, 1, 50176), cols=_log_int(rng, 64, 8192), type=rng.choice(["f32", "f16", "bf16"]))
            if op != "quant":
                case["residual"] = rng.random() < 0.7
            if op == "norm":
                case["q8"] = rng.random() < 0.5
        case["pad"] = rng.choice([0, 0, 0, 16, rng.randrange(1, 33)])
        w = work(case)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return case


def _wide(rows, cols, pad, dtype):
    """A (rows, cols) view of a buffer whose rows are cols + pad apart."""
    return torch.empty((rows, cols + pad), dtype=dtype, device="cuda")[:, :cols]


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pad, dtype = case["pad"], DTYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def fill(values, dt=dtype):
        t = _wide(values.shape[0], values.shape[1], pad, dt)
        t.copy_(values)
        return t

    s = {}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        # rows quantised from near-normal values: a spread of about a quarter of the range
        s["x"] = fill((normal(m, k) * 32).round_().clamp_(-127, 127), torch.int8)
        s["w"] = fill((normal(n, k) * 32).round_().clamp_(-127, 127), torch.int8)
        s["x_scale"] = 0.01 + 0.02 * torch.rand(m, generator=g, device="cuda")
        s["w_scale"] = (0.5 + torch.rand(n, generator=g, device="cuda")) * (0.03 / math.sqrt(k))
        s["bias"] = normal(n) * 0.1 if case["bias"] else None
        return s
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "quant":
        # normalised pixels, some of them erased to zero
        u = torch.randint(0, 256, (rows, cols), generator=g, device="cuda").float()
        v = (u / 255 - 0.45) / 0.226
        v[torch.rand((rows, cols), generator=g, device="cuda") < 0.1] = 0
        s["x"] = fill(v)
        return s
    s["weight"] = 1 + 0.1 * normal(cols)
    if case["op"] == "norm":
        s["x"] = fill(normal(rows, cols))
        # the stream has a few channels that are much larger than the rest
        loud = 1 + 7 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
        s["residual"] = fill(normal(rows, cols) * loud) if case["residual"] else None
    else:
        s["h"] = fill(normal(rows, cols) * 1.5)
        s["dy"] = fill(normal(rows, cols) * 0.1)
        s["dresidual"] = fill(normal(rows, cols) * 0.1) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    pad, dtype = case["pad"], DTYPES[case["type"]]
    # the buffers a program keeps beside its inputs
    if case["op"] == "product":
        s["y"] = _wide(case["m"], case["n"], pad, dtype)
        need = 0
        if own:
            import image_preprocessing_gb300 as trfn
            need = trfn.tr_int8_matmul_workspace_bytes(case["m"], case["n"], case["k"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return s
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "quant" or case.get("q8"):
        s["q"] = _wide(rows, cols, pad, torch.int8)
        s["scale"] = torch.empty(rows, device="cuda")
        s["back"] = _wide(rows, cols, pad, torch.float16)
    if case["op"] == "norm":
        s["y"] = None if case["q8"] else _wide(rows, cols, pad, dtype)
        s["h_out"] = _wide(rows, cols, pad, dtype) if case["residual"] else None
    if case["op"] == "grad":
        s["dx"] = _wide(rows, cols, pad, dtype)
        s["dweight"] = torch.empty(cols, device="cuda")
        need = 0
        if own:
            import image_preprocessing_gb300 as trfn
            need = trfn.tr_rms_norm_backward_workspace_bytes(rows, cols)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import image_preprocessing_gb300 as trfn
    case = s["case"]
    op = case["op"]
    if op == "product":
        trfn.tr_int8_matmul(s["x"], s["x_scale"], s["w"], s["w_scale"], s["y"], bias=s["bias"], workspace=s["workspace"])
        return {"y": s["y"]}
    if op == "quant":
        trfn.tr_quantize_rows(s["x"], s["q"], s["scale"])
        trfn.tr_dequantize_rows(s["q"], s["scale"], s["back"])
        return {"back": s["back"], "scale": s["scale"]}
    if op == "grad":
        trfn.tr_rms_norm_backward(s["dy"], s["h"], s["dx"], weight=s["weight"], dweight=s["dweight"],
                                  dresidual=s["dresidual"], eps=EPS, workspace=s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if case["q8"]:
        trfn.tr_rms_norm(s["x"], s["q"], weight=s["weight"], residual=s["residual"], residual_out=s["h_out"],
                         scale=s["scale"], eps=EPS)
        trfn.tr_dequantize_rows(s["q"], s["scale"], s["back"])
        out = {"back": s["back"], "scale": s["scale"]}
    else:
        trfn.tr_rms_norm(s["x"], s["y"], weight=s["weight"], residual=s["residual"], residual_out=s["h_out"], eps=EPS)
        out = {"y": s["y"]}
    if s["h_out"] is not None:
        out["h"] = s["h_out"]
    return out


def _plain_q8(v):
    """Rows in 8 bits, read back as binary16, and their scales."""
    top = v.abs().amax(1, keepdim=True)
    some = top >= TINY
    inverse = torch.where(some, 127 / top, torch.zeros_like(top))
    scale = torch.where(some, top / 127, torch.zeros_like(top))
    q = (v * inverse).round().clamp(-127, 127)
    return (q * scale).to(torch.float16), scale.squeeze(1)


def _run_plain(s):
    case = s["case"]
    op, dtype = case["op"], DTYPES[case["type"]]
    if op == "product":
        sums = s["x"].float() @ s["w"].float().t()
        y = sums * s["x_scale"][:, None] * s["w_scale"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(dtype)}
    if op == "quant":
        back, scale = _plain_q8(s["x"].float())
        return {"back": back, "scale": scale}
    if op == "grad":
        h, dy, n = s["h"].float(), s["dy"].float(), case["cols"]
        inverse = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        g = dy * s["weight"]
        unit = h * inverse
        dx = inverse * (g - unit * ((g * unit).sum(1, keepdim=True) / n))
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].float()
        return {"dx": dx.to(dtype), "dweight": (dy * unit).sum(0)}
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"]
    if case["q8"]:
        back, scale = _plain_q8(y)
        out = {"back": back, "scale": scale}
    else:
        out = {"y": y.to(dtype)}
    if s["residual"] is not None:
        out["h"] = h.to(dtype)
    return out


def work(case):
    b = SIZE[case["type"]]
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * b + 4 * (m + n) + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    e = rows * cols
    if case["op"] == "quant":   # the values, their 8-bit form and what is read back of it
        return {"bytes": e * (b + 1 + 2) + 4 * rows, "flops": 5 * e}
    if case["op"] == "grad":
        return {"bytes": e * b * (4 if case["residual"] else 3) + 8 * cols, "flops": 12 * e}
    out = 1 + 2 if case["q8"] else b
    return {"bytes": e * (b * (3 if case["residual"] else 1) + out) + 4 * cols + (4 * rows if case["q8"] else 0),
            "flops": (9 if case["q8"] else 5) * e}


def exact(case, seed):
    s = _inputs(case, seed)
    wide = {k: v.double() for k, v in s.items() if v is not None}
    if case["op"] == "product":
        w = wide["w"]
        parts = []
        for x, sx in zip(wide["x"].split(4096), wide["x_scale"].split(4096)):   # blocks of tokens, to bound memory
            part = torch.einsum("mk,nk->mn", x, w) * torch.outer(sx, wide["w_scale"])
            parts.append(part + wide["bias"] if "bias" in wide else part)
        return {"y": torch.cat(parts)}

    def eight_bits(v):
        top = torch.linalg.vector_norm(v, ord=float("inf"), dim=1, keepdim=True)
        step = torch.where(top < TINY, torch.ones_like(top), top / 127)
        q = torch.round(v / step)
        step = torch.where(top < TINY, torch.zeros_like(top), step)
        return q * step, step.flatten()

    if case["op"] == "quant":
        back, scale = eight_bits(wide["x"])
        return {"back": back, "scale": scale}
    n = case["cols"]
    if case["op"] == "grad":
        h, dy, weight = wide["h"], wide["dy"], wide["weight"]
        rms = torch.sqrt(torch.einsum("rc,rc->r", h, h) / n + EPS)[:, None]
        along = torch.einsum("rc,rc,c->r", dy, h, weight)[:, None]
        dx = dy * weight / rms - h * along / (n * rms ** 3)
        if "dresidual" in wide:
            dx += wide["dresidual"]
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, h / rms)}
    h = wide["x"] + wide["residual"] if "residual" in wide else wide["x"]
    rms = torch.sqrt(torch.einsum("rc,rc->r", h, h) / n + EPS)[:, None]
    y = h / rms * wide["weight"]
    out = {}
    if case["q8"]:
        out["back"], out["scale"] = eight_bits(y)
    else:
        out["y"] = y
    if "residual" in wide:
        out["h"] = h
    return out
