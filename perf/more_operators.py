"""Timed cases of what a transformer block over token rows has between its products: layer norm with the residual's
addition (also with an 8-bit output) and its gradients, rotary positions, and attention over packed sequences.

Tokens are the 16x16 patches of normalised image batches (196 to a 224x224x3 image, 256 images to a batch) and the
hidden rows a network makes of them, or the tokens of prompts; serving takes one token at a time of each sequence.
"""
import math
import random

import torch

own = False

EPS = 1e-5
TINY = 2.0 ** -119   # rows whose largest magnitude is below this hold zeros in 8 bits
TRAINED = 4096       # positions that frequencies scaled by parts were trained on
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token of a serving step: residual stream and norm, latency alone counts
        {"name": "layer_norm_token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "residual": True, "q8": False, "pad": 0},
        # hidden rows of a training batch: 256 images x 196 patches
        {"name": "layer_norm_batch", "op": "norm", "rows": 50176, "cols": 1024, "type": "f16", "residual": True, "q8": False, "pad": 0},
        # norm in front of an 8-bit product, 64 images; the 8-bit rows are read back as binary16
        {"name": "layer_norm_q8_batch", "op": "norm", "rows": 12544, "cols": 4096, "type": "bf16", "residual": True, "q8": True, "pad": 0},
        # training: the norm's gradients over the batch, with the gradient that arrives along the residual stream
        {"name": "layer_norm_grad_batch", "op": "grad", "rows": 50176, "cols": 1024, "type": "f16", "residual": True, "pad": 0},
        # training: an odd width inside a wider buffer, binary32
        {"name": "layer_norm_grad_odd", "op": "grad", "rows": 1777, "cols": 999, "type": "f32", "residual": False, "pad": 5},
        # one token's query and key heads in a serving step, far into a sequence
        {"name": "rotary_token", "op": "rotary", "tokens": 1, "heads": 40, "dim": 128, "rot": 128, "layout": "halves",
         "scaling": "none", "factor": 1.0, "start": 70001, "period": 1, "inverse": False, "type": "bf16", "pad": 0},
        # query and key heads of the batch's patches, which lie in a wider matrix with the values
        {"name": "rotary_batch", "op": "rotary", "tokens": 50176, "heads": 24, "dim": 64, "rot": 64, "layout": "pairs",
         "scaling": "none", "factor": 1.0, "start": 0, "period": 196, "inverse": False, "type": "f16", "pad": 768},
        # training on long prompts: the gradient of half of each head, frequencies scaled by parts, far positions
        {"name": "rotary_grad_far", "op": "rotary", "tokens": 8192, "heads": 40, "dim": 128, "rot": 64, "layout": "halves",
         "scaling": "parts", "factor": 32.0, "start": 100000, "period": 8192, "inverse": True, "type": "bf16", "pad": 0},
        # the patches of each image attend to one another
        {"name": "attention_images", "op": "attention", "mode": "prompt", "sequences": 256, "longest": 196, "lengths": 0, "new": 0,
         "heads": 12, "kv_heads": 12, "dim": 64, "causal": False, "type": "f16", "pad": 1536},
        # prompts of different lengths, packed, grouped heads
        {"name": "attention_packed", "op": "attention", "mode": "prompt", "sequences": 16, "longest": 4096, "lengths": 7, "new": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16", "pad": 0},
        # one long prompt
        {"name": "attention_prompt", "op": "attention", "mode": "prompt", "sequences": 1, "longest": 8192, "lengths": 0, "new": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16", "pad": 0},
        # a serving step: one new token for each of some sequences, keys and values in slots of one length
        {"name": "attention_tokens", "op": "attention", "mode": "tokens", "sequences": 32, "longest": 8192, "lengths": 3, "new": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16", "pad": 0},
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
        op = rng.choice(["norm", "grad", "rotary", "rotary", "attention", "attention", "attention"])
        case = {"op": op}
        if op in ("norm", "grad"):
            case.update(rows=_log_int(rng, 1, 50176), cols=_log_int(rng, 64, 8192), type=rng.choice(["f32", "f16", "bf16"]),
                        residual=rng.random() < 0.7)
            if op == "norm":
                case["q8"] = rng.random() < 0.5
            case["pad"] = rng.choice([0, 0, 0, 16, rng.randrange(1, 33)])
        elif op == "rotary":
            dim = rng.choice([64, 64, 128, 128, 2 * rng.randrange(8, 129)])
            case.update(tokens=_log_int(rng, 1, 50176), heads=_log_int(rng, 1, 80), dim=dim,
                        rot=rng.choice([dim, dim, 2 * rng.randrange(1, dim // 2 + 1)]), layout=rng.choice(["halves", "pairs"]),
                        scaling=rng.choice(["none", "linear", "base", "parts"]), factor=1.0 + 31 * rng.random(),
                        start=rng.choice([0, _log_int(rng, 1, 1000000)]), period=_log_int(rng, 1, 50176),
                        inverse=rng.random() < 0.4, type=rng.choice(["f32", "f16", "bf16"]),
                        pad=rng.choice([0, 0, dim, rng.randrange(1, 33)]))
            if case["rot"] < 4 or case["scaling"] == "none":
                case.update(scaling="none", factor=1.0)
        else:
            kv_heads, group = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 1, 2, 3, 4, 5, 8])
            mode = rng.choice(["prompt", "prompt", "tokens"])
            case.update(mode=mode, sequences=_log_int(rng, 1, 64 if mode == "prompt" else 128), longest=_log_int(rng, 1, 16384),
                        lengths=rng.choice([0, rng.randrange(1, 1000)]), new=rng.choice([1, 1, 1, 2, 5]) if mode == "tokens" else 0,
                        heads=kv_heads * group, kv_heads=kv_heads, dim=rng.choice([64, 64, 128, 128, 8 * rng.randrange(2, 17)]),
                        causal=mode == "tokens" or rng.random() < 0.6, type=rng.choice(["f16", "bf16"]), pad=rng.choice([0, 0, 8, 64]))
            if mode == "tokens":
                case["longest"] = max(case["longest"], case["new"])
        w = work(case)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return case


def _lengths(case):
    """Queries and keys of each sequence."""
    n, longest = case["sequences"], case["longest"]
    keys = [longest] * n
    if case["lengths"]:
        # one of them is the longest; with some sequences, one has a single token and one none
        rng = random.Random(case["lengths"])
        keys = [longest] + [_log_int(rng, 1, longest) for _ in range(n - 1)]
        if n > 4:
            keys[1], keys[2] = 1, 0
        rng.shuffle(keys)
    if case["mode"] == "prompt":
        return keys, keys
    return [case["new"]] * n, [max(k, case["new"]) if k else 0 for k in keys]


def _seen(case):
    """Pairs of a query and a key that it sees, in all."""
    total = 0
    for lq, lk in zip(*_lengths(case)):
        if not case["causal"]:
            total += lq * lk
        else:   # query i sees i + 1 + lk - lq keys, where that is a number of keys
            first = max(0, lq - lk)
            total += (lq - first) * lk - (lq - first) * (lq - first - 1) // 2
    return total


def _frequencies(rot, scaling, factor):
    """Angle for each position of every pair, and what the turned values are scaled by."""
    base, magnitude = 10000.0, 1.0
    if scaling == "base":
        base *= factor ** (rot / (rot - 2))
    freqs = [base ** (-2.0 * k / rot) for k in range(rot // 2)]
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    if scaling == "parts":
        # pairs with 32 and more turns over the trained positions stay, those with less than one are stretched
        for k, f in enumerate(freqs):
            keep = min(1.0, max(0.0, (TRAINED * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
            freqs[k] = f * (keep + (1 - keep) / factor)
        magnitude = 1.0 + 0.1 * math.log(factor)
    return freqs, magnitude


def _wide(rows, cols, pad, dtype):
    """A (rows, cols) view of a buffer whose rows are cols + pad apart."""
    return torch.empty((rows, cols + pad), dtype=dtype, device="cuda")[:, :cols]


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pad, dtype = case["pad"], DTYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def fill(values):
        t = _wide(values.shape[0], values.shape[1], pad, dtype)
        t.copy_(values)
        return t

    s = {}
    if case["op"] == "rotary":
        # far positions are exact in 32-bit integers alone
        s["positions"] = (case["start"] + torch.arange(case["tokens"], device="cuda") % case["period"]).to(torch.int32)
        s["x"] = fill(normal(case["tokens"], case["heads"] * case["dim"]))
        return s
    if case["op"] == "attention":
        lq, lk = _lengths(case)
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        slot = case["longest"] if case["mode"] == "tokens" else None
        # heads from wide ones to ones that look at few tokens; some channels of the values are much larger
        sharp = (0.5 + 2.5 * torch.rand(hq, generator=g, device="cuda")).repeat_interleave(d)
        s["q"] = fill(normal(sum(lq), hq * d) * sharp)
        rows = slot * len(lk) if slot else sum(lk)
        s["k"] = fill(normal(rows, hk * d))
        loud = 1 + 7 * (torch.rand(hk * d, generator=g, device="cuda") < 0.01)
        s["v"] = fill(normal(rows, hk * d) * loud)
        return s
    rows, cols = case["rows"], case["cols"]
    s["weight"] = 1 + 0.1 * normal(cols)
    loud = 1 + 7 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
    if case["op"] == "norm":
        s["bias"] = 0.1 * normal(cols)
        s["x"] = fill(normal(rows, cols))
        # the stream has a few channels that are much larger than the rest, and a mean of its own
        s["residual"] = fill(normal(rows, cols) * loud + 0.5) if case["residual"] else None
    else:
        s["h"] = fill(normal(rows, cols) * 1.5 * loud + 0.5)
        s["dy"] = fill(normal(rows, cols) * 0.1)
        s["dresidual"] = fill(normal(rows, cols) * 0.1) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    pad, dtype = case["pad"], DTYPES[case["type"]]
    trfn = None
    if own:
        import image_preprocessing_gb300 as trfn
    # the buffers, sequences and frequencies a program keeps beside its inputs
    if case["op"] == "rotary":
        s["out"] = _wide(case["tokens"], case["heads"] * case["dim"], pad, dtype)
        s["freqs"], s["magnitude"] = _frequencies(case["rot"], case["scaling"], case["factor"])
        if own:
            kind = {"none": trfn.ROTARY_UNSCALED, "linear": trfn.ROTARY_LINEAR, "base": trfn.ROTARY_BASE, "parts": trfn.ROTARY_PARTS}
            s["freqs"], s["magnitude"] = trfn.tr_rotary_frequencies(case["rot"], scaling=kind[case["scaling"]],
                                                                    factor=case["factor"], trained=TRAINED)
        return s
    if case["op"] == "attention":
        lq, lk = _lengths(case)

        def starts(lengths):
            return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")

        s["lq"], s["lk"] = lq, lk
        s["q_starts"] = starts(lq)
        if case["mode"] == "tokens":
            s["k_starts"] = torch.arange(len(lk) + 1, dtype=torch.int32, device="cuda") * case["longest"]
            s["k_lengths"] = torch.tensor(lk, dtype=torch.int32, device="cuda")
        else:
            s["k_starts"], s["k_lengths"] = s["q_starts"], None
        s["out"] = _wide(sum(lq), case["heads"] * case["dim"], pad, dtype)
        need = 0
        if own:
            need = trfn.tr_attention_workspace_bytes(sum(lq), len(lq), case["heads"], case["kv_heads"], case["dim"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return s
    rows, cols = case["rows"], case["cols"]
    if case.get("q8"):
        s["q"] = _wide(rows, cols, pad, torch.int8)
        s["scale"] = torch.empty(rows, device="cuda")
        s["back"] = _wide(rows, cols, pad, torch.float16)
    if case["op"] == "norm":
        s["y"] = None if case["q8"] else _wide(rows, cols, pad, dtype)
        s["h_out"] = _wide(rows, cols, pad, dtype) if case["residual"] else None
    else:
        s["dx"] = _wide(rows, cols, pad, dtype)
        s["dweight"], s["dbias"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        need = trfn.tr_layer_norm_backward_workspace_bytes(rows, cols) if own else 0
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import image_preprocessing_gb300 as trfn
    case = s["case"]
    op = case["op"]
    if op == "rotary":
        trfn.tr_rotary(s["x"], s["out"], case["heads"], s["freqs"], positions=s["positions"],
                       layout=trfn.ROTARY_HALVES if case["layout"] == "halves" else trfn.ROTARY_PAIRS,
                       magnitude=s["magnitude"], inverse=case["inverse"])
        return {"out": s["out"]}
    if op == "attention":
        trfn.tr_attention(s["q"], s["k"], s["v"], s["out"], case["heads"], case["kv_heads"], s["q_starts"], s["k_starts"],
                          k_lengths=s["k_lengths"], causal=case["causal"], workspace=s["workspace"])
        return {"out": s["out"]}
    if op == "grad":
        trfn.tr_layer_norm_backward(s["dy"], s["h"], s["dx"], weight=s["weight"], dweight=s["dweight"], dbias=s["dbias"],
                                    dresidual=s["dresidual"], eps=EPS, workspace=s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if case["q8"]:
        trfn.tr_layer_norm(s["x"], s["q"], weight=s["weight"], bias=s["bias"], residual=s["residual"], residual_out=s["h_out"],
                           scale=s["scale"], eps=EPS)
        trfn.tr_dequantize_rows(s["q"], s["scale"], s["back"])
        out = {"back": s["back"], "scale": s["scale"]}
    else:
        trfn.tr_layer_norm(s["x"], s["y"], weight=s["weight"], bias=s["bias"], residual=s["residual"],
                           residual_out=s["h_out"], eps=EPS)
        out = {"y": s["y"]}
    if s["h_out"] is not None:
        out["h"] = s["h_out"]
    return out


def _plain_rotary(s):
    case = s["case"]
    heads, dim, rot = case["heads"], case["dim"], case["rot"]
    # angles of far positions need more than 32 bits
    angle = s["positions"].double()[:, None] * torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
    cos = (angle.cos() * s["magnitude"]).float()[:, None, :]
    sin = (angle.sin() * s["magnitude"]).float()[:, None, :]
    if case["inverse"]:
        sin = -sin
    x = s["x"].float().view(case["tokens"], heads, dim)
    turned = x[:, :, :rot]
    if case["layout"] == "halves":
        a, b = turned[:, :, :rot // 2], turned[:, :, rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    else:
        a, b = turned[:, :, 0::2], turned[:, :, 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    return {"out": torch.cat([turned, x[:, :, rot:]], 2).flatten(1).to(DTYPES[case["type"]])}


def _plain_attention(s):
    case = s["case"]
    hq, hk, d, dtype = case["heads"], case["kv_heads"], case["dim"], DTYPES[case["type"]]
    group = hq // hk
    out = torch.zeros((sum(s["lq"]), hq * d), dtype=dtype, device="cuda")
    q0 = k0 = 0
    for lq, lk in zip(s["lq"], s["lk"]):
        k = s["k"][k0:k0 + lk].float().view(lk, hk, d).permute(1, 2, 0)
        v = s["v"][k0:k0 + lk].float().view(lk, hk, d).transpose(0, 1)
        step = max(1, (1 << 29) // max(1, hq * lk))   # queries at a time, to bound memory
        for i0 in range(0, lq if lk else 0, step):
            n = min(step, lq - i0)
            q = s["q"][q0 + i0:q0 + i0 + n].float().view(n, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * n, d)
            scores = ((q @ k) * (1 / math.sqrt(d))).view(hk, group, n, lk)
            if case["causal"]:
                last = torch.arange(i0, i0 + n, device="cuda") + (lk - lq)
                scores = scores.masked_fill(torch.arange(lk, device="cuda") > last[:, None], float("-inf"))
            top = scores.amax(3, keepdim=True)
            p = torch.exp(scores - torch.where(top == float("-inf"), torch.zeros_like(top), top))
            total = p.sum(3, keepdim=True)
            o = (p.view(hk, group * n, lk) @ v).view(hk, group, n, d) / torch.where(total == 0, torch.ones_like(total), total)
            out[q0 + i0:q0 + i0 + n] = o.permute(2, 0, 1, 3).reshape(n, hq * d).to(dtype)
        q0 += lq
        k0 += case["longest"] if case["mode"] == "tokens" else lk
    return {"out": out}


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
    if op == "rotary":
        return _plain_rotary(s)
    if op == "attention":
        return _plain_attention(s)
    if op == "grad":
        h, dy = s["h"].float(), s["dy"].float()
        apart = h - h.mean(1, keepdim=True)
        inverse = torch.rsqrt((apart * apart).mean(1, keepdim=True) + EPS)
        unit = apart * inverse
        g = dy * s["weight"]
        dx = inverse * (g - g.mean(1, keepdim=True) - unit * (g * unit).mean(1, keepdim=True))
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].float()
        return {"dx": dx.to(dtype), "dweight": (dy * unit).sum(0), "dbias": dy.sum(0)}
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    apart = h - h.mean(1, keepdim=True)
    y = apart * torch.rsqrt((apart * apart).mean(1, keepdim=True) + EPS) * s["weight"] + s["bias"]
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
    if case["op"] == "rotary":
        e = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * e * b + 4 * case["tokens"], "flops": 6 * case["tokens"] * case["heads"] * (case["rot"] // 2)}
    if case["op"] == "attention":
        lq, lk = _lengths(case)
        d = case["dim"]
        # scores and weighted values, two operations a product
        return {"bytes": b * d * (2 * sum(lq) * case["heads"] + 2 * sum(lk) * case["kv_heads"]) + 8 * len(lq),
                "flops": 4 * d * case["heads"] * _seen(case)}
    rows, cols = case["rows"], case["cols"]
    e = rows * cols
    if case["op"] == "grad":
        return {"bytes": e * b * (4 if case["residual"] else 3) + 12 * cols, "flops": 16 * e}
    out = 1 + 2 if case["q8"] else b
    return {"bytes": e * (b * (3 if case["residual"] else 1) + out) + 8 * cols + (4 * rows if case["q8"] else 0),
            "flops": (12 if case["q8"] else 8) * e}


def _exact_rotary(case, s):
    freqs, magnitude = _frequencies(case["rot"], case["scaling"], case["factor"])
    tokens, heads, dim, half = case["tokens"], case["heads"], case["dim"], case["rot"] // 2
    turn = torch.outer(s["positions"].double(), torch.tensor(freqs, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(turn, magnitude), -turn if case["inverse"] else turn)
    out = s["x"].double().reshape(tokens, heads, dim).clone()
    at = torch.arange(half, device="cuda")
    first, second = (at, at + half) if case["layout"] == "halves" else (2 * at, 2 * at + 1)
    z = torch.complex(out[:, :, first], out[:, :, second]) * turn[:, None]
    out[:, :, first], out[:, :, second] = z.real, z.imag
    return {"out": out.reshape(tokens, heads * dim)}


def _exact_attention(case, s):
    lq, lk = _lengths(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros((sum(lq), hq, d), dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(lq, lk):
        if nq and nk:
            q = s["q"][q0:q0 + nq].double().reshape(nq, hq, d)
            k = s["k"][k0:k0 + nk].double().reshape(nk, hk, d)
            v = s["v"][k0:k0 + nk].double().reshape(nk, hk, d)
            sees = torch.ones((nq, nk), dtype=torch.bool, device="cuda")
            if case["causal"]:
                sees = sees.tril(nk - nq)
            some = sees.any(1)
            for h in range(hq):
                a = torch.einsum("id,jd->ij", q[:, h], k[:, h // (hq // hk)]) / d ** 0.5
                a = torch.softmax(torch.where(sees, a, -math.inf)[some], 1)
                out[q0:q0 + nq, h][some] = torch.einsum("ij,jd->id", a, v[:, h // (hq // hk)])
        q0 += nq
        k0 += case["longest"] if case["mode"] == "tokens" else nk
    return {"out": out.reshape(-1, hq * d)}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    wide = {k: v.double() for k, v in s.items() if v is not None}

    def eight_bits(v):
        top = torch.linalg.vector_norm(v, ord=float("inf"), dim=1, keepdim=True)
        step = torch.where(top < TINY, torch.ones_like(top), top / 127)
        q = torch.round(v / step)
        step = torch.where(top < TINY, torch.zeros_like(top), step)
        return q * step, step.flatten()

    n = case["cols"]
    if case["op"] == "grad":
        h, dy, weight = wide["h"], wide["dy"], wide["weight"]
        h = h - (h.sum(1) / n)[:, None]
        std = torch.sqrt(torch.einsum("rc,rc->r", h, h) / n + EPS)[:, None]
        along = torch.einsum("rc,rc,c->r", dy, h, weight)[:, None]
        level = torch.einsum("rc,c->r", dy, weight)[:, None] / n
        dx = (dy * weight - level) / std - h * along / (n * std ** 3)
        if "dresidual" in wide:
            dx += wide["dresidual"]
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, h / std), "dbias": torch.einsum("rc->c", dy)}
    h = wide["x"] + wide["residual"] if "residual" in wide else wide["x"]
    var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
    y = torch.addcmul(wide["bias"], (h - mean) / torch.sqrt(var + EPS), wide["weight"])
    out = {}
    if case["q8"]:
        out["back"], out["scale"] = eight_bits(y)
    else:
        out["y"] = y
    if "residual" in wide:
        out["h"] = h
    return out
