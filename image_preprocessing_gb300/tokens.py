"""Python face of the token-row operators (include/tr_token_ops.h); the
functions carry the C entry points' names.

Matrices are 2-D CUDA tensors with unit column stride (any row stride);
outputs and workspaces are the caller's, as everywhere in this package.  Each
call enqueues on `stream` (the current one if None) and raises TrError on a
refusal.  The tensors are on the current device, all of them: the library
launches there, and a tensor elsewhere is refused.
"""
import ctypes

from ._native import TrError, check, lib

ELEM_F32, ELEM_F16, ELEM_BF16, ELEM_I8 = 0, 1, 2, 3
MAX_ROW, MAX_INT8_K = 32768, 131071   # TR_MAX_ROW, TR_MAX_INT8_K
ROTARY_HALVES, ROTARY_PAIRS = 0, 1
ROTARY_UNSCALED, ROTARY_LINEAR, ROTARY_BASE, ROTARY_PARTS = 0, 1, 2, 3

_INT32 = 4            # no tr_elem: positions and sequences
_codes = {}           # torch dtypes, filled when the first tensor comes
_current_stream = _current_device = None


def _prepare():
    global _current_stream, _current_device
    import torch
    _codes.update({torch.float32: ELEM_F32, torch.float16: ELEM_F16, torch.bfloat16: ELEM_BF16,
                   torch.int8: ELEM_I8, torch.int32: _INT32})
    # the handle alone: a stream object costs a microsecond a call
    _current_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice


def _elem(t):
    if not _codes:
        _prepare()
    return _codes.get(t.dtype, -1)


def _stream(stream, device, where):
    """The stream's handle, for tensors on this device, which has to be the current one."""
    if device < 0:
        raise TrError(1, where, "the tensors must be CUDA tensors")
    if device != _current_device():
        raise TrError(1, where, "the tensors are on cuda:%d, the current device is cuda:%d" % (device, _current_device()))
    if stream is None:
        return _current_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _elsewhere(t, where, name):
    return TrError(1, where, "%s %s" % (name, "must be a CUDA tensor" if t.get_device() < 0 else
                                        "is not on the device of the other tensors"))


def _matrix(t, shape, elem, device, where, name):
    """Address and row stride of a matrix of this shape (any if None) and element type (any if -1) on this CUDA device."""
    if shape is not None and t.shape != shape:
        raise TrError(1, where, "%s must be a %s matrix" % (name, tuple(shape)))
    if elem >= 0 and _codes.get(t.dtype, -1) != elem:
        raise TrError(1, where, "%s has another type" % name)
    if t.get_device() != device:
        raise _elsewhere(t, where, name)
    row, col = t.stride()
    if col != 1 and t.shape[1] > 1:
        raise TrError(1, where, "%s must have unit column stride" % name)
    return t.data_ptr(), row


def _integers(t, n, device, where, name):
    """Address of n contiguous int32 values on this CUDA device; None for None."""
    if t is None:
        return None
    if _codes.get(t.dtype, -1) != _INT32 or t.numel() != n or not t.is_contiguous():
        raise TrError(1, where, "%s must be %d contiguous int32 values" % (name, n))
    if t.get_device() != device:
        raise _elsewhere(t, where, name)
    return t.data_ptr()


def _vector(t, n, device, where, name):
    """Address of n contiguous binary32 values on this CUDA device; None for None."""
    if t is None:
        return None
    if _codes.get(t.dtype, -1) != ELEM_F32 or t.numel() != n or not t.is_contiguous():
        raise TrError(1, where, "%s must be %d contiguous float32 values" % (name, n))
    if t.get_device() != device:
        raise _elsewhere(t, where, name)
    return t.data_ptr()


def _workspace(ws, need, device, where):
    if need == 0:
        return None
    if ws is None or ws.numel() * ws.element_size() < need or not ws.is_contiguous():
        raise TrError(1, where, "needs a contiguous CUDA workspace of at least %d bytes" % need)
    if ws.get_device() != device:
        raise _elsewhere(ws, where, "workspace")
    return ws.data_ptr()


def _shape(t, where, name):
    shape = t.shape
    if len(shape) != 2:
        raise TrError(1, where, "%s must be a matrix" % name)
    return shape


def tr_rms_norm(x, out, weight=None, residual=None, residual_out=None, scale=None, eps=1e-6, stream=None):
    """h = x + residual; out = h / sqrt(mean(h^2) + eps) * weight, row by row.

    x, residual: float32, float16 or bfloat16 of one shape; out: of x's type,
    or int8, then with scale (rows float32) receiving max|row| / 127;
    residual_out: h in x's type (may be x or residual); weight: cols float32,
    or None for ones."""
    where = "tr_rms_norm"
    shape = _shape(x, where, "x")
    rows, cols = shape
    dt = _elem(x)
    device = x.get_device()
    pr, sr = (None, 0) if residual is None else _matrix(residual, shape, dt, device, where, "residual")
    ph, sh = (None, 0) if residual_out is None else _matrix(residual_out, shape, dt, device, where, "residual_out")
    px, sx = _matrix(x, None, -1, device, where, "x")
    po, so = _matrix(out, shape, -1, device, where, "out")
    rc = lib().tr_rms_norm(px, pr, _vector(weight, cols, device, where, "weight"), po, ph,
                           _vector(scale, rows, device, where, "scale"), rows, cols, sx, sr, so, sh, dt, _elem(out), eps,
                           _stream(stream, device, where))
    if rc:
        check(rc, where)


def tr_rms_norm_backward_workspace_bytes(rows, cols):
    """Bytes of a workspace for the dweight of up to this many rows of this length."""
    return int(lib().tr_rms_norm_backward_workspace_bytes(rows, cols))


def tr_rms_norm_backward(dy, h, dx, weight=None, dweight=None, dresidual=None, eps=1e-6, workspace=None,
                         stream=None):
    """Gradients of tr_rms_norm's out (in h's type) at h, the forward's
    residual_out (or its x where there was no residual).

    dx receives the gradient of h, hence of x and of residual, dresidual (the
    gradient that reaches h along the residual stream) included; it may be dy,
    h or dresidual.  dweight: cols float32, overwritten, or None; it needs a
    workspace of tr_rms_norm_backward_workspace_bytes(rows, cols) bytes."""
    where = "tr_rms_norm_backward"
    shape = _shape(h, where, "h")
    rows, cols = shape
    dt = _elem(h)
    device = h.get_device()
    py, sy = _matrix(dy, shape, dt, device, where, "dy")
    ph, sh = _matrix(h, None, -1, device, where, "h")
    px, sx = _matrix(dx, shape, dt, device, where, "dx")
    pr, sr = (None, 0) if dresidual is None else _matrix(dresidual, shape, dt, device, where, "dresidual")
    ws = None
    if dweight is not None and rows > 0:
        ws = _workspace(workspace, lib().tr_rms_norm_backward_workspace_bytes(rows, cols), device, where)
    rc = lib().tr_rms_norm_backward(py, ph, _vector(weight, cols, device, where, "weight"), pr, px,
                                    _vector(dweight, cols, device, where, "dweight"), rows, cols, sy, sh, sr, sx, dt, eps,
                                    ws, _stream(stream, device, where))
    if rc:
        check(rc, where)


def tr_layer_norm(x, out, weight=None, bias=None, residual=None, residual_out=None, scale=None, eps=1e-5, stream=None):
    """h = x + residual; out = (h - mean(h)) / sqrt(mean((h - mean(h))^2) + eps) * weight + bias, row by row.

    bias: cols float32, or None for zeros; the others as tr_rms_norm's."""
    where = "tr_layer_norm"
    shape = _shape(x, where, "x")
    rows, cols = shape
    dt = _elem(x)
    device = x.get_device()
    pr, sr = (None, 0) if residual is None else _matrix(residual, shape, dt, device, where, "residual")
    ph, sh = (None, 0) if residual_out is None else _matrix(residual_out, shape, dt, device, where, "residual_out")
    px, sx = _matrix(x, None, -1, device, where, "x")
    po, so = _matrix(out, shape, -1, device, where, "out")
    rc = lib().tr_layer_norm(px, pr, _vector(weight, cols, device, where, "weight"), _vector(bias, cols, device, where, "bias"),
                             po, ph, _vector(scale, rows, device, where, "scale"), rows, cols, sx, sr, so, sh, dt, _elem(out),
                             eps, _stream(stream, device, where))
    if rc:
        check(rc, where)


def tr_layer_norm_backward_workspace_bytes(rows, cols):
    """Bytes of a workspace for the dweight and dbias of up to this many rows of this length."""
    return int(lib().tr_layer_norm_backward_workspace_bytes(rows, cols))


def tr_layer_norm_backward(dy, h, dx, weight=None, dweight=None, dbias=None, dresidual=None, eps=1e-5, workspace=None,
                           stream=None):
    """Gradients of tr_layer_norm's out (in h's type) at h, as tr_rms_norm_backward's.

    dweight, dbias: cols float32 each, overwritten, or None; either needs a
    workspace of tr_layer_norm_backward_workspace_bytes(rows, cols) bytes."""
    where = "tr_layer_norm_backward"
    shape = _shape(h, where, "h")
    rows, cols = shape
    dt = _elem(h)
    device = h.get_device()
    py, sy = _matrix(dy, shape, dt, device, where, "dy")
    ph, sh = _matrix(h, None, -1, device, where, "h")
    px, sx = _matrix(dx, shape, dt, device, where, "dx")
    pr, sr = (None, 0) if dresidual is None else _matrix(dresidual, shape, dt, device, where, "dresidual")
    ws = None
    if (dweight is not None or dbias is not None) and rows > 0:
        ws = _workspace(workspace, lib().tr_layer_norm_backward_workspace_bytes(rows, cols), device, where)
    rc = lib().tr_layer_norm_backward(py, ph, _vector(weight, cols, device, where, "weight"), pr, px,
                                      _vector(dweight, cols, device, where, "dweight"),
                                      _vector(dbias, cols, device, where, "dbias"), rows, cols, sy, sh, sr, sx, dt, eps, ws,
                                      _stream(stream, device, where))
    if rc:
        check(rc, where)


def tr_quantize_rows(x, q, scale, stream=None):
    """Rows of x (float32, float16, bfloat16) in 8 bits: q int8 of x's shape,
    scale rows float32; q * scale stands for x."""
    where = "tr_quantize_rows"
    shape = _shape(x, where, "x")
    rows, cols = shape
    dt = _elem(x)
    device = x.get_device()
    pq, sq = _matrix(q, shape, ELEM_I8, device, where, "q")
    px, sx = _matrix(x, None, -1, device, where, "x")
    rc = lib().tr_quantize_rows(px, pq, _vector(scale, rows, device, where, "scale"), rows, cols, sx, sq, dt,
                                _stream(stream, device, where))
    if rc:
        check(rc, where)


def tr_dequantize_rows(q, scale, out, stream=None):
    """out = q * scale, row by row, in out's type."""
    where = "tr_dequantize_rows"
    shape = _shape(q, where, "q")
    rows, cols = shape
    dt = _elem(out)
    device = q.get_device()
    pq, sq = _matrix(q, shape, ELEM_I8, device, where, "q")
    po, so = _matrix(out, shape, -1, device, where, "out")
    rc = lib().tr_dequantize_rows(pq, _vector(scale, rows, device, where, "scale"), po, rows, cols, sq, so, dt,
                                  _stream(stream, device, where))
    if rc:
        check(rc, where)


def tr_int8_matmul_workspace_bytes(M, N, K):
    """Bytes of a workspace for products of up to M tokens with this N and K."""
    return int(lib().tr_int8_matmul_workspace_bytes(M, N, K))


def tr_int8_matmul(x, x_scale, w, w_scale, y, bias=None, workspace=None, stream=None):
    """y = (x @ w.T) * x_scale[:, None] * w_scale + bias, the products summed
    exactly in integers.

    x: int8 (M, K), x_scale: M float32; w: int8 (N, K), w_scale: N float32;
    bias: N float32 or None; y: (M, N) float32, float16 or bfloat16; workspace:
    tr_int8_matmul_workspace_bytes(M, N, K) bytes, for this M or a larger one."""
    where = "tr_int8_matmul"
    M, K = _shape(x, where, "x")
    N = _shape(w, where, "w")[0]
    dt = _elem(y)
    device = x.get_device()
    px, sx = _matrix(x, None, ELEM_I8, device, where, "x")
    pw, sw = _matrix(w, (N, K), ELEM_I8, device, where, "w")
    py, sy = _matrix(y, (M, N), -1, device, where, "y")
    L = lib()
    # the size holds for up to M tokens: this M may do without, which the library knows
    need = L.tr_int8_matmul_workspace_bytes(M, N, K)
    given = not need or (workspace is not None and workspace.numel() * workspace.element_size() >= need)
    ws = _workspace(workspace, need, device, where) if given else None
    rc = L.tr_int8_matmul(px, _vector(x_scale, M, device, where, "x_scale"), pw,
                          _vector(w_scale, N, device, where, "w_scale"), _vector(bias, N, device, where, "bias"), py,
                          M, N, K, sx, sw, sy, dt, ws, _stream(stream, device, where))
    if rc:
        if rc == 1 and not given:
            raise TrError(1, where, "needs a contiguous CUDA workspace of at least %d bytes, or another argument is invalid" % need)
        check(rc, where)


def tr_rotary_frequencies(rot, base=10000.0, scaling=ROTARY_UNSCALED, factor=1.0, trained=0):
    """(freqs, magnitude) for tr_rotary: rot / 2 frequencies (a ctypes array of
    doubles, radians for each position) and what the turned values are scaled by.

    scaling: for contexts `factor` times as long as the `trained` positions:
    ROTARY_LINEAR, ROTARY_BASE or ROTARY_PARTS."""
    where = "tr_rotary_frequencies"
    if rot < 2 or rot > 512:   # (the size of the array)
        raise TrError(1 if rot < 2 else 2, where, "rot is between 2 and 512")
    freqs, magnitude = (ctypes.c_double * (rot // 2))(), ctypes.c_float()
    rc = lib().tr_rotary_frequencies(rot, base, scaling, factor, trained, freqs, ctypes.byref(magnitude))
    if rc:
        check(rc, where)
    return freqs, magnitude.value


def tr_rotary(x, out, heads, freqs, positions=None, layout=ROTARY_HALVES, magnitude=1.0, inverse=False, stream=None):
    """Rotary positions of every head of x (tokens, heads * dim), into out (may be x).

    freqs: of tr_rotary_frequencies, or a sequence of numbers: a head's first
    2 * len(freqs) values turn, the rest are copied; positions: tokens int32, or
    None for 0, 1, ...; inverse: turns back, which is the gradient (dx of dout)."""
    where = "tr_rotary"
    shape = _shape(x, where, "x")
    tokens, cols = shape
    if heads < 1 or cols % heads:
        raise TrError(1, where, "x must have heads * dim columns")
    dt = _elem(x)
    device = x.get_device()
    px, sx = _matrix(x, None, -1, device, where, "x")
    po, so = _matrix(out, shape, dt, device, where, "out")
    if not isinstance(freqs, ctypes.Array) or freqs._type_ is not ctypes.c_double:
        freqs = (ctypes.c_double * len(freqs))(*freqs)
    rc = lib().tr_rotary(px, po, _integers(positions, tokens, device, where, "positions"), freqs, tokens, heads, cols // heads,
                         2 * len(freqs), sx, so, dt, layout, magnitude, bool(inverse), _stream(stream, device, where))
    if rc:
        check(rc, where)


def tr_attention_workspace_bytes(q_rows, sequences, heads, kv_heads, dim):
    """Bytes of a workspace for attention of up to this many rows of q and sequences."""
    return int(lib().tr_attention_workspace_bytes(q_rows, sequences, heads, kv_heads, dim))


def tr_attention(q, k, v, out, heads, kv_heads, q_starts, k_starts=None, q_lengths=None, k_lengths=None, causal=False,
                 scale=None, workspace=None, stream=None):
    """Attention of packed sequences, head by head.

    q, out: (rows, heads * dim), k, v: (rows, kv_heads * dim), of one type
    (float32, float16 or bfloat16); q_starts: sequences + 1 int32, sequence s is
    the rows q_starts[s] .. q_starts[s + 1], or with q_lengths (sequences int32)
    the first so many from q_starts[s] on; k_starts, k_lengths: of the keys and
    values (None, None: those of the queries).  causal: the last query sees every
    key, the one before it all but the last, and so on.  scale: None for
    1 / sqrt(dim); workspace: tr_attention_workspace_bytes(...) bytes."""
    where = "tr_attention"
    shape = _shape(q, where, "q")
    rows, cols = shape
    if heads < 1 or cols % heads or kv_heads < 1 or heads % kv_heads:
        raise TrError(1, where, "q must have heads * dim columns, heads a multiple of kv_heads")
    dim = cols // heads
    dt = _elem(q)
    device = q.get_device()
    k_rows = _shape(k, where, "k")[0]
    pq, sq = _matrix(q, None, -1, device, where, "q")
    pk, sk = _matrix(k, (k_rows, kv_heads * dim), dt, device, where, "k")
    pv, sv = _matrix(v, (k_rows, kv_heads * dim), dt, device, where, "v")
    po, so = _matrix(out, shape, dt, device, where, "out")
    if k_starts is None:
        if k_lengths is not None:
            raise TrError(1, where, "k_lengths needs k_starts")
        k_starts, k_lengths = q_starts, q_lengths
    sequences = q_starts.numel() - 1
    if sequences < 0:
        raise TrError(1, where, "q_starts must hold sequences + 1 values")
    qs = _integers(q_starts, sequences + 1, device, where, "q_starts")
    ks = _integers(k_starts, sequences + 1, device, where, "k_starts")
    ql = _integers(q_lengths, sequences, device, where, "q_lengths")
    kl = _integers(k_lengths, sequences, device, where, "k_lengths")
    L = lib()
    ws = _workspace(workspace, L.tr_attention_workspace_bytes(rows, sequences, heads, kv_heads, dim), device, where)
    rc = L.tr_attention(pq, pk, pv, po, qs, ks, ql, kl, rows, k_rows, sequences, heads, kv_heads, dim, sq, sk, sv, so, dt,
                        dim ** -0.5 if scale is None else scale, bool(causal), ws, _stream(stream, device, where))
    if rc:
        check(rc, where)
