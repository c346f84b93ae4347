"""Python face of the token-row operators (include/tr_token_ops.h); the
functions carry the C entry points' names.

Matrices are 2-D CUDA tensors with unit column stride (any row stride);
outputs and workspaces are the caller's, as everywhere in this package.  Each
call enqueues on `stream` (the current one if None) and raises TrError on a
refusal.  The tensors are on the current device, all of them: the library
launches there, and a tensor elsewhere is refused.
"""
from ._native import TrError, check, lib

ELEM_F32, ELEM_F16, ELEM_BF16, ELEM_I8 = 0, 1, 2, 3
MAX_ROW, MAX_INT8_K = 32768, 131071   # TR_MAX_ROW, TR_MAX_INT8_K

_codes = {}           # torch dtypes, filled when the first tensor comes
_current_stream = _current_device = None


def _prepare():
    global _current_stream, _current_device
    import torch
    _codes.update({torch.float32: ELEM_F32, torch.float16: ELEM_F16, torch.bfloat16: ELEM_BF16,
                   torch.int8: ELEM_I8})
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
