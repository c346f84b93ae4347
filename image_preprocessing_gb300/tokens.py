"""Python face of the token-row operators (include/tr_token_ops.h); the
functions carry the C entry points' names.

Matrices are 2-D CUDA tensors with unit column stride (any row stride);
outputs and workspaces are the caller's, as everywhere in this package.  Each
call enqueues on `stream` (the current one if None) and raises TrError on a
refusal.
"""
from ._native import TrError, check, lib
from .api import _stream_handle

ELEM_F32, ELEM_F16, ELEM_BF16, ELEM_I8 = 0, 1, 2, 3
MAX_ROW, MAX_INT8_K = 32768, 131071   # TR_MAX_ROW, TR_MAX_INT8_K

_codes = {}


def _elem(t):
    if not _codes:
        import torch
        _codes.update({torch.float32: ELEM_F32, torch.float16: ELEM_F16, torch.bfloat16: ELEM_BF16,
                       torch.int8: ELEM_I8})
    return _codes.get(t.dtype, -1)


def _matrix(t, rows, cols, where, name):
    """Address and row stride of a (rows, cols) CUDA matrix; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dim() != 2 or t.size(0) != rows or t.size(1) != cols:
        raise TrError(1, where, "%s must be a (%d, %d) matrix" % (name, rows, cols))
    if not t.is_cuda:
        raise TrError(1, where, "%s must be a CUDA tensor" % name)
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise TrError(1, where, "%s must have unit column stride" % name)
    return t.data_ptr(), row


def _vector(t, n, where, name):
    """Address of n contiguous binary32 values; None for None."""
    if t is None:
        return None
    if _elem(t) != ELEM_F32 or t.numel() != n or not t.is_contiguous():
        raise TrError(1, where, "%s must be %d contiguous float32 values" % (name, n))
    if not t.is_cuda:
        raise TrError(1, where, "%s must be a CUDA tensor" % name)
    return t.data_ptr()


def _workspace(ws, need, where):
    if need == 0:
        return None
    if ws is None or ws.numel() * ws.element_size() < need or not ws.is_cuda or not ws.is_contiguous():
        raise TrError(1, where, "needs a contiguous CUDA workspace of at least %d bytes" % need)
    return ws.data_ptr()


def _types(where, dtype, *tensors):
    for name, t in tensors:
        if t is not None and _elem(t) != dtype:
            raise TrError(1, where, "%s has another type" % name)


def tr_rms_norm(x, out, weight=None, residual=None, residual_out=None, scale=None, eps=1e-6, stream=None):
    """h = x + residual; out = h / sqrt(mean(h^2) + eps) * weight, row by row.

    x, residual: float32, float16 or bfloat16 of one shape; out: of x's type,
    or int8, then with scale (rows float32) receiving max|row| / 127;
    residual_out: h in x's type (may be x or residual); weight: cols float32,
    or None for ones."""
    where = "tr_rms_norm"
    if x.dim() != 2:
        raise TrError(1, where, "x must be a matrix")
    rows, cols = x.shape
    dt, odt = _elem(x), _elem(out)
    _types(where, dt, ("residual", residual), ("residual_out", residual_out))
    px, sx = _matrix(x, rows, cols, where, "x")
    pr, sr = _matrix(residual, rows, cols, where, "residual")
    po, so = _matrix(out, rows, cols, where, "out")
    ph, sh = _matrix(residual_out, rows, cols, where, "residual_out")
    check(lib().tr_rms_norm(px, pr, _vector(weight, cols, where, "weight"), po, ph,
                            _vector(scale, rows, where, "scale"), rows, cols, sx, sr, so, sh, dt, odt, eps,
                            _stream_handle(stream)), where)


def tr_rms_norm_backward_workspace_bytes(rows, cols):
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
    if h.dim() != 2:
        raise TrError(1, where, "h must be a matrix")
    rows, cols = h.shape
    dt = _elem(h)
    _types(where, dt, ("dy", dy), ("dx", dx), ("dresidual", dresidual))
    py, sy = _matrix(dy, rows, cols, where, "dy")
    ph, sh = _matrix(h, rows, cols, where, "h")
    pr, sr = _matrix(dresidual, rows, cols, where, "dresidual")
    px, sx = _matrix(dx, rows, cols, where, "dx")
    ws = None
    if dweight is not None and rows > 0:
        ws = _workspace(workspace, lib().tr_rms_norm_backward_workspace_bytes(rows, cols), where)
    check(lib().tr_rms_norm_backward(py, ph, _vector(weight, cols, where, "weight"), pr, px,
                                     _vector(dweight, cols, where, "dweight"), rows, cols, sy, sh, sr, sx, dt, eps,
                                     ws, _stream_handle(stream)), where)


def tr_quantize_rows(x, q, scale, stream=None):
    """Rows of x (float32, float16, bfloat16) in 8 bits: q int8 of x's shape,
    scale rows float32; q * scale stands for x."""
    where = "tr_quantize_rows"
    if x.dim() != 2:
        raise TrError(1, where, "x must be a matrix")
    rows, cols = x.shape
    _types(where, ELEM_I8, ("q", q))
    px, sx = _matrix(x, rows, cols, where, "x")
    pq, sq = _matrix(q, rows, cols, where, "q")
    check(lib().tr_quantize_rows(px, pq, _vector(scale, rows, where, "scale"), rows, cols, sx, sq, _elem(x),
                                 _stream_handle(stream)), where)


def tr_dequantize_rows(q, scale, out, stream=None):
    """out = q * scale, row by row, in out's type."""
    where = "tr_dequantize_rows"
    if q.dim() != 2:
        raise TrError(1, where, "q must be a matrix")
    rows, cols = q.shape
    _types(where, ELEM_I8, ("q", q))
    pq, sq = _matrix(q, rows, cols, where, "q")
    po, so = _matrix(out, rows, cols, where, "out")
    check(lib().tr_dequantize_rows(pq, _vector(scale, rows, where, "scale"), po, rows, cols, sq, so, _elem(out),
                                   _stream_handle(stream)), where)


def tr_int8_matmul_workspace_bytes(M, N, K):
    return int(lib().tr_int8_matmul_workspace_bytes(M, N, K))


def tr_int8_matmul(x, x_scale, w, w_scale, y, bias=None, workspace=None, stream=None):
    """y = (x @ w.T) * x_scale[:, None] * w_scale + bias, the products summed
    exactly in integers.

    x: int8 (M, K), x_scale: M float32; w: int8 (N, K), w_scale: N float32;
    bias: N float32 or None; y: (M, N) float32, float16 or bfloat16; workspace:
    tr_int8_matmul_workspace_bytes(M, N, K) bytes."""
    where = "tr_int8_matmul"
    if x.dim() != 2 or w.dim() != 2:
        raise TrError(1, where, "x and w must be matrices")
    M, K = x.shape
    N = w.size(0)
    _types(where, ELEM_I8, ("x", x), ("w", w))
    px, sx = _matrix(x, M, K, where, "x")
    pw, sw = _matrix(w, N, K, where, "w")
    py, sy = _matrix(y, M, N, where, "y")
    ws = _workspace(workspace, lib().tr_int8_matmul_workspace_bytes(M, N, K), where)
    check(lib().tr_int8_matmul(px, _vector(x_scale, M, where, "x_scale"), pw, _vector(w_scale, N, where, "w_scale"),
                               _vector(bias, N, where, "bias"), py, M, N, K, sx, sw, sy, _elem(y), ws,
                               _stream_handle(stream)), where)
