"""The memory layer's operators around the lookup-decode (C ABI: include/cp.h).

Training a table's rows before they are encoded: ``embed`` and ``embed_grad``.
Bringing rows into the residual stream: ``rms_norm`` and ``rms_norm_grad``.
Projecting them in 8 bits: ``rms_norm_fp8``, ``quantize_fp8`` and ``matmul_fp8``.

Argument marshalling only: every step runs in libcp's kernels.  Tensors lie on the
current device, with rows of unit stride; a row stride may exceed the row (a slice
of a wider tensor) and, for inputs, be zero (an expanded row).  ``stream`` is the
``torch.cuda.Stream`` to queue on (default: the current one): outputs that the call
allocates, and its workspace, belong to that stream.  A caller that hands in tensors
made on another stream, or uses the outputs on one, orders the streams as for any
PyTorch operation.  Wrong types, shapes or strides raise ValueError before anything
is queued; what the library itself refuses raises CPError.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import CP_ERR_INVALID_ARG, CPError, _check, lib

__all__ = ["CP_F32", "CP_F16", "CP_BF16", "embed", "embed_grad", "embed_grad_workspace",
           "rms_norm", "rms_norm_fp8", "rms_norm_grad", "rms_norm_grad_workspace",
           "quantize_fp8", "matmul_fp8", "matmul_fp8_status"]

CP_F32, CP_F16, CP_BF16 = 0, 1, 2
_CODE = {torch.float32: CP_F32, torch.float16: CP_F16, torch.bfloat16: CP_BF16}
_E4M3 = torch.float8_e4m3fn
_declared = None


def _lib():
    """libcp with this module's argument types declared."""
    global _declared
    if _declared is None:
        L = lib()
        vp, u64, u32, i32, f32 = C.c_void_p, C.c_uint64, C.c_uint32, C.c_int, C.c_float
        L.cp_embed.argtypes = [vp, i32, u64, u32, u64, vp, u64, f32, vp, u64, vp, vp]
        L.cp_embed_grad_workspace_bytes.argtypes = [u64, u64, u32]
        L.cp_embed_grad_workspace_bytes.restype = u64
        L.cp_embed_grad.argtypes = [vp, i32, u64, vp, u64, u64, u32, f32, i32, vp, i32, u64, vp,
                                    vp, u64, vp]
        L.cp_rms_norm.argtypes = [vp, u64, vp, u64, i32, vp, i32, u64, u32, f32, vp, vp, vp]
        L.cp_rms_norm_fp8.argtypes = [vp, u64, vp, u64, i32, vp, i32, u64, u32, f32, vp, vp, vp,
                                      vp]
        L.cp_rms_norm_grad_workspace_bytes.argtypes = [u64, u32]
        L.cp_rms_norm_grad_workspace_bytes.restype = u64
        L.cp_rms_norm_grad.argtypes = [vp, u64, vp, u64, vp, u64, i32, vp, i32, u64, u32, f32, vp,
                                       vp, vp, u64, vp]
        L.cp_quantize_fp8.argtypes = [vp, u64, i32, u64, u32, u32, vp, vp, vp]
        L.cp_matmul_fp8.argtypes = [vp, u64, vp, vp, u64, vp, u64, u64, u64, vp, i32, u64, vp]
        L.cp_matmul_fp8_status.argtypes = [vp]
        L.cp_matmul_fp8_status.restype = i32
        for f in (L.cp_embed, L.cp_embed_grad, L.cp_rms_norm, L.cp_rms_norm_fp8,
                  L.cp_rms_norm_grad, L.cp_quantize_fp8, L.cp_matmul_fp8):
            f.restype = i32
        _declared = L
    return _declared


def _stream(stream, device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if stream.device != device:
        raise ValueError("stream and tensors must be on the same device")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An allocation that belongs to the stream the kernels run on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _float(t: torch.Tensor, name: str) -> int:
    code = _CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16")
    return code


def _here(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return t


def _rows(t: torch.Tensor, name: str) -> tuple[torch.Tensor, int]:
    """t as [rows, d] and its row stride (leading dimensions are flattened, as a view)."""
    _here(t, name)
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{name} must have at least one dimension")
        try:
            t = t.view(-1, t.shape[-1]) if t.shape[-1] else t.view(0, 0)
        except RuntimeError:
            raise ValueError(f"{name}: leading dimensions must be mergeable without a copy"
                             ) from None
    d = t.shape[1]
    if d > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return t, (t.stride(0) if t.shape[0] > 1 else d)


def _ids(ids: torch.Tensor) -> int:
    if ids.dtype != torch.int64 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int64 CUDA tensor")
    _here(ids, "ids")
    return ids.numel()


def _status_ptr(status):
    if status is None:
        return None
    if status.dtype != torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 CUDA tensor")
    return _here(status, "status").data_ptr()


def _out(out, shape, dtype, device, stream, name) -> tuple[torch.Tensor, int]:
    """The caller's output, checked, or a new one; and its row stride."""
    shape = tuple(shape)
    if out is None:
        return _empty(shape, dtype, device, stream), shape[-1]
    if out.dtype != dtype or tuple(out.shape) != shape:
        raise ValueError(f"{name} must be {dtype} of shape {shape}")
    t, stride = _rows(out, name)
    if t.shape[0] > 1 and stride < t.shape[1]:
        raise ValueError(f"{name}'s rows must not overlap")
    return out, stride


def _whole(out, shape, dtype, device, stream, name) -> torch.Tensor:
    """The same for outputs that have to be contiguous."""
    if out is not None and not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _out(out, shape, dtype, device, stream, name)[0]


def _workspace(workspace, nbytes: int, device, stream) -> torch.Tensor:
    if workspace is None:
        return _empty(nbytes, torch.uint8, device, stream)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() \
            or workspace.numel() < nbytes:
        raise ValueError(f"workspace must be a contiguous uint8 CUDA tensor of {nbytes} bytes")
    return _here(workspace, "workspace")


def embed(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
          out: torch.Tensor | None = None, status: torch.Tensor | None = None,
          stream=None) -> torch.Tensor:
    """scale * weight[ids], ids.shape + (d,) in weight's type (fp32 product, rounded once).

    An id outside the table gives a row of zeros and, where `status` (one int32 on the
    device) is given, sets its bit 0."""
    code = _float(weight, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must be [n_rows, d]")
    w, stride = _rows(weight, "weight")
    n = _ids(ids)
    d = w.shape[1]
    out, out_stride = _out(out, ids.shape + (d,), w.dtype, w.device, stream, "out")
    _check(_lib().cp_embed(w.data_ptr(), code, w.shape[0], d, stride, ids.data_ptr(), n, scale,
                           out.data_ptr(), out_stride, _status_ptr(status),
                           _stream(stream, w.device)), "cp_embed")
    return out


def embed_grad_workspace(n: int, n_rows: int, d: int) -> torch.Tensor:
    """A workspace for embed_grad calls of these sizes (uint8, on the current device)."""
    nbytes = int(_lib().cp_embed_grad_workspace_bytes(n, n_rows, d))
    if nbytes == 0 and (n or n_rows):
        raise CPError(CP_ERR_INVALID_ARG, "cp_embed_grad_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def embed_grad(dy: torch.Tensor, ids: torch.Tensor, n_rows: int, scale: float = 1.0,
               dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
               accumulate: bool = False, status: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of embed by its table: [n_rows, d], row r = scale * the sum of dy over
    the lookups of r (fp32, in an order fixed by the ids), in `dtype` (default: dy's).

    accumulate=True adds to `out` instead of overwriting it and touches only the rows that
    ids name (with scale = -rate: a step of gradient descent on the table `out`)."""
    code = _float(dy, "dy")
    n = _ids(ids)
    g, dy_stride = _rows(dy, "dy")
    d = g.shape[1]
    if tuple(dy.shape) != tuple(ids.shape) + (d,):
        raise ValueError("dy must be ids.shape + (d,)")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if out is not None and dtype is not None and out.dtype != dtype:
        raise ValueError("out and dtype differ")
    out, out_stride = _out(out, (n_rows, d), out.dtype if out is not None else dtype or dy.dtype,
                           g.device, stream, "out")
    out_code = _float(out, "out")
    L = _lib()
    nbytes = L.cp_embed_grad_workspace_bytes(n, n_rows, d)
    ws = _workspace(workspace, nbytes, g.device, stream)
    _check(L.cp_embed_grad(g.data_ptr(), code, dy_stride, ids.data_ptr(), n, n_rows, d, scale,
                           1 if accumulate else 0, out.data_ptr(), out_code, out_stride,
                           _status_ptr(status), ws.data_ptr(), ws.numel(),
                           _stream(stream, g.device)), "cp_embed_grad")
    return out


def _weight(weight: torch.Tensor, d: int) -> int:
    code = _float(weight, "weight")
    if weight.dim() != 1 or weight.shape[0] != d or not weight.is_contiguous():
        raise ValueError("weight must be contiguous, one value per column")
    _here(weight, "weight")
    return code


def _norm_inputs(x, weight, residual, residual_out, stream):
    code = _float(x, "x")
    x2, x_stride = _rows(x, "x")
    wcode = _weight(weight, x2.shape[1])
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return code, wcode, x2, x_stride, None, 0, None
    if residual.dtype != x.dtype or residual.shape != x.shape:
        raise ValueError("residual must have x's type and shape")
    r2, r_stride = _rows(residual, "residual")
    h = _whole(residual_out, x.shape, x.dtype, x.device, stream, "residual_out")
    return code, wcode, x2, x_stride, r2.data_ptr(), r_stride, h


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
             residual_out: torch.Tensor | None = None, stream=None):
    """y = s * weight / sqrt(mean(s^2) + eps) over the last dimension, s = x + residual.

    Returns y, and with a residual (y, h), h = s rounded to x's type (`residual_out` may be
    the residual itself: the stream is then updated in place)."""
    code, wcode, x2, xs, rp, rs, h = _norm_inputs(x, weight, residual, residual_out, stream)
    y = _whole(out, x.shape, x.dtype, x.device, stream, "out")
    _check(_lib().cp_rms_norm(x2.data_ptr(), xs, rp, rs, code, weight.data_ptr(), wcode,
                              x2.shape[0], x2.shape[1], eps, y.data_ptr(),
                              None if h is None else h.data_ptr(), _stream(stream, x.device)),
           "cp_rms_norm")
    return y if h is None else (y, h)


def rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                 stream=None):
    """The same norm left in 8 bits: (q, scales) or, with a residual, (q, scales, h).

    q is float8_e4m3fn of x's shape; scales fp32, one for each 128 columns of a row
    (x.shape[:-1] + (ceil(d / 128),)): y is about q * scales."""
    code, wcode, x2, xs, rp, rs, h = _norm_inputs(x, weight, residual, residual_out, stream)
    rows, d = x2.shape
    q = _whole(out, x.shape, _E4M3, x.device, stream, "out")
    sc = _whole(scales, x.shape[:-1] + ((d + 127) // 128,), torch.float32, x.device, stream,
                "scales")
    _check(_lib().cp_rms_norm_fp8(x2.data_ptr(), xs, rp, rs, code, weight.data_ptr(), wcode, rows,
                                  d, eps, q.data_ptr(), sc.data_ptr(),
                                  None if h is None else h.data_ptr(),
                                  _stream(stream, x.device)), "cp_rms_norm_fp8")
    return (q, sc) if h is None else (q, sc, h)


def rms_norm_grad_workspace(rows: int, d: int) -> torch.Tensor:
    """A workspace for rms_norm_grad calls of these sizes (uint8, on the current device)."""
    nbytes = int(_lib().cp_rms_norm_grad_workspace_bytes(rows, d))
    if nbytes == 0:
        raise CPError(CP_ERR_INVALID_ARG, "cp_rms_norm_grad_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def rms_norm_grad(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                  dres: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                  dw: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(dx, dw) of y = rms_norm at its summed input h: dx is the gradient by x and by the
    residual alike (`dres`, the gradient that reaches h past the norm, is added), dw the
    gradient by weight in weight's type.  `dx` may be `dres` or `dy` itself."""
    code = _float(h, "h")
    h2, hs = _rows(h, "h")
    rows, d = h2.shape
    wcode = _weight(weight, d)
    if dy.dtype != h.dtype or dy.shape != h.shape:
        raise ValueError("dy must have h's type and shape")
    g2, gs = _rows(dy, "dy")
    rp, rs = None, 0
    if dres is not None:
        if dres.dtype != h.dtype or dres.shape != h.shape:
            raise ValueError("dres must have h's type and shape")
        r2, rs = _rows(dres, "dres")
        rp = r2.data_ptr()
    dx = _whole(dx, h.shape, h.dtype, h.device, stream, "dx")
    dw = _whole(dw, (d,), weight.dtype, h.device, stream, "dw")
    L = _lib()
    ws = _workspace(workspace, L.cp_rms_norm_grad_workspace_bytes(rows, d), h.device, stream)
    _check(L.cp_rms_norm_grad(g2.data_ptr(), gs, h2.data_ptr(), hs, rp, rs, code,
                              weight.data_ptr(), wcode, rows, d, eps, dx.data_ptr(),
                              dw.data_ptr(), ws.data_ptr(), ws.numel(),
                              _stream(stream, h.device)), "cp_rms_norm_grad")
    return dx, dw


def quantize_fp8(x: torch.Tensor, block_rows: int = 1, out: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, stream=None):
    """(q, scales) of x [rows, d]: float8_e4m3fn, and one fp32 scale for each block of
    block_rows x 128 (1: activations, 128: weights), amax / 448."""
    code = _float(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [rows, d]")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    x2, xs = _rows(x, "x")
    rows, d = x2.shape
    q = _whole(out, (rows, d), _E4M3, x.device, stream, "out")
    sc = _whole(scales, (-(-rows // block_rows), -(-d // 128)), torch.float32, x.device, stream,
                "scales")
    _check(_lib().cp_quantize_fp8(x2.data_ptr(), xs, code, rows, d, block_rows, q.data_ptr(),
                                  sc.data_ptr(), _stream(stream, x.device)), "cp_quantize_fp8")
    return q, sc


def _scaled(t, scales, rows, name):
    if t.dtype != _E4M3 or t.dim() != 2:
        raise ValueError(f"{name} must be float8_e4m3fn, [rows, k]")
    t2, stride = _rows(t, name)
    want = (rows(t.shape[0]), -(-t.shape[1] // 128))
    if scales.dtype != torch.float32 or tuple(scales.shape) != want \
            or not scales.is_contiguous():
        raise ValueError(f"{name}_scales must be contiguous float32 of shape {want}")
    _here(scales, f"{name}_scales")
    return t2, stride


def matmul_fp8(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
               dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """a @ w.T for a [m, k] and w [n, k] in float8_e4m3fn with scales for each block of 128
    along k (a_scales [m, ceil(k/128)], w_scales [ceil(n/128), ceil(k/128)], fp32), summed in
    fp32 and rounded once to `dtype`."""
    a2, lda = _scaled(a, a_scales, lambda m: m, "a")
    w2, ldw = _scaled(w, w_scales, lambda n: -(-n // 128), "w")
    m, k = a2.shape
    n = w2.shape[0]
    if w2.shape[1] != k:
        raise ValueError("a and w must have the same number of columns")
    if out is not None:
        dtype = out.dtype
    code = _CODE.get(dtype)
    if code is None:
        raise ValueError("the output must be float32, float16 or bfloat16")
    out, ldo = _out(out, (m, n), dtype, a.device, stream, "out")
    _check(_lib().cp_matmul_fp8(a2.data_ptr(), lda, a_scales.data_ptr(), w2.data_ptr(), ldw,
                                w_scales.data_ptr(), m, n, k, out.data_ptr(), code, ldo,
                                _stream(stream, a.device)), "cp_matmul_fp8")
    return out


def matmul_fp8_status(stream=None) -> int:
    """Synchronise the stream; CP_ERR_CUDA if a wait inside a matmul_fp8 since the last call
    ran out of time (its output is then not valid), else CP_OK."""
    stream = torch.cuda.current_stream() if stream is None else stream
    return int(_lib().cp_matmul_fp8_status(stream.cuda_stream))
