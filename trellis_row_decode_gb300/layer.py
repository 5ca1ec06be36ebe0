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
PyTorch operation.  No call records anything for torch.autograd: a result is cut off from
inputs that require gradients, and the caller chains embed_grad and rms_norm_grad by hand, as
examples/memory_layer.py does.  Wrong types, shapes or strides raise ValueError before anything
is queued; what the library itself refuses raises CPError.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import CP_ERR_INVALID_ARG, CPError, _check, lib

__all__ = ["CP_F32", "CP_F16", "CP_BF16", "embed", "embed_grad", "embed_grad_workspace",
           "rms_norm", "rms_norm_fp8", "rms_norm_grad", "rms_norm_grad_workspace",
           "quantize_fp8", "matmul_fp8", "matmul_fp8_workspace", "matmul_fp8_status"]

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
        L.cp_embed_grad.argtypes = [vp, i32, u64, vp, u64, u32, u64, u32, f32, i32, vp, i32, u64,
                                    vp, vp, u64, vp]
        L.cp_rms_norm.argtypes = [vp, u64, vp, u64, i32, vp, i32, u64, u32, f32, vp, vp, vp]
        L.cp_rms_norm_fp8.argtypes = [vp, u64, vp, u64, i32, vp, i32, u64, u32, f32, vp, vp, vp,
                                      vp]
        L.cp_rms_norm_grad_workspace_bytes.argtypes = [u64, u32]
        L.cp_rms_norm_grad_workspace_bytes.restype = u64
        L.cp_rms_norm_grad.argtypes = [vp, u64, vp, u64, vp, u64, i32, vp, i32, u64, u32, f32, vp,
                                       vp, vp, u64, vp]
        L.cp_quantize_fp8.argtypes = [vp, u64, i32, u64, u32, u32, vp, vp, vp]
        L.cp_matmul_fp8_workspace_bytes.argtypes = [vp, u64, vp, u64, u64, u64, u64]
        L.cp_matmul_fp8_workspace_bytes.restype = u64
        L.cp_matmul_fp8.argtypes = [vp, u64, vp, vp, u64, vp, u64, u64, u64, vp, i32, u64, vp, u64,
                                    vp]
        L.cp_matmul_fp8_status.argtypes = [vp]
        L.cp_matmul_fp8_status.restype = i32
        for f in (L.cp_embed, L.cp_embed_grad, L.cp_rms_norm, L.cp_rms_norm_fp8,
                  L.cp_rms_norm_grad, L.cp_quantize_fp8, L.cp_matmul_fp8):
            f.restype = i32
        _declared = L
    return _declared


def _device(t: torch.Tensor, name: str) -> int:
    """The index of t's device, which has to be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return dev


def _on(t: torch.Tensor, dev: int, name: str) -> int:
    """t's address; t has to lie on device `dev`."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same CUDA device as the others")
    return t.data_ptr()


def _stream(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError("stream and tensors must be on the same device")
    return stream.cuda_stream


def _empty(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """An allocation that belongs to the stream the kernels run on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _float(dtype: torch.dtype, name: str) -> int:
    code = _CODE.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16")
    return code


def _u32(value: int, name: str) -> int:
    """A size that the library takes in 32 bits: ctypes would cut a larger one without a word."""
    if not 0 <= value < 1 << 32:
        raise ValueError(f"{name} must be at least 0 and below 2^32")
    return value


def _rows(t: torch.Tensor, name: str) -> tuple[int, int, int]:
    """(rows, d, row stride) of t with its leading dimensions merged (as a view)."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 0:
        raise ValueError(f"{name} must have at least one dimension")
    if shape[-1] >> 32:
        raise ValueError(f"{name}'s rows must be shorter than 2^32")
    if len(shape) != 2:
        if len(shape) == 1:
            if shape[0] > 1 and strides[0] != 1:
                raise ValueError(f"{name} must have unit stride in its last dimension")
            return 1, shape[0], shape[0]
        try:
            t = t.view(-1, shape[-1]) if shape[-1] else t.view(0, 0)
        except RuntimeError:
            raise ValueError(f"{name}: leading dimensions must be mergeable without a copy"
                             ) from None
        shape, strides = t.shape, t.stride()
    rows, d = shape
    if d > 1 and strides[1] != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return rows, d, (strides[0] if rows > 1 else d)


def _ids(ids: torch.Tensor) -> int:
    if ids.dtype != torch.int64 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int64 CUDA tensor")
    return ids.numel()


def _status_ptr(status, dev: int):
    if status is None:
        return None
    if status.dtype != torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 CUDA tensor")
    return _on(status, dev, "status")


def _check_out(out: torch.Tensor, shape, dtype, dev: int, name: str) -> int:
    """The row stride of the caller's output, whose rows may lie apart."""
    if out.dtype != dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}")
    rows, d, stride = _rows(out, name)
    if rows > 1 and stride < d:
        raise ValueError(f"{name}'s rows must not overlap")
    _on(out, dev, name)
    return stride


def _whole(out, shape, dtype, like: torch.Tensor, dev: int, stream, name: str) -> torch.Tensor:
    """The caller's output, which has to be contiguous, or a new one."""
    if out is None:
        return _empty(shape, dtype, like, stream)
    if not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _check_out(out, shape, dtype, dev, name)
    return out


def _workspace(workspace, nbytes: int, like: torch.Tensor, dev: int, stream) -> torch.Tensor:
    if workspace is None:
        return _empty(nbytes, torch.uint8, like, stream)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() \
            or workspace.numel() < nbytes:
        raise ValueError(f"workspace must be a contiguous uint8 CUDA tensor of {nbytes} bytes")
    _on(workspace, dev, "workspace")
    return workspace


def embed(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
          out: torch.Tensor | None = None, status: torch.Tensor | None = None,
          stream=None) -> torch.Tensor:
    """scale * weight[ids], ids.shape + (d,) in weight's type (fp32 product, rounded once).

    An id outside the table gives a row of zeros and, where `status` (one int32 on the
    device) is given, sets its bit 0."""
    code = _float(weight.dtype, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must be [n_rows, d]")
    dev = _device(weight, "weight")
    n_rows, d, stride = _rows(weight, "weight")
    n = _ids(ids)
    shape = ids.shape + (d,)
    if out is None:
        out, out_stride = _empty(shape, weight.dtype, weight, stream), d
    else:
        out_stride = _check_out(out, shape, weight.dtype, dev, "out")
    _check(_lib().cp_embed(weight.data_ptr(), code, n_rows, d, stride, _on(ids, dev, "ids"), n,
                           scale, out.data_ptr(), out_stride, _status_ptr(status, dev),
                           _stream(stream, dev)), "cp_embed")
    return out


def embed_grad_workspace(n: int, n_rows: int, d: int) -> torch.Tensor:
    """A workspace for embed_grad calls of these sizes (uint8, on the current device)."""
    nbytes = int(_lib().cp_embed_grad_workspace_bytes(n, n_rows, _u32(d, "d")))
    if nbytes == 0 and (n or n_rows):
        raise CPError(CP_ERR_INVALID_ARG, "cp_embed_grad_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def embed_grad(dy: torch.Tensor, ids: torch.Tensor, n_rows: int, scale: float = 1.0,
               dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
               accumulate: bool = False, group: int = 1, status: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of embed by its table: [n_rows, d], row r = scale * the sum of dy over
    the lookups of r (fp32, in an order fixed by the ids), in `dtype` (default: dy's).

    dy has a row per lookup, or, with `group`, one for each `group` consecutive lookups (the
    gradient of their sum).

    accumulate=True adds to `out` instead of overwriting it and touches only the rows that
    ids name (with scale = -rate: a step of gradient descent on the table `out`)."""
    code = _float(dy.dtype, "dy")
    dev = _device(dy, "dy")
    n = _ids(ids)
    rows, d, dy_stride = _rows(dy, "dy")
    if _u32(group, "group") < 1 or rows * group != n:
        raise ValueError("dy must have one row for each `group` ids")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        dtype = dtype or dy.dtype
        out_code = _float(dtype, "the gradient")
        out, out_stride = _empty((n_rows, d), dtype, dy, stream), d
    else:
        if dtype is not None and out.dtype != dtype:
            raise ValueError("out and dtype differ")
        out_code = _float(out.dtype, "out")
        out_stride = _check_out(out, (n_rows, d), out.dtype, dev, "out")
    L = _lib()
    nbytes = L.cp_embed_grad_workspace_bytes(n, n_rows, d)
    ws = _workspace(workspace, nbytes, dy, dev, stream)
    _check(L.cp_embed_grad(dy.data_ptr(), code, dy_stride, _on(ids, dev, "ids"), n, group, n_rows,
                           d, scale, 1 if accumulate else 0, out.data_ptr(), out_code, out_stride,
                           _status_ptr(status, dev), ws.data_ptr(), ws.numel(),
                           _stream(stream, dev)), "cp_embed_grad")
    return out


def _weight(weight: torch.Tensor, d: int) -> int:
    if weight.dim() != 1 or weight.shape[0] != d or not weight.is_contiguous():
        raise ValueError("weight must be contiguous, one value per column")
    return _float(weight.dtype, "weight")


def _norm_inputs(x, weight, residual, residual_out, stream):
    code = _float(x.dtype, "x")
    dev = _device(x, "x")
    rows, d, xs = _rows(x, "x")
    wcode = _weight(weight, d)
    args = [x.data_ptr(), xs, None, 0, code, _on(weight, dev, "weight"), wcode, rows, d]
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return dev, args, None
    if residual.dtype != x.dtype or residual.shape != x.shape:
        raise ValueError("residual must have x's type and shape")
    args[3] = _rows(residual, "residual")[2]
    args[2] = _on(residual, dev, "residual")
    return dev, args, _whole(residual_out, x.shape, x.dtype, x, dev, stream, "residual_out")


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
             residual_out: torch.Tensor | None = None, stream=None):
    """y = s * weight / sqrt(mean(s^2) + eps) over the last dimension, s = x + residual.

    Returns y, and with a residual (y, h), h = s rounded to x's type (`residual_out` may be
    the residual itself: the stream is then updated in place)."""
    dev, args, h = _norm_inputs(x, weight, residual, residual_out, stream)
    y = _whole(out, x.shape, x.dtype, x, dev, stream, "out")
    _check(_lib().cp_rms_norm(*args, eps, y.data_ptr(), None if h is None else h.data_ptr(),
                              _stream(stream, dev)), "cp_rms_norm")
    return y if h is None else (y, h)


def rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                 stream=None):
    """The same norm left in 8 bits: (q, scales) or, with a residual, (q, scales, h).

    q is float8_e4m3fn of x's shape; scales fp32, one for each 128 columns of a row
    (x.shape[:-1] + (ceil(d / 128),)): y is about q * scales."""
    dev, args, h = _norm_inputs(x, weight, residual, residual_out, stream)
    q = _whole(out, x.shape, _E4M3, x, dev, stream, "out")
    sc = _whole(scales, x.shape[:-1] + ((args[8] + 127) // 128,), torch.float32, x, dev, stream,
                "scales")
    _check(_lib().cp_rms_norm_fp8(*args, eps, q.data_ptr(), sc.data_ptr(),
                                  None if h is None else h.data_ptr(), _stream(stream, dev)),
           "cp_rms_norm_fp8")
    return (q, sc) if h is None else (q, sc, h)


def rms_norm_grad_workspace(rows: int, d: int) -> torch.Tensor:
    """A workspace for rms_norm_grad calls of these sizes (uint8, on the current device)."""
    nbytes = int(_lib().cp_rms_norm_grad_workspace_bytes(rows, _u32(d, "d")))
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
    code = _float(h.dtype, "h")
    dev = _device(h, "h")
    rows, d, hs = _rows(h, "h")
    wcode = _weight(weight, d)
    if dy.dtype != h.dtype or dy.shape != h.shape:
        raise ValueError("dy must have h's type and shape")
    gs = _rows(dy, "dy")[2]
    rp, rs = None, 0
    if dres is not None:
        if dres.dtype != h.dtype or dres.shape != h.shape:
            raise ValueError("dres must have h's type and shape")
        rs = _rows(dres, "dres")[2]
        rp = _on(dres, dev, "dres")
    dx = _whole(dx, h.shape, h.dtype, h, dev, stream, "dx")
    dw = _whole(dw, (d,), weight.dtype, h, dev, stream, "dw")
    L = _lib()
    ws = _workspace(workspace, L.cp_rms_norm_grad_workspace_bytes(rows, d), h, dev, stream)
    _check(L.cp_rms_norm_grad(_on(dy, dev, "dy"), gs, h.data_ptr(), hs, rp, rs, code,
                              _on(weight, dev, "weight"), wcode, rows, d, eps, dx.data_ptr(),
                              dw.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream, dev)),
           "cp_rms_norm_grad")
    return dx, dw


def quantize_fp8(x: torch.Tensor, block_rows: int = 1, out: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, stream=None):
    """(q, scales) of x: float8_e4m3fn of x's shape, and one fp32 scale for each block of
    block_rows x 128, amax / 448.  block_rows 1 (activations): x [..., d], scales
    [..., ceil(d / 128)]; 128 (weights): x [rows, d], scales [ceil(rows / 128), ceil(d / 128)]."""
    code = _float(x.dtype, "x")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    if x.dim() != 2 and (x.dim() < 2 or block_rows != 1):
        raise ValueError("x must be [rows, d], or [..., d] for blocks of one row")
    dev = _device(x, "x")
    rows, d, xs = _rows(x, "x")
    q = _whole(out, x.shape, _E4M3, x, dev, stream, "out")
    lead = x.shape[:-1] if block_rows == 1 else (-(-rows // 128),)
    sc = _whole(scales, lead + (-(-d // 128),), torch.float32, x, dev, stream, "scales")
    _check(_lib().cp_quantize_fp8(x.data_ptr(), xs, code, rows, d, block_rows, q.data_ptr(),
                                  sc.data_ptr(), _stream(stream, dev)), "cp_quantize_fp8")
    return q, sc


def _scaled(t: torch.Tensor, scales: torch.Tensor, block: int, dev: int, name: str):
    """(rows, k, row stride) of an e4m3 operand whose scales fit it: [..., k] with blocks of one
    row, [rows, k] with larger ones."""
    if t.dtype != _E4M3 or (t.dim() != 2 and (t.dim() < 2 or block != 1)):
        raise ValueError(f"{name} must be float8_e4m3fn, {'[..., k]' if block == 1 else '[n, k]'}")
    rows, k, stride = _rows(t, name)
    want = (t.shape[:-1] if block == 1 else (-(-rows // block),)) + (-(-k // 128),)
    if scales.dtype != torch.float32 or scales.shape != want or not scales.is_contiguous():
        raise ValueError(f"{name}_scales must be contiguous float32 of shape {want}")
    return rows, k, stride


def matmul_fp8(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
               dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """a @ w.T, [..., n], for a [..., k] and w [n, k] in float8_e4m3fn with scales for each block
    of 128 along k (a_scales [..., ceil(k/128)], w_scales [ceil(n/128), ceil(k/128)], fp32),
    summed in fp32 and rounded once to `dtype` (to out's type where `out` is given).

    Rows that do not start on 16-byte boundaries are copied to such rows in `workspace`
    (matmul_fp8_workspace; allocated where it is not given), but for the smallest products."""
    dev = _device(a, "a")
    m, k, lda = _scaled(a, a_scales, 1, dev, "a")
    n, kw, ldw = _scaled(w, w_scales, 128, dev, "w")
    if kw != k:
        raise ValueError("a and w must have the same number of columns")
    if out is None:
        code = _float(dtype, "the output")
        out, ldo = _empty(a.shape[:-1] + (n,), dtype, a, stream), n
    else:
        code = _float(out.dtype, "the output")
        ldo = _check_out(out, a.shape[:-1] + (n,), out.dtype, dev, "out")
    pa, pw, ws = a.data_ptr(), _on(w, dev, "w"), None
    if (pa | pw | lda | ldw) & 15 or lda == 0 or ldw == 0:
        nbytes = _lib().cp_matmul_fp8_workspace_bytes(pa, lda, pw, ldw, m, n, k)
        if nbytes:
            ws = _workspace(workspace, nbytes, a, dev, stream)
    _check(_lib().cp_matmul_fp8(pa, lda, _on(a_scales, dev, "a_scales"), pw, ldw,
                                _on(w_scales, dev, "w_scales"), m, n, k, out.data_ptr(), code, ldo,
                                None if ws is None else ws.data_ptr(),
                                0 if ws is None else ws.numel(), _stream(stream, dev)),
           "cp_matmul_fp8")
    return out


def matmul_fp8_workspace(a: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """A workspace for matmul_fp8 calls on these operands (uint8; empty where nothing has to be
    copied)."""
    dev = _device(a, "a")
    m, k, lda = _rows(a, "a")
    n, kw, ldw = _rows(w, "w")
    if kw != k:
        raise ValueError("a and w must have the same number of columns")
    nbytes = _lib().cp_matmul_fp8_workspace_bytes(a.data_ptr(), lda, _on(w, dev, "w"), ldw, m, n, k)
    return torch.empty(int(nbytes), dtype=torch.uint8, device=a.device)


def matmul_fp8_status(stream=None) -> int:
    """Synchronise the stream; CP_ERR_CUDA if a wait inside a matmul_fp8 since the last call
    ran out of time (its output is then not valid), else CP_OK."""
    stream = torch.cuda.current_stream() if stream is None else stream
    return int(_lib().cp_matmul_fp8_status(stream.cuda_stream))
