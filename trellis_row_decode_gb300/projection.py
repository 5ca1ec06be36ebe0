"""The memory layer's projection in 16 bits and dropout (C ABI: include/cp.h).

``linear`` and ``linear_grad`` train the projection that ``matmul_fp8`` serves: bias, activation,
dropout and the residual's addition happen where the product's sums are.  ``dropout`` and
``dropout_grad`` mask rows anywhere else; a mask is made again from (p, seed, offset), not stored.

The conventions are those of the operators in ``layer``: argument marshalling only, tensors on the
current device with rows of unit stride, ``stream`` to queue on, no record for torch.autograd
(the caller chains ``linear_grad`` and ``dropout_grad`` by hand), ValueError for wrong types, shapes
or strides and CPError for what the library itself refuses.
"""
from __future__ import annotations

import ctypes as C
import importlib.machinery
import importlib.util
import warnings

import torch

from . import CP_ERR_INVALID_ARG, LIB_PATH, CPError, _check, lib
from . import layer as _layer
from .layer import (CP_BF16, CP_F16, CP_F32, _check_out, _device, _empty, _float, _on, _rows, _stream,
                    _workspace)

__all__ = ["ACTIVATIONS", "linear", "linear_workspace", "linear_grad", "linear_grad_workspace",
           "linear_status", "dropout", "dropout_grad"]

ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_ACT = {name: i for i, name in enumerate(ACTIVATIONS)}
_HALF = {torch.float16: CP_F16, torch.bfloat16: CP_BF16}
_CALLS_PATH = LIB_PATH.with_name("_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])
_declared = None
_calls = None


class _Checked:
    """What stands for the calls' common forms where the compiled code is not there: every call takes
    the checked way."""

    @staticmethod
    def dropout(*args):
        return NotImplemented

    linear = linear_grad = dropout


def _common():
    """The calls' common forms in compiled code (csrc/cp_calls.cpp), built beside libcp.so for this
    Python."""
    global _calls
    if _calls is None:
        lib()                                     # (raises where nothing has been built)
        path = str(_CALLS_PATH)
        loader = importlib.machinery.ExtensionFileLoader("_calls", path)
        try:
            calls = importlib.util.module_from_spec(
                importlib.util.spec_from_file_location("_calls", path, loader=loader))
            loader.exec_module(calls)
        except (ImportError, AttributeError) as e:    # none, another Python's, or another PyTorch's
            warnings.warn(f"calls of linear, linear_grad and dropout go through ctypes alone: {e}",
                          RuntimeWarning, stacklevel=3)
            calls = _Checked
        _calls = calls
    return _calls


def _lib():
    """libcp with this module's argument types declared."""
    global _declared
    if _declared is None:
        L = _layer._lib()
        vp, u64, u32, i32, f64 = C.c_void_p, C.c_uint64, C.c_uint32, C.c_int, C.c_double
        L.cp_dropout.argtypes = [vp, u64, vp, u64, i32, u64, u32, f64, u64, u64, vp, vp, u64, vp]
        L.cp_linear_workspace_bytes.argtypes = [vp, u64, vp, u64, u64, u64, u64]
        L.cp_linear.argtypes = [vp, u64, vp, u64, i32, u64, u64, u64, vp, i32, i32, f64, u64, u64,
                                vp, vp, u64, vp, i32, u64, vp, u64, vp, u64, vp]
        L.cp_linear_grad_workspace_bytes.argtypes = [u64, u64, u64]
        L.cp_linear_grad.argtypes = [vp, i32, u64, vp, u64, vp, u64, i32, vp, u64, u64, u64, u64,
                                     i32, f64, u64, u64, vp, i32, vp, u64, vp, i32, u64, vp, i32,
                                     vp, u64, vp]
        L.cp_linear_status.argtypes = [vp]
        L.cp_linear_grad_call_bytes.argtypes = [vp, i32, u64, vp, u64, vp, u64, i32, u64, u64, u64,
                                                i32, f64]
        for f in (L.cp_linear_workspace_bytes, L.cp_linear_grad_workspace_bytes,
                  L.cp_linear_grad_call_bytes):
            f.restype = u64
        for f in (L.cp_dropout, L.cp_linear, L.cp_linear_grad, L.cp_linear_status):
            f.restype = i32
        _declared = L
    return _declared


def _half(t: torch.Tensor, name: str) -> int:
    code = _HALF.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float16 or bfloat16")
    return code


def _activation(name: str) -> int:
    code = _ACT.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    return code


def _rng(seed: int, offset: int, rng, dev: int):
    """rng's address, and seed and offset checked: ctypes would cut larger ones without a word."""
    if (seed | offset) >> 64:                     # (a negative one too: its sign stays)
        raise ValueError("seed and offset must be at least 0 and below 2^64")
    if rng is None:
        return None
    if rng.dtype != torch.int64 or rng.numel() != 2 or not rng.is_contiguous():
        raise ValueError("rng must be a contiguous int64 CUDA tensor of two values")
    return _on(rng, dev, "rng")


def dropout(x: torch.Tensor, p: float, seed: int = 0, offset: int = 0,
            rng: torch.Tensor | None = None, residual: torch.Tensor | None = None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """residual + D(x) in x's type (without a residual D(x)): element [i, j] of x's rows (its
    leading dimensions merged) is kept and multiplied by 1 / (1 - p), or dropped, as word
    j mod 4 of Philox4x32-10 at (j / 4, i, offset) under the key `seed` says.

    The mask depends on p, seed, offset and the rows' shape alone: the backward pass makes it
    again (dropout_grad).  Each use of a mask wants an offset of its own.  `rng` (int64 [2] on the
    device: a seed, and what is added to `offset`) is read by the kernel as it runs, so that the
    replays of a captured graph draw masks of their own.  `out` may be x or the residual."""
    if out is None and stream is None:
        made = _common().dropout(x, residual, p, seed, offset, rng)
        if made is not NotImplemented:
            return made
    code = _float(x.dtype, "x")
    dev = _device(x, "x")
    rows, d, xs = _rows(x, "x")
    rp, rs = None, 0
    if residual is not None:
        if residual.dtype != x.dtype or residual.shape != x.shape:
            raise ValueError("residual must have x's type and shape")
        rs = _rows(residual, "residual")[2]
        rp = _on(residual, dev, "residual")
    gp = _rng(seed, offset, rng, dev)
    if out is None:
        out, ldo = _empty(x.shape, x.dtype, x, stream), d
    else:
        ldo = _check_out(out, x.shape, x.dtype, dev, "out")
    _check(_lib().cp_dropout(x.data_ptr(), xs, rp, rs, code, rows, d, p, seed, offset, gp,
                             out.data_ptr(), ldo, _stream(stream, dev)), "cp_dropout")
    return out


def dropout_grad(dy: torch.Tensor, p: float, seed: int = 0, offset: int = 0,
                 rng: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """The gradient of dropout by x: dy under the same mask (p, seed, offset and rng of the forward
    call).  The residual's gradient is dy itself."""
    return dropout(dy, p, seed, offset, rng, out=out, stream=stream)


def _operands(x: torch.Tensor, weight: torch.Tensor):
    """(device, type, m, n, k, row strides) of a projection."""
    code = _half(x, "x")
    if weight.dtype != x.dtype or weight.dim() != 2:
        raise ValueError("weight must be [n, k] of x's type")
    dev = _device(x, "x")
    m, k, ldx = _rows(x, "x")
    n, kw, ldw = _rows(weight, "weight")
    if kw != k:
        raise ValueError("x and weight must have the same number of columns")
    return dev, code, m, n, k, ldx, ldw


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
           activation: str = "none", residual: torch.Tensor | None = None, p: float = 0.0,
           seed: int = 0, offset: int = 0, rng: torch.Tensor | None = None,
           dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
           pre: bool | torch.Tensor = False, workspace: torch.Tensor | None = None, stream=None):
    """residual + D(act(x @ weight.T + bias)), [..., n], for x [..., k] and weight [n, k] in float16
    or bfloat16; everything in fp32 up to one rounding to `dtype` (default x's; out's where
    `out` is given; the residual has it too).  D: dropout with probability p, as ``dropout`` makes
    it on the output's rows.

    `out` may be the residual (the stream is updated in place); neither it nor `pre` may lie on x or
    weight.  With `pre` (True, or a tensor to fill) returns (out, pre): the sums in front of the
    activation in x's type, for linear_grad.  Operands off 16-byte boundaries and sums of a split k
    need `workspace` (linear_workspace; allocated where it is not given)."""
    act = _activation(activation)
    if out is None and stream is None and workspace is None and (pre is False or pre is True):
        made = _common().linear(x, weight, bias, act, residual, dtype, pre, p, seed, offset, rng)
        if made is not NotImplemented:
            return made
    dev, code, m, n, k, ldx, ldw = _operands(x, weight)
    shape = x.shape[:-1] + (n,)
    if out is None:
        dtype = dtype or x.dtype
        ocode = _float(dtype, "the output")
        out, ldo = _empty(shape, dtype, x, stream), n
    else:
        if dtype is not None and out.dtype != dtype:
            raise ValueError("out and dtype differ")
        ocode = _float(out.dtype, "out")
        ldo = _check_out(out, shape, out.dtype, dev, "out")
    bp, bcode = None, 0
    if bias is not None:
        if bias.dim() != 1 or bias.shape[0] != n or not bias.is_contiguous():
            raise ValueError("bias must be contiguous, one value per row of weight")
        bp, bcode = _on(bias, dev, "bias"), _float(bias.dtype, "bias")
    rp, rs = None, 0
    if residual is not None:
        if residual.dtype != out.dtype or residual.shape != shape:
            raise ValueError("residual must have the output's type and shape")
        rs = _rows(residual, "residual")[2]
        rp = _on(residual, dev, "residual")
    pp, ps = None, 0
    keep = pre is not False and pre is not None
    if keep:
        if pre is True:
            pre, ps = _empty(shape, x.dtype, x, stream), n
        else:
            ps = _check_out(pre, shape, x.dtype, dev, "pre")
        pp = pre.data_ptr()
    gp = _rng(seed, offset, rng, dev)
    L = _lib()
    xp, wp, sp, nbytes = x.data_ptr(), _on(weight, dev, "weight"), None, 0
    # (few rows on 16-byte boundaries, the form for single tokens, need none)
    if m > 128 or (xp | wp | 2 * (ldx | ldw)) & 15 or not ldx or not ldw:
        nbytes = L.cp_linear_workspace_bytes(xp, ldx, wp, ldw, m, n, k)
        if nbytes:
            workspace = _workspace(workspace, nbytes, x, dev, stream)
            sp = workspace.data_ptr()
    _check(L.cp_linear(xp, ldx, wp, ldw, code, m, n, k, bp, bcode, act, p, seed, offset, gp, rp, rs,
                       out.data_ptr(), ocode, ldo, pp, ps, sp, nbytes, _stream(stream, dev)),
           "cp_linear")
    return (out, pre) if keep else out


def linear_workspace(x: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """A workspace for linear calls on these operands (uint8; empty where none is needed)."""
    dev, _, m, n, k, ldx, ldw = _operands(x, weight)
    nbytes = _lib().cp_linear_workspace_bytes(x.data_ptr(), ldx, _on(weight, dev, "weight"), ldw,
                                              m, n, k)
    return torch.empty(nbytes, dtype=torch.uint8, device=x.device)


def linear_grad(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, activation: str = "none",
                pre: torch.Tensor | None = None, p: float = 0.0, seed: int = 0, offset: int = 0,
                rng: torch.Tensor | None = None, need_dx: bool = True, need_dw: bool = True,
                need_db: bool = True, accumulate: bool = False, dx: torch.Tensor | None = None,
                dw: torch.Tensor | None = None, db: torch.Tensor | None = None,
                dw_dtype: torch.dtype | None = None, db_dtype: torch.dtype | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """(dx, dw, db) of linear: with dz = D(dy) act'(pre), dx = dz @ weight in x's type,
    dw = dz.T @ x in `dw_dtype` (default weight's), db = the sum of dz over the rows in `db_dtype`
    (default weight's); None in the place of one that is not needed.

    dy has x's type, or float32 (that of linear's output); the residual's gradient is dy itself.
    activation, p, seed, offset and rng are those of the forward call, `pre` what it left.  The
    products take dz rounded to x's type (dy itself without activation and dropout).
    accumulate=True adds to the `dw` and `db` that are given (gradients of several batches); `dx` and
    `dw` may not lie on x, weight, or a dy that is taken as it is."""
    act = _activation(activation)
    if (need_dx and need_dw and need_db and not accumulate and dx is None and dw is None
            and db is None and workspace is None and stream is None):
        made = _common().linear_grad(dy, x, weight, act, pre, dw_dtype, db_dtype, p, seed, offset,
                                     rng)
        if made is not NotImplemented:
            return made
    dev, code, m, n, k, ldx, ldw = _operands(x, weight)
    if dy.dtype != x.dtype and dy.dtype != torch.float32:
        raise ValueError("dy must have x's type or float32")
    if dy.shape != x.shape[:-1] + (n,):
        raise ValueError("dy must have x's leading dimensions and one column per row of weight")
    lddy = _rows(dy, "dy")[2]
    pp, ps = None, 0
    if act != 0:
        if pre is None or pre.dtype != x.dtype or pre.shape != dy.shape:
            raise ValueError("an activation needs pre, of dy's shape and x's type")
        ps = _rows(pre, "pre")[2]
        pp = _on(pre, dev, "pre")
    elif pre is not None:
        raise ValueError("pre goes with an activation")
    if accumulate and ((need_dw and dw is None) or (need_db and db is None)):
        raise ValueError("accumulate needs dw and db where they are wanted")
    dxp, dxs = None, 0
    if need_dx:
        if dx is None:
            dx, dxs = _empty(x.shape, x.dtype, x, stream), k
        else:
            dxs = _check_out(dx, x.shape, x.dtype, dev, "dx")
        dxp = dx.data_ptr()
    elif dx is not None:
        raise ValueError("dx is given, but not needed")
    dwp, dws, dwc = None, 0, 0
    if need_dw:
        if dw is None:
            dw, dws = _empty((n, k), dw_dtype or weight.dtype, x, stream), k
        else:
            if dw_dtype is not None and dw.dtype != dw_dtype:
                raise ValueError("dw and dw_dtype differ")
            dws = _check_out(dw, (n, k), dw.dtype, dev, "dw")
        dwp, dwc = dw.data_ptr(), _float(dw.dtype, "dw")
    elif dw is not None:
        raise ValueError("dw is given, but not needed")
    dbp, dbc = None, 0
    if need_db:
        if db is None:
            db = _empty((n,), db_dtype or weight.dtype, x, stream)
        else:
            if db_dtype is not None and db.dtype != db_dtype:
                raise ValueError("db and db_dtype differ")
            if not db.is_contiguous():
                raise ValueError("db must be contiguous")
            _check_out(db, (n,), db.dtype, dev, "db")
        dbp, dbc = db.data_ptr(), _float(db.dtype, "db")
    elif db is not None:
        raise ValueError("db is given, but not needed")
    gp = _rng(seed, offset, rng, dev)
    L = _lib()
    gradient = (_on(dy, dev, "dy"), code if dy.dtype == x.dtype else CP_F32, lddy, x.data_ptr(),
                ldx, _on(weight, dev, "weight"), ldw, code)
    nbytes, sp = L.cp_linear_grad_call_bytes(*gradient, m, n, k, act, p), None
    if nbytes:
        workspace = _workspace(workspace, nbytes, x, dev, stream)
        sp = workspace.data_ptr()
    _check(L.cp_linear_grad(*gradient, pp, ps, m, n, k, act, p, seed, offset, gp,
                            1 if accumulate else 0, dxp, dxs, dwp, dwc, dws, dbp, dbc, sp, nbytes,
                            _stream(stream, dev)), "cp_linear_grad")
    return dx, dw, db


def linear_grad_workspace(m: int, n: int, k: int) -> torch.Tensor:
    """A workspace for linear_grad calls of these sizes (m rows, weight [n, k]; uint8, on the
    current device)."""
    nbytes = int(_lib().cp_linear_grad_workspace_bytes(m, n, k))
    if nbytes == 0:
        raise CPError(CP_ERR_INVALID_ARG, "cp_linear_grad_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def linear_status(stream=None) -> int:
    """Synchronise the stream; CP_ERR_CUDA if a wait inside linear or linear_grad ran out since the
    last call."""
    dev = torch.cuda.current_device()
    return int(_lib().cp_linear_status(_stream(stream, dev)))
