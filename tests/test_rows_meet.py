"""Outputs that lie on what a call reads while it writes them are refused, before any CUDA call (so this
runs without a GPU); the rule is plain C++ (cp_geometry.h), held against counting the bytes."""
import ctypes as C
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent
CSRC = ROOT / "trellis_row_decode_gb300" / "csrc"
BAD = 1          # CP_ERR_INVALID_ARG


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_rows_meet_where_their_bytes_do(tmp_path):
    exe = tmp_path / "meet"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", "-o", str(exe),
                    str(ROOT / "tests" / "sanitize" / "meet_main.cpp")], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stderr
    assert "meet ok" in run.stdout


@pytest.fixture(scope="module")
def L():
    import trellis_row_decode_gb300 as cp
    from trellis_row_decode_gb300 import build_ext, projection
    if not cp.LIB_PATH.exists():
        build_ext.build()
    return projection._lib()


@pytest.fixture(scope="module")
def p():
    buf = (C.c_uint8 * (1 << 16))()
    yield (C.addressof(buf) + 63) & ~63
    del buf


def refused(L, status, why):
    return status == BAD and why in L.cp_last_error().decode()


def test_linear_refuses_outputs_on_its_inputs(L, p):
    """bf16, x and out [4][64]: each pair of arrays that meets, whole or in part, in one buffer of rows."""
    m, n, k = 4, 64, 64

    def call(x, w, out, xs=64, os=64, res=None, rs=0, pre=None, ps=64):
        return L.cp_linear(x, xs, w, 64, 2, m, n, k, None, 0, 0, 0.0, 0, 0, None, res, rs, out, 2, os,
                           pre, ps, None, 0, None)
    far, far2 = p + 32768, p + 49152
    on_x = "out or pre lies on x or w"
    for args in [dict(x=p, w=far, out=p), dict(x=p, w=far, out=p, res=p, rs=64),
                 dict(x=p, w=far, out=p + 128), dict(x=p + 256, w=far, out=p),
                 dict(x=far, w=p, out=p), dict(x=far, w=p, out=p + 64 * 127),
                 dict(x=p, w=far, out=far2, pre=p), dict(x=far2, w=p, out=far, pre=p + 128),
                 dict(x=p, xs=160, w=far, out=p + 96, os=160)]:
        assert refused(L, call(**args), on_x), args
    on_residual = "out lies on part of the residual"
    for args in [dict(x=far, w=far2, out=p, res=p + 128, rs=64),
                 dict(x=far, w=far2, out=p, res=p, rs=0),
                 dict(x=far, w=far2, out=p, pre=p), dict(x=far, w=far2, out=p, pre=p + 256),
                 dict(x=far, w=far2, out=p, res=p + 4096, rs=64, pre=p + 4096)]:
        assert refused(L, call(**args), on_residual), args


def test_linear_grad_refuses_outputs_on_its_inputs(L, p):
    m, n, k = 8, 64, 64
    dy, x, w, o, ws = p, p + 8192, p + 16384, p + 32768, p + 49152

    def call(dx=None, dw=None, pre=None, act=0, prob=0.0, dwt=2, wb=1 << 14):
        return L.cp_linear_grad(dy, 2, 64, x, 64, w, 64, 2, pre, 64 if pre else 0, m, n, k, act, prob,
                                0, 0, None, 0, dx, 64, dw, dwt, 64, None, 0, ws, wb, None)
    why = "dx or dw lies on dy, x or w"
    for args in [dict(dx=dy), dict(dw=dy), dict(dw=x), dict(dx=x, dw=o), dict(dx=w), dict(dx=o, dw=w),
                 dict(dx=dy + 128), dict(dx=x + 128, dw=o), dict(dx=o, dw=w + 1024),
                 dict(dx=x, dw=o, pre=o + 8192, act=2), dict(dx=w, pre=o, act=2, prob=0.5)]:
        assert refused(L, call(**args), why), args


def test_dropout_refuses_outputs_on_part_of_its_inputs(L, p):
    def call(x, out, res=None, xs=64, os=64, rs=64):
        return L.cp_dropout(x, xs, res, rs, 2, 4, 64, 0.5, 1, 2, None, out, os, None)
    far = p + 32768
    for args in [dict(x=p, out=p + 128), dict(x=p + 2, out=p), dict(x=far, res=p, out=p + 64),
                 dict(x=p, res=far, out=p + 384)]:
        assert refused(L, call(**args), "out lies on part of x or of the residual"), args
