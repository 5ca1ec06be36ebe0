"""Host-side argument checks of cp_linear, cp_linear_grad and cp_dropout (refused before any CUDA
call, so they run without a GPU), and the generator's known answers for the tests' own form of it."""
import ctypes as C

import numpy as np
import pytest

from linear_util import mask64, philox

BAD = 1          # CP_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    import trellis_row_decode_gb300 as cp
    from trellis_row_decode_gb300 import build_ext, projection
    if not cp.LIB_PATH.exists():
        build_ext.build()
    return projection._lib()


@pytest.fixture(scope="module")
def p():
    buf = (C.c_uint8 * 4096)()
    at = (C.addressof(buf) + 63) & ~63
    yield at
    del buf


def test_generator_known_answers():
    """Published with the generator: counter and key of zeros, of ones, and of pi's digits."""
    f = 0xFFFFFFFF
    for args, want in [((0,) * 6, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
                       ((f,) * 6, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
                       ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344, 0xa4093822, 0x299f31d0),
                        "d16cfe09 94fdcceb 5001e420 24126ea1")]:
        assert " ".join(f"{int(w):08x}" for w in philox(*args)) == want
    assert mask64(3, 9, 0.0, 5, 6).all() and not mask64(3, 9, 1.0, 5, 6).any()
    assert np.isclose(mask64(200, 500, 0.3, 1 << 63, 1 << 40).double().mean(), 0.7, atol=0.01)


def test_dropout_arguments(L, p):
    ok = dict(x=p, xs=8, r=None, rs=0, t=0, m=2, d=8, p=0.5, seed=1, off=2, rng=None, o=p, os=8)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_dropout(a["x"], a["xs"], a["r"], a["rs"], a["t"], a["m"], a["d"], a["p"],
                            a["seed"], a["off"], a["rng"], a["o"], a["os"], None)
    for kw in [dict(t=3), dict(t=-1), dict(xs=7), dict(os=7), dict(os=0), dict(r=p, rs=7),
               dict(m=1 << 31), dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(rng=p + 4),
               dict(x=None), dict(o=None), dict(x=p + 2), dict(o=p + 2), dict(r=p + 1, rs=8),
               dict(t=2, x=p + 1)]:
        assert call(**kw) == BAD, kw
    assert call(m=0) == 0 and call(d=0) == 0 and call(m=0, x=None, o=None) == 0


def test_linear_arguments(L, p):
    ok = dict(x=p, xs=8, w=p, ws=8, t=2, m=2, n=3, k=8, b=None, bt=0, act=0, p=0.0, rng=None,
              r=None, rs=0, o=p, ot=0, os=3, pre=None, ps=0, wk=None, wb=0)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_linear(a["x"], a["xs"], a["w"], a["ws"], a["t"], a["m"], a["n"], a["k"], a["b"],
                           a["bt"], a["act"], a["p"], 0, 0, a["rng"], a["r"], a["rs"], a["o"],
                           a["ot"], a["os"], a["pre"], a["ps"], a["wk"], a["wb"], None)
    big = dict(m=300, n=2000, k=16, xs=16, ws=16, os=2000)
    for kw in [dict(t=0), dict(t=3), dict(ot=3), dict(b=p, bt=4), dict(xs=7), dict(ws=7),
               dict(os=2), dict(os=0), dict(m=1 << 31), dict(n=1 << 31), dict(k=1 << 30),
               dict(r=p, rs=2), dict(pre=p, ps=2), dict(act=5), dict(act=-1), dict(p=-1.0),
               dict(p=float("nan")), dict(rng=p + 4), dict(x=None), dict(w=None), dict(o=None),
               dict(x=p + 1), dict(w=p + 1), dict(o=p + 2), dict(b=p + 2), dict(r=p + 2, rs=3),
               dict(pre=p + 1, ps=3), dict(xs=9), dict(x=p + 2), dict(ws=0),
               dict(xs=9, wk=p, wb=31), dict(xs=9, wk=p + 8, wb=4096),
               dict(big, x=p + 2, wk=p, wb=300 * 32 - 1)]:
        assert call(**kw) == BAD, kw
    assert call(m=0) == 0 and call(n=0) == 0 and call(m=0, x=None, o=None) == 0


def test_linear_grad_arguments(L, p):
    ok = dict(dy=p, dt=2, ds=8, x=p, xs=16, w=p, ws=16, t=2, pre=None, ps=0, m=2, n=8, k=16, act=0,
              p=0.0, rng=None, acc=0, dx=p, dxs=16, dw=p, dwt=0, dws=16, db=p, dbt=0, wk=p,
              wb=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_linear_grad(a["dy"], a["dt"], a["ds"], a["x"], a["xs"], a["w"], a["ws"], a["t"],
                                a["pre"], a["ps"], a["m"], a["n"], a["k"], a["act"], a["p"], 0, 0,
                                a["rng"], a["acc"], a["dx"], a["dxs"], a["dw"], a["dwt"], a["dws"],
                                a["db"], a["dbt"], a["wk"], a["wb"], None)
    for kw in [dict(t=0), dict(t=1), dict(dt=1), dict(dwt=3), dict(dbt=-1), dict(ds=7), dict(xs=15),
               dict(ws=15), dict(dxs=15), dict(dxs=0), dict(dws=15), dict(m=1 << 30),
               dict(n=1 << 30), dict(k=1 << 30), dict(acc=2), dict(act=1), dict(act=9, pre=p, ps=8),
               dict(pre=p, ps=8), dict(act=2, pre=p, ps=7), dict(act=2, pre=p + 1, ps=8),
               dict(p=1.5), dict(rng=p + 1), dict(dy=None), dict(x=None), dict(w=None),
               dict(dy=p + 1), dict(x=p + 1), dict(w=p + 1), dict(dx=p + 1), dict(dw=p + 2),
               dict(db=p + 2), dict(dt=0, dy=p + 2)]:
        assert call(**kw) == BAD, kw
    # an activation, dropout, dy in 32 bits or off 16 bytes, x or w off them: each wants a workspace
    for kw in [dict(act=2, pre=p, ps=8), dict(p=0.5), dict(dt=0), dict(ds=9), dict(xs=17),
               dict(w=p + 2), dict(m=600, ds=8)]:
        for ws in [dict(wk=None), dict(wk=p + 8), dict(wb=16)]:
            assert call(**kw, **ws) == BAD, (kw, ws)
    assert call(dx=None, dw=None, db=None) == 0 and call(n=0, dx=None, db=None, k=0, dw=None) == 0


def test_linear_workspace_sizes(L, p):
    """Copies of operands off 16-byte boundaries and sums of a split k, nothing else."""
    need = L.cp_linear_workspace_bytes
    assert need(p, 504, p, 504, 100, 200, 500) == 0
    assert need(p, 500, p, 504, 100, 200, 500) == 100 * 504 * 2
    assert need(p + 2, 504, p, 0, 100, 200, 500) == 300 * 504 * 2
    assert need(p, 8192, p, 8192, 4096, 4096, 8192) == 0
    split = need(p, 1 << 16, p, 1 << 16, 300, 40, 1 << 16)
    assert split > 0 and (split - 16) % (4 * 300 * 64) == 0
    assert need(p, 1, p, 1, 1 << 31, 4, 1) == 0 and need(p, 8, p, 8, 0, 4, 8) == 0
    # the largest sizes do not wrap
    m = (1 << 31) - 1
    assert need(p, 1, p, 1, m, m, (1 << 30) - 1) == 2 * m * 2 * (1 << 30)
    grad = L.cp_linear_grad_workspace_bytes
    m = (1 << 30) - 1
    assert grad(1 << 30, 4, 4) == 0 and grad(4, 1 << 30, 4) == 0 and grad(4, 4, 1 << 30) == 0
    assert 6 * m * (m + 1) <= grad(m, m, m) < 1 << 63
    assert grad(0, 0, 0) == 16 and grad(0, 5, 7) >= 16
    one = L.cp_linear_grad_call_bytes
    assert one(p, 2, 504, p, 64, p, 64, 2, 100, 500, 64, 0, 0.0) == 0
    assert one(p, 2, 504, p, 64, p, 64, 2, 100, 500, 64, 0, 0.1) >= 100 * 504 * 2
    assert one(p, 2, 500, p, 65, p, 64, 2, 100, 500, 65, 0, 0.0) >= (504 + 72) * 200
    for m, n, k in [(1, 1, 1), (100, 500, 65), (5000, 64, 3000), (300, 4000, 20000)]:
        for dy, act in [(p, 0), (p + 2, 0), (p, 2)]:
            assert one(dy, 2, n, p + 2, k, p + 2, k, 2, m, n, k, act, 0.0) <= grad(m, n, k)


def test_compiled_calls_leave_other_forms_alone():
    """What is not of the common form is answered NotImplemented, with no error left behind: host
    tensors, views, wrong objects, wrong counts of arguments."""
    import torch
    from trellis_row_decode_gb300 import build_ext, projection
    if not build_ext.CALLS.exists():
        build_ext.build()
    calls = projection._common()
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for args in [(), (x,), (x, None, 0.1, 1, 2, None), (x.T, None, 0.1, 1, 2, None),
                 (None, None, 0.1, 1, 2, None), (3, x, 0.1, 1, 2, None),
                 (x, None, "p", 1, 2, None), (x, None, 0.1, -1, 2, None),
                 (x, None, 0.1, 1 << 70, 2, None)]:
        assert calls.dropout(*args) is NotImplemented
    for args in [(), (x, x, None, 0, None, None, False, 0.0, 0, 0, None),
                 (x, None, None, 0, None, None, False, 0.0, 0, 0, None),
                 (x, x, x, "silu", x, torch.float32, True, 0.0, 0, 0, x)]:
        assert calls.linear(*args) is NotImplemented
    for args in [(x,), (x, x, x, 0, None, None, None, 0.0, 0, 0, None),
                 (None,) * 11, (x, x, x, 1 << 80, None, None, None, 0.0, 0, 0, None)]:
        assert calls.linear_grad(*args) is NotImplemented
