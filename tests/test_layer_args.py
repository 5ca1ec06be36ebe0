"""Host-side argument checks of the memory layer's entry points: refused before any CUDA
call, so they run without a GPU."""
import ctypes as C

import pytest

BAD = 1          # CP_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    import trellis_row_decode_gb300 as cp
    from trellis_row_decode_gb300 import build_ext, layer
    if not cp.LIB_PATH.exists():
        build_ext.build()
    return layer._lib()


@pytest.fixture(scope="module")
def p():
    buf = (C.c_uint8 * 4096)()
    at = (C.addressof(buf) + 63) & ~63
    yield at
    del buf


def test_embed_arguments(L, p):
    ok = dict(w=p, t=0, rows=4, d=8, ws=8, ids=p, n=2, out=p, os=8, st=None)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_embed(a["w"], a["t"], a["rows"], a["d"], a["ws"], a["ids"], a["n"], 1.0,
                          a["out"], a["os"], a["st"], None)
    for kw in [dict(t=3), dict(t=-1), dict(d=0), dict(d=(1 << 20) + 1), dict(ws=7), dict(os=7),
               dict(n=1 << 31), dict(w=None), dict(ids=None), dict(out=None), dict(w=p + 2),
               dict(out=p + 1), dict(ids=p + 4), dict(st=p + 1), dict(t=2, w=p + 1)]:
        assert call(**kw) == BAD, kw
    assert call(n=0) == 0 and call(n=0, ids=None, out=None) == 0


def test_embed_grad_arguments(L, p):
    big = 1 << 30
    ok = dict(dy=p, t=0, ds=8, ids=p, n=2, grp=1, rows=4, d=8, acc=0, g=p, gt=0, gs=8, st=None, ws=p,
              wb=big)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_embed_grad(a["dy"], a["t"], a["ds"], a["ids"], a["n"], a["grp"], a["rows"], a["d"],
                               1.0, a["acc"], a["g"], a["gt"], a["gs"], a["st"], a["ws"], a["wb"], None)
    for kw in [dict(t=5), dict(gt=9), dict(d=0), dict(ds=7), dict(gs=7), dict(gs=0),
               dict(n=1 << 31), dict(rows=1 << 31), dict(acc=2), dict(grp=0), dict(grp=3), dict(dy=None), dict(ids=None),
               dict(g=None), dict(dy=p + 2), dict(g=p + 1), dict(ids=p + 4), dict(ws=None),
               dict(ws=p + 8), dict(wb=16)]:
        assert call(**kw) == BAD, kw
    assert call(n=0, acc=1) == 0
    assert call(n=0, rows=0) == 0
    assert L.cp_embed_grad_workspace_bytes(1 << 31, 4, 8) == 0
    assert L.cp_embed_grad_workspace_bytes(4, 4, 0) == 0
    for n, rows, d in [(1, 1, 1), (196608, 1 << 17, 1024), (5, (1 << 31) - 1, 64),
                       ((1 << 31) - 1, 7, 8), (1 << 20, 1 << 24, 4096)]:
        need = L.cp_embed_grad_workspace_bytes(n, rows, d)
        # sorted pairs twice, and at most 268 MB of parts and marks beside them
        assert 16 * n <= need <= 16 * n + (300 << 20), (n, rows, d, need)


def test_norm_arguments(L, p):
    ok = dict(x=p, xs=8, r=None, rs=0, t=0, w=p, wt=0, m=2, d=8, eps=0.0, y=p, h=None)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_rms_norm(a["x"], a["xs"], a["r"], a["rs"], a["t"], a["w"], a["wt"], a["m"],
                             a["d"], a["eps"], a["y"], a["h"], None)

    def call8(**kw):
        a = {**ok, "sc": p, **kw}
        return L.cp_rms_norm_fp8(a["x"], a["xs"], a["r"], a["rs"], a["t"], a["w"], a["wt"],
                                 a["m"], a["d"], a["eps"], a["y"], a["sc"], a["h"], None)
    for kw in [dict(t=3), dict(wt=3), dict(d=0), dict(d=49153, xs=49153), dict(xs=7),
               dict(m=1 << 31), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(w=None),
               dict(y=None), dict(x=p + 2), dict(w=p + 2), dict(r=p), dict(h=p),
               dict(r=p, h=p, rs=5), dict(r=p + 1, h=p, rs=8)]:
        assert call(**kw) == BAD, kw
        assert call8(**kw) == BAD, kw
    assert call(y=p + 2) == BAD
    assert call8(sc=None) == BAD and call8(sc=p + 2) == BAD
    assert call(m=0) == 0 and call8(m=0) == 0


def test_norm_grad_arguments(L, p):
    ok = dict(dy=p, ds=8, h=p, hs=8, r=None, rs=0, t=0, w=p, wt=0, m=2, d=8, eps=0.0, dx=p, dw=p,
              ws=p, wb=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_rms_norm_grad(a["dy"], a["ds"], a["h"], a["hs"], a["r"], a["rs"], a["t"],
                                  a["w"], a["wt"], a["m"], a["d"], a["eps"], a["dx"], a["dw"],
                                  a["ws"], a["wb"], None)
    for kw in [dict(t=3), dict(wt=-1), dict(d=0), dict(ds=7), dict(hs=7), dict(r=p, rs=7),
               dict(m=1 << 31), dict(eps=-1.0), dict(dy=None), dict(h=None), dict(w=None),
               dict(dx=None), dict(dw=None), dict(dy=p + 2), dict(dx=p + 1), dict(dw=p + 2),
               dict(ws=None), dict(ws=p + 4), dict(wb=4)]:
        assert call(**kw) == BAD, kw
    assert L.cp_rms_norm_grad_workspace_bytes(4, 49153) == 0
    assert L.cp_rms_norm_grad_workspace_bytes(0, 8) > 0


def test_quantize_arguments(L, p):
    ok = dict(x=p, xs=8, t=0, m=2, d=8, b=1, q=p, sc=p)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_quantize_fp8(a["x"], a["xs"], a["t"], a["m"], a["d"], a["b"], a["q"], a["sc"],
                                 None)
    for kw in [dict(t=3), dict(b=2), dict(b=0), dict(xs=7), dict(m=1 << 31), dict(x=None),
               dict(q=None), dict(sc=None), dict(x=p + 1), dict(sc=p + 2)]:
        assert call(**kw) == BAD, kw
    assert call(m=0) == 0 and call(d=0) == 0


def test_matmul_arguments(L, p):
    ok = dict(a=p, la=8, sa=p, w=p, lw=8, sw=p, m=2, n=3, k=8, o=p, t=0, lo=3, ws=None, wb=0)

    def call(**kw):
        a = {**ok, **kw}
        return L.cp_matmul_fp8(a["a"], a["la"], a["sa"], a["w"], a["lw"], a["sw"], a["m"], a["n"],
                               a["k"], a["o"], a["t"], a["lo"], a["ws"], a["wb"], None)
    for kw in [dict(t=3), dict(la=7), dict(lw=7), dict(lo=2), dict(m=1 << 31), dict(n=1 << 31),
               dict(k=1 << 31), dict(a=None), dict(w=None), dict(sa=None), dict(sw=None),
               dict(o=None), dict(o=p + 2), dict(sa=p + 2), dict(sw=p + 1), dict(m=17),
               dict(m=17, ws=p, wb=16 * 20 - 1), dict(m=17, ws=p + 8, wb=1 << 20)]:
        assert call(**kw) == BAD, kw
    assert call(m=0) == 0 and call(n=0) == 0


def test_matmul_workspace_sizes(L, p):
    """One 16-byte-aligned copy of each operand whose rows need it, but for few rows of a and
    little of w."""
    need = L.cp_matmul_fp8_workspace_bytes
    assert need(p, 512, p, 512, 300, 200, 500) == 0
    assert need(p, 500, p, 512, 300, 200, 500) == 300 * 512
    assert need(p, 512, p + 1, 512, 300, 200, 500) == 200 * 512
    assert need(p, 0, p, 513, 300, 200, 512) == 500 * 512
    assert need(p + 8, 500, p, 500, 16, 200, 500) == 0
    assert need(p, 500, p, 77, 17, 1, 500) == 17 * 512
    assert need(p, 4096, p, 4097, 16, 4096, 4096) == 4096 * 4096
    assert need(p, 1, p, 1, 1 << 31, 4, 1) == 0 and need(p, 0, p, 0, 40, 4, 0) == 0
    assert need(p, (1 << 31) + 1, p, 1, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 200) == \
        2 * ((1 << 31) - 1) * (((1 << 31) - 200 + 15) // 16 * 16)
