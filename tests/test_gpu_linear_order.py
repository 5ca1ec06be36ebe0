"""Calls one behind another and side by side: what one call leaves is not what the next one reads."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import gen, randn

pytestmark = pytest.mark.gpu
SIZES = [(1, 256, 512), (40, 300, 200), (200, 96, 4000), (300, 513, 129), (1000, 640, 64),
         (130, 2048, 1024)]


def _args(m, n, k):
    g = gen(m + n + k)
    t = [randn(g, *s, dtype=torch.bfloat16).cuda() for s in ((m, k), (n, k), (n,), (m, n), (m, n))]
    return t


def _run(t, stream=None):
    x, w, b, res, dy = t
    out, pre = cp.linear(x, w, b, "gelu", residual=res, p=0.2, seed=x.shape[0], pre=True,
                         stream=stream)
    grads = cp.linear_grad(dy, x, w, "gelu", pre, p=0.2, seed=x.shape[0], stream=stream)
    return [out, pre, *grads, cp.dropout(out, 0.3, 4, residual=pre, stream=stream)]


def test_calls_one_behind_another():
    """Kernels start while the ones before them end: results do not depend on what ran before."""
    ts = [_args(*s) for s in SIZES]
    want = []
    for t in ts:
        want.append(_run(t))
        torch.cuda.synchronize()
    for _ in range(20):
        got = [_run(t) for t in ts]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert cp.linear_status() == cp.CP_OK


def test_calls_feed_one_another():
    """Each product reads what the one before wrote, in place of the residual, without a wait."""
    g = gen(3)
    w = [randn(g, 256, 256, dtype=torch.bfloat16, std=0.06).cuda() for _ in range(8)]
    for m in (3, 200, 700):
        x0 = randn(g, m, 256, dtype=torch.bfloat16).cuda()
        slow, fast = x0.clone(), x0.clone()
        for i in range(8):
            torch.cuda.synchronize()
            cp.linear(slow.clone(), w[i], None, "silu", residual=slow, out=slow)
            torch.cuda.synchronize()
        for i in range(8):
            cp.linear(fast.clone(), w[i], None, "silu", residual=fast, out=fast)
        assert torch.equal(slow, fast)


def test_calls_on_two_streams():
    ts = [_args(*s) for s in SIZES]
    want = [_run(t) for t in ts]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [[_run(t, s) for t in ts] for s in streams]
        torch.cuda.synchronize()
        for one in got:
            for a, b in zip(one, want):
                assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_two_graphs_share_a_workspace_in_turn():
    """Captured calls with one workspace, replayed one after the other on one stream."""
    a, b = _args(200, 96, 4000), _args(300, 513, 129)
    ws = torch.empty(max(cp.linear_workspace(a[0], a[1]).numel(),
                         cp.linear_workspace(b[0], b[1]).numel(),
                         cp.linear_grad_workspace(200, 96, 4000).numel(),
                         cp.linear_grad_workspace(300, 513, 129).numel()), dtype=torch.uint8,
                     device="cuda")
    outs, graphs, want = [], [], []
    for x, w, bias, _, dy in (a, b):
        want.append([cp.linear(x, w, bias), *cp.linear_grad(dy, x, w)])
        o = [torch.empty_like(t) for t in want[-1]]

        def call():
            cp.linear(x, w, bias, out=o[0], workspace=ws)
            cp.linear_grad(dy, x, w, dx=o[1], dw=o[2], db=o[3], workspace=ws)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        outs.append(o)
        graphs.append(graph)
    for i in (0, 1, 1, 0, 0, 1):
        ws.fill_(0xFF)
        for t in outs[i]:
            t.fill_(float("nan"))
        graphs[i].replay()
        assert all(torch.equal(u, v) for u, v in zip(outs[i], want[i]))


def test_same_form_from_compiled_calls_and_checked_ones():
    """The calls' common form and the form with a stream given are one operation."""
    s = torch.cuda.current_stream()
    for size in SIZES:
        t = _args(*size)
        assert all(torch.equal(u, v) for u, v in zip(_run(t), _run(t, s)))
