"""examples/memory_block.py: embed, dropout, the norm and two projections, forward, backward and
captured, as they are used together."""
import importlib.util
import math
from pathlib import Path

import pytest
import torch

import trellis_row_decode_gb300 as cp

from linear_util import mask64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    path = Path(__file__).resolve().parent.parent / "examples" / "memory_block.py"
    spec = importlib.util.spec_from_file_location("memory_block_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_memory_block_runs(m):
    block, loss, one = m.main(tokens=200, steps=4)
    assert math.isfinite(loss) and bool(torch.isfinite(one).all())
    assert bool(torch.isfinite(block.w1).all()) and bool(torch.isfinite(block.rows).all())


def _inputs(block, tokens):
    g = torch.Generator().manual_seed(5)
    d = block.rows.shape[1]
    ids = torch.randint(0, block.n_rows, (tokens, block.group), generator=g)
    return ids, torch.randn(tokens, d, generator=g).bfloat16(), \
        (0.1 * torch.randn(tokens, d, generator=g)).bfloat16()


def _step64(m, block, ids, residual, dout, seed, offset):
    """(out, gradients) of the block in 64 bits, by automatic differentiation."""
    leaves = [t.detach().cpu().double().requires_grad_() for t in
              (residual, block.rows, block.gain, block.w1, block.b1, block.w2, block.b2)]
    res, rows, gain, w1, b1, w2, b2 = leaves

    def drop(v, at):
        return v * mask64(*v.shape, block.p, seed, offset + at).double() / (1 - block.p)
    stream = res + drop(rows[ids].sum(1), 0)
    y = stream / torch.sqrt(stream.square().mean(-1, keepdim=True) + m.EPS) * gain
    a = drop(torch.nn.functional.silu(y @ w1.T + b1), 1)
    out = stream + drop(a @ w2.T + b2, 2)
    out.backward(dout.double())
    return out.detach(), [t.grad for t in leaves]


def test_memory_block_gradients(m):
    """Against automatic differentiation in 64 bits.  Between an input and a gradient lie at most 12
    roundings to bf16 of whole tensors, each off by at most 2^-8 relative to a term, and the slopes
    stay within 1.13: 12 * 1.13 * 2^-8 = 0.053 of a norm."""
    block = m.MemoryBlock(n_rows=300, d=96, hidden=160, group=3, p=0.25, seed=3)
    ids, residual, dout = _inputs(block, 150)
    rng = torch.tensor([77, 1 << 35], dtype=torch.int64, device="cuda")
    out, kept = block.forward(residual.cuda(), ids.cuda(), rng)
    got = block.backward(dout.cuda(), kept)
    want, grads = _step64(m, block, ids, residual, dout, 77, 1 << 35)
    for u, v in zip([out, *got], [want, *grads]):
        assert float((u.cpu().double() - v).norm()) <= 0.053 * float(v.norm())
    assert cp.linear_status() == cp.CP_OK


def test_memory_block_captured_replays_what_it_does_eagerly(m):
    """Forward and backward in one graph, its offset moved between replays: the eager calls' bits."""
    block = m.MemoryBlock(n_rows=300, d=128, hidden=256, group=4, p=0.1, seed=4)
    ids, residual, dout = (t.cuda() for t in _inputs(block, 260))
    rng = torch.tensor([5, 0], dtype=torch.int64, device="cuda")

    def run():
        out, kept = block.forward(residual, ids, rng)
        return [out, *block.backward(dout, kept)]
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for offset in (0, 3, 6):
        rng[1] = offset
        want = run()
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_memory_block_single_token_is_a_row_of_many(m):
    """The forms for one row, few rows and many agree to their last rounding's reach: three
    roundings to bf16 (the kept activations, the stream, the output) of values below 2^3 and the
    second product's share, 4 * 2^-8 * 8."""
    block = m.MemoryBlock(n_rows=300, d=128, hidden=256, group=4, seed=6)
    ids, residual, _ = (t.cuda() for t in _inputs(block, 300))
    many, _ = block.forward(residual, ids)
    for t in (1, 3, 40):
        few, _ = block.forward(residual[:t], ids[:t])
        assert float((few.float() - many[:t].float()).abs().max()) <= 4 * 2.0 ** -8 * 8
