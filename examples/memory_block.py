"""A block around a memory layer trained in 16 bits on one GPU, and its step as a CUDA graph.

Each token looks up a group of rows of a table in training; their sum, under dropout, joins the
residual stream, which is normed and passes two projections, silu and dropout between them and the
stream added behind.  Every product, with what surrounds it, is one call (linear), and so is its
gradient (linear_grad); masks are made again from a seed and offsets, not stored.  One token is
the same forward pass without dropout.  Synthetic data; run it with

    python examples/memory_block.py
"""
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import trellis_row_decode_gb300 as cp  # noqa: E402

EPS = 1e-6
BF16 = torch.bfloat16


class MemoryBlock:
    def __init__(self, n_rows=4096, d=512, hidden=1024, group=8, p=0.1, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*size, std):
            return (std * torch.randn(size, device="cuda", generator=g)).to(BF16)
        self.n_rows, self.group, self.p = n_rows, group, p
        self.rows = normal(n_rows, d, std=0.3)
        self.gain = torch.ones(d, device="cuda")
        self.w1, self.b1 = normal(hidden, d, std=d ** -0.5), normal(hidden, std=0.1)
        self.w2, self.b2 = normal(d, hidden, std=hidden ** -0.5), normal(d, std=0.1)

    def forward(self, residual, ids, rng=None):
        """(out, what backward needs) of tokens [t, d] with their ids [t, group]; dropout where
        `rng` (int64 [2] on the device: a seed and the step's first offset) is given."""
        p = self.p if rng is not None else 0.0
        summed = cp.embed(self.rows, ids).sum(1)
        if p:
            summed = cp.dropout(summed, p, offset=0, rng=rng)
        y, stream = cp.rms_norm(summed, self.gain, EPS, residual=residual)
        a, pre = cp.linear(y, self.w1, self.b1, "silu", p=p, offset=1, rng=rng, pre=True)
        out = cp.linear(a, self.w2, self.b2, residual=stream, p=p, offset=2, rng=rng)
        return out, (ids, p, rng, y, stream, a, pre)

    def backward(self, dout, kept):
        """The gradients by the residual, rows, gain, w1, b1, w2 and b2."""
        ids, p, rng, y, stream, a, pre = kept
        da, dw2, db2 = cp.linear_grad(dout, a, self.w2, p=p, offset=2, rng=rng)
        dy, dw1, db1 = cp.linear_grad(da, y, self.w1, "silu", pre, p=p, offset=1, rng=rng)
        dstream, dgain = cp.rms_norm_grad(dy, stream, self.gain, EPS, dres=dout)
        dsum = cp.dropout_grad(dstream, p, offset=0, rng=rng) if p else dstream
        drows = cp.embed_grad(dsum, ids, self.n_rows, group=self.group)
        return dstream, drows, dgain, dw1, db1, dw2, db2

    def step(self, residual, ids, target, rate, rng):
        """One step of gradient descent on everything; returns the loss."""
        out, kept = self.forward(residual, ids, rng)
        diff = out.float() - target
        dout = (diff * (2.0 / diff.numel())).to(BF16)
        grads = self.backward(dout, kept)[1:]
        for weight, grad in zip((self.rows, self.gain, self.w1, self.b1, self.w2, self.b2), grads):
            weight.sub_(rate * grad.to(weight.dtype))
        rng[1] += 3                                # three masks a step: offsets 0 to 2
        return diff.square().mean()


def main(tokens=512, steps=20, seed=0):
    block = MemoryBlock(seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    d = block.rows.shape[1]
    ids = torch.randint(0, block.n_rows, (tokens, block.group), device="cuda", generator=g)
    residual = torch.randn(tokens, d, device="cuda", generator=g).to(BF16)
    target = torch.randn(tokens, d, device="cuda", generator=g)
    rng = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")
    first = block.step(residual, ids, target, 5.0, rng)            # (before the capture: warm-up)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = block.step(residual, ids, target, 5.0, rng)
    for _ in range(steps):
        graph.replay()
    one, _ = block.forward(residual[:1], ids[:1])                    # a single token, served
    torch.cuda.synchronize()
    assert cp.linear_status() == cp.CP_OK
    print(f"loss {float(first):.4f} -> {float(loss):.4f} in {steps} replayed steps; "
          f"one token: {tuple(one.shape)}")
    return block, float(loss), one


if __name__ == "__main__":
    main()
