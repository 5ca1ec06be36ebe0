"""A memory layer trained, compressed and served on one GPU.

Each token looks up a group of rows of a hashed memory table; their sum joins the residual
stream, which is normed and projected.  The table is trained as plain rows (embed,
rms_norm, their gradients, embed_grad as a step of gradient descent), encoded to 2-bit
records (encode_rows) and served in 8 bits: the decoded rows' sums (lookup_decode_reduce),
the norm with the residual's addition left in e4m3 (rms_norm_fp8), and the projection with a
scale for each block of 128 (quantize_fp8 once, matmul_fp8).  Synthetic data; run it with

    python examples/memory_layer.py
"""
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import trellis_row_decode_gb300 as cp  # noqa: E402

EPS = 1e-6


class MemoryLayer:
    def __init__(self, n_rows=2048, d=256, group=24, n_out=384, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n_rows, self.d, self.group = n_rows, d, group
        self.rows = 0.1 * torch.randn(n_rows, d, device="cuda", generator=g)
        self.gain = torch.ones(d, device="cuda")
        self.proj = torch.randn(n_out, d, device="cuda", generator=g) / d ** 0.5

    def forward(self, residual, ids):
        """(projected, stream) of tokens [t, d] with their ids [t, group]."""
        gathered = cp.embed(self.rows, ids)
        y, stream = cp.rms_norm(gathered.sum(1), self.gain, EPS, residual=residual)
        return y @ self.proj.T, stream

    def step(self, residual, ids, target, rate):
        """One step of gradient descent on the rows and the gain; returns the loss."""
        out, stream = self.forward(residual, ids)
        diff = out - target
        loss = diff.square().mean()
        dy = (2.0 / diff.numel()) * diff @ self.proj
        dsum, dgain = cp.rms_norm_grad(dy, stream, self.gain, EPS)
        # every row of a group has the sum's gradient; the step lands on the rows met
        cp.embed_grad(dsum, ids, self.n_rows, -rate, out=self.rows, accumulate=True,
                      group=self.group)
        self.gain -= 1e-3 * rate * dgain
        return loss

    def compress(self, bits_per_step=4):
        """The table as records (b = bits_per_step / 2 bits a coordinate), the projection in
        e4m3 with a scale for each 128 x 128 block."""
        records, _ = cp.encode_rows(self.rows, bits_per_step)
        table = cp.load_table(records.view(-1), self.n_rows, self.d, bits_per_step)
        return table, cp.quantize_fp8(self.proj, 128)


def serve(layer, table, proj, residual, ids):
    """The same tokens from the compressed table, bf16 stream, 8-bit projection."""
    q_proj, s_proj = proj
    summed = cp.lookup_decode_reduce(table, ids.view(-1), layer.group)
    q, scales, stream = cp.rms_norm_fp8(summed, layer.gain, EPS, residual=residual)
    return cp.matmul_fp8(q, scales, q_proj, s_proj), stream


def main(tokens=512, steps=60, seed=0):
    layer = MemoryLayer(seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    ids = torch.randint(0, layer.n_rows, (tokens, layer.group), device="cuda", generator=g)
    residual = torch.randn(tokens, layer.d, device="cuda", generator=g)
    target = torch.randn(tokens, layer.proj.shape[0], device="cuda", generator=g)
    losses = [float(layer.step(residual, ids, target, rate=2000.0)) for _ in range(steps)]
    out, _ = layer.forward(residual, ids)
    table, proj = layer.compress()
    got, _ = serve(layer, table, proj, residual.bfloat16(), ids)
    assert cp.get_status(table) == cp.CP_OK
    one, _ = serve(layer, table, proj, residual[:1].bfloat16(), ids[:1])      # a single token
    table.close()
    off = float((got.float() - out).norm() / out.norm())
    off_one = float((one.float() - out[:1]).norm() / out[:1].norm())
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps; served from 2-bit records "
          f"in 8 bits: {off:.3f} off the trained layer, one token {off_one:.3f}")
    return losses, off, off_one


if __name__ == "__main__":
    main()
