"""Calls queued back to back: each reads what the kernel in front of it, still ending when it starts,
has written (ids, weights, scales, rows), into buffers that held other values a moment before."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import E4M3, gen, randn

pytestmark = pytest.mark.gpu
TURNS = 24


@pytest.mark.parametrize("tokens,d,n_out", [(1, 1024, 512), (9, 512, 700), (40, 1000, 4096), (300, 1024, 640)])
def test_a_chain_reads_its_own_turn(tokens, d, n_out):
    """Product sizes for the few-row kernel, the thin one, copies in front of it, and the pairs."""
    g = gen(tokens)
    n_rows = 500
    tables = [randn(g, n_rows, d, dtype=torch.bfloat16).cuda() for _ in range(3)]
    all_ids = torch.randint(0, n_rows, (TURNS, tokens), generator=g).cuda()
    gains = randn(g, TURNS, d).cuda()
    projs = [randn(g, n_out, d, dtype=torch.bfloat16).cuda() for _ in range(3)]
    # buffers that every turn reuses
    table, ids = torch.zeros_like(tables[0]), torch.zeros_like(all_ids[0])
    x = torch.zeros(tokens, d, dtype=torch.bfloat16, device="cuda")
    gain = torch.zeros(d, device="cuda")
    groups, blocks = -(-d // 128), -(-n_out // 128)
    q, sc = torch.zeros(tokens, d, device="cuda").to(E4M3), torch.zeros(tokens, groups, device="cuda")
    w, sw = torch.zeros(n_out, d, device="cuda").to(E4M3), torch.zeros(blocks, groups, device="cuda")
    grad = torch.zeros(n_rows, d, device="cuda")

    def turn(i, wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        table.copy_(tables[i % 3])
        ids.copy_(all_ids[i])
        pause()
        cp.embed(table, ids, 0.5, out=x)
        pause()
        gain.copy_(gains[i])
        pause()
        cp.quantize_fp8(projs[i % 3], 128, out=w, scales=sw)
        pause()
        cp.rms_norm_fp8(x, gain, out=q, scales=sc)
        pause()
        y = cp.matmul_fp8(q, sc, w, sw, dtype=torch.float32)
        pause()
        q8 = cp.quantize_fp8(y)
        pause()
        cp.embed_grad(x, ids, n_rows, out=grad)
        pause()
        back, dgain = cp.rms_norm_grad(x, x, gain)
        return y, q8[0].view(torch.uint8), q8[1], grad.clone(), back, dgain

    queued = [turn(i, False) for i in range(TURNS)]
    torch.cuda.synchronize()
    for i, got in enumerate(queued):
        for a, b in zip(got, turn(i, True)):
            assert torch.equal(a, b), i
