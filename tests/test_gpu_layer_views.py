"""Views that the memory layer's calls take as they are: expanded rows, leading dimensions."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import DTYPES, E4M3, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [16, 33, 1024])
def test_embed_of_an_expanded_row(d, dtype):
    """A table whose rows are one row (stride 0), as every input may be."""
    g = gen(d)
    row = randn(g, 1, d, dtype=dtype).cuda()
    ids = torch.tensor([0, 9, -1, 4, 10], device="cuda")
    got = cp.embed(row.expand(10, d), ids, 2.0)
    assert torch.equal(got, cp.embed(row.expand(10, d).contiguous(), ids, 2.0))
    assert torch.equal(got[1], 2 * row[0]) and not got[[2, 4]].any()


def _same(a, b):
    return torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))


@pytest.mark.parametrize("d", [256, 300])
def test_a_batched_stream_goes_through_the_chain(d):
    """[batch, token, d] from the norm and the quantiser to the product, as the merged rows do."""
    g = gen(d)
    x = randn(g, 3, 7, d, dtype=torch.bfloat16).cuda()
    gain, proj = randn(g, d).cuda(), randn(g, 200, d).cuda()
    w, sw = cp.quantize_fp8(proj, 128)
    for q, sc in (cp.rms_norm_fp8(x, gain), cp.quantize_fp8(x)):
        assert q.shape == (3, 7, d) and sc.shape == (3, 7, -(-d // 128))
        flat = cp.matmul_fp8(q.view(21, d), sc.view(21, -1), w, sw)
        got = cp.matmul_fp8(q, sc, w, sw)
        assert got.shape == (3, 7, 200) and torch.equal(got.view(21, 200), flat)
        one = cp.matmul_fp8(q[1:2, 4:5], sc[1:2, 4:5].contiguous(), w, sw)    # a single token
        ref = cp.matmul_fp8(q[1, 4:5], sc[1, 4:5], w, sw)
        assert one.shape == (1, 1, 200) and torch.equal(one[0], ref)
        buf = torch.full((3, 7, 208), 5.0, device="cuda")
        cp.matmul_fp8(q, sc, w, sw, out=buf[..., 4:204])
        assert torch.equal(buf[..., 4:204], cp.matmul_fp8(q, sc, w, sw, dtype=torch.float32))
        assert bool((buf[..., :4] == 5).all()) and bool((buf[..., 204:] == 5).all())
    q, sc = cp.quantize_fp8(x)
    q2, sc2 = cp.quantize_fp8(x.view(21, d))
    assert _same(q, q2) and _same(sc, sc2)
    wide = randn(g, 3, 7, d + 40).cuda()[..., 8:8 + d]           # rows apart, leading dimensions merge
    q, sc = cp.quantize_fp8(wide)
    q2, sc2 = cp.quantize_fp8(wide.contiguous())
    assert _same(q, q2) and _same(sc, sc2)
    none = torch.empty(2, 0, d, device="cuda")
    q, sc = cp.quantize_fp8(none)
    assert q.shape == (2, 0, d) and sc.shape == (2, 0, -(-d // 128))
    assert cp.matmul_fp8(q, sc, w, sw).shape == (2, 0, 200)


def test_leading_dimensions_refusals():
    x = torch.zeros(2, 128, 128, device="cuda")
    q, sc = cp.quantize_fp8(x)
    w, sw = cp.quantize_fp8(x[0], 128)
    for call in [
        lambda: cp.quantize_fp8(x, 128),                         # a block would span matrices
        lambda: cp.quantize_fp8(x[0, 0]),
        lambda: cp.quantize_fp8(x[:, ::2][:, :5]),               # rows that do not merge
        lambda: cp.quantize_fp8(x, out=torch.empty(256, 128, device="cuda").to(E4M3)),
        lambda: cp.matmul_fp8(q, sc.view(256, 1), w, sw),
        lambda: cp.matmul_fp8(q[0, 0], sc[0, 0], w, sw),
        lambda: cp.matmul_fp8(q, sc, q, sw),
        lambda: cp.matmul_fp8(q, sc, w, sw, out=torch.empty(256, 128, device="cuda")),
    ]:
        with pytest.raises(ValueError):
            call()
