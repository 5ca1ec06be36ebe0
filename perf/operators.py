"""Timed cases of the memory layer's operators around the lookup-decode.

A memory table is trained as plain rows (``embed`` and its gradient), normed into
the residual stream (``rms_norm`` and its gradient), and served in 8 bits: the
normed rows and the projection's weights leave as e4m3 with fp32 scales
(``rms_norm_fp8``, ``quantize_fp8``) and the projection multiplies them
(``matmul_fp8``, one scale for each block of 128).

With ``own`` false, ``run`` computes an operator from elementary torch operations
in 32 bits, rounded once at the end; with ``own`` true it makes the library's
calls.  Formulas (all sums in 32 bits or more):

embed       out[j] = scale * weight[ids[j]], a row of zeros where ids[j] is no row
embed_grad  grad[r] = scale * sum of dy[j] over the j with ids[j] = r
norm        h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight;
            scales[i, g] = max(amax |y| over group g, 1e-30) / 448;  q = e4m3(y / scale)
norm_grad   of y: dx = dres + r (dy w - n mean(dy w n)), dw = sum of dy n over the
            rows, with r = 1 / sqrt(mean(h^2) + eps), n = h r
quantize    the same scales over groups of 1 x 128 or blocks of 128 x 128
matmul      out[i, j] = sum over k of a[i, k] sa[i, k/128] w[j, k] sw[j/128, k/128]
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
AMAX_MIN = 1e-30
EPS = 1e-6


def _up(n, m):
    return -(-n // m)


def listed():
    return [
        # a prompt of 4,096 tokens gathers 48 rows a token from a table in training
        {"name": "embed_replay", "op": "embed", "n": 196608, "rows": 1 << 20, "d": 1024,
         "type": "bf16", "ids": "zipf"},
        # the gradient of a small table of uniform ids (a unit test's or a toy model's size)
        {"name": "embed_grad_tiny", "op": "embed_grad", "n": 4096, "rows": 4096, "d": 256,
         "type": "f32", "out": "f32", "ids": "uniform"},
        # the gradient of that prompt's rows, skewed ids: the hottest row is met in 1 of 12 lookups
        {"name": "embed_grad_replay", "op": "embed_grad", "n": 196608, "rows": 1 << 17,
         "d": 1024, "type": "bf16", "out": "bf16", "ids": "zipf"},
        # decode of one sequence: one token's row
        {"name": "norm_token", "op": "norm", "m": 1, "d": 1024, "type": "bf16"},
        # a prompt's residual stream, handed to an 8-bit projection
        {"name": "norm_prompt", "op": "norm", "m": 4096, "d": 4096, "type": "bf16"},
        # the same stream's backward pass
        {"name": "norm_grad_prompt", "op": "norm_grad", "m": 4096, "d": 4096, "type": "bf16"},
        # a decode step of 2,048 sequences: rows to be projected, not normed
        {"name": "quantize_rows", "op": "quantize", "m": 2048, "k": 1024, "block": 1,
         "type": "bf16"},
        # a projection's weights as they are loaded, 24 rows of 1,024 wide
        {"name": "quantize_weights", "op": "quantize", "m": 4096, "k": 24576, "block": 128,
         "type": "bf16"},
        # decode of one sequence: one token's 24 rows projected
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": 4096, "k": 24576, "out": "bf16"},
        # a small batch of sequences
        {"name": "matmul_batch", "op": "matmul", "m": 48, "n": 4096, "k": 24576, "out": "bf16"},
        # ragged in every direction: the last block of 128 is part full
        {"name": "matmul_ragged", "op": "matmul", "m": 333, "n": 1000, "k": 2320, "out": "f32"},
        # a prompt of 4,096 tokens
        {"name": "matmul_prompt", "op": "matmul", "m": 4096, "n": 4096, "k": 24576,
         "out": "bf16"},
    ]


def _kept(n, step=1):
    """n, or the size below it where n is one that no configuration of this library has."""
    return n - step if n == 3072 else n


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return _kept(max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))))


def _ragged(rng, n, step):
    """n brought to a multiple of step, or left as it fell one time in four."""
    return n if rng.random() < 0.25 else _kept(max(step, n // step * step), step)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "quantize", "matmul", "matmul"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "embed":
        d = _ragged(rng, _spread(rng, 8, 4096), 8)
        n = _spread(rng, 1, min(196608, 196608 * 1024 // d))
        return {"op": op, "n": n, "rows": _spread(rng, 100, min(1 << 20, (1 << 30) // d)), "d": d,
                "type": kind, "ids": rng.choice(["zipf", "uniform"])}
    if op == "embed_grad":
        d = _ragged(rng, _spread(rng, 8, 4096), 8)
        n = _spread(rng, 1, min(196608, 196608 * 1024 // d))
        return {"op": op, "n": n, "rows": _spread(rng, 100, min(1 << 20, (1 << 27) // d)), "d": d,
                "type": kind, "out": rng.choice([kind, "f32"]), "ids": rng.choice(["zipf", "uniform"])}
    if op in ("norm", "norm_grad"):
        d = _ragged(rng, _spread(rng, 64, 16384), 128)
        return {"op": op, "m": _spread(rng, 1, (1 << 24) // d), "d": d, "type": kind}
    if op == "quantize":
        k = _ragged(rng, _spread(rng, 64, 24576), 128)
        return {"op": op, "m": _spread(rng, 1, (1 << 26) // k), "k": k,
                "block": rng.choice([1, 128]), "type": kind}
    k = _ragged(rng, _spread(rng, 128, 24576), 16)
    n = _spread(rng, 64, 4096)
    return {"op": op, "m": _spread(rng, 1, 4096), "n": n, "k": k, "out": rng.choice(["bf16", "bf16", "f32"])}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *size, dtype=torch.float32, std=1.0):
    # in slabs: a table's fp32 draw is never held whole beside its own copy
    if len(size) == 1 or size[0] * size[1] <= 1 << 28:
        return torch.randn(size, generator=g, device="cuda").mul_(std).to(dtype)
    out = torch.empty(size, dtype=dtype, device="cuda")
    for r in range(0, size[0], 1 << 16):
        out[r:r + (1 << 16)] = torch.randn(out[r:r + (1 << 16)].shape, generator=g,
                                           device="cuda").mul_(std)
    return out


def _ids(g, case):
    """Row ids: uniform, or Zipf(1) ranks scattered over the table by a multiplication; about
    one in 64 is -1, the lookup of a position that has no n-gram yet."""
    n, rows = case["n"], case["rows"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if case["ids"] == "zipf":
        rank = (torch.exp(u * math.log(rows + 1)) - 1).long().clamp_(0, rows - 1)
        p = 2654435761
        while math.gcd(p, rows) != 1:
            p += 2
        ids = rank * p % rows
    else:
        ids = (u * rows).long().clamp_(0, rows - 1)
    return torch.where(torch.rand(n, generator=g, device="cuda") < 1 / 64, -1, ids)


def _stream(g, m, d, dtype):
    """A residual stream and what a layer adds to it: a few strong channels, and rows that the
    memory left at zero."""
    gain = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    gain = torch.where(torch.rand(d, generator=g, device="cuda") < 1 / 256, 20 * gain, gain)
    residual = (_normal(g, m, d) * gain).to(dtype)
    x = _normal(g, m, d, std=0.5)
    x = torch.where(torch.rand(m, 1, generator=g, device="cuda") < 1 / 64, 0.0, x).to(dtype)
    return x, residual


def _blocks(x, block):
    """x [m, k] padded with zeros to whole blocks, as [m / block, block, k / 128, 128]."""
    m, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % 128, 0, -m % block))
    return x.view(_up(m, block), block, _up(k, 128), 128)


def _quantize(x, block):
    m, k = x.shape
    b = _blocks(x, block)
    scales = b.abs().amax((1, 3)).clamp(min=AMAX_MIN) / E4M3_MAX
    q = (b / scales[:, None, :, None]).to(E4M3)
    return q.view(b.shape[0] * block, -1)[:m, :k].contiguous(), scales


def _spread_scales(scales, block, m, k):
    return scales.repeat_interleave(block, 0)[:m].repeat_interleave(128, 1)[:, :k]


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op == "embed":
        s["weight"] = _normal(g, case["rows"], case["d"], dtype=DTYPES[case["type"]])
        s["ids"] = _ids(g, case)
        s["scale"] = math.sqrt(case["d"])
    elif op == "embed_grad":
        s["dy"] = _normal(g, case["n"], case["d"], dtype=DTYPES[case["type"]], std=0.02)
        s["ids"] = _ids(g, case)
        s["scale"] = math.sqrt(case["d"])
    elif op == "norm":
        s["x"], s["residual"] = _stream(g, case["m"], case["d"], DTYPES[case["type"]])
        s["weight"] = 1 + _normal(g, case["d"], std=0.2)
    elif op == "norm_grad":
        x, residual = _stream(g, case["m"], case["d"], torch.float32)
        s["h"] = (x + residual).to(DTYPES[case["type"]])
        s["weight"] = 1 + _normal(g, case["d"], std=0.2)
        s["dy"] = _normal(g, case["m"], case["d"], dtype=DTYPES[case["type"]], std=0.02)
        s["dres"] = _normal(g, case["m"], case["d"], dtype=DTYPES[case["type"]], std=0.02)
    elif op == "quantize":
        s["x"] = _normal(g, case["m"], case["k"], dtype=DTYPES[case["type"]])
    elif op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _quantize(_normal(g, m, k), 1)
        s["w"], s["sw"] = _quantize(_normal(g, n, k, std=1 / math.sqrt(k)), 128)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import trellis_row_decode_gb300 as cp
    c = s["case"]
    op = c["op"]
    if op == "embed":
        return cp.embed(s["weight"], s["ids"], s["scale"])
    if op == "embed_grad":
        return cp.embed_grad(s["dy"], s["ids"], c["rows"], s["scale"], dtype=DTYPES[c["out"]])
    if op == "norm":
        return cp.rms_norm_fp8(s["x"], s["weight"], EPS, residual=s["residual"])
    if op == "norm_grad":
        return cp.rms_norm_grad(s["dy"], s["h"], s["weight"], EPS, dres=s["dres"])
    if op == "quantize":
        return cp.quantize_fp8(s["x"], c["block"])
    return cp.matmul_fp8(s["a"], s["sa"], s["w"], s["sw"], dtype=DTYPES[c["out"]])


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "embed":
        ids, weight = s["ids"], s["weight"]
        row = (ids >= 0) & (ids < weight.shape[0])
        out = weight[torch.where(row, ids, 0)].float() * s["scale"]
        return torch.where(row[:, None], out, 0.0).to(weight.dtype)
    if op == "embed_grad":
        ids, rows = s["ids"], c["rows"]
        row = (ids >= 0) & (ids < rows)
        grad = torch.zeros(rows + 1, c["d"], dtype=torch.float32, device=ids.device)
        grad.index_add_(0, torch.where(row, ids, rows), s["dy"].float())
        return (grad[:rows] * s["scale"]).to(DTYPES[c["out"]])
    if op == "norm":
        h = s["x"].float() + s["residual"].float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
        q, scales = _quantize(y, 1)
        return q, scales, h.to(s["x"].dtype)
    if op == "norm_grad":
        h, dy = s["h"].float(), s["dy"].float()
        r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
        n, t = h * r, dy * s["weight"]
        dx = s["dres"].float() + r * (t - n * (t * n).mean(-1, keepdim=True))
        return dx.to(s["h"].dtype), (dy * n).sum(0)
    if op == "quantize":
        return _quantize(s["x"].float(), c["block"])
    a = s["a"].float() * _spread_scales(s["sa"], 1, c["m"], c["k"])
    w = s["w"].float() * _spread_scales(s["sw"], 128, c["n"], c["k"])
    return (a @ w.T).to(DTYPES[c["out"]])


def _distinct(case):
    """Rows that n lookups are expected to meet at least once."""
    n, rows = case["n"], case["rows"]
    if case["ids"] == "uniform":
        return rows * -math.expm1(n * math.log1p(-1 / rows))
    rank = torch.arange(1, rows + 1, dtype=torch.float64)
    p = torch.log1p(1 / rank) / math.log(rows + 1)
    return float(-torch.expm1(n * torch.log1p(-p)).sum())


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        n, rows, d, b = case["n"], case["rows"], case["d"], BYTES[case["type"]]
        if op == "embed":  # ids, each distinct row once, the output
            return {"bytes": 8 * n + int(_distinct(case) + n) * d * b, "flops": n * d}
        return {"bytes": 8 * n + n * d * b + rows * d * BYTES[case["out"]], "flops": n * d}
    if op == "norm":  # x and the residual in; h, q and the scales out
        e = case["m"] * case["d"]
        return {"bytes": e * (3 * BYTES[case["type"]] + 1) + 4 * case["m"] * _up(case["d"], 128),
                "flops": 6 * e}
    if op == "norm_grad":  # dy, h and dres in; dx out
        e = case["m"] * case["d"]
        return {"bytes": 4 * e * BYTES[case["type"]] + 8 * case["d"], "flops": 14 * e}
    if op == "quantize":
        e = case["m"] * case["k"]
        return {"bytes": e * (BYTES[case["type"]] + 1)
                + 4 * _up(case["m"], case["block"]) * _up(case["k"], 128), "flops": 3 * e}
    m, n, k = case["m"], case["n"], case["k"]
    kb = _up(k, 128)
    return {"bytes": (m + n) * k + 4 * kb * (m + _up(n, 128)) + m * n * BYTES[case["out"]],
            "flops": 2 * m * n * k}


def _groups64(y, block):
    """Scales and unrounded quotients of y in 64 bits: each block's largest magnitude by
    scattered maxima, and each value over its own block's scale."""
    m, k = y.shape
    i = torch.arange(m, device=y.device) // block
    j = torch.arange(k, device=y.device) // 128
    nb = _up(k, 128)
    at = i[:, None] * nb + j[None, :]
    amax = torch.zeros(_up(m, block) * nb, dtype=torch.float64, device=y.device)
    amax.scatter_reduce_(0, at.reshape(-1), y.abs().reshape(-1), "amax")
    scales = torch.maximum(amax, torch.full_like(amax, AMAX_MIN)) / E4M3_MAX
    return y / scales[at], scales.view(-1, nb)


def exact(case, seed):
    """The definitions in 64 bits.  An e4m3 output is held against the quotient that it rounds."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        ids, w = s["ids"], s["weight"]
        out = torch.zeros(ids.numel(), case["d"], dtype=torch.float64, device=ids.device)
        at = torch.nonzero((ids >= 0) & (ids < w.shape[0]))[:, 0]
        out.index_copy_(0, at, w.index_select(0, ids[at]).double() * s["scale"])
        return out
    if op == "embed_grad":
        # running sums of the rows in the order of their ids, and differences at the ids' ends
        at = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["rows"]))[:, 0]
        ids, order = torch.sort(s["ids"][at], stable=True)
        run_sums = torch.cumsum(s["dy"][at[order]].double(), 0)
        run_sums = torch.nn.functional.pad(run_sums, (0, 0, 1, 0))
        r = torch.arange(case["rows"], device=ids.device)
        lo, hi = torch.searchsorted(ids, r), torch.searchsorted(ids, r, right=True)
        return (run_sums[hi] - run_sums[lo]) * s["scale"]
    if op == "norm":
        h = torch.add(s["x"].double(), s["residual"].double())
        size = torch.linalg.vector_norm(h, dim=1, keepdim=True)
        y = torch.einsum("ij,j->ij", h / torch.sqrt(size * size / case["d"] + EPS),
                         s["weight"].double())
        q, scales = _groups64(y, 1)
        return q, scales, h
    if op == "norm_grad":
        # by the chain rule through u = mean(h^2) + eps: y = h w u^(-1/2)
        h, dy, w = s["h"].double(), s["dy"].double(), s["weight"].double()
        u = (torch.einsum("ij,ij->i", h, h) / case["d"] + EPS)[:, None]
        along = torch.einsum("ij,ij,j->i", dy, h, w)[:, None]
        dx = s["dres"].double() + dy * w / torch.sqrt(u) - h * along / (case["d"] * u ** 1.5)
        return dx, torch.einsum("ij,ij->j", dy, h / torch.sqrt(u))
    if op == "quantize":
        return _groups64(s["x"].double(), case["block"])
    # block by block of 128 along k: the products of the values, scaled afterwards
    m, n, k = case["m"], case["n"], case["k"]
    out = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    rows_of = torch.arange(n, device="cuda") // 128
    for b in range(_up(k, 128)):
        part = s["a"][:, 128 * b:128 * b + 128].double() @ s["w"][:, 128 * b:128 * b + 128].double().T
        out += part * s["sa"][:, b, None].double() * s["sw"][rows_of, b][None, :].double()
    return out
