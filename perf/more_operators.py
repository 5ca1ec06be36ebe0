"""Timed cases of the 16-bit projection with its epilogue, its gradient, and dropout.

Beside the 8-bit projection that serves a compressed table stands the one that trains it:
``linear`` multiplies 16-bit rows with 16-bit weights and finishes the sums where they are
(bias, activation, dropout, the residual stream's addition), ``linear_grad`` is its backward
pass, and ``dropout`` masks rows from a counter-based generator, so that no mask is stored.

With ``own`` false, ``run`` computes an operator from elementary torch operations in 32 bits,
rounded once at the end; with ``own`` true it makes the library's calls.  Formulas (all sums in
32 bits or more):

linear       z = x w^T + b;  out = residual + D(act(z));  pre = z, where it is kept
linear_grad  dz = D(dy) act'(pre);  dx = dz w;  dw = dz^T x;  db = sum of dz over the rows
dropout      out = residual + D(x)
D            D(v)[i, j] = v[i, j] / (1 - p) where word j mod 4 of Philox4x32-10 with the counter
             (j / 4, i, offset, offset / 2^32) and the key (seed, seed / 2^32) is below
             round((1 - p) 2^32), zero elsewhere.  (Salmon, Moraes, Dror and Shaw, "Parallel
             random numbers: as easy as 1, 2, 3", 2011.)  Its gradient is D itself.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
LOW = 0xFFFFFFFF


def _linear(name, m, n, k, type="bf16", out=None, act="none", bias=True, residual=True, p=0.0,
            pre=False):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "type": type,
            "out": out or type, "act": act, "bias": bias, "residual": residual, "p": p, "pre": pre}


def _grad(name, m, n, k, type="bf16", dw=None, act="none", p=0.0):
    return {"name": name, "op": "linear_grad", "m": m, "n": n, "k": k, "type": type,
            "dw": dw or type, "act": act, "p": p}


def _dropout(name, m, d, type="bf16", p=0.1, residual=True, rng=False):
    return {"name": name, "op": "dropout", "m": m, "d": d, "type": type, "p": p,
            "residual": residual, "rng": rng}


def listed():
    return [
        # decode of one sequence: the summed row of one token joins the residual stream
        _linear("linear_token", 1, 4096, 1024, act="silu"),
        # a small batch of sequences, 24 rows of 1,024 a token
        _linear("linear_batch", 48, 4096, 24576),
        # ragged in every direction, no row on a 16-byte boundary
        _linear("linear_ragged", 333, 1001, 2321, type="f16", out="f32", act="gelu",
                residual=False),
        # a training step's forward pass over 4,096 tokens: the sums before the activation are kept
        _linear("linear_train", 4096, 4096, 1024, act="silu", p=0.1, pre=True),
        # a prompt of 4,096 tokens, 24 rows of 1,024 a token
        _linear("linear_prompt", 4096, 4096, 24576),
        # the gradient of a toy layer (the example's sizes)
        _grad("linear_grad_tiny", 512, 384, 256, dw="f32"),
        # ragged in every direction
        _grad("linear_grad_ragged", 1237, 699, 901, type="f16", act="gelu_tanh", p=0.25),
        # the training step's backward pass
        _grad("linear_grad_train", 4096, 4096, 1024, act="silu", p=0.1),
        # a wide projection's backward pass
        _grad("linear_grad_wide", 4096, 4096, 4096, dw="f32"),
        # 48 tokens' rows
        _dropout("dropout_batch", 48, 1024),
        # rows of odd length in 32 bits; the seed lies on the device, as a captured step keeps it
        _dropout("dropout_ragged", 9001, 813, type="f32", p=0.5, residual=False, rng=True),
        # a prompt's gathered rows, 48 a token
        _dropout("dropout_replay", 196608, 1024, residual=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _ragged(rng, n, step):
    """n brought to a multiple of step, or left as it fell one time in four."""
    return n if rng.random() < 0.25 else max(step, n // step * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "linear_grad", "dropout"])
    kind = rng.choice(["bf16", "bf16", "f16"])
    p = rng.choice([0.0, 0.1, 0.5, rng.uniform(0.01, 0.9)])
    if op == "dropout":
        d = _ragged(rng, _spread(rng, 8, 16384), 8)
        return {"op": op, "m": _spread(rng, 1, min(196608, (1 << 27) // d)), "d": d,
                "type": rng.choice([kind, kind, "f32"]), "p": p or 0.2,
                "residual": rng.random() < 0.5, "rng": rng.random() < 0.5}
    act = rng.choice(ACTS)
    n = _ragged(rng, _spread(rng, 64, 4096), 16)
    if op == "linear":
        k = _ragged(rng, _spread(rng, 64, 24576), 16)
        return {"op": op, "m": _spread(rng, 1, 4096), "n": n, "k": k, "type": kind,
                "out": rng.choice([kind, kind, "f32"]), "act": act, "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.5, "p": rng.choice([0.0, p]),
                "pre": act != "none" and rng.random() < 0.5}
    k = _ragged(rng, _spread(rng, 64, 4096), 16)
    # the products' operands have 16 bits; a gradient that is used in 32 comes from dy as it is
    plain = rng.random() < 0.4
    return {"op": op, "m": _spread(rng, 1, 8192), "n": n, "k": k, "type": kind,
            "dw": rng.choice([kind, "f32"]) if plain else kind, "act": "none" if plain else act,
            "p": 0.0 if plain else rng.choice([0.0, p])}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *size, dtype=torch.float32, std=1.0):
    return torch.randn(size, generator=g, device="cuda").mul_(std).to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    op, kind = case["op"], DTYPES[case["type"]]
    s = {"case": case, "seed": (int(seed) * 0x9E3779B97F4A7C15 + 1) % (1 << 63),
         "offset": int(seed) % 1000003 + (1 << 33)}
    if op == "dropout":
        s["x"] = _normal(g, case["m"], case["d"], dtype=kind)
        if case["residual"]:
            s["residual"] = _normal(g, case["m"], case["d"], dtype=kind)
        if case["rng"]:
            s["rng"] = torch.tensor([s["seed"], s["offset"]], dtype=torch.int64, device="cuda")
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["x"] = _normal(g, m, k, dtype=kind)
    s["weight"] = _normal(g, n, k, dtype=kind, std=1 / math.sqrt(k))
    if op == "linear":
        if case["bias"]:
            s["bias"] = _normal(g, n, dtype=kind, std=0.1)
        if case["residual"]:
            s["residual"] = _normal(g, m, n, dtype=DTYPES[case["out"]])
        return s
    s["dy"] = _normal(g, m, n, dtype=kind, std=0.02)
    if case["act"] != "none":
        s["pre"] = _normal(g, m, n, dtype=kind)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import trellis_row_decode_gb300 as cp
    c = s["case"]
    if c["op"] == "dropout":
        if c["rng"]:
            return cp.dropout(s["x"], c["p"], rng=s["rng"], residual=s.get("residual"))
        return cp.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s.get("residual"))
    if c["op"] == "linear":
        return cp.linear(s["x"], s["weight"], s.get("bias"), c["act"], residual=s.get("residual"),
                         p=c["p"], seed=s["seed"], offset=s["offset"], dtype=DTYPES[c["out"]],
                         pre=c["pre"])
    return cp.linear_grad(s["dy"], s["x"], s["weight"], c["act"], pre=s.get("pre"), p=c["p"],
                          seed=s["seed"], offset=s["offset"], dw_dtype=DTYPES[c["dw"]],
                          db_dtype=torch.float32)


def _seed_of(s):
    """(seed, offset): whole numbers, or elements of the state on the device."""
    if "rng" in s:
        return s["rng"][0], s["rng"][1]
    return s["seed"], s["offset"]


def _kept(m, d, p, seed, offset):
    """Whether element [i, j] is kept.  The generator's 32-bit words are held in int64; a product
    of two of them wraps, which leaves its bits as they are."""
    dev = "cuda"
    c0 = torch.arange((d + 3) // 4, device=dev)[None, :]
    c1 = torch.arange(m, device=dev)[:, None]
    c2 = torch.zeros(1, 1, dtype=torch.int64, device=dev) + (offset & LOW)
    c3 = torch.zeros(1, 1, dtype=torch.int64, device=dev) + ((offset >> 32) & LOW)
    k0, k1 = seed & LOW, (seed >> 32) & LOW
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & LOW) ^ c1 ^ k0, b & LOW, ((a >> 32) & LOW) ^ c3 ^ k1, a & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    words = torch.stack(torch.broadcast_tensors(c0, c1, c2, c3), -1).view(m, -1)[:, :d]
    return words < int((1.0 - p) * 2.0 ** 32 + 0.5)


def _drop(v, p, seed, offset):
    if p == 0.0:
        return v
    return torch.where(_kept(*v.shape, p, seed, offset), v * (1.0 / (1.0 - p)), 0.0)


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, 0.0, z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) \
            + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _run_plain(s):
    c = s["case"]
    seed, offset = _seed_of(s)
    if c["op"] == "dropout":
        out = _drop(s["x"].float(), c["p"], seed, offset)
        if c["residual"]:
            out = out + s["residual"].float()
        return out.to(s["x"].dtype)
    if c["op"] == "linear":
        z = s["x"].float() @ s["weight"].float().T
        if c["bias"]:
            z = z + s["bias"].float()
        out = _drop(_act(z, c["act"]), c["p"], seed, offset)
        if c["residual"]:
            out = out + s["residual"].float()
        out = out.to(DTYPES[c["out"]])
        return (out, z.to(s["x"].dtype)) if c["pre"] else out
    dz = _drop(s["dy"].float(), c["p"], seed, offset)
    if c["act"] != "none":
        dz = dz * _slope(s["pre"].float(), c["act"])
    dx = (dz @ s["weight"].float()).to(s["x"].dtype)
    dw = (dz.T @ s["x"].float()).to(DTYPES[c["dw"]])
    return dx, dw, dz.sum(0)


def work(case):
    b = BYTES[case["type"]]
    if case["op"] == "dropout":
        e = case["m"] * case["d"]
        return {"bytes": e * b * (3 if case["residual"] else 2), "flops": 2 * e}
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "linear":
        o = BYTES[case["out"]]
        return {"bytes": b * (m + n) * k + (b * n if case["bias"] else 0)
                + m * n * (o * (2 if case["residual"] else 1) + (b if case["pre"] else 0)),
                "flops": 2 * m * n * k}
    return {"bytes": b * (2 * m * k + n * k + m * n * (1 if case["act"] == "none" else 2))
            + n * k * BYTES[case["dw"]] + 4 * n, "flops": 4 * m * n * k}


def _mask64(m, d, p, seed, offset):
    """The mask in 64 bits, row block by row block, with the generator's products made of 16-bit
    halves, so that nothing wraps."""
    def product(c, hi16, lo16):
        low = c * lo16
        mid = c * hi16 + (low >> 16)
        return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)

    keep = torch.empty(m, d, dtype=torch.bool, device="cuda")
    limit = math.floor((1.0 - p) * 4294967296.0 + 0.5)
    step = max(1, (1 << 24) // d)
    for r in range(0, m, step):
        rows = min(step, m - r)
        i = torch.arange(r, r + rows, device="cuda").repeat_interleave((d + 3) // 4)
        j = torch.arange((d + 3) // 4, device="cuda").repeat(rows)
        x = [j, i, torch.full_like(i, offset % (1 << 32)), torch.full_like(i, offset >> 32)]
        for t in range(10):
            ka = (seed + t * 0x9E3779B9) % (1 << 32)
            kb = ((seed >> 32) + t * 0xBB67AE85) % (1 << 32)
            (h0, l0), (h1, l1) = product(x[0], 0xD251, 0x1F53), product(x[2], 0xCD9E, 0x8D57)
            x = [torch.bitwise_xor(torch.bitwise_xor(h1, x[1]), ka), l1,
                 torch.bitwise_xor(torch.bitwise_xor(h0, x[3]), kb), l0]
        for w in range(4):
            at = keep[r:r + rows, w::4]
            at.copy_((x[w].view(rows, -1) < limit)[:, :at.shape[1]])
    return keep


def _masked64(v, case, s):
    if case["p"] == 0.0:
        return v
    keep = _mask64(*v.shape, case["p"], s["seed"], s["offset"])
    return (v / (1.0 - case["p"])).masked_fill(~keep, 0.0)


def exact(case, seed):
    """The definitions in 64 bits; the activations through error functions and exponentials of
    torch.special, their slopes by automatic differentiation."""
    s = prepare(case, seed)
    act = {"none": lambda z: z, "relu": torch.relu, "silu": lambda z: z * torch.special.expit(z),
           "gelu": lambda z: z * torch.special.ndtr(z),
           "gelu_tanh": lambda z: z * torch.special.expit(
               2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))}[case.get("act", "none")]
    if case["op"] == "dropout":
        out = _masked64(s["x"].double(), case, s)
        return out.add_(s["residual"].double()) if case["residual"] else out
    x, w = s["x"].double(), s["weight"].double()
    if case["op"] == "linear":
        z = torch.einsum("ik,jk->ij", x, w)
        if case["bias"]:
            z += s["bias"].double()[None, :]
        out = _masked64(act(z), case, s)
        if case["residual"]:
            out = out + s["residual"].double()
        return (out, z) if case["pre"] else out
    dz = _masked64(s["dy"].double(), case, s)
    if case["act"] != "none":
        pre = s["pre"].double().requires_grad_()
        dz, = torch.autograd.grad(act(pre), pre, dz)
    return torch.einsum("ij,jk->ik", dz, w), torch.einsum("ij,ik->jk", dz, x), \
        torch.einsum("ij->j", dz)
