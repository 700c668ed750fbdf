"""The cases that measure the many-tensor AdamW step and the microscaled 4-bit products.

Operators:
  adamw    one AdamW step over a list of tensors: finite check, global norm, clipping, update, with
           moments in 8 bits (blocks of 64 under a shared exponent) or in 32
  quantize a matrix in 4-bit elements under shared exponents of 32, along its rows, its columns or both
  product  C = s A B^T of two such matrices, written or added to fp32
  linear   a linear layer's forward and backward pass on them; the weight's gradient is added to an
           error buffer

Shapes are those of the package's own workloads (a resblock's per-GPU shard at d_model 3968, the
unsharded resblock, sequences of 1280 tokens, the small groups of its tests) or generic. With `own`
false `run` computes each operator from elementary torch operations; with `own` true it calls the
package.
"""
import math

import numpy as np
import torch

own = False

D_MODEL = 3968
SEQ = 1280
SHARD = (3968 * 1488, 496 * 3968, 3968 * 1984, 1984 * 3968)              # one resblock on one of 8 GPUs
FULL = (3968 * 11904, 3968 * 3968, 3968 * 15872, 15872 * 3968)           # one resblock, unsharded
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
LR, EPS, DECAY = (float(np.float32(v)) for v in (1e-3, 1e-8, 0.01))
BETA1, BETA2 = float(np.float32(0.9)), float(np.float32(0.999))
GROUP = 64              # elements under one exponent in the 8-bit moments
BLOCK = 32              # elements under one exponent in the 4-bit matrices
PANEL = 128             # columns of a panel of the 4-bit matrices
MASK = 0xFFFFFFFF


def _sizes(case):
    return [int(n) for s in case["sizes"].split(",") for n, k in [s.split("x")] for _ in range(int(k))]


def _list(sizes, count=1):
    return ",".join("%dx%d" % (n, count) for n in sizes)


def listed():
    return [
        # gains and biases of 64 resblocks: many small fp32 tensors, latency
        {"name": "adamw8_gains_f32", "op": "adamw", "sizes": _list((7936, 1488, 1984, 496), 64), "param": "f32", "grad": "f32",
         "bits": 8, "stochastic": True, "max_norm": 1.0, "bad": False},
        # a resblock shard's 16-bit parameters, gradients as decompressed
        {"name": "adamw8_resblock_bf16", "op": "adamw", "sizes": _list(SHARD), "param": "bf16", "grad": "f32",
         "bits": 8, "stochastic": True, "max_norm": 1.0, "bad": False},
        # odd sizes end to end, so that most start off a 16-byte boundary; moments in 32 bits
        {"name": "adamw32_ragged_f16", "op": "adamw", "sizes": "777777x3,1x5,1001x7,65537x9,130x11", "param": "f16", "grad": "f16",
         "bits": 32, "stochastic": False, "max_norm": 0.5, "bad": False},
        # the unsharded resblock: the largest list of parameters
        {"name": "adamw8_unsharded_f32", "op": "adamw", "sizes": _list(FULL), "param": "f32", "grad": "bf16",
         "bits": 8, "stochastic": True, "max_norm": 1.0, "bad": False},
        # one sequence's activations, for the forward product alone
        {"name": "quantize_seq_f16", "op": "quantize", "m": SEQ, "n": D_MODEL, "in": "f16", "row": True, "col": False, "stochastic": False},
        # the gradient of sixteen sequences, for both products of the backward pass
        {"name": "quantize_batch_bf16", "op": "quantize", "m": 16 * SEQ, "n": D_MODEL, "in": "bf16", "row": True, "col": True,
         "stochastic": True},
        # sixteen tokens through the unsharded attention input weights: a decoding step
        {"name": "product_tokens_bf16", "op": "product", "m": 16, "n": 11904, "k": D_MODEL, "out": "bf16", "accumulate": False},
        # odd sizes that no tile divides
        {"name": "product_ragged_f16", "op": "product", "m": 333, "n": 2049, "k": 1001, "out": "f16", "accumulate": False},
        # a shard's weight gradient over sixteen sequences, added to its error buffer
        {"name": "product_wgrad_f32", "op": "product", "m": D_MODEL, "n": 1488, "k": 16 * SEQ, "out": "f32", "accumulate": True},
        # the unsharded first MLP weight over sixteen sequences
        {"name": "product_unsharded_bf16", "op": "product", "m": 16 * SEQ, "n": 15872, "k": D_MODEL, "out": "bf16", "accumulate": False},
        # forward and backward of a shard's first MLP weight, one sequence
        {"name": "linear_seq_bf16", "op": "linear", "t": SEQ, "in": D_MODEL, "out": 1984, "dtype": "bf16"},
        # and over sixteen sequences
        {"name": "linear_batch_f16", "op": "linear", "t": 16 * SEQ, "in": 1984, "out": D_MODEL, "dtype": "f16"},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "quantize", "product", "linear"])
    kinds = ["f32", "f16", "bf16"]
    if op == "adamw":
        total, sizes = _logint(rng, 1000, 2.5e7), []
        for _ in range(rng.randint(1, 6)):
            n = _logint(rng, 1, total)
            sizes.append("%dx%d" % (n, rng.randint(1, max(1, min(60, total // n)))))
        return {"op": op, "sizes": ",".join(sizes), "param": rng.choice(kinds), "grad": rng.choice(kinds), "bits": rng.choice([8, 8, 32]),
                "stochastic": rng.random() < 0.6, "max_norm": rng.choice([0.0, 0.5, 100.0]), "bad": rng.random() < 0.1}
    if op == "quantize":
        way = rng.choice([(True, False), (False, True), (True, True)])
        return {"op": op, "m": _logint(rng, 1, 16 * SEQ), "n": _logint(rng, 1, D_MODEL), "in": rng.choice(kinds), "row": way[0], "col": way[1],
                "stochastic": rng.random() < 0.5}
    if op == "product":
        out = rng.choice(kinds)
        return {"op": op, "m": _logint(rng, 1, 8192), "n": _logint(rng, 8, 8192), "k": _logint(rng, 16, 16384), "out": out,
                "accumulate": out == "f32" and rng.random() < 0.5}
    return {"op": op, "t": _logint(rng, 1, 8192), "in": _logint(rng, 16, 4096), "out": _logint(rng, 16, 4096), "dtype": rng.choice(kinds)}


# ---- random numbers: a counter's hash ------------------------------------------------------
def _mix(x):
    x = x & MASK
    x = ((x ^ (x >> 16)) * 0xA54FF53B) & MASK
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & MASK
    return x ^ (x >> 16)


def _key(seed, step, tensor):
    """Of Python numbers or int64 tensors."""
    k = _mix((seed & MASK) ^ 0x9E3779B9)
    k = _mix(k ^ (seed >> 32))
    return _mix(_mix(step ^ k) ^ tensor)


def _bits(key, i):
    """32 random bits of element i (int64 tensor)."""
    return _mix((i & MASK) ^ _mix((i >> 32) ^ key))


def _more_bits(r):
    t = ((r ^ (r >> 15)) * 0x9E3779B1) & MASK
    return t ^ (t >> 16)


# ---- the 8-bit moments ----------------------------------------------------------------------
# A code is a sign and 4 exponent and 3 fraction bits (first moment), or 5 exponent and 3 fraction bits
# (second moment, never negative), with subnormals; the block's exponent byte is that of the
# largest exponent a code can have.
def _top(second):
    return 31 if second else 15


def _decode8(codes, exps, second):
    c = codes.to(torch.int64).view(-1, GROUP)
    mag = c if second else c & 127
    field, frac = mag >> 3, mag & 7
    e = torch.clamp(field, min=1) + exps.to(torch.int64)[:, None] - _top(second)
    v = (frac + 8 * (field > 0)).double() * torch.exp2((e - 130).double())
    v = v if second else torch.where(c > 127, -v, v)
    return torch.where(exps[:, None] == 255, torch.full_like(v, math.nan), v).float().view(-1)


def _encode8(v, r, second, stochastic):
    """Codes and exponents of fp32 values (whole groups), r: 16 random bits a value."""
    v = v.view(-1, GROUP)
    high = v.abs().amax(1).view(torch.int32).to(torch.int64)
    exps = torch.clamp((high + 0xFFFFF) >> 23, 1, 255)
    b = (v.abs().double() * torch.exp2((_top(second) - exps).double())[:, None]).float().view(torch.int32).to(torch.int64)
    b = b + (((r.view(-1, GROUP) << 4) | 8) if stochastic else 0x7FFFF + ((b >> 20) & 1))
    c = b >> 20
    c = torch.where((v > 0) & (c == 0), torch.ones_like(c), c) if second else c | ((v < 0).to(torch.int64) << 7)
    return torch.where(exps[:, None] == 255, torch.zeros_like(c), c).to(torch.uint8).view(-1), exps.to(torch.uint8)


def _store16(v, r2, kind, stochastic):
    if kind == "f32" or not stochastic:
        return v.to(DTYPES[kind])
    if kind == "bf16":
        b = (v.view(torch.int32).to(torch.int64) & MASK) + (r2 >> 16)
        w = torch.where(b >= 1 << 31, b - (1 << 32), b).to(torch.int32) & -65536
        return torch.where(torch.isfinite(v), w.view(torch.float32), v).to(torch.bfloat16)
    b = (v.abs().double() * 2.0 ** -112).float().view(torch.int32).to(torch.int64) + (r2 >> 19)
    c = torch.clamp(b >> 13, max=0x7C00) | ((v < 0).to(torch.int64) << 15)
    w = torch.where(c >= 1 << 15, c - (1 << 16), c).to(torch.int16).view(torch.float16)
    return torch.where(torch.isfinite(v), w, v.to(torch.float16))


# ---- the 4-bit matrices ---------------------------------------------------------------------
# Rows of k elements, padded with zeros to panels of 128 columns; a panel holds 64 bytes of codes a
# row (the even element in the low nibble). After all panels come the exponents: per panel and 64 rows
# 256 bytes, ordered by block of the panel, row % 16, row / 16.
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _panels(k):
    return -(-k // PANEL)


def _quantize4(x, r, stochastic):
    """Values q (of the 4-bit grid, signed) and exponent bytes of fp32 rows of whole panels."""
    v = x.view(x.shape[0], -1, BLOCK)
    high = v.abs().amax(2).view(torch.int32).to(torch.int64)
    exps = torch.clamp(((high + (0x3FFFFF if stochastic else 0x200000)) >> 23) - 2, min=1)
    a = v.abs() * torch.exp2((127 - exps).double()).float()[:, :, None]
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    if stochastic:
        q = (torch.floor(a.double() / step + (r.view(v.shape) >> 10).double() * 2.0 ** -22) * step).float()
    else:
        q = torch.round(a / step) * step
    q = torch.where(v < 0, -q, q).clamp(-6, 6)
    nan = high >= 0x7F800000
    return torch.where(nan[:, :, None], torch.zeros_like(q), q), torch.where(nan, torch.full_like(exps, 255), exps)


def _values4(q, exps):
    s = torch.where(exps == 255, math.nan, torch.exp2((exps - 127).double()))
    return (q.double() * s[:, :, None]).view(q.shape[0], -1)


def _pack4(q, exps):
    """The bytes of a quantised matrix."""
    rows = q.shape[0]
    level = torch.bucketize(q.abs().view(rows, -1), torch.tensor(VALUES, device=q.device))
    code = (level + 8 * torch.signbit(q).view(rows, -1)).view(rows, -1, PANEL // 2, 2)
    codes = (code[..., 0] + 16 * code[..., 1]).view(rows, -1, PANEL // 2).transpose(0, 1)
    exps = torch.nn.functional.pad(exps, (0, 0, 0, -rows % 64), value=1).view(-1, 4, 16, codes.shape[0], 4).permute(3, 0, 4, 2, 1)
    return torch.cat([codes.reshape(-1), exps.reshape(-1)]).to(torch.uint8)


def _unpack4(data, rows, k):
    """fp32 values [rows, k] of a quantised matrix."""
    p = _panels(k)
    codes = data[:p * rows * 64].view(p, rows, 64).transpose(0, 1).to(torch.int64)
    exps = data[p * rows * 64:].view(p, -1, 4, 16, 4).permute(1, 4, 3, 0, 2).reshape(-1, 4 * p)[:rows].to(torch.int64)
    grid = torch.tensor(VALUES + tuple(-v for v in VALUES), device=data.device)
    q = grid[torch.stack([codes & 15, codes >> 4], 3).view(rows, -1, BLOCK)]
    s = torch.where(exps == 255, math.nan, torch.exp2((exps - 127).double())).float()
    return (q * s[:, :, None]).view(rows, -1)[:, :k]


def _pad(x):
    return torch.nn.functional.pad(x, (0, _panels(x.shape[1]) * PANEL - x.shape[1]))


def _pair_bits(m, n, seed):
    """32 random bits of each element of an m x n matrix: a hash for two neighbours, the second's turned by 16."""
    h = _bits(_key(seed, 0, 0), torch.arange(m * ((n + 1) // 2), device="cuda")).view(m, -1)
    return torch.stack([h, ((h << 16) & MASK) | (h >> 16)], 2).view(m, -1)[:, :n]


def _random4(x, seed, flip):
    """The random bits of a matrix, of its transpose where `flip`, padded."""
    r = _pair_bits(*x.shape, seed)
    return _pad(r.t() if flip else r)


def _round4(x, stochastic, seed, flip=False):
    """x (its transpose where `flip`) as quantised values q and exponents."""
    y = _pad((x.t() if flip else x).float()).contiguous()
    return _quantize4(y, _random4(x, seed, flip) if stochastic else None, stochastic)


# ---- inputs ---------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(m, n, g, dtype):
    """Rows of different size and a few columns that are much larger, as in a trained model."""
    x = torch.randn(m, n, device="cuda", generator=g)
    x *= torch.exp(torch.empty(m, 1, device="cuda").uniform_(math.log(0.2), 0.0, generator=g))
    x *= 1.0 + 20.0 * (torch.rand(1, n, device="cuda", generator=g) < 0.01)
    return x.to(dtype)


def _gradients(m, n, g, dtype):
    """A gradient: rows over several decades."""
    x = torch.randn(m, n, device="cuda", generator=g) * 1e-2
    return (x * torch.exp(torch.empty(m, 1, device="cuda").uniform_(math.log(1e-3), 0.0, generator=g))).to(dtype)


def _adamw_inputs(case, g, seed):
    sizes = torch.tensor(_sizes(case), dtype=torch.int64)
    padded = (sizes + GROUP - 1) // GROUP * GROUP
    total, room = int(sizes.sum()), int(padded.sum())
    sizes, padded = sizes.cuda(), padded.cuda()
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), sizes)
    place = torch.arange(total, device="cuda") - torch.repeat_interleave(torch.cumsum(sizes, 0) - sizes, sizes)
    st = {"tensor": tensor, "place": place, "at": place + torch.repeat_interleave(torch.cumsum(padded, 0) - padded, sizes)}
    st["param"] = (torch.randn(total, device="cuda", generator=g) * 0.02).to(DTYPES[case["param"]])
    size = torch.exp(torch.empty(total, device="cuda").uniform_(math.log(1e-3), 0.0, generator=g)) * 1e-2
    grad = torch.randn(total, device="cuda", generator=g) * size
    if case["bad"]:
        grad[total // 2] = math.nan
    st["grad"] = grad.to(DTYPES[case["grad"]])
    m1 = torch.zeros(room, device="cuda")
    m2 = torch.zeros(room, device="cuda")
    m1[st["at"]] = 0.3 * size * torch.randn(total, device="cuda", generator=g)
    m2[st["at"]] = (size * (0.5 + torch.rand(total, device="cuda", generator=g))).square()
    if case["bits"] == 8:
        st["m1"], st["e1"] = _encode8(m1, None, False, False)
        st["m2"], st["e2"] = _encode8(m2, None, True, False)
    else:
        st["m1"], st["m2"] = m1, m2
    st["step"] = torch.full((1,), 1 + seed % 500, dtype=torch.int32, device="cuda")
    st["skip"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    st["norm"] = torch.zeros(2, device="cuda")
    return st


def _linear_inputs(case, g):
    t, n_in, n_out, dtype = case["t"], case["in"], case["out"], DTYPES[case["dtype"]]
    return {"x": _activations(t, n_in, g, dtype), "dy": _gradients(t, n_out, g, dtype),
            "w": (torch.randn(n_in, n_out, device="cuda", generator=g) * 0.02).to(dtype),
            "err": torch.randn(n_in, n_out, device="cuda", generator=g) * 1e-3,
            "scale": torch.rand(1, device="cuda", generator=g) + 0.5}


def _inputs(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "adamw":
        return _adamw_inputs(case, g, seed)
    if op == "quantize":
        return {"x": _activations(case["m"], case["n"], g, DTYPES[case["in"]])}
    if op == "linear":
        return _linear_inputs(case, g)
    st = {"a": _pack4(*_round4(_activations(case["m"], case["k"], g, torch.float32), False, 0)),
          "b": _pack4(*_round4(torch.randn(case["n"], case["k"], device="cuda", generator=g) * 0.02, False, 0)),
          "scale": torch.rand(1, device="cuda", generator=g) + 0.5}
    st["c"] = torch.randn(case["m"], case["n"], device="cuda", generator=g).to(DTYPES[case["out"]])
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"], st["seed"] = case, seed
    op = case["op"]
    if op == "linear":
        st["wr"] = _pack4(*_round4(st["w"], False, 0))
        st["wc"] = _pack4(*_round4(st["w"], False, 0, True))
    if not own:
        return st
    import rank_gradient_compression_powersgd_amd as psgd
    if op == "adamw":
        sizes = _sizes(case)
        st["group"] = psgd.AdamWGroup(torch.split(st["param"], sizes), torch.split(st["grad"], sizes), bits=case["bits"], seed=seed,
                                      stochastic=case["stochastic"],
                                      moments=(st["m1"], st["m2"], st["e1"], st["e2"]) if case["bits"] == 8 else (st["m1"], st["m2"]))
        st["group"].step_count.copy_(st["step"])
        st["hp"] = psgd.psgd_adam_hparams(LR, BETA1, BETA2, EPS, DECAY)
        return st
    st["ctx"] = psgd.psgd_create(0, 1)
    if op == "quantize":
        m, n = case["m"], case["n"]
        st["row"] = psgd.MxTensor(m, n, "cuda") if case["row"] else None
        st["col"] = psgd.MxTensor(n, m, "cuda") if case["col"] else None
    elif op == "product":
        st["a"], st["b"] = psgd.MxTensor(case["m"], case["k"], data=st["a"]), psgd.MxTensor(case["n"], case["k"], data=st["b"])
        st["workspace"] = torch.empty(psgd.psgd_mx_product_workspace(case["m"], case["n"], case["k"]), dtype=torch.uint8, device="cuda")
    else:
        st["layer"] = psgd.MxLinear(st["w"], seed=seed)
    return st


# ---- one pass -------------------------------------------------------------------------------
def _plain_adamw(st):
    case = st["case"]
    g = st["grad"].float()
    total = g.double().square().sum()
    fine = torch.isfinite(total)
    norm = total.sqrt()
    clip = torch.where(norm > case["max_norm"], case["max_norm"] / norm, 1.0) if case["max_norm"] > 0 else torch.ones_like(norm)
    st["skip"].copy_(~fine)
    st["step"].add_(fine)
    st["norm"].copy_(torch.where(fine, torch.stack([norm, clip]).float(), st["norm"]))
    t = st["step"].double()
    one = torch.ones((), dtype=torch.float64, device="cuda")
    rbc1, rbc2 = ((1.0 / (1.0 - (one * b) ** t)).float() for b in (BETA1, BETA2))
    r = _bits(_key(st["seed"], st["step"].to(torch.int64), torch.arange(len(_sizes(case)), device="cuda"))[st["tensor"]], st["place"])
    at, low = st["at"], case["bits"] == 8
    m1 = (_decode8(st["m1"], st["e1"], False) if low else st["m1"])[at]
    m2 = (_decode8(st["m2"], st["e2"], True) if low else st["m2"])[at]
    g = g * clip.float()
    m1 = m1 * BETA1 + g * (1.0 - BETA1)
    m2 = m2 * BETA2 + g * g * (1.0 - BETA2)
    p = st["param"].float()
    new = p - ((m1 * rbc1) / (torch.sqrt(m2 * rbc2) + EPS) + p * DECAY) * LR
    st["param"].copy_(torch.where(fine, _store16(new, _more_bits(r), case["param"], case["stochastic"]), st["param"]))
    place = lambda v: torch.zeros(st["m1"].numel(), dtype=v.dtype, device="cuda").index_copy_(0, at, v)  # noqa: E731
    if low:
        (c1, e1), (c2, e2) = (_encode8(place(v), place(u), s, case["stochastic"]) for v, u, s in ((m1, r >> 16, False), (m2, r & 0xFFFF, True)))
        st["m1"].copy_(torch.where(fine, c1, st["m1"]))
        st["e1"].copy_(torch.where(fine, e1, st["e1"]))
        st["m2"].copy_(torch.where(fine, c2, st["m2"]))
        st["e2"].copy_(torch.where(fine, e2, st["e2"]))
        m1, m2 = _decode8(st["m1"], st["e1"], False).bfloat16(), _decode8(st["m2"], st["e2"], True).bfloat16()
    else:
        m1 = st["m1"].copy_(torch.where(fine, place(m1), st["m1"]))
        m2 = st["m2"].copy_(torch.where(fine, place(m2), st["m2"]))
    return {"param": st["param"], "m1": m1, "m2": m2, "step": st["step"], "skip": st["skip"], "norm": st["norm"]}


def _plain_linear(st):
    case, dtype = st["case"], DTYPES[st["case"]["dtype"]]
    t, n_in, n_out = case["t"], case["in"], case["out"]
    values = lambda x, stochastic, flip: _values4(*_round4(x, stochastic, st["seed"], flip)).float()  # noqa: E731
    y = values(st["x"], False, False)[:, :n_in] @ _unpack4(st["wc"], n_out, n_in).t()
    dx = values(st["dy"], True, False)[:, :n_out] @ _unpack4(st["wr"], n_in, n_out).t()
    dw = values(st["x"], False, True)[:, :t] @ values(st["dy"], True, True)[:, :t].t()
    st["err"] += st["scale"] * dw
    return {"y": y.to(dtype), "dx": dx.to(dtype), "err": st["err"]}


def _plain(st):
    case = st["case"]
    if case["op"] == "adamw":
        return _plain_adamw(st)
    if case["op"] == "linear":
        return _plain_linear(st)
    if case["op"] == "quantize":
        out = {}
        if case["row"]:
            out["row"] = _values4(*_round4(st["x"], case["stochastic"], st["seed"]))[:, :case["n"]].bfloat16()
        if case["col"]:
            out["col"] = _values4(*_round4(st["x"], case["stochastic"], st["seed"], True))[:, :case["m"]].bfloat16()
        return out
    c = st["scale"] * (_unpack4(st["a"], case["m"], case["k"]) @ _unpack4(st["b"], case["n"], case["k"]).t())
    return st["c"].copy_(st["c"] + c if case["accumulate"] else c)


def run(st):
    if not own:
        return _plain(st)
    import rank_gradient_compression_powersgd_amd as psgd
    case = st["case"]
    op = case["op"]
    if op == "adamw":
        group = st["group"]
        group.step(st["hp"], max_norm=case["max_norm"])
        m1, m2 = group.moments()
        return {"param": st["param"], "m1": m1, "m2": m2, "step": group.step_count, "skip": group.skip, "norm": group.norm}
    if op == "quantize":
        psgd.psgd_mx_quantize(st["ctx"], st["x"], st["row"], st["col"], stochastic=case["stochastic"], seed=st["seed"])
        out = {}
        if case["row"]:
            out["row"] = torch.empty(case["m"], case["n"], dtype=torch.bfloat16, device="cuda")
            psgd.psgd_mx_dequantize(st["ctx"], st["row"], out["row"])
        if case["col"]:
            out["col"] = torch.empty(case["n"], case["m"], dtype=torch.bfloat16, device="cuda")
            psgd.psgd_mx_dequantize(st["ctx"], st["col"], out["col"])
        return out
    if op == "product":
        psgd.psgd_mx_product(st["ctx"], st["a"], st["b"], st["c"], scale=st["scale"], accumulate=case["accumulate"], workspace=st["workspace"])
        return st["c"]
    layer = st["layer"]
    y = layer.forward(st["x"])
    dx = layer.backward(st["dy"], st["err"], st["scale"])
    return {"y": y, "dx": dx, "err": st["err"]}


# ---- the definition in 64 bits --------------------------------------------------------------
def _exponent(v):
    """floor(log2 v), of 0: very small."""
    e = torch.frexp(v).exponent.double() - 1.0
    return torch.where(v > 0, e, torch.full_like(e, -1e4))


def _exact_round(v, step, u):
    """|v| to a multiple of step, with u in [0, 1) added before rounding down; to nearest even without."""
    w = v.abs() / step
    return torch.sign(v) * step * (torch.round(w) if u is None else torch.floor(w + u))


def _exact8(v, u, fields):
    w = v.view(-1, GROUP)
    big = w.abs().amax(1, keepdim=True)
    e = _exponent(big)
    e = torch.clamp(e + (big > 1.875 * torch.exp2(e)), min=-126.0)
    low = e - (fields - 2)                                   # exponent of the lowest normal code
    step = torch.exp2(torch.maximum(_exponent(w.abs()), low) - 3.0)
    q = _exact_round(w, step, None if u is None else u.view(-1, GROUP))
    return torch.where((w > 0) & (q == 0) & (fields == 32), torch.exp2(low - 3.0), q).view(-1)


def _exact16(v, r2, kind):
    """A parameter's rounding up or down by random bits."""
    bits, drop, low = (7, 16, -126.0) if kind == "bf16" else (10, 19, -14.0)
    step = torch.exp2(torch.clamp(_exponent(v.abs()), min=low) - bits)
    return _exact_round(v, step, (r2 >> drop).double() * 2.0 ** (drop - 32))


def _exact_adamw(case, seed):
    st = _inputs(case, seed)
    at, low = st["at"], case["bits"] == 8
    g = st["grad"].double()
    norm = torch.linalg.vector_norm(g)
    m1, m2 = (_decode8(st["m1"], st["e1"], False).double(), _decode8(st["m2"], st["e2"], True).double()) if low else (st["m1"].double(), st["m2"].double())
    p = st["param"].double()
    if case["bad"]:
        return {"param": p, "m1": m1, "m2": m2, "step": None, "skip": None, "norm": st["norm"].double()}
    t = 2 + seed % 500
    clip = min(1.0, case["max_norm"] / float(norm)) if case["max_norm"] > 0 else 1.0
    g = clip * g
    m1[at] = BETA1 * m1[at] + (1.0 - BETA1) * g
    m2[at] = BETA2 * m2[at] + (1.0 - BETA2) * g * g
    ratio = (m1[at] / (1.0 - BETA1 ** t)) / (torch.sqrt(m2[at] / (1.0 - BETA2 ** t)) + EPS)
    p = p - LR * (ratio + DECAY * p)
    r = _bits(_key(seed, t, st["tensor"]), st["place"])
    if case["stochastic"] and case["param"] != "f32":
        p = _exact16(p, _more_bits(r), case["param"])
    if low:
        u1 = u2 = None
        if case["stochastic"]:
            u1, u2 = torch.zeros_like(m1), torch.zeros_like(m2)
            u1[at], u2[at] = ((r >> 16).double() + 0.5) / 65536, ((r & 0xFFFF).double() + 0.5) / 65536
        m1, m2 = _exact8(m1, u1, 16), _exact8(m2, u2, 32)
    return {"param": p, "m1": m1, "m2": m2, "step": None, "skip": None, "norm": torch.tensor([float(norm), clip], dtype=torch.float64)}


def _exact4(x, stochastic, seed, flip=False):
    v = x.double()
    r = _pair_bits(*v.shape, seed) if stochastic else None
    v = v.t() if flip else v
    k = v.shape[1]
    pad = -k % BLOCK
    v = torch.nn.functional.pad(v, (0, pad)).reshape(v.shape[0], -1, BLOCK)
    big = v.abs().amax(2, keepdim=True)
    e = _exponent(big)
    e = torch.clamp(e + ((big > 1.5 * torch.exp2(e)) if stochastic else (big >= 1.75 * torch.exp2(e))), min=-124.0)
    step = torch.exp2(torch.maximum(_exponent(v.abs()), e - 2.0) - 1.0)
    u = None
    if stochastic:
        r = torch.nn.functional.pad(r.t() if flip else r, (0, pad)).reshape(v.shape)
        u = (r >> 10).double() * 2.0 ** -22
    q = _exact_round(v, step, u)
    top = 1.5 * torch.exp2(e)
    return torch.maximum(torch.minimum(q, top), -top).reshape(v.shape[0], -1)[:, :k]


def exact(case, seed):
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(case, seed)
    st = _inputs(case, seed)
    if op == "quantize":
        out = {}
        if case["row"]:
            out["row"] = _exact4(st["x"], case["stochastic"], seed)
        if case["col"]:
            out["col"] = _exact4(st["x"], case["stochastic"], seed, True)
        return out
    if op == "product":
        g = _generator(seed)
        a = _exact4(_activations(case["m"], case["k"], g, torch.float32), False, 0)
        b = _exact4(torch.randn(case["n"], case["k"], device="cuda", generator=g) * 0.02, False, 0)
        c = torch.mm(a, b.t().contiguous()) * st["scale"].double()
        return st["c"].double() + c if case["accumulate"] else c
    y = torch.mm(_exact4(st["x"], False, 0), _exact4(st["w"], False, 0, True).t().contiguous())
    dx = torch.mm(_exact4(st["dy"], True, seed), _exact4(st["w"], False, 0).t().contiguous())
    dw = torch.mm(_exact4(st["x"], False, 0, True), _exact4(st["dy"], True, seed, True).t().contiguous())
    return {"y": y, "dx": dx, "err": st["err"].double() + st["scale"].double() * dw}


# ---- what a pass cannot do without ----------------------------------------------------------
def _bytes4(rows, k):
    return _panels(k) * (rows * 64 + -(-rows // 64) * 256)


def work(case):
    op = case["op"]
    if op == "adamw":
        sizes = _sizes(case)
        n = sum(sizes)
        room = sum(-(-s // GROUP) for s in sizes) * GROUP
        state = room * (2 * 2 * (1 + 1 / GROUP) + 2 * 2) if case["bits"] == 8 else 16 * n       # 8 bits: the values are written too
        return {"bytes": n * (2 * SIZE[case["param"]] + SIZE[case["grad"]]) + state, "flops": 20 * n}
    if op == "quantize":
        m, n = case["m"], case["n"]
        out = (_bytes4(m, n) + 2 * m * n) * case["row"] + (_bytes4(n, m) + 2 * m * n) * case["col"]
        return {"bytes": m * n * SIZE[case["in"]] + out, "flops": 4 * m * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _bytes4(m, k) + _bytes4(n, k) + m * n * SIZE[case["out"]] * (2 if case["accumulate"] else 1), "flops": 2 * m * n * k}
    t, i, o = case["t"], case["in"], case["out"]
    moved = 2 * t * (i + o) * SIZE[case["dtype"]] + _bytes4(i, o) + _bytes4(o, i) + 8 * i * o
    return {"bytes": moved, "flops": 6 * t * i * o}
