"""The cases that measure the optimizer's Newton-Schulz and embedding operators.

Operators:
  newton_schulz  a group of update matrices orthogonalised by Newton-Schulz products
  muon           momentum, Newton-Schulz and parameter update of a plan's matrices
  embed_lookup   scaled embedding rows of a batch of tokens
  embed_grad     the embedding's gradient from the activations' gradient

Shapes are those of the package's own workloads (a resblock's per-GPU shard at d_model 3968, the
unsharded resblock, the small groups of its tests) or generic. With `own` false `run` computes
each operator from elementary torch operations; with `own` true it calls the package.
"""
import math

import torch

own = False

D_MODEL = 3968
SHARD = ((3968, 1488), (496, 3968), (3968, 1984), (1984, 3968))          # one resblock on one of 8 GPUs
FULL = ((3968, 11904), (3968, 3968), (3968, 15872), (15872, 3968))       # one resblock, unsharded
COEF = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-20
MUON = dict(lr=2e-3, momentum=0.95, weight_decay=0.01)
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
RANK = 112


def _flat(shapes):
    return ",".join("%dx%d" % s for s in shapes)


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def listed():
    return [
        # one attention-output shard of a resblock, as a step that updates layer by layer calls it
        {"name": "ns_attn_out_bf16", "op": "newton_schulz", "shapes": "496x3968", "in": "f32", "out": "bf16"},
        # a resblock shard whose orthogonal update is kept in fp32
        {"name": "ns_resblock_f32", "op": "newton_schulz", "shapes": _flat(SHARD), "in": "f32", "out": "f32"},
        # odd sizes that no tile divides, 16-bit updates
        {"name": "ns_ragged_f16", "op": "newton_schulz", "shapes": "1001x777,333x2049,130x511,17x1025", "in": "bf16", "out": "f16"},
        # the smallest step: two small matrices, latency
        {"name": "muon_small_bf16", "op": "muon", "shapes": "496x256,130x512", "param": "bf16", "nesterov": True, "adjust": 0},
        # four resblock shards in one call, bf16 parameters
        {"name": "muon_4_resblocks_bf16", "op": "muon", "shapes": _flat(SHARD * 4), "param": "bf16", "nesterov": True, "adjust": 1},
        # fp32 parameters, one resblock shard, plain momentum
        {"name": "muon_resblock_f32", "op": "muon", "shapes": _flat(SHARD), "param": "f32", "nesterov": False, "adjust": 1},
        # the unsharded resblock: the largest matrices
        {"name": "muon_unsharded_f16", "op": "muon", "shapes": _flat(FULL), "param": "f16", "nesterov": True, "adjust": 1},
        # one decoding step's tokens
        {"name": "lookup_tokens_f16", "op": "embed_lookup", "n": 16, "vocab": 8192, "dim": D_MODEL, "table": "f32", "out": "f16",
         "ids": "i64", "zipf": False, "pad": 0.0, "scale": 1.0},
        # sixteen sequences of 1280 tokens
        {"name": "lookup_batch_bf16", "op": "embed_lookup", "n": 16 * 1280, "vocab": 32768, "dim": D_MODEL, "table": "f32", "out": "bf16",
         "ids": "i64", "zipf": True, "pad": 0.05, "scale": 63.0},
        # the gradient of a short sequence into a small table
        {"name": "grad_short_f32", "op": "embed_grad", "n": 333, "vocab": 1031, "dim": 1000, "dx": "f32", "ids": "i32",
         "zipf": False, "pad": 0.0, "scale": 1.0, "accumulate": False},
        # the gradient of sixteen sequences, tokens as skewed as text
        {"name": "grad_batch_f32", "op": "embed_grad", "n": 16 * 1280, "vocab": 32768, "dim": D_MODEL, "dx": "f32", "ids": "i64",
         "zipf": True, "pad": 0.05, "scale": 63.0, "accumulate": False},
        # many tokens, a small table, added to the gradient a tied unembedding left there
        {"name": "grad_tied_bf16", "op": "embed_grad", "n": 65537, "vocab": 8195, "dim": 1032, "dx": "bf16", "ids": "i64",
         "zipf": True, "pad": 0.0, "scale": 1.0, "accumulate": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["newton_schulz", "muon", "embed_lookup", "embed_grad"])
    if op == "newton_schulz":
        shapes = [(_logint(rng, 16, 4500), _logint(rng, 16, 4500)) for _ in range(rng.randint(1, 6))]
        return {"op": op, "shapes": _flat(shapes), "in": rng.choice(["f32", "f16", "bf16"]), "out": rng.choice(["f32", "f16", "bf16"])}
    if op == "muon":
        shapes = [(_logint(rng, 16, 4500), 8 * _logint(rng, 2, 560)) for _ in range(rng.randint(1, 6))]
        return {"op": op, "shapes": _flat(shapes), "param": rng.choice(["f32", "f16", "bf16"]), "nesterov": rng.random() < 0.5,
                "adjust": rng.randint(0, 1)}
    case = {"op": op, "n": _logint(rng, 1, 65536), "vocab": _logint(rng, 2, 65536), "dim": _logint(rng, 8, 4096),
            "ids": rng.choice(["i32", "i64"]), "zipf": rng.random() < 0.5, "pad": rng.choice([0.0, 0.1]),
            "scale": rng.choice([1.0, 0.37, 63.0])}
    if op == "embed_lookup":
        case.update(table=rng.choice(["f32", "f16", "bf16"]), out=rng.choice(["f32", "f16", "bf16"]))
    else:
        case.update(dx=rng.choice(["f32", "f16", "bf16"]), accumulate=rng.random() < 0.5)
    return case


# ---- inputs ------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _update(m, n, g, dtype):
    """A gradient as the path meets it: rows of very different size, and a few strong directions."""
    rows = torch.exp(torch.empty(m, 1, device="cuda").uniform_(math.log(1e-3), 0.0, generator=g))
    x = torch.randn(m, n, device="cuda", generator=g) * rows
    k = min(8, m, n)
    x += torch.randn(m, k, device="cuda", generator=g) @ torch.randn(k, n, device="cuda", generator=g)
    return (x * 1e-2).to(dtype)


def _low_rank(m, n, g):
    """A decompressed gradient: rank 112 at most, with a falling spectrum."""
    r = min(RANK, m, n)
    s = torch.exp(torch.linspace(0.0, -4.0, r, device="cuda"))
    return (torch.randn(m, r, device="cuda", generator=g) * s) @ torch.randn(r, n, device="cuda", generator=g) * 1e-2


def _weights(case):
    v = case["vocab"]
    w = torch.ones(v, dtype=torch.float64)
    return 1.0 / (torch.arange(v, dtype=torch.float64) + 2.7) if case["zipf"] else w


def _tokens(case, g):
    w = _weights(case).cuda()
    c = torch.cumsum(w, 0)
    u = torch.rand(case["n"], device="cuda", generator=g, dtype=torch.float64) * c[-1]
    ids = torch.searchsorted(c, u).clamp_(max=case["vocab"] - 1)
    ids = torch.randperm(case["vocab"], device="cuda", generator=g)[ids]
    pad = torch.rand(case["n"], device="cuda", generator=g) < case["pad"]
    ids = torch.where(pad, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)


def _inputs(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "newton_schulz":
        ins = [_update(m, n, g, DTYPES[case["in"]]) for m, n in _shapes(case)]
        return {"in": ins, "out": [torch.empty(x.shape, dtype=DTYPES[case["out"]], device="cuda") for x in ins]}
    if op == "muon":
        st = {"grad": [], "mom": [], "param": []}
        for m, n in _shapes(case):
            st["grad"].append(_low_rank(m, n, g))
            st["mom"].append(_update(m, n, g, torch.float32) + 3.0 * _low_rank(m, n, g))
            st["param"].append((torch.randn(m, n, device="cuda", generator=g) * 0.02).to(DTYPES[case["param"]]))
        st["skip"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["norm"] = torch.rand(2, device="cuda", generator=g) * 0.5 + 0.5       # global norm, clipping factor
        return st
    st = {"ids": _tokens(case, g)}
    n, v, d = case["n"], case["vocab"], case["dim"]
    if op == "embed_lookup":
        st["table"] = (torch.randn(v, d, device="cuda", generator=g) * 0.02).to(DTYPES[case["table"]])
        st["out"] = torch.empty(n, d, dtype=DTYPES[case["out"]], device="cuda")
    else:
        st["dx"] = (torch.randn(n, d, device="cuda", generator=g) * 1e-3).to(DTYPES[case["dx"]])
        st["dtable"] = torch.randn(v, d, device="cuda", generator=g) * 1e-3
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if not own:
        return st
    import rank_gradient_compression_powersgd_amd as psgd
    op = case["op"]
    if op == "newton_schulz":
        st["group"] = psgd.NewtonSchulzGroup(st["in"], st["out"])
    elif op == "muon":
        grads = st["grad"]
        rank = min(RANK, min(min(x.shape) for x in grads))
        st["group"] = psgd.PowerSGDGroup([None] * len(grads), [0] * len(grads), torch.ones(1, device="cuda"), rank,
                                         [torch.zeros(x.shape[1], rank) for x in grads], [torch.zeros_like(x) for x in grads])
        for o, x in zip(st["group"].out, grads):
            o.copy_(x)
        st["group"].attach_muon(st["param"], st["mom"])
        st["hp"] = psgd.muon_hparams(nesterov=case["nesterov"], adjust=case["adjust"], eps=EPS, **MUON)
    else:
        st["ctx"] = psgd.psgd_create(0, 1)
        if op == "embed_grad":
            need = psgd.psgd_embed_grad_workspace(case["n"], case["vocab"], case["dim"])
            st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return st


# ---- one pass ----------------------------------------------------------------------------
def _factor(case, m, n):
    return 0.2 * math.sqrt(max(m, n)) if case["adjust"] else math.sqrt(max(1.0, m / n))


def _plain_newton_schulz(u):
    a, b, c = COEF
    norm = u.double().square().sum().sqrt().clamp(min=EPS)
    x = (u / norm).float()
    flip = x.shape[0] > x.shape[1]
    if flip:
        x = x.t().contiguous()
    for _ in range(STEPS):
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if flip else x


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "newton_schulz":
        for x, o in zip(st["in"], st["out"]):
            o.copy_(_plain_newton_schulz(x.float()))
        return st["out"]
    if op == "muon":
        mu, lr, wd = MUON["momentum"], MUON["lr"], MUON["weight_decay"]
        for g, m, p in zip(st["grad"], st["mom"], st["param"]):
            g = g * st["norm"][1]
            m.mul_(mu).add_(g)
            o = _plain_newton_schulz(g + mu * m if case["nesterov"] else m)
            t = p.float()
            p.copy_(t - lr * (_factor(case, *p.shape) * o + wd * t))
        return {"param": st["param"], "momentum": st["mom"]}
    ids = st["ids"].long()
    ok = (ids >= 0) & (ids < case["vocab"])
    if op == "embed_lookup":
        rows = st["table"][ids.clamp(0, case["vocab"] - 1)].float() * case["scale"]
        st["out"].copy_(torch.where(ok[:, None], rows, torch.zeros_like(rows)))
        return st["out"]
    # one slot past the table takes the rows that belong to no token
    total = torch.zeros(case["vocab"] + 1, case["dim"], device="cuda")
    total.index_add_(0, torch.where(ok, ids, torch.full_like(ids, case["vocab"])), st["dx"].float())
    total = total[:-1] * case["scale"]
    st["dtable"].copy_(st["dtable"] + total if case["accumulate"] else total)
    return st["dtable"]


def run(st):
    if not own:
        return _plain(st)
    import rank_gradient_compression_powersgd_amd as psgd
    case = st["case"]
    op = case["op"]
    if op == "newton_schulz":
        st["group"].run()
        return st["out"]
    if op == "muon":
        group = st["group"]
        psgd.psgd_muon_update(group.ctx, group.plan, st["skip"], st["norm"], st["hp"])
        return {"param": st["param"], "momentum": st["mom"]}
    if op == "embed_lookup":
        psgd.psgd_embed_lookup(st["ctx"], st["table"], st["ids"], st["out"], case["scale"])
        return st["out"]
    psgd.psgd_embed_grad(st["ctx"], st["dx"], st["ids"], st["dtable"], case["scale"], case["accumulate"], st["workspace"])
    return st["dtable"]


# ---- the definition in 64 bits -----------------------------------------------------------
def _exact_orthogonal(u):
    """Newton-Schulz on the tall side: X (a I + b W + c W^2), W = X^T X."""
    a, b, c = COEF
    x = u / max(float(torch.linalg.vector_norm(u)), EPS)
    wide = x.shape[1] > x.shape[0]
    x = x.mT.contiguous() if wide else x
    eye = torch.eye(x.shape[1], dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        w = torch.mm(x.mT.contiguous(), x)
        x = torch.mm(x, torch.mm(w, c * w + b * eye) + a * eye)
    return x.mT if wide else x


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "newton_schulz":
        return [_exact_orthogonal(x.double()).contiguous() for x in st["in"]]
    if op == "muon":
        clip, mu = float(st["norm"][1]), MUON["momentum"]
        moms = [mu * m.double() + clip * g.double() for g, m in zip(st["grad"], st["mom"])]
        params = []
        for g, m, p in zip(st["grad"], moms, st["param"]):
            o = _exact_orthogonal(clip * g.double() + mu * m if case["nesterov"] else m)
            rows, cols = p.shape
            params.append(p.double() * (1.0 - MUON["lr"] * MUON["weight_decay"]) - MUON["lr"] * _factor(case, rows, cols) * o)
        return {"param": params, "momentum": moms}
    ids = st["ids"].long()
    keep = torch.nonzero((ids >= 0) & (ids < case["vocab"]))[:, 0]
    if op == "embed_lookup":
        out = torch.zeros(case["n"], case["dim"], dtype=torch.float64, device="cuda")
        out[keep] = st["table"].index_select(0, ids[keep]).double() * case["scale"]
        return out
    total = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
    total.scatter_add_(0, ids[keep][:, None].expand(-1, case["dim"]).contiguous(), case["scale"] * st["dx"][keep].double())
    return st["dtable"].double() + total if case["accumulate"] else total


# ---- what a pass cannot do without -------------------------------------------------------
def _distinct(case):
    p = _weights(case)
    p = p / p.sum() * (1.0 - case["pad"])
    return float((1.0 - (1.0 - p) ** case["n"]).sum())


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    op = case["op"]
    if op in ("newton_schulz", "muon"):
        nbytes = flops = 0
        for m, n in _shapes(case):
            s, l = min(m, n), max(m, n)
            flops += STEPS * (3 * s * s * l + s * s * s)         # symmetric products count once
            if op == "muon":
                nbytes += m * n * (4 + 8 + 2 * size[case["param"]])
            else:
                nbytes += m * n * (size[case["in"]] + size[case["out"]])
        return {"bytes": nbytes, "flops": flops}
    n, v, d = case["n"], case["vocab"], case["dim"]
    idb = n * (4 if case["ids"] == "i32" else 8)
    if op == "embed_lookup":
        return {"bytes": idb + d * (_distinct(case) * size[case["table"]] + n * size[case["out"]]), "flops": n * d}
    table = 8 * _distinct(case) if case["accumulate"] else 4 * v
    return {"bytes": idb + d * (n * (1.0 - case["pad"]) * size[case["dx"]] + table), "flops": n * d}
