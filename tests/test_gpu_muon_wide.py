"""Newton-Schulz and the Muon step on groups whose products take 128- and 256-wide tiles, alone and
split along K, against the iteration itself in float64 on the device.

Tolerances, as a share of the orthogonal factor's Frobenius norm:
  fast      2e-3, what the header states for updates of ordinary spectra (random ones here).
  accurate  5.8e-6. In the mean square (0.58 of the largest rounding), in units of 2^-24: each factor's
            22 bits 4 * 0.58 = 2.3; lo lo, left out, 1; 12 MFMAs on one accumulator per 128 k, each
            rounding the growing sum, 0.58 sqrt(3 (1 + 4 + 9 + 16) / 16) = 1.4; the sums of these over
            15872 k at most, 0.58 sqrt(124 / 3) = 3.7. A product: sqrt(2 * 2.3^2 + 1 + 1.4^2 + 3.7^2)
            = 5.2, with its own storage 5.7: 3.4e-7. A step multiplies A's error by 4.8 * 1.46 = 7 (the
            bound of B's derivative times X's of A), B's by 2.8 and adds B X's own: sqrt(7^2 + 2.8^2 + 1)
            * 3.4e-7 = 2.6e-6; five independent steps sqrt(5) times that.
Parameters and 16-bit outputs add their type's half step of what is stored, fp32 arithmetic around them
three of 2^-24.
"""
from __future__ import annotations

import pytest

import oracle
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu

FAST_TOL, ACC_TOL = 2e-3, 5.8e-6
EPS2 = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _dt(code):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[code]


def _direct(u, coef=oracle.muon.QUINTIC, steps=5):
    """The iteration in float64."""
    import torch
    x = u.double()
    x = x / torch.linalg.vector_norm(x)
    x = x.t().contiguous() if x.shape[0] > x.shape[1] else x
    for _ in range(steps):
        a = x @ x.t().contiguous()
        x = coef[0] * x + (coef[1] * a + coef[2] * (a @ a)) @ x
    return x.t() if u.shape[0] > u.shape[1] else x


def _updates(shapes, dtype="f32", seed=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1000 + len(shapes) + seed)
    return [(torch.randn(m, n, device="cuda", generator=gen) * (0.05 + torch.rand(m, 1, device="cuda", generator=gen))).to(_dt(dtype))
            for m, n in shapes]


def _off(got, want):
    import torch
    return float(torch.linalg.vector_norm(got.double() - want)), float(torch.linalg.vector_norm(want))


# Which product takes which tile (A, B, update) and whether A and B are split: what the group is here for
GROUPS = {
    "128 128 128": [(1200, 1104)] * 4,
    "256 256 256": [(1030, 2048)] * 16,
    "accurate: 64 64 128, split": [(1500, 1500)],
    "128 128 256, split": [(3000, 3000)],
    "one resblock shard: A split at 128, accurate B too": [(3968, 1488), (496, 3968), (3968, 1984), (1984, 3968)],
    "unsharded resblock: split at 256": [(3968, 11904), (3968, 3968), (15872, 3968)],
}


@pytest.mark.parametrize("accurate", [False, True])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", list(GROUPS))
def test_outputs_of_every_type(name, out, accurate):
    import torch
    from rank_gradient_compression_powersgd_amd import NewtonSchulzGroup
    ups = _updates(GROUPS[name])
    outs = [torch.empty(u.shape, dtype=_dt(out), device="cuda") for u in ups]
    log(f"newton-schulz {name} -> {out} accurate={accurate}")
    g = NewtonSchulzGroup(ups, outs, accurate)
    g.run()
    torch.cuda.synchronize()
    for i, (u, o) in enumerate(zip(ups, outs)):
        if i >= 4:
            break
        err, norm = _off(o, _direct(u))
        log(f"  {tuple(u.shape)}: {err / norm:.2e}")
        assert err <= ((ACC_TOL if accurate else FAST_TOL) + EPS2[out]) * norm, (i, err / norm)
    g.close()


@pytest.mark.parametrize("shapes", [[(1500, 4096)] * 8, [(512, 4096)] * 40, [(128, 4096)] * 3])
def test_rounded_sums_of_long_products(shapes):
    """One step of X <- A X on positive elements: nothing cancels, and the elements' sums, all about as
    large, round alike, so that what a long sum loses shows. In units of 2^-24, mean square: A
    sqrt(1.4^2 + 1.9^2) = 2.4, A X over up to 1500 k sqrt(1.4^2 + 1.2^2) = 1.8, the stores of A, B and X
    1.2 each: together 3.7, 2.2e-7. One chain over all k: 6.6 and 4.0, 4.6e-7."""
    import torch
    from rank_gradient_compression_powersgd_amd import NewtonSchulzGroup, ns_hparams
    gen = torch.Generator(device="cuda").manual_seed(5)
    ups = [torch.rand(s, device="cuda", generator=gen) + 0.5 for s in shapes]
    outs = [torch.empty_like(u) for u in ups]
    g = NewtonSchulzGroup(ups, outs, accurate=True)
    g.run(ns_hparams(0.0, 1.0, 0.0, steps=1))
    torch.cuda.synchronize()
    for i in (0, len(ups) - 1):
        err, norm = _off(outs[i], _direct(ups[i], (0.0, 1.0, 0.0), 1))
        log(f"  {shapes[i]}: {err / norm:.2e}")
        assert err <= 2.2e-7 * norm, (i, err / norm)
    g.close()


# ---- the Muon step ---------------------------------------------------------------------------
MUON = {"64": [(300, 200), (130, 264)], "128": [(1200, 1104)] * 4, "256": [(1030, 2048)] * 16, "split": [(3000, 3000)]}


def _params(shapes, pdt, form, gen):
    """(parameter, its buffer, True where the buffer is the parameter's): contiguous; a slice of odd pitch;
    contiguous rows from an address that is aligned to one element only."""
    import torch
    out = []
    for m, n in shapes:
        if form == "odd pitch":
            buf = torch.full((m + 2, n + 3), 7.0, dtype=_dt(pdt), device="cuda")
            mine = torch.zeros_like(buf, dtype=torch.bool)
            view, inside = buf[1:m + 1, 1:n + 1], mine[1:m + 1, 1:n + 1]
        elif form == "one element off":
            buf = torch.full((m * n + 9,), 7.0, dtype=_dt(pdt), device="cuda")
            mine = torch.zeros_like(buf, dtype=torch.bool)
            view, inside = buf[1:1 + m * n].view(m, n), mine[1:1 + m * n].view(m, n)
        else:
            buf = torch.empty(m, n, dtype=_dt(pdt), device="cuda")
            mine = torch.zeros_like(buf, dtype=torch.bool)
            view, inside = buf, mine
        view.copy_(torch.randn(m, n, device="cuda", generator=gen) * 0.02)
        inside.fill_(True)
        out.append((view, buf, mine))
    return out


@pytest.mark.parametrize("pdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", ["contiguous", "odd pitch", "one element off"])
@pytest.mark.parametrize("name", list(MUON))
def test_muon_step(name, form, pdt):
    """Every tile width of the last product, which reads and writes the parameter, with parameters that
    it takes four elements at a time and one at a time; what lies around a parameter stays."""
    import torch
    from rank_gradient_compression_powersgd_amd import PowerSGDGroup, muon_hparams, psgd_muon_update
    shapes, accurate = MUON[name], pdt == "f32"
    gen = torch.Generator(device="cuda").manual_seed(77)
    k = len(shapes)
    g = PowerSGDGroup([None] * k, [0] * k, torch.ones(1, device="cuda"), 4, [torch.zeros(n, 4) for _, n in shapes],
                      [torch.zeros(s, device="cuda") for s in shapes])
    for o, x in zip(g.out, _updates(shapes, seed=1)):
        o.copy_(x)
    params = _params(shapes, pdt, form, gen)
    mom = [torch.randn(s, device="cuda", generator=gen) for s in shapes]
    g.attach_muon([p for p, _, _ in params], mom)
    hp = muon_hparams(0.5, 0.9, 0.1, nesterov=form != "odd pitch", adjust=1)
    clip = 0.25
    old = [(p.double().clone(), m.double().clone()) for (p, _, _), m in list(zip(params, mom))[:4]]
    log(f"muon {name} {form} {pdt}")
    psgd_muon_update(g.ctx, g.plan, g.skip, torch.tensor([4.0, clip], device="cuda"), hp)
    torch.cuda.synchronize()
    for i, (p0, m0) in enumerate(old):
        grad = clip * g.out[i].double()
        want_m = hp.momentum * m0 + grad
        # two products and a sum, each rounded once
        bound = 2.01 * 2.0 ** -24 * (grad.abs() + (hp.momentum * m0).abs())
        assert bool(((mom[i].double() - want_m).abs() <= bound).all()), i
        factor = oracle.muon_factor(*shapes[i], 1)
        upd = hp.lr * factor * _direct(grad + hp.momentum * want_m if hp.nesterov else want_m)
        want_p = p0 * (1.0 - hp.lr * hp.weight_decay) - upd
        err, norm = _off(params[i][0], want_p)
        tol = (ACC_TOL if accurate else FAST_TOL) * float(torch.linalg.vector_norm(upd)) + \
            (EPS2[pdt] + 3 * 2.0 ** -24) * (norm + float(torch.linalg.vector_norm(p0)))
        if i == 0:
            log(f"  {shapes[i]}: {err / norm:.2e}, allowed {tol / norm:.2e}")
        assert err <= tol, (i, err, tol)
    for _, buf, mine in params:
        assert bool((buf[~mine] == 7.0).all())
    g.close()
