"""float64 Newton-Schulz orthogonalisation, the Muon step and the embedding's gradient (numpy).

Newton-Schulz is written by its action on singular values: X0 = U / max(||U||_F, eps) = V S W^T
keeps V and W while each step maps s -> a s + b s^3 + c s^5, so no product of the iteration is
repeated here. A direction whose singular value is lost to float64 rounding contributes nothing.
"""
from __future__ import annotations

import numpy as np

__all__ = ["QUINTIC", "embed_grad", "embed_lookup", "muon_factor", "muon_step", "newton_schulz"]

QUINTIC = (3.4445, -4.7750, 2.0315)


def newton_schulz(u, coef=QUINTIC, steps: int = 5, eps: float = 1e-20) -> np.ndarray:
    u = np.asarray(u, np.float64)
    if not np.isfinite(u).all():
        return np.full(u.shape, np.nan)
    norm = max(float(np.linalg.norm(u)), eps)
    v, s, wt = np.linalg.svd(u / norm, full_matrices=False)
    a, b, c = coef
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return (v * s) @ wt


def muon_factor(m: int, n: int, adjust: int) -> float:
    return 0.2 * np.sqrt(max(m, n)) if adjust else float(np.sqrt(max(1.0, m / n)))


def muon_step(param, momentum, grad, clip, lr, mu, weight_decay, nesterov, adjust, coef=QUINTIC, steps=5,
              eps=1e-20):
    """(param, momentum) after one step, unrounded."""
    g = clip * np.asarray(grad, np.float64)
    mom = mu * np.asarray(momentum, np.float64) + g
    o = newton_schulz(g + mu * mom if nesterov else mom, coef, steps, eps)
    th = np.asarray(param, np.float64)
    return th - lr * (muon_factor(*th.shape, adjust) * o + weight_decay * th), mom


def embed_lookup(table, ids, scale) -> np.ndarray:
    table = np.asarray(table, np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < table.shape[0]:
            out[t] = scale * table[i]
    return out


def embed_grad(dx, ids, vocab, scale, base=None) -> np.ndarray:
    dx = np.asarray(dx, np.float64)
    out = np.zeros((vocab, dx.shape[1])) if base is None else np.asarray(base, np.float64).copy()
    for t, i in enumerate(ids):
        if 0 <= i < vocab:
            out[i] += scale * dx[t]
    return out
