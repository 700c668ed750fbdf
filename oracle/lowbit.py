"""AdamW with 8-bit moments and microscaled 4-bit matrices (numpy): hashes and codes bit by bit,
everything else in float64.

The moments' arithmetic is also here operation by operation in float32 (`moments32`), because their codes
are defined on those numbers.
"""
from __future__ import annotations

import numpy as np

__all__ = ["adamw_param", "bias_free", "carried8", "code_values", "decode8", "encode8", "hash_bits", "hash_key", "hash_more", "moments32",
           "mx_quantize", "mx_unpack", "mx_values", "round16"]

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---- random bits -----------------------------------------------------------------------------
def _mix(x):
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    for shift, factor in ((16, 0xA54FF53B), (15, 0xBB67AE85)):
        x = ((x ^ (x >> np.uint64(shift))) * np.uint64(factor)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def hash_key(seed: int, step: int, tensor: int):
    seed &= 0xFFFFFFFFFFFFFFFF
    k = _mix((seed & 0xFFFFFFFF) ^ 0x9E3779B9)
    k = _mix(k ^ np.uint64(seed >> 32))
    return _mix(_mix(np.uint64(step) ^ k) ^ np.uint64(tensor))


def hash_bits(key, index):
    index = np.asarray(index, np.uint64)
    return _mix((index & np.uint64(0xFFFFFFFF)) ^ _mix((index >> np.uint64(32)) ^ key)).astype(np.uint32)


def hash_more(r):
    r = np.asarray(r, np.uint64)
    t = ((r ^ (r >> np.uint64(15))) * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)
    return (t ^ (t >> np.uint64(16))).astype(np.uint32)


# ---- 8-bit moments -----------------------------------------------------------------------------
def code_values(second: bool) -> np.ndarray:
    """Magnitudes of the codes of a group whose exponent is 0 (byte 127): fields 0.. with 3 fraction bits."""
    top = 31 if second else 15
    c = np.arange(256 if second else 128)
    field, frac = c >> 3, c & 7
    return np.where(field > 0, 8 + frac, frac) * 2.0 ** (np.maximum(field, 1) - top - 3)


def decode8(codes, exps, second: bool) -> np.ndarray:
    c = np.asarray(codes, np.int64).reshape(-1, 64)
    e = np.asarray(exps, np.int64)[:, None]
    v = code_values(second)[c if second else c & 127]
    v = v if second else np.where(c > 127, -v, v)
    with np.errstate(over="ignore"):
        return np.where(e == 255, np.nan, v * 2.0 ** (e - 127.0)).reshape(-1)


def carried8(c1, e1, c2, e2):
    """(m1, m2) as a step takes them up: those of a group whose m2 were lost (byte 255) as 0 and the format's largest
    value, lost m1 as 0."""
    m1, m2 = decode8(c1, e1, False), decode8(c2, e2, True)
    lost1, lost2 = (np.repeat(np.asarray(e) == 255, 64) for e in (e1, e2))
    return np.where(lost1 | lost2, 0.0, m1), np.where(lost2, 1.875 * 2.0 ** 127, m2)


def encode8(v, second: bool, u=None):
    """Codes and exponent bytes of values (whole groups of 64). u: per element a number in [0, 1) added before
    rounding down, or None: to nearest even."""
    v = np.asarray(v, np.float64).reshape(-1, 64)
    big = np.abs(v).max(1)
    _, e = np.frexp(big)
    e = e - 1                                                     # big in [2^e, 2^(e + 1))
    e = np.where(big > 1.875 * 2.0 ** e, e + 1, e)
    e = np.where(big == 0, -126, np.maximum(e, -126))
    unit = np.abs(v) / 2.0 ** e[:, None]
    top = 31 if second else 15
    _, x = np.frexp(unit)
    step = 2.0 ** (np.maximum(x - 1, 1 - top) - 3)                # distance of the neighbours
    q = np.rint(unit / step) if u is None else np.floor(unit / step + np.asarray(u).reshape(v.shape))
    q = q * step
    c = np.searchsorted(code_values(second), q)
    if second:
        c = np.where((v > 0) & (c == 0), 1, c)
    else:
        c = c | (np.where(v < 0, 128, 0))
    return c.astype(np.uint8).reshape(-1), (e + 127).astype(np.uint8)


def bias_free(beta: float, t: int) -> float:
    return 1.0 / (1.0 - float(np.float32(beta)) ** t)


def moments32(m1, m2, g, clip, b1, b2):
    """The new moments with every operation rounded to float32."""
    f = np.float32
    g = np.asarray(g, f) * f(clip)
    m1 = np.asarray(m1, f) * f(b1) + g * (f(1.0) - f(b1))
    m2 = np.asarray(m2, f) * f(b2) + (g * g) * (f(1.0) - f(b2))
    assert m1.dtype == f and m2.dtype == f
    return m1, m2


def adamw_param(param, m1, m2, t, lr, b1, b2, eps, wd):
    """The parameter after step t from the new moments, unrounded; hyperparameters as float32 holds them."""
    lr, eps, wd = (float(np.float32(x)) for x in (lr, eps, wd))
    p = np.asarray(param, np.float64)
    return p - lr * (m1 * bias_free(b1, t) / (np.sqrt(m2 * bias_free(b2, t)) + eps) + wd * p)


def round16(v, kind: str, u) -> np.ndarray:
    """v to fp16 or bf16 numbers, u in [0, 1) of their distance added before rounding towards zero."""
    bits, low = (10, -14) if kind == "f16" else (7, -126)
    v = np.asarray(v, np.float64)
    _, x = np.frexp(np.abs(v))
    step = 2.0 ** (np.maximum(x - 1, low) - bits)
    return np.sign(v) * np.floor(np.abs(v) / step + u) * step


# ---- 4-bit matrices ------------------------------------------------------------------------------
def mx_quantize(x, u=None):
    """(values, exponent bytes [rows, blocks]) of a matrix quantised along its rows; u as in encode8."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    pad = -k % 32
    v = np.pad(x, ((0, 0), (0, pad))).reshape(rows, -1, 32)
    bad = ~np.isfinite(v).all(2)
    v = np.where(bad[:, :, None], 0.0, v)
    big = np.abs(v).max(2)
    _, e = np.frexp(big)
    e = e - 1
    e = np.where(big > 1.5 * 2.0 ** e, e + 1, e) if u is not None else np.where(big >= 1.75 * 2.0 ** e, e + 1, e)
    s = np.where(big == 0, 1, np.maximum(e - 2 + 127, 1))
    a = np.abs(v) / 2.0 ** (s[:, :, None] - 127.0)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    if u is None:
        q = np.minimum(np.rint(a / step) * step, 6.0)
    else:
        q = np.floor(a / step + np.pad(u, ((0, 0), (0, pad))).reshape(v.shape)) * step
    out = np.sign(v) * q * 2.0 ** (s[:, :, None] - 127.0)
    out = np.where(bad[:, :, None], np.nan, out).reshape(rows, -1)[:, :k]
    return out, np.where(bad, 255, s).astype(np.uint8)


def mx_unpack(data, rows: int, k: int):
    """(codes [rows, 128 P], exponent bytes [rows, 4 P]) of a matrix's buffer, padding included."""
    data = np.asarray(data, np.uint8)
    p, g = -(-k // 128), -(-rows // 64)
    b = data[:p * rows * 64].reshape(p, rows, 64).transpose(1, 0, 2).reshape(rows, -1)
    codes = np.stack([b & 15, b >> 4], 2).reshape(rows, -1)
    s = data[p * rows * 64:p * (rows * 64 + g * 256)].reshape(p, g, 4, 16, 4)     # panel, group, block, row % 16, row / 16
    return codes, s.transpose(1, 4, 3, 0, 2).reshape(g * 64, 4 * p)[:rows]


def mx_values(data, rows: int, k: int) -> np.ndarray:
    codes, s = mx_unpack(data, rows, k)
    v = GRID[codes & 7] * np.where(codes > 7, -1.0, 1.0)
    f = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127.0))
    return (v.reshape(rows, -1, 32) * f[:, :, None]).reshape(rows, -1)[:, :k]
