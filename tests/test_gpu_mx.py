"""Microscaled 4-bit matrices and their products against the float64 oracle.

Codes and exponents are compared bit by bit, padding included. A product's operands are the decoded
matrices. Every product of two elements is exact in fp32 (2 + 2 significant bits); a panel's 128 are
added by one instruction into an fp32 sum, at worst one after another: 128 P additions of 2^-24 of what
has been added so far, so the error is at most 128 P 2^-24 sum |a b|; of random signs it is far less, and
(P + 8) 2^-23 sum |a b| is asked for here, 8 for the instruction's own additions and the joins. The
scale, the addition and the storage round once each, by half a step.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import lowbit as L
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu


def _dt(k):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[k]


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.fixture(scope="module")
def ctx():
    from rank_gradient_compression_powersgd_amd import psgd_create, psgd_destroy
    c = psgd_create(0, 1)
    yield c
    psgd_destroy(c)


def _matrix(m, n, kind, seed, skew=0, ld=None):
    """A matrix on the device (a view with row stride ld that starts `skew` elements in) and its values."""
    import torch
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, n)) * np.exp(rng.uniform(np.log(1e-3), np.log(30.0), (m, 1)))
    x[rng.random((m, n)) < 0.05] *= 20
    ld = ld or n
    flat = torch.full((skew + m * ld + 8,), float("nan"), dtype=_dt(kind), device="cuda")
    t = torch.as_strided(flat, (m, n), (ld, 1), skew)
    t.copy_(torch.from_numpy(x))
    return t, _np(t)


def _bits(m, n, seed, step=0):
    """u in [0, 1) of every element."""
    half = (n + 1) // 2
    h = L.hash_bits(L.hash_key(seed, step, 0), np.arange(m * half, dtype=np.uint64)).reshape(m, half)
    both = np.stack([h, (h << np.uint32(16)) | (h >> np.uint32(16))], 2).reshape(m, -1)[:, :n]
    return (both >> np.uint32(10)) * 2.0 ** -22


def _check(mx, x, u, what):
    """An MxTensor against its matrix's values."""
    rows, k = x.shape
    want, s = L.mx_quantize(x, u)
    data = mx.data.cpu().numpy()
    codes, exps = L.mx_unpack(data, rows, k)
    pad = exps[:, s.shape[1]:]
    assert np.array_equal(exps[:, :s.shape[1]], s), what
    assert (pad == 1).all() and (codes[:, k:] == 0).all(), what
    got = L.mx_values(data, rows, k)
    bad = np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))
    assert len(bad) == 0, (what, bad[:6], [(got[tuple(b)], want[tuple(b)]) for b in bad[:6]])
    nan = np.repeat(s == 255, 32, axis=1)[:, :k]
    assert (codes[:, :k][nan] == 0).all(), what


SHAPES = [(1, 1), (1, 128), (3, 33), (64, 127), (65, 129), (31, 2), (200, 300), (129, 1000), (1, 4097), (333, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("stochastic", [False, True])
def test_both_directions(ctx, shape, kind, stochastic):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_quantize
    m, n = shape
    seed = 77 + (5 << 40)
    log(f"quantize {shape} {kind} {stochastic}")
    for skew, ld in ((0, None), (1, n + 3)):
        t, x = _matrix(m, n, kind, m * 31 + n, skew, ld)
        u = _bits(m, n, seed) if stochastic else None
        keep = 64
        outs = {}
        for ways in ("row", "col", "both"):
            mk = lambda r, k: MxTensor(r, k, data=torch.full((MxTensor(r, k).data.numel() + keep,), 0xA5, dtype=torch.uint8, device="cuda"))  # noqa: E731
            row, col = (mk(m, n) if ways != "col" else None), (mk(n, m) if ways != "row" else None)
            psgd_mx_quantize(ctx, t, row, col, stochastic=stochastic, seed=seed)
            for name, mx, v, w in (("row", row, x, u), ("col", col, x.T, None if u is None else u.T)):
                if mx is None:
                    continue
                _check(mx, v, w, (shape, kind, ways, name, skew))
                assert (mx.data[-keep:] == 0xA5).all()
                if name in outs:                                          # padding of the exponents' rows aside
                    a, b = (L.mx_unpack(d.data.cpu().numpy(), mx.rows, mx.k) for d in (mx, outs[name]))
                    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
                outs[name] = mx


def test_the_step_count_is_part_of_the_bits(ctx):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_quantize
    t, x = _matrix(70, 260, "f32", 1)
    step = torch.tensor([41], dtype=torch.int32, device="cuda")
    row, col = MxTensor(70, 260), MxTensor(260, 70)
    psgd_mx_quantize(ctx, t, row, col, stochastic=True, seed=9, step=step)
    u = _bits(70, 260, 9, 41)
    _check(row, x, u, "row")
    _check(col, x.T, u.T, "col")
    psgd_mx_quantize(ctx, t, row, stochastic=True, seed=9, step=step)
    _check(row, x, u, "row alone")


def _special():
    x = np.zeros((40, 96), np.float64)
    x[0, :8] = [7.0, 6.99, 5.0, 3.5, 2.5, 1.75, 0.75, 0.25]
    x[1, :8] = [6.0, -5.0, 1.25, -1.25, 0.25, -0.25, 0.2500001, 4.999]
    x[2, :4] = [6.0000005, -0.0, 1e-9, 3.0]
    x[3, 5] = np.inf
    x[4, 40] = -np.inf
    x[5, 70] = np.nan
    x[6, :3] = [3.4e38, -1e38, 1e30]
    x[7, :4] = [1.1e-38, 2e-39, 6e-39, 1e-45]                               # fp32 subnormals
    x[8, :3] = [3e-38, 1.2e-38, 4e-39]
    x[9, :2] = [1e-45, -1e-45]
    x[10] = 6.0
    x[11] = -np.exp2(np.arange(96) % 40 - 60)
    return x


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_ties_borders_and_special_values(ctx, kind, stochastic):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_dequantize, psgd_mx_quantize
    t = torch.from_numpy(_special()).to("cuda", _dt(kind))                   # fp16: some become infinities, some 0
    x = _np(t)
    row, col = MxTensor(40, 96), MxTensor(96, 40)
    psgd_mx_quantize(ctx, t, row, col, stochastic=stochastic, seed=3)
    u = _bits(40, 96, 3) if stochastic else None
    _check(row, x, u, "row")
    _check(col, x.T, None if u is None else u.T, "col")
    for mx in (row, col):
        out = torch.empty(mx.rows, mx.k, device="cuda")
        psgd_mx_dequantize(ctx, mx, out)
        # 3.4e38 is 1.998 2^127, off the top of its binade: 4 2^126 = 2^128, in fp32 an infinity
        want = torch.from_numpy(L.mx_values(mx.data.cpu().numpy(), mx.rows, mx.k)).float().double().numpy()
        assert np.array_equal(_np(out), want, equal_nan=True)


@pytest.mark.parametrize("shape", [(1, 1), (65, 129), (200, 300), (3, 4097)], ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_values_come_back(ctx, shape, kind):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_dequantize, psgd_mx_quantize
    m, n = shape
    t, x = _matrix(m, n, "bf16", 3)
    mx = MxTensor(m, n)
    psgd_mx_quantize(ctx, t, mx)
    want, _ = L.mx_quantize(x)
    flat = torch.full((m * (n + 5) + 1,), 9.0, dtype=_dt(kind), device="cuda")
    out = torch.as_strided(flat, (m, n), (n + 5, 1), 1)
    psgd_mx_dequantize(ctx, mx, out)
    assert np.array_equal(_np(out), _np(torch.from_numpy(want).to(_dt(kind))))       # exact in fp32 and bf16, rounded once in fp16
    out.fill_(9.0)
    assert (flat == 9).all()                                                 # nothing between the rows


def _operand(rows, k, seed, spread=4):
    """An MxTensor of random codes and exponents, and its values."""
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor
    rng = np.random.default_rng(seed)
    mx = MxTensor(rows, k)
    p, g = -(-k // 128), -(-rows // 64)
    codes = rng.integers(0, 256, (p, rows, 64), dtype=np.uint8)
    nib = np.arange(128)[None, :] + 128 * np.arange(p)[:, None] < k         # elements that exist
    codes &= (np.where(nib[:, 0::2], 15, 0) | np.where(nib[:, 1::2], 240, 0)).astype(np.uint8)[:, None, :]
    exps = rng.integers(127 - spread, 128 + spread, p * g * 256).astype(np.uint8)
    mx.data.copy_(torch.from_numpy(np.concatenate([codes.reshape(-1), exps])))
    return mx, L.mx_values(mx.data.cpu().numpy(), rows, k)


def _product(ctx, m, n, k, kind="f32", scale=None, accumulate=False, skew=0, ld=None, seed=0):
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_mx_product
    a, av = _operand(m, k, 1 + seed)
    b, bv = _operand(n, k, 2 + seed)
    ld = ld or n
    flat = torch.full((skew + m * ld + 8,), 5.0, dtype=_dt(kind), device="cuda")
    c = torch.as_strided(flat, (m, n), (ld, 1), skew)
    if accumulate:
        c.copy_(torch.from_numpy(np.random.default_rng(9).standard_normal((m, n)) * 10))
    c0 = _np(c)
    s = None if scale is None else torch.tensor([scale], device="cuda")
    psgd_mx_product(ctx, a, b, c, scale=s, accumulate=accumulate)
    f = 1.0 if scale is None else float(np.float32(scale))
    want = f * (av @ bv.T)
    sums = abs(f) * (np.abs(av) @ np.abs(bv).T)
    tol = ((-(-k // 128) + 8) * 2.0 ** -23) * sums + 2.0 ** -24 * np.abs(want)
    if accumulate:
        want = want + c0
        tol = tol + 2.0 ** -24 * np.abs(want)
    if kind != "f32":
        tol = tol + np.maximum({"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind] * (np.abs(want) + tol), 2.0 ** -25)
    got = _np(c)
    if kind == "f16":                                                        # from 65520 on fp16 rounds to infinity
        past = np.abs(want) + tol >= 65520
        assert (np.abs(got[past]) >= 65504 * (1 - 2.0 ** -9)).all() and (np.sign(got[past]) == np.sign(want[past])).all()
        got, want, tol = got[~past], want[~past], tol[~past]
    worst = float((np.abs(got - want) / np.maximum(tol, 1e-300)).max()) if got.size else 0.0
    log(f"  product {m} x {n} x {k} {kind}: {worst:.3f} of what is allowed")
    assert worst <= 1.0, (m, n, k, kind)
    c.fill_(5.0)
    assert (flat == 5).all(), "written outside of C"


FEW = [(1, 1, 1), (1, 16, 128), (1, 4099, 4097), (7, 100, 129), (16, 1000, 3968), (17, 33, 5000), (33, 65, 700), (64, 130, 9000), (50, 17, 256)]
MANY = [(65, 1, 128), (65, 63, 1), (100, 200, 300), (128, 128, 128), (129, 130, 640), (333, 2049, 1001), (257, 255, 513), (1000, 64, 1152)]


@pytest.mark.parametrize("mnk", FEW + MANY, ids=lambda s: "%dx%dx%d" % s)
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_products(ctx, mnk, kind):
    _product(ctx, *mnk, kind=kind)


@pytest.mark.parametrize("mnk", [(1, 70, 300), (40, 70, 300), (333, 250, 700), (130, 1300, 257)], ids=lambda s: "%dx%dx%d" % s)
def test_products_added_scaled_and_off_alignment(ctx, mnk):
    m, n, k = mnk
    _product(ctx, m, n, k, scale=0.3, accumulate=True)
    _product(ctx, m, n, k, scale=-2.5, skew=1, ld=n + 3)
    _product(ctx, m, n, k, accumulate=True, skew=3, ld=n + 1)
    _product(ctx, m, n, k, kind="bf16", scale=0.3, skew=1, ld=n + 1)
    _product(ctx, m, n, k, kind="f16", scale=0.3, skew=3, ld=n + 2)


@pytest.mark.parametrize("mnk", [(2048, 6200, 500), (4100, 4100, 130), (1500, 1500, 1500), (3968, 1488, 2560), (130, 130, 20000), (300, 496, 30000)],
                         ids=lambda s: "%dx%dx%d" % s)
def test_products_of_full_tiles_and_long_sums(ctx, mnk):
    _product(ctx, *mnk)
    _product(ctx, *mnk, scale=0.5, accumulate=True)


@pytest.mark.parametrize("mnk,kind", [((64, 20000, 1001), "bf16"), ((1, 32768, 4096), "f16"), ((4090, 4090, 2050), "bf16"),
                                      ((4090, 4090, 2050), "f32"), ((8192, 8192, 600), "f16"), ((8192, 8192, 600), "f32")],
                         ids=lambda v: v if isinstance(v, str) else "%dx%dx%d" % v)
def test_products_of_few_rows_with_many_and_of_several_tiles_a_workgroup(ctx, mnk, kind):
    _product(ctx, *mnk, kind=kind, accumulate=kind == "f32")


def test_products_of_very_long_sums_in_parts(ctx):
    """Against a product in 64 bits of the values that psgd_mx_dequantize gives."""
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_dequantize, psgd_mx_product, psgd_mx_quantize
    from rank_gradient_compression_powersgd_amd import binding
    m, n, k = 2000, 2040, 131067
    assert binding.psgd_mx_product_workspace(m, n, k) >= 2 * 4 * m * n
    want, sums = (torch.zeros(m, n, dtype=torch.float64, device="cuda") for _ in range(2))
    values = []
    for rows in (m, n):
        x, mx = torch.randn(rows, k, device="cuda"), MxTensor(rows, k)
        psgd_mx_quantize(ctx, x, mx)
        psgd_mx_dequantize(ctx, mx, x)
        values.append((mx, x))
    (a, av), (b, bv) = values
    for i in range(0, k, 16384):
        p, q = av[:, i:i + 16384].double(), bv[:, i:i + 16384].double().t().contiguous()
        want += p @ q
        sums += p.abs() @ q.abs()
    c = torch.full((m, n), 3.0, device="cuda")
    psgd_mx_product(ctx, a, b, c)
    tol = ((-(-k // 128) + 8) * 2.0 ** -23) * sums + 2.0 ** -24 * want.abs()
    assert ((c.double() - want).abs() <= tol).all()


def test_products_of_very_long_sums_in_parts_of_middle_tiles(ctx):
    """Exactly: on values of one magnitude fp32 sums below 2^24 of them round nothing."""
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_product, psgd_mx_quantize
    from rank_gradient_compression_powersgd_amd import binding
    m, n, k = 1000, 1020, 200059
    assert binding.psgd_mx_product_workspace(m, n, k) == 4 * 4 * m * n
    x, w = (torch.randint(-1, 2, (r, k), device="cuda").to(torch.bfloat16) for r in (m, n))
    a, b = MxTensor(m, k), MxTensor(n, k)
    psgd_mx_quantize(ctx, x, a)
    psgd_mx_quantize(ctx, w, b)
    c = torch.full((m, n), 3.0, device="cuda")
    psgd_mx_product(ctx, a, b, c)
    want = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for i in range(0, k, 16384):
        want += x[:, i:i + 16384].double() @ w[:, i:i + 16384].double().t().contiguous()
    assert torch.equal(c.double(), want)


@pytest.mark.parametrize("m", [5, 200])
def test_empty_products(ctx, m):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_dequantize, psgd_mx_product, psgd_mx_quantize
    c = torch.ones(m, 9, device="cuda")
    psgd_mx_product(ctx, MxTensor(m, 0), MxTensor(9, 0), c, accumulate=True)
    assert (c == 1).all()
    psgd_mx_product(ctx, MxTensor(m, 0), MxTensor(9, 0), c)
    assert (c == 0).all()
    b, _ = _operand(9, 100, 1)
    psgd_mx_product(ctx, MxTensor(0, 100), b, torch.ones(0, 9, device="cuda"))
    psgd_mx_product(ctx, b, MxTensor(0, 100), torch.ones(9, 0, device="cuda"))
    psgd_mx_quantize(ctx, torch.ones(0, m, device="cuda"), MxTensor(0, m), MxTensor(m, 0))
    psgd_mx_dequantize(ctx, MxTensor(m, 0), torch.ones(m, 0, device="cuda"))


@pytest.mark.parametrize("m,n", [(20, 40), (200, 300), (300, 30)])
def test_a_bad_block_reaches_its_own_row_only(ctx, m, n):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_product, psgd_mx_quantize
    x, w = torch.randn(m, 260, device="cuda"), torch.randn(n, 260, device="cuda")
    x[3, 200], w[7, 0], w[9, 259] = float("nan"), float("inf"), float("-inf")
    a, b = MxTensor(m, 260), MxTensor(n, 260)
    psgd_mx_quantize(ctx, x, a)
    psgd_mx_quantize(ctx, w, b)
    c = torch.empty(m, n, device="cuda")
    psgd_mx_product(ctx, a, b, c)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[3], bad[:, 7], bad[:, 9] = True, True, True
    assert torch.equal(torch.isnan(c), bad) and torch.isfinite(c[~bad]).all()


def test_results_do_not_depend_on_what_memory_held(ctx):
    """The exponents' padding rows and the workspace are never part of a result."""
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_product, psgd_mx_product_workspace, psgd_mx_quantize
    for m, n, k in ((5, 70, 300), (130, 130, 20000), (333, 65, 200)):
        x, w = torch.randn(m, k, device="cuda"), torch.randn(n, k, device="cuda")
        got = []
        for fill in (0x00, 0xFF):
            a, b = MxTensor(m, k), MxTensor(n, k)
            a.data.fill_(fill)
            b.data.fill_(fill)
            psgd_mx_quantize(ctx, x, a)
            psgd_mx_quantize(ctx, w, b)
            ws = torch.full((psgd_mx_product_workspace(m, n, k) + 16,), fill, dtype=torch.uint8, device="cuda")
            c = torch.empty(m, n, device="cuda")
            psgd_mx_product(ctx, a, b, c, workspace=ws)
            assert (ws[-16:] == fill).all()
            got.append(c)
        assert torch.equal(*got) and torch.isfinite(got[0]).all()


def test_products_past_32_bit_offsets(ctx):
    """Codes of 4 GiB and more on one side, and a C of more than 2^31 elements: the last rows against a product of
    their own."""
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_product, psgd_mx_quantize
    m, k, n = 2 ** 21 + 70, 4096, 1032
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[-100:] = torch.randn(100, k, device="cuda")
    w = torch.randn(n, k, device="cuda")
    a, tail, b = MxTensor(m, k), MxTensor(100, k), MxTensor(n, k)
    assert a.data.numel() > 2 ** 32
    psgd_mx_quantize(ctx, x, a)
    psgd_mx_quantize(ctx, x[-100:], tail)
    psgd_mx_quantize(ctx, w, b)
    c = torch.full((m, n), 3.0, dtype=torch.bfloat16, device="cuda")
    psgd_mx_product(ctx, a, b, c)
    want = torch.empty(100, n, device="cuda")
    psgd_mx_product(ctx, tail, b, want)
    assert not c[:-100].any()
    # the two sizes may take their panels in parts or not: both are fp32 sums of the same products
    assert ((c[-100:].float() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-3).all()
    back = MxTensor(k, m)
    psgd_mx_quantize(ctx, x, None, back)
    assert not back.data[:k * 64].any()                                       # the first panel's codes
    last = (m - 1) // 128
    t2 = MxTensor(k, m - 128 * last)
    psgd_mx_quantize(ctx, x[128 * last:], None, t2)
    assert torch.equal(back.data[last * k * 64:(last + 1) * k * 64], t2.data[:k * 64])


def test_graph_replays_match_eager(ctx):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_product, psgd_mx_product_workspace, psgd_mx_quantize
    m, n, k = 130, 130, 20000                                                # panels in parts
    x = [torch.randn(m, k, device="cuda") for _ in range(4)]
    w = torch.randn(n, k, device="cuda")
    live = x[0].clone()
    step = torch.zeros(1, dtype=torch.int32, device="cuda")

    def bufs():
        return MxTensor(m, k), MxTensor(n, k), torch.zeros(m, n, device="cuda"), \
            torch.empty(psgd_mx_product_workspace(m, n, k) + 16, dtype=torch.uint8, device="cuda")

    def go(a, b, c, ws):
        psgd_mx_quantize(ctx, live, a, stochastic=True, seed=1, step=step)
        psgd_mx_quantize(ctx, w, b)
        psgd_mx_product(ctx, a, b, c, accumulate=True, workspace=ws)

    eager, cap = bufs(), bufs()
    go(*bufs())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go(*cap)
    torch.cuda.synchronize()
    for t in range(4):
        live.copy_(x[t])
        step.fill_(t)
        go(*eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager[2], cap[2]), t


def test_two_streams_at_once(ctx):
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_mx_product
    a, _ = _operand(130, 20000, 1)
    b, _ = _operand(140, 20000, 2)
    want = torch.empty(130, 140, device="cuda")
    psgd_mx_product(ctx, a, b, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros(130, 140, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    for i, c in enumerate(outs):
        psgd_mx_product(ctx, a, b, c, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for c in outs)


# ---- a layer, and a whole step ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t,n_in,n_out", [(1, 40, 24), (77, 200, 130), (300, 333, 65)])
def test_linear_forward_and_backward(kind, t, n_in, n_out):
    import torch
    from rank_gradient_compression_powersgd_amd import MxLinear
    rng = np.random.default_rng(t)
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s)).to("cuda", _dt(kind))  # noqa: E731
    w, x, dy = mk(n_in, n_out), mk(t, n_in), mk(t, n_out)
    layer = MxLinear(w, seed=17)
    err = torch.from_numpy(rng.standard_normal((n_in, n_out)).astype(np.float32)).cuda()
    e0, s = _np(err), torch.tensor([0.25], device="cuda")
    step = torch.tensor([6], dtype=torch.int32, device="cuda")
    y = layer.forward(x)
    dx = layer.backward(dy, err, s, step=step)
    u = _bits(t, n_out, 17, 6)
    q = lambda v, r=None: L.mx_quantize(v, r)[0]  # noqa: E731
    xv, wv, dv = _np(x), _np(w), _np(dy)
    for got, a, b, base, f in ((y, q(xv), q(wv.T), 0.0, 1.0), (dx, q(dv, u), q(wv), 0.0, 1.0), (err, q(xv.T), q(dv.T, u.T), e0, 0.25)):
        want = base + f * (a @ b.T)
        k = a.shape[1]
        tol = (-(-k // 128) + 8) * 2.0 ** -23 * f * (np.abs(a) @ np.abs(b).T) + 2.0 ** -23 * np.abs(want)
        if got.dtype != torch.float32:
            tol = tol + np.maximum({"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind] * (np.abs(want) + tol), 2.0 ** -25)
        assert (np.abs(_np(got) - want) <= tol).all()


def test_gradients_are_the_differences_of_the_forward_pass():
    """On values that 4 bits hold exactly (every block's largest is 6) forward and backward are exact: the
    gradient of sum(dy * y) is its difference over one step of the grid either way."""
    import torch
    from rank_gradient_compression_powersgd_amd import MxLinear
    rng = np.random.default_rng(5)
    t, n_in, n_out = 64, 96, 64
    draw = lambda m, n: rng.choice([-3.0, -1.5, -1.0, 0.0, 0.5, 1.0, 2.0], (m, n))  # noqa: E731
    x, w, dy = draw(t, n_in), draw(n_in, n_out), draw(t, n_out)
    for v in (x, w, dy):                                                     # a 6 in every block of 32 of rows and of columns
        for i in range(v.shape[0]):
            v[i, i % 32::32] = 6.0
    dev = lambda v: torch.from_numpy(v).float().cuda()  # noqa: E731
    layer = MxLinear(dev(w))
    layer.forward(dev(x))
    err = torch.zeros(n_in, n_out, device="cuda")
    dx = layer.backward(dev(dy), err)

    def loss(xv, wv):
        return float((_np(MxLinear(dev(wv)).forward(dev(xv))) * dy).sum())

    for i, j in ((0, 3), (17, 90), (63, 2), (40, 41)):
        for base, grad, first in ((x, dx, True), (w, err, False)):
            if j >= base.shape[1] or base[i, j] == 6.0:
                continue
            hi, lo = base.copy(), base.copy()
            hi[i, j], lo[i, j] = 4.0, -4.0
            d = (loss(hi, w) - loss(lo, w)) if first else (loss(x, hi) - loss(x, lo))
            assert d / 8.0 == float(grad[i, j]), (i, j, first)


def test_a_layer_takes_leading_dimensions_and_single_tokens():
    import torch
    from rank_gradient_compression_powersgd_amd import MxLinear, binding as B
    layer = MxLinear(torch.randn(40, 24, device="cuda").bfloat16())
    x = torch.randn(3, 5, 40, device="cuda").bfloat16()
    y = layer.forward(x)
    assert y.shape == (3, 5, 24) and torch.equal(y.reshape(15, 24), layer.forward(x.reshape(15, 40)))
    one = layer.forward(x[1, 2:3], train=False)
    assert torch.equal(one[0], y[1, 2])
    assert layer.forward(x[:0], train=False).shape == (0, 5, 24)
    dx = layer.backward(torch.randn(3, 5, 24, device="cuda").bfloat16(), torch.zeros(40, 24, device="cuda"))
    assert dx.shape == (3, 5, 40)
    with pytest.raises(B.PsgdError):
        layer.backward(torch.randn(4, 24, device="cuda"), torch.zeros(40, 24, device="cuda"))       # of other tokens
    with pytest.raises(B.PsgdError):
        layer.forward(torch.randn(4, 24, device="cuda"))


@pytest.mark.parametrize("bits", [8, 32])
def test_a_whole_training_step(bits):
    """Two layers: forward, backward into the error buffers of an in-place group, compression, decompression, AdamW
    on the decompressed gradients, new 4-bit weights. Against the oracle's step on the same error buffers."""
    import torch
    import oracle
    from rank_gradient_compression_powersgd_amd import AdamWGroup, MxLinear, PowerSGDGroup, psgd_adam_hparams
    rng = np.random.default_rng(31)
    dims, t, rank = [(264, 136), (136, 200)], 96, 24
    ws = [torch.from_numpy(rng.standard_normal(d) * 0.1).to("cuda", torch.bfloat16) for d in dims]
    layers = [MxLinear(w, seed=50 + i) for i, w in enumerate(ws)]
    scale = torch.tensor([0.5, 2.0], device="cuda")
    q0 = [rng.standard_normal((d[1], rank)).astype(np.float32) for d in dims]
    errs = [torch.zeros(d, device="cuda") for d in dims]
    group = PowerSGDGroup([None, None], [0, 1], scale, rank, [torch.from_numpy(q) for q in q0], err=errs)
    opt = AdamWGroup(ws, group.out, bits=bits, seed=3)
    x = torch.from_numpy(rng.standard_normal((t, 264))).to("cuda", torch.bfloat16)
    hp = psgd_adam_hparams(1e-3, 0.9, 0.999, 1e-8, 0.01)

    def half(step_no, poison=False):
        y1 = layers[0].forward(x)
        y2 = layers[1].forward(y1)
        dy = torch.from_numpy(np.random.default_rng(step_no).standard_normal((t, 200))).to("cuda", torch.bfloat16)
        if poison:
            dy[5, 7] = float("inf")
        d1 = layers[1].backward(dy, group.err[1], scale[1:2], step=opt.step_count)
        layers[0].backward(d1, group.err[0], scale[0:1], step=opt.step_count)

    half(0)
    m = [_np(e).astype(np.float32) for e in errs]
    before = [w.clone() for w in ws]
    st = oracle.step_group([np.zeros(d, np.float32) for d in dims], [a.astype(np.float64) for a in m], q0, [0, 1],
                           np.ones(2, np.float32), [])
    group.step()
    opt.step(hp, max_norm=1.0, skip=group.skip)
    assert group.skip.item() == 0 and opt.skip.item() == 0 and opt.step_count.item() == 1
    for i in range(2):
        assert np.linalg.norm(_np(group.out[i]) - st.D[i]) <= 2e-3 * np.linalg.norm(st.D[i])
    norm = np.sqrt(sum(np.square(_np(o)).sum() for o in group.out))
    assert abs(opt.norm[0].item() - norm) <= 2.0 ** -22 * norm
    # first step: the update is lr sign(g) where the gradient is not tiny, to what bf16 holds of a weight
    for w, b, o in zip(ws, before, group.out):
        big = o.abs() * opt.norm[1] > 1e-5
        d = (w.float() - b.float() + 1e-3 * (torch.sign(o) + 0.01 * b.float()))[big]
        assert (d.abs() <= 2.0 ** -7 * b.float().abs()[big] + 2e-5).all()
    for layer in layers:
        layer.refresh()
    assert not any(torch.equal(a, b) for a, b in zip(before, ws))
    # a poisoned step is skipped as a whole: error buffers cleared, weights and moments kept
    keep = [w.clone() for w in ws] + [s.clone() for s in opt.state()]
    half(1, poison=True)
    group.step()
    opt.step(hp, max_norm=1.0, skip=group.skip)
    assert group.skip.item() == 1 and opt.skip.item() == 1 and opt.step_count.item() == 1
    assert all(torch.equal(a, b) for a, b in zip(keep, [*ws, *opt.state()])) and not any(e.any() for e in errs)
    half(2)
    group.step()
    opt.step(hp, max_norm=1.0, skip=group.skip)
    assert opt.step_count.item() == 2 and all(torch.isfinite(w).all() for w in ws)


def test_refusals(ctx):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, binding as B

    def refused(status, fn):
        with pytest.raises(B.PsgdError) as ei:
            fn()
        assert ei.value.status == status, str(ei.value)

    x = torch.zeros(10, 20, device="cuda")
    row = MxTensor(10, 20)
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_quantize(ctx, x))
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_quantize(ctx, x, MxTensor(20, 10)))
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_quantize(ctx, x, None, row))
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_quantize(ctx, x.t(), MxTensor(20, 10)))
    refused(B.PSGD_EDTYPE, lambda: B.psgd_mx_quantize(ctx, x.double(), row))
    refused(B.PSGD_EDTYPE, lambda: B.psgd_mx_quantize(ctx, x, row, step=torch.zeros(1, device="cuda")))
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_quantize(ctx, x, MxTensor(10, 20, data=torch.empty(9999, dtype=torch.uint8, device="cuda")[1:])))
    refused(B.PSGD_EINVAL, lambda: MxTensor(10, 20, data=torch.empty(100, dtype=torch.uint8, device="cuda")))
    refused(B.PSGD_EINVAL, lambda: MxTensor(-1, 20))
    refused(B.PSGD_EINVAL, lambda: MxTensor(2 ** 25 + 1, 1))
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_dequantize(ctx, row, torch.zeros(10, 21, device="cuda")))
    refused(B.PSGD_EDTYPE, lambda: B.psgd_mx_dequantize(ctx, row, torch.zeros(10, 20, dtype=torch.int32, device="cuda")))
    b = MxTensor(30, 20)
    c = torch.zeros(10, 30, device="cuda")
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_product(ctx, row, MxTensor(30, 21), c))
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_product(ctx, row, b, c.t()))
    refused(B.PSGD_EDTYPE, lambda: B.psgd_mx_product(ctx, row, b, c.half(), accumulate=True))
    refused(B.PSGD_EDTYPE, lambda: B.psgd_mx_product(ctx, row, b, c, scale=torch.ones(1, device="cuda").half()))
    big = [MxTensor(130, 20000) for _ in range(2)]
    need = B.psgd_mx_product_workspace(130, 130, 20000)
    assert need > 0
    c = torch.zeros(130, 130, device="cuda")
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_product(ctx, *big, c, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda")))
    refused(B.PSGD_EINVAL, lambda: B.psgd_mx_product(ctx, *big, c, workspace=torch.empty(need + 16, dtype=torch.uint8, device="cuda")[4:]))
    lib = B.load_library()
    assert lib.psgd_mx_quantize(ctx, x.data_ptr(), 19, 10, 20, 3, B._mx(row), None, 0, 0, None, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_quantize(ctx, x.data_ptr(), 20, 10, 20, 3, B._mx(row), None, 2, 0, None, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_quantize(ctx, x.data_ptr() + 2, 20, 10, 20, 3, B._mx(row), None, 0, 0, None, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_quantize(ctx, x.data_ptr(), 20, 10, 20, 9, B._mx(row), None, 0, 0, None, None) == B.PSGD_EDTYPE
    assert lib.psgd_mx_product(ctx, B._mx(row), B._mx(b), None, c.data_ptr(), 29, 3, 0, None, 0, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_product(ctx, B._mx(row), None, None, c.data_ptr(), 30, 3, 0, None, 0, None) == B.PSGD_EINVAL


def test_overlapping_buffers_are_refused(ctx):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, binding as B
    flat = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")

    def at(rows, k, offset):
        return MxTensor(rows, k, data=flat[offset:offset + B.psgd_mx_bytes(rows, k)])

    def refused(fn):
        with pytest.raises(B.PsgdError) as ei:
            fn()
        assert ei.value.status == B.PSGD_EINVAL and "overlap" in str(ei.value)

    m, n, k = 100, 200, 300
    size = B.psgd_mx_bytes(m, k)
    x = flat[4096:4096 + 4 * m * k].view(torch.float32).view(m, k)
    end = 4096 + 4 * m * k
    refused(lambda: B.psgd_mx_quantize(ctx, x, at(m, k, 4080)))
    refused(lambda: B.psgd_mx_quantize(ctx, x, None, at(k, m, end - 16)))
    refused(lambda: B.psgd_mx_quantize(ctx, x, at(m, k, end), at(k, m, end + size - 16)))
    refused(lambda: B.psgd_mx_dequantize(ctx, at(m, k, 4080), x))
    B.psgd_mx_quantize(ctx, x, at(m, k, end), at(k, m, end + (size + 15) // 16 * 16))      # neighbours
    B.psgd_mx_dequantize(ctx, at(m, k, end), x)
    a, b = at(m, k, 0), at(n, k, 1 << 19)
    c = flat[(1 << 19) - 4 * m * n:1 << 19].view(torch.float32).view(m, n)
    B.psgd_mx_product(ctx, a, b, c)
    refused(lambda: B.psgd_mx_product(ctx, a, b, flat[(1 << 19) - 4 * m * n + 4:(1 << 19) + 4].view(torch.float32).view(m, n)))
    refused(lambda: B.psgd_mx_product(ctx, a, b, flat[size - 16:size - 16 + 4 * m * n].view(torch.float32).view(m, n)))
    refused(lambda: B.psgd_mx_product(ctx, a, b, c, scale=c[5, 7:8]))
    B.psgd_mx_product(ctx, a, a, torch.empty(m, m, device="cuda"))                         # an operand may be both
    p, q = MxTensor(130, 20000), MxTensor(130, 20000)
    need = B.psgd_mx_product_workspace(130, 130, 20000)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    refused(lambda: B.psgd_mx_product(ctx, p, q, ws[:4 * 130 * 130].view(torch.float32).view(130, 130), workspace=ws))
    refused(lambda: B.psgd_mx_product(ctx, p, q, torch.empty(130, 130, device="cuda"), workspace=p.data))


def test_no_columns_to_sum_over_and_more_rows_than_a_launch_has_workgroups(ctx):
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_product
    m = 2 ** 24 + 70
    c = torch.full((m, 3), 7.0, device="cuda", dtype=torch.float16)
    psgd_mx_product(ctx, MxTensor(m, 0), MxTensor(3, 0), c)
    assert not c.any()


def test_backward_uses_up_its_forward_and_may_run_on_another_stream():
    import torch
    from rank_gradient_compression_powersgd_amd import MxLinear, binding as B
    layer = MxLinear(torch.randn(264, 130, device="cuda").bfloat16())
    x, dy = torch.randn(200, 264, device="cuda").bfloat16(), torch.randn(200, 130, device="cuda").bfloat16()
    want, err = torch.zeros(264, 130, device="cuda"), torch.zeros(264, 130, device="cuda")
    layer.forward(x)
    layer.backward(dy)                                       # the gradient of x alone leaves it
    layer.backward(dy, want)
    with pytest.raises(B.PsgdError):
        layer.backward(dy, err)
    other = torch.cuda.Stream()
    layer.forward(x)
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        layer.backward(dy, err)
    torch.cuda.synchronize()
    assert torch.equal(err, want)


def test_refusals_of_a_layer():
    import torch
    from rank_gradient_compression_powersgd_amd import MxLinear, binding as B

    def refused(status, fn):
        with pytest.raises(B.PsgdError) as ei:
            fn()
        assert ei.value.status == status, str(ei.value)

    layer = MxLinear(torch.randn(40, 24, device="cuda"))
    x, dy, err = torch.randn(5, 40, device="cuda"), torch.randn(5, 24, device="cuda"), torch.zeros(40, 24, device="cuda")
    refused(B.PSGD_EINVAL, lambda: layer.forward(x.cpu()))
    refused(B.PSGD_EDTYPE, lambda: layer.forward(x.double()))
    refused(B.PSGD_EINVAL, lambda: layer.forward(torch.randn(40, 5, device="cuda").t()))
    refused(B.PSGD_EINVAL, lambda: layer.forward(x[0]))
    layer.forward(x)
    refused(B.PSGD_EINVAL, lambda: layer.backward(dy.cpu(), err))
    refused(B.PSGD_EINVAL, lambda: layer.backward(dy, err.cpu()))
    refused(B.PSGD_EINVAL, lambda: layer.backward(dy, err.t()))
    refused(B.PSGD_EDTYPE, lambda: layer.backward(dy, err.half()))
    refused(B.PSGD_EDTYPE, lambda: layer.backward(dy, err, torch.ones(1, device="cuda", dtype=torch.float64)))
    refused(B.PSGD_EDTYPE, lambda: layer.backward(dy, err, step=torch.ones(1, device="cuda", dtype=torch.int64)))
    refused(B.PSGD_EDTYPE, lambda: layer.backward(dy.double(), err))
    assert not err.any()
    layer.backward(dy, err)                                  # no refusal used up the forward
    assert err.any()


def test_a_captured_layer_replays_as_the_eager_one():
    import torch
    from rank_gradient_compression_powersgd_amd import MxLinear
    w = torch.randn(333, 200, device="cuda").bfloat16()
    x, dy = torch.zeros(150, 333, device="cuda").bfloat16(), torch.zeros(150, 200, device="cuda").bfloat16()
    step, scale = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0.5], device="cuda")
    err, want = torch.zeros(333, 200, device="cuda"), torch.zeros(333, 200, device="cuda")
    captured, eager = MxLinear(w, seed=9), MxLinear(w, seed=9)

    def both(layer, e):
        layer.refresh()
        return layer.forward(x), layer.backward(dy, e, scale, step=step)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(captured, err)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = both(captured, err)
    err.zero_()
    for t in range(1, 5):
        x.copy_(torch.randn(150, 333, device="cuda"))
        dy.copy_(torch.randn(150, 200, device="cuda"))
        w.copy_(torch.randn(333, 200, device="cuda"))
        step.fill_(t)
        y2, dx2 = both(eager, want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(err, want) and want.any(), t


@pytest.mark.parametrize("m,n,k", [(64, 64, 131067), (1, 70, 400001), (40, 513, 70000), (16, 33, 262144)])
def test_products_of_few_rows_and_columns_and_very_long_sums(ctx, m, n, k):
    """Exactly: sums of -1, 0 and 1 below 2^24 round nothing in fp32."""
    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_product, psgd_mx_quantize
    from rank_gradient_compression_powersgd_amd import binding
    assert binding.psgd_mx_product_workspace(m, n, k) >= 2 * 4 * m * n
    x, w = (torch.randint(-1, 2, (r, k), device="cuda").to(torch.bfloat16) for r in (m, n))
    a, b = MxTensor(m, k), MxTensor(n, k)
    psgd_mx_quantize(ctx, x, a)
    psgd_mx_quantize(ctx, w, b)
    c = torch.full((m, n), 3.0, device="cuda")
    psgd_mx_product(ctx, a, b, c, accumulate=True)
    want = 3.0 + x.double() @ w.double().t().contiguous()
    assert torch.equal(c.double(), want)


def test_random_bits_of_pairs_past_32_bits(ctx):
    """The last rows of a matrix whose pairs of neighbours pass 2^32, in the middle of a lane's four pairs of a row (rows
    alone) and of its 32 rows (columns, and rows with them), bit by bit."""
    import types

    import torch
    from rank_gradient_compression_powersgd_amd import MxTensor, psgd_mx_quantize
    n, half, first = 4100, 2050, 2095104 - 128                              # first: a whole panel's and group's
    cross = 2 ** 32 // half                                                  # the row whose pairs pass it
    m, at = cross + 200, 2 ** 32 - cross * half
    assert cross % 32 != 0 and at % 4 == 2 and first % 128 == 0 and first < cross // 32 * 32
    x = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    tail, _ = _matrix(m - first, n, "bf16", 5)
    x[first:] = tail
    xv = _np(x[first:])
    h = L.hash_bits(L.hash_key(13, 0, 0), np.arange(first * half, m * half, dtype=np.uint64)).reshape(m - first, half)
    u = (np.stack([h, (h << np.uint32(16)) | (h >> np.uint32(16))], 2).reshape(m - first, n) >> np.uint32(10)) * 2.0 ** -22

    def rows_of(mx):
        p, g = -(-n // 128), -(-m // 64)
        codes, exps = mx.data[:p * m * 64].view(p, m, 64)[:, first:], mx.data[p * m * 64:p * (m * 64 + g * 256)].view(p, g, 256)[:, first // 64:]
        return types.SimpleNamespace(data=torch.cat([codes.reshape(-1), exps.reshape(-1)]))

    def columns_of(mx):
        p, g = -(-m // 128), -(-n // 64)
        codes, exps = mx.data[:p * n * 64].view(p, n * 64)[first // 128:], mx.data[p * n * 64:p * (n * 64 + g * 256)].view(p, g * 256)[first // 128:]
        return types.SimpleNamespace(data=torch.cat([codes.reshape(-1), exps.reshape(-1)]))

    row, col = MxTensor(m, n), MxTensor(n, m)
    psgd_mx_quantize(ctx, x, row, stochastic=True, seed=13)
    _check(rows_of(row), xv, u, "rows alone")
    row.data.zero_()
    psgd_mx_quantize(ctx, x, row, col, stochastic=True, seed=13)
    _check(rows_of(row), xv, u, "rows with columns")
    _check(columns_of(col), xv.T, u.T, "columns with rows")
    col.data.zero_()
    psgd_mx_quantize(ctx, x, None, col, stochastic=True, seed=13)
    _check(columns_of(col), xv.T, u.T, "columns alone")
