"""The scaled embedding lookup and its gradient by sorted tokens against the float64 oracle.

The lookup rounds scale * W once in fp32 and once to the output: 2^-24 and eps/2 of each element.
The gradient of a token seen k times is a sum of k fp32 terms in any grouping, then one product
and, when accumulating, one more sum: at most (k + 2) 2^-24 of scale * sum |dx| (+ |dtable|)."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu

EPS2 = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _dt(code):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}[code]


def _np(t):
    return t.detach().cpu().double().numpy()


@pytest.fixture()
def ctx():
    import rank_gradient_compression_powersgd_amd as psgd
    c = psgd.psgd_create(0, 1)
    yield c
    psgd.psgd_destroy(c)


@pytest.mark.parametrize("tt,ot,it", [("f32", "f32", "i64"), ("f32", "f16", "i32"), ("f32", "bf16", "i64"), ("f16", "f16", "i64"),
                                      ("bf16", "f32", "i32"), ("f16", "bf16", "i32")])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (5, 3, 7), (16, 1000, 3968), (333, 77, 1000), (4, 9, 2056)])
def test_lookup(ctx, tt, ot, it, n, vocab, dim):
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_lookup
    rng = np.random.default_rng(n * 31 + dim)
    table = torch.from_numpy(rng.standard_normal((vocab, dim))).to(_dt(tt)).cuda()
    ids = torch.from_numpy(rng.integers(-2, vocab + 2, n)).to(_dt(it)).cuda()
    ids[0] = vocab - 1
    out = torch.full((n, dim), 7.0, dtype=_dt(ot), device="cuda")
    for scale in (1.0, -0.37, 63.0):
        log(f"lookup {tt}->{ot} {it} n={n} vocab={vocab} dim={dim} scale={scale}")
        psgd_embed_lookup(ctx, table, ids, out, scale)
        torch.cuda.synchronize()
        want = oracle.embed_lookup(_np(table), ids.cpu().numpy(), float(np.float32(scale)))
        # half a step of fp16's smallest (2^-25) where a product is subnormal there
        bound = (EPS2[ot] + 2.0 ** -24) * np.abs(want) * 1.001 + (2.0 ** -25 if ot == "f16" else 0.0)
        assert np.all(np.abs(_np(out) - want) <= bound)
        gone = (ids < 0) | (ids >= vocab)
        assert not bool(torch.signbit(out[gone]).any()) and bool((out[gone] == 0).all())


def test_lookup_strides_shapes_and_untouched_memory(ctx):
    """A table and an output that are slices of wider buffers (rows not 16-byte aligned), ids of two
    dimensions, NaN rows that no token names, and no token at all."""
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_lookup
    rng = np.random.default_rng(4)
    wide = torch.full((10, 45), float("nan"), device="cuda")
    table = wide[:, 3:43]
    table[:9].copy_(torch.from_numpy(rng.standard_normal((9, 40))))
    ids = torch.from_numpy(rng.integers(0, 9, (3, 4))).cuda()
    buf = torch.full((14, 50), 5.0, device="cuda")
    out = buf[1:13, 5:45]
    psgd_embed_lookup(ctx, table, ids, out, 2.0)
    torch.cuda.synchronize()
    assert torch.equal(out, 2.0 * table[ids.flatten()])
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:13, 5:45] = False
    assert bool((buf[keep] == 5.0).all())
    full = torch.empty(3, 4, 40, device="cuda")
    psgd_embed_lookup(ctx, table, ids, full, 2.0)
    assert torch.equal(full, 2.0 * table[ids])
    psgd_embed_lookup(ctx, table, ids[:0], buf[:0, :40])
    torch.cuda.synchronize()


def _grad_case(ctx, n, vocab, dim, dt, it, scale, accumulate, ids_np, ld_pad=0, seed=0):
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_grad
    rng = np.random.default_rng(seed + n + dim)
    dxb = torch.from_numpy(rng.standard_normal((n, dim + ld_pad))).to(_dt(dt)).cuda()
    dx = dxb[:, :dim]
    ids = torch.from_numpy(ids_np).to(_dt(it)).cuda()
    wide = torch.full((vocab, dim + ld_pad), 3.0, device="cuda")
    dtable = wide[:, :dim]
    dtable.copy_(torch.from_numpy(rng.standard_normal((vocab, dim))))
    base = _np(dtable) if accumulate else None
    start = dtable.clone()
    log(f"grad {dt} {it} n={n} vocab={vocab} dim={dim} accumulate={accumulate} pad={ld_pad}")
    psgd_embed_grad(ctx, dx, ids, dtable, scale, accumulate)
    torch.cuda.synchronize()
    s = float(np.float32(scale))
    want = oracle.embed_grad(_np(dx), ids_np, vocab, s, base)
    mag = oracle.embed_grad(np.abs(_np(dx)), ids_np, vocab, abs(s), None if base is None else np.abs(base))
    k = np.bincount(ids_np[(ids_np >= 0) & (ids_np < vocab)], minlength=vocab)[:, None]
    got = _np(dtable)
    assert np.all(np.abs(got - want) <= (k + 2) * 2.0 ** -24 * mag)
    if not accumulate:
        assert np.all(got[k[:, 0] == 0] == 0)
    if ld_pad:
        assert bool((wide[:, dim:] == 3.0).all())
    first = dtable.clone()
    dtable.copy_(start)
    psgd_embed_grad(ctx, dx, ids, dtable, scale, accumulate)
    torch.cuda.synchronize()
    assert torch.equal(first, dtable)                # the same bits again


@pytest.mark.parametrize("dt,it", [("f32", "i64"), ("bf16", "i32"), ("f16", "i64")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (31, 5, 33), (333, 1031, 100), (2000, 17, 64), (4097, 900, 28), (65, 40000, 12)])
def test_grad(ctx, dt, it, accumulate, n, vocab, dim):
    rng = np.random.default_rng(n)
    _grad_case(ctx, n, vocab, dim, dt, it, 0.37, accumulate, rng.integers(-1, vocab + 1, n))


@pytest.mark.parametrize("n", [700, 30000])
def test_grad_largest_vocabulary(ctx, n):
    rng = np.random.default_rng(n)
    vocab = 2 ** 20
    ids = np.where(np.arange(n) % 3 == 0, rng.integers(0, 40, n), rng.integers(0, vocab, n))
    ids[0], ids[1] = vocab - 1, vocab
    _grad_case(ctx, n, vocab, 4, "f32", "i64", -1.5, False, ids)
    _grad_case(ctx, n, vocab, 3, "bf16", "i32", 1.0, True, ids)


def test_lookup_most_tokens(ctx):
    """2^25 tokens, the most a call takes, and a table past 2^31 elements."""
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_lookup
    n, vocab, dim = 2 ** 25, 2 ** 22 + 3, 520
    table = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda")
    table.copy_((torch.arange(vocab, device="cuda") % 251).to(torch.bfloat16)[:, None])       # whole numbers below 256: exact
    ids = torch.arange(n, device="cuda") * 7919 % vocab
    out = torch.empty(n, 1, dtype=torch.float32, device="cuda")
    psgd_embed_lookup(ctx, table[:, :1], ids, out)
    assert torch.equal(out[:, 0], (ids % 251).float())
    few = ids[:1000].clone()
    few[5] = vocab - 1
    rows = torch.empty(1000, dim, dtype=torch.float32, device="cuda")
    psgd_embed_lookup(ctx, table, few, rows)
    assert torch.equal(rows, (few % 251).float()[:, None].expand(1000, dim))


@pytest.mark.parametrize("kind", ["one token", "two tokens in turn", "descending", "skewed", "all outside", "last id"])
def test_grad_token_orders(ctx, kind):
    """Every token the same, alternating, reversed, heavily skewed (runs over many chunks of the
    sorted order and runs ending at their borders), none valid."""
    n, vocab, dim = 3000, 700, 36
    rng = np.random.default_rng(8)
    ids = {"one token": np.full(n, 5), "two tokens in turn": np.arange(n) % 2, "descending": (n - 1 - np.arange(n)) // 5,
           "skewed": np.minimum(rng.geometric(0.02, n) - 1, vocab - 1), "all outside": np.full(n, vocab),
           "last id": np.full(n, vocab - 1)}[kind]
    _grad_case(ctx, n, vocab, dim, "f32", "i64", 1.0, False, ids)
    _grad_case(ctx, n, vocab, dim, "f32", "i32", 1.0, True, ids)


@pytest.mark.parametrize("count", [31, 32, 33, 64, 65, 1024, 1025])
def test_grad_runs_at_chunk_borders(ctx, count):
    """Token runs that begin and end at, before and behind the borders of the sorted chunks."""
    ids = np.concatenate([np.full(count, 1), np.full(32, 3), np.full(7, 4), np.full(count, 6), [9]])
    _grad_case(ctx, len(ids), 10, 20, "f32", "i64", 2.0, False, np.random.default_rng(count).permutation(ids))


def test_grad_unaligned_rows(ctx):
    rng = np.random.default_rng(3)
    _grad_case(ctx, 500, 50, 40, "bf16", "i64", 1.0, True, rng.integers(0, 50, 500), ld_pad=3)
    _grad_case(ctx, 500, 50, 37, "f32", "i64", 1.0, False, rng.integers(0, 50, 500), ld_pad=1)


def test_grad_is_the_lookups_gradient(ctx):
    """<lookup(W), dx> has the gradient <dW, .>: central differences along a direction, both sides
    linear in W, so only rounding separates them."""
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_grad, psgd_embed_lookup
    rng = np.random.default_rng(12)
    vocab, dim, n = 30, 48, 200
    w, h = (torch.from_numpy(rng.standard_normal((vocab, dim))).float().cuda() for _ in range(2))
    ids = torch.from_numpy(rng.integers(-1, vocab, n)).cuda()
    dx = torch.from_numpy(rng.standard_normal((n, dim))).float().cuda()
    dw, xp, xm = torch.empty_like(w), torch.empty_like(dx), torch.empty_like(dx)
    psgd_embed_grad(ctx, dx, ids, dw, 1.5)
    psgd_embed_lookup(ctx, w + h, ids, xp, 1.5)
    psgd_embed_lookup(ctx, w - h, ids, xm, 1.5)
    torch.cuda.synchronize()
    diff = float((((xp.double() - xm.double()) / 2) * dx.double()).sum())
    lin = float((dw.double() * h.double()).sum())
    size = float((dw.double().abs() * h.double().abs()).sum())
    # the rows w +- h and the lookups round by 2^-24 of |w| + |h|, the sums by 20 of them
    assert abs(diff - lin) <= 64 * 2.0 ** -24 * size * 4, (diff, lin)


def test_grad_non_finite_and_nothing(ctx):
    """A NaN row reaches its token only; no token clears the table, or leaves it when accumulating."""
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_grad
    dx = torch.ones(100, 16, device="cuda")
    ids = (torch.arange(100, device="cuda") % 10).to(torch.int64)
    dx[13, 2] = float("nan")
    dx[24, 3] = float("inf")
    ids[55] = -1
    dx[55] = float("nan")
    d = torch.empty(12, 16, device="cuda")
    psgd_embed_grad(ctx, dx, ids, d)
    torch.cuda.synchronize()
    want = torch.full((12, 16), 10.0)
    want[5] = 9.0
    want[10:] = 0.0
    want[3, 2], want[4, 3] = float("nan"), float("inf")
    assert torch.equal(torch.nan_to_num(d.cpu(), nan=-7.0, posinf=-9.0), torch.nan_to_num(want, nan=-7.0, posinf=-9.0))
    keep = d.nan_to_num_().clone()
    psgd_embed_grad(ctx, dx[:0], ids[:0], d, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(d, keep)
    psgd_embed_grad(ctx, dx[:0], ids[:0], d)
    torch.cuda.synchronize()
    assert bool((d == 0).all())


def test_two_calls_at_once_and_graph_replays(ctx):
    """Two gradients on two streams with a workspace each, and a captured lookup and gradient replayed
    with new tokens, equal the calls made one after another."""
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_grad, psgd_embed_grad_workspace, psgd_embed_lookup
    rng = np.random.default_rng(33)
    n, vocab, dim = 5000, 300, 256
    dx = [torch.from_numpy(rng.standard_normal((n, dim))).float().cuda() for _ in range(2)]
    ids = [torch.from_numpy(rng.integers(0, vocab, n)).cuda() for _ in range(2)]
    ref, got = ([torch.empty(vocab, dim, device="cuda") for _ in range(2)] for _ in range(2))
    for i in range(2):
        psgd_embed_grad(ctx, dx[i], ids[i], ref[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        psgd_embed_grad(ctx, dx[i], ids[i], got[i], stream=streams[i])
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    for i, stream in enumerate((0, streams[1].cuda_stream)):    # raw stream handles
        got[i].zero_()
        torch.cuda.synchronize()
        psgd_embed_grad(ctx, dx[i], ids[i], got[i], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(ref[i], got[i])
    need = psgd_embed_grad_workspace(n, vocab, dim)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    x, xr = torch.empty(n, dim, device="cuda"), torch.empty(n, dim, device="cuda")
    psgd_embed_lookup(ctx, ref[0], ids[0], xr)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        psgd_embed_lookup(ctx, ref[0], ids[0], x)
        psgd_embed_grad(ctx, x, ids[0], got[0], workspace=ws[0])
    for t in range(3):
        ids[0].copy_(torch.from_numpy(rng.integers(-1, vocab, n)))
        graph.replay()
        psgd_embed_lookup(ctx, ref[0], ids[0], xr)
        psgd_embed_grad(ctx, xr, ids[0], got[1], workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(x, xr) and torch.equal(got[0], got[1]), t


@pytest.mark.parametrize("n,vocab", [(16385, 3000), (24576, 3000), (24577, 3000), (40001, 9000), (300000, 130), (30000, 300001)])
def test_grad_long_batches(ctx, n, vocab):
    """Both sides of the length from which tokens are dealt to ranges by several workgroups, shares of
    several sizes, and a vocabulary of more ranges than they deal to; half of the tokens are one."""
    rng = np.random.default_rng(n)
    ids = rng.integers(-1, vocab + 1, n)
    ids[rng.random(n) < 0.5] = vocab // 2
    _grad_case(ctx, n, vocab, 8, "f32", "i64", 1.0, False, ids)
    _grad_case(ctx, n, vocab, 8, "bf16", "i32", 0.5, True, ids)
