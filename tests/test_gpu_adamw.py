"""AdamW over a list of tensors against the float64 oracle.

Codes and exponents of 8-bit moments are compared bit by bit: they are defined on moments computed in
float32 operation by operation, which the oracle does too. Parameters: from those moments, float32
arithmetic moves the exact result by at most
    2^-23 |p'| + lr (2^-21 |m1'| rbc1 / (sqrt(m2' rbc2) + eps) + 2^-22 wd |p|)
(in units of 2^-24: the last subtraction 1 of p'; rbc1 1, its product 1, rbc2 and its product 1 together
under the root, root 2, sum 1, reciprocal 2 at most, its product 1, the sum with wd p 1, the product with
lr 1: below 8 of the quotient + 1 that the subtraction's operand has left; wd p: product 1, sum 1, lr 1),
and a radicand among fp32's subnormals is off by half of 2^-149 more. The rounding to storage never
falls: it moves the ends of that interval to the ends of what is allowed.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import lowbit as L
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu

HP = (2e-3, 0.9, 0.999, 1e-8, 0.01)


def _dt(k):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[k]


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _hp(v=HP):
    from rank_gradient_compression_powersgd_amd import psgd_adam_hparams
    return psgd_adam_hparams(*v)


def _pad(v):
    return np.pad(v, (0, -len(v) % 64))


class Case:
    """A list of tensors with state on the device and its copy on the host."""

    def __init__(self, sizes, param, grad, bits, stochastic, seed=11, step=3, scale=1.0, skew=0):
        import torch
        from rank_gradient_compression_powersgd_amd import AdamWGroup
        rng = np.random.default_rng(seed)
        self.sizes, self.param, self.bits, self.stochastic, self.seed, self.t = sizes, param, bits, stochastic, seed + (seed << 33), step
        total = sum(sizes)
        size = scale * np.exp(rng.uniform(np.log(1e-4), 0, total))
        flat = lambda v, k: torch.from_numpy(np.concatenate([np.zeros(skew), v])).to("cuda", _dt(k))[skew:]  # noqa: E731
        self.p_all = flat(rng.standard_normal(total) * 0.05, param)
        self.g_all = flat(rng.standard_normal(total) * size, grad)
        self.params, self.grads = list(torch.split(self.p_all, sizes)), list(torch.split(self.g_all, sizes))
        m1 = [_pad((rng.standard_normal(n) * 0.3 * scale).astype(np.float32).astype(np.float64)) for n in sizes]
        m2 = [_pad((np.square(rng.standard_normal(n)) * np.square(np.float64(scale))).astype(np.float32).astype(np.float64)) for n in sizes]
        if bits == 8:
            (c1, e1), (c2, e2) = L.encode8(np.concatenate(m1), False), L.encode8(np.concatenate(m2), True)
            st = [c1, c2, e1, e2]
        else:
            st = [np.concatenate(m1).astype(np.float32), np.concatenate(m2).astype(np.float32)]
        self.group = AdamWGroup(self.params, self.grads, bits=bits, stochastic=stochastic, seed=self.seed,
                                moments=[torch.from_numpy(x).cuda() for x in st])
        self.group.step_count.fill_(step)

    def moments(self):
        """float64 (m1, m2) per tensor, padding included."""
        g = self.group
        if self.bits == 8:
            m1 = L.decode8(g.m1.cpu().numpy(), g.e1.cpu().numpy(), False)
            m2 = L.decode8(g.m2.cpu().numpy(), g.e2.cpu().numpy(), True)
        else:
            m1, m2 = _np(g.m1), _np(g.m2)
        ends = [o + len(_pad(np.zeros(n))) for o, n in zip(g.offsets, self.sizes)]
        return [(m1[o:e], m2[o:e]) for o, e in zip(g.offsets, ends)]

    def step_and_check(self, max_norm=0.0, hp=HP):
        lr, b1, b2, eps, wd = hp
        p0, g0, before = [_np(p) for p in self.params], [_np(g) for g in self.grads], self.moments()
        self.group.step(_hp(hp), max_norm=max_norm)
        self.t += 1
        norm, clip = self.group.norm.tolist()
        want = np.sqrt(sum(np.square(g).sum() for g in g0))
        assert self.group.skip.item() == 0 and self.group.step_count.item() == self.t
        assert abs(norm - want) <= 2.0 ** -23 * want
        c = min(1.0, max_norm / want) if max_norm > 0 and want > max_norm else 1.0
        assert abs(clip - c) <= 2.0 ** -23 * c
        flat = [x.cpu().numpy() for x in self.group.state()]
        for i, n in enumerate(self.sizes):
            if n == 0:
                continue
            o, room = self.group.offsets[i], len(before[i][0])
            r = L.hash_bits(L.hash_key(self.seed, self.t, i), np.arange(n))
            w1, w2 = L.moments32(before[i][0][:n], before[i][1][:n], g0[i], clip, b1, b2)
            if self.bits == 8:
                sr = self.stochastic
                u1 = _pad(((r >> 16) + 0.5) / 65536.0) if sr else None
                u2 = _pad(((r & 0xFFFF) + 0.5) / 65536.0) if sr else None
                for j, (w, second, u) in enumerate(((w1, False, u1), (w2, True, u2))):
                    code, exp = L.encode8(_pad(w), second, u)
                    assert np.array_equal(flat[2 + j][o // 64:(o + room) // 64], exp), (i, j)
                    bad = np.flatnonzero(flat[j][o:o + room] != code)
                    assert bad.size == 0, (i, j, bad[:8], flat[j][o:o + room][bad[:8]], code[bad[:8]])
            else:
                assert np.array_equal(flat[0][o:o + room], _pad(w1)) and np.array_equal(flat[1][o:o + room], _pad(w2))
            w1, w2 = w1.astype(np.float64), w2.astype(np.float64)
            x = L.adamw_param(p0[i], w1, w2, self.t, lr, b1, b2, eps, wd)
            radicand = w2 * L.bias_free(b2, self.t)
            quotient = np.abs(w1) * L.bias_free(b1, self.t) / (np.sqrt(radicand) + np.float32(eps))
            below = np.where(radicand < 2.0 ** -126, 2.0 ** -149 / np.maximum(radicand, 2.0 ** -149), 0.0)
            tol = 2.0 ** -23 * np.abs(x) + lr * ((2.0 ** -21 + below) * quotient + 2.0 ** -22 * wd * np.abs(p0[i]))
            if self.param == "f32":
                store = lambda v: v  # noqa: E731
            elif self.stochastic:
                drop = 16 if self.param == "bf16" else 19
                u = (L.hash_more(r) >> drop) * 2.0 ** (drop - 32)
                store = lambda v: L.round16(v, self.param, u)  # noqa: E731
            else:
                import torch
                store = lambda v: _np(torch.from_numpy(v).to(_dt(self.param)))  # noqa: E731
            got = _np(self.params[i])
            lo, hi = store(x - tol), store(x + tol)
            out = np.flatnonzero((got < lo) | (got > hi))
            assert out.size == 0, (i, out[:8], got[out[:8]], lo[out[:8]], hi[out[:8]])


SIZES = [[1], [63, 64, 65], [4095, 4096, 4097, 3], [0, 5, 0], [20000], [130, 1001, 7, 9000, 1, 511, 64 * 70 + 1]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "_".join(map(str, s)))
@pytest.mark.parametrize("bits,stochastic", [(8, True), (8, False), (32, False)])
@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16"), ("f32", "bf16")])
def test_two_steps_of_a_list(sizes, bits, stochastic, param, grad):
    log(f"adamw {sizes} {param} {grad} {bits} {stochastic}")
    c = Case(sizes, param, grad, bits, stochastic)
    c.step_and_check(max_norm=0.5)
    c.step_and_check(max_norm=0.0)


@pytest.mark.parametrize("param", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("grad", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits,stochastic", [(8, True), (32, True), (32, False)])
def test_every_pair_of_types_off_alignment(param, grad, bits, stochastic):
    log(f"adamw types {param} {grad} {bits}")
    Case([777, 4100, 33], param, grad, bits, stochastic, seed=5, skew=1).step_and_check(max_norm=1.0)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e-8, 1e8, 1e15])
@pytest.mark.parametrize("stochastic", [True, False])
def test_moments_over_the_range_of_fp32(scale, stochastic):
    """Second moments from fp32's subnormals (and 0) to 1e30."""
    log(f"adamw scale {scale}")
    c = Case([3000, 65], "f32", "f32", 8, stochastic, seed=9, scale=scale)
    c.step_and_check(hp=(2e-3, 0.9, 0.999, 1e-30, 0.0))


def test_first_step_from_zero_state():
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    for bits in (8, 32):
        p = torch.ones(1000, device="cuda")
        g = torch.cat([torch.zeros(500), torch.full((500,), 1e-3)]).cuda()
        group = AdamWGroup([p], [g], bits=bits)
        group.step(_hp((0.1, 0.9, 0.999, 1e-8, 0.0)))
        assert torch.equal(p[:500], torch.ones(500, device="cuda"))
        # |update| is 1 up to the codes' 2^-4 (8 bits) of the quotient's parts, which are not used before they are stored
        assert (p[500:] - 0.9).abs().max().item() < 1e-5
        m1, m2 = group.moments(torch.float32)
        assert not m1[:500].any() and not m2[:500].any() and (m2[500:1000] > 0).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("grad", ["f32", "f16", "bf16"])
def test_a_bad_gradient_changes_nothing(bits, bad, grad):
    c = Case([4097, 100, 3], "bf16", grad, bits, True, seed=2)
    keep = [x.clone() for x in (c.p_all, *c.group.state(), c.group.norm, c.group.step_count)]
    good = c.grads[1][57].clone()
    c.grads[1][57] = bad
    c.group.step(_hp(), max_norm=1.0)
    assert c.group.skip.item() == 1
    assert all((a == b).all() for a, b in zip(keep, (c.p_all, *c.group.state(), c.group.norm, c.group.step_count)))
    c.grads[1][57] = good
    c.step_and_check(max_norm=1.0)


def test_a_skip_word_decided_before_is_kept():
    import torch
    c = Case([300], "f32", "f32", 8, True)
    keep = c.p_all.clone()
    c.group.step(_hp(), skip=torch.ones(1, dtype=torch.int32, device="cuda"))
    assert c.group.skip.item() == 1 and torch.equal(c.p_all, keep) and c.group.step_count.item() == 3
    c.group.step(_hp(), skip=c.group.skip)                         # in and out may be one word
    assert c.group.skip.item() == 1 and torch.equal(c.p_all, keep)
    c.group.step(_hp(), skip=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert c.group.skip.item() == 0 and not torch.equal(c.p_all, keep)


def test_a_moment_past_the_codes_is_nan_in_its_group_only():
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    p, g = torch.zeros(192, device="cuda"), torch.ones(192, device="cuda")
    g[70] = 1e25                                                   # its square is past fp32
    group = AdamWGroup([p], [g])
    group.step(_hp())
    m1, m2 = group.moments(torch.float32)
    assert group.skip.item() == 0 and torch.isfinite(m1).all()
    assert torch.isnan(m2[64:128]).all() and torch.isfinite(m2[:64]).all() and torch.isfinite(m2[128:]).all()


def test_moments_move_as_their_expectation_says():
    """1000 steps of a constant gradient at b2 = 0.999: rounded to nearest the second moment stands still,
    rounded stochastically its mean over 2^16 elements follows 1 - b2^t. A step moves an element by at most
    1e-3, its rounding by at most an eighth of it either way: a variance of at most 1e-3 / 8 a step and
    0.125 in all, 0.0014 in the standard deviation of the mean; six of them."""
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    n = 1 << 16
    end = {}
    for stochastic in (True, False):
        p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
        group = AdamWGroup([p], [g], stochastic=stochastic, seed=4)
        for _ in range(1000):
            group.step(_hp((1e-3, 0.9, 0.999, 1e-8, 0.0)))
        end[stochastic] = group.moments(torch.float32)[1].double().mean().item()
    log(f"  second moment after 1000 steps: stochastic {end[True]:.4f}, nearest {end[False]:.4f}")
    assert abs(end[True] - (1 - 0.999 ** 1000)) < 0.0084
    assert end[False] < 0.1


def test_moments_as_bf16_and_fp32():
    import torch
    c = Case([5, 100, 64], "f32", "f32", 8, False)
    for dtype in (torch.bfloat16, torch.float32):
        m1, m2 = c.group.moments(dtype)
        assert m1.dtype == m2.dtype == dtype
        for (w1, w2), o in zip(c.moments(), c.group.offsets):
            assert np.array_equal(_np(m1)[o:o + len(w1)], w1) and np.array_equal(_np(m2)[o:o + len(w2)], w2)
    out = torch.full((2, 20), 7.0, device="cuda")
    from rank_gradient_compression_powersgd_amd import psgd_adamw_moments
    g = c.group
    psgd_adamw_moments(g.ctx, g.m1, g.e1, g.m2, g.e2, out[0, :5], out[1, :5])      # an odd count ends where it says
    assert np.array_equal(_np(out[0, :5]), c.moments()[0][0][:5]) and (out[:, 5:] == 7).all()


def test_same_bits_twice_and_other_bits_with_another_seed():
    import torch
    runs = []
    for seed in (11, 11, 12):
        c = Case([9000, 70], "bf16", "f32", 8, True, seed=11)
        c.group.seed = seed
        for _ in range(3):
            c.group.step(_hp(), max_norm=1.0)
        runs.append([c.p_all, *c.group.state()])
    assert all(torch.equal(a, b) for a, b in zip(runs[0], runs[1]))
    assert not torch.equal(runs[0][1], runs[2][1])


@pytest.mark.parametrize("bits", [8, 32])
def test_graph_replays_match_eager(bits):
    import torch
    sizes = [5000, 33, 4096]
    eager, cap = (Case(sizes, "bf16", "f32", bits, True, seed=6) for _ in range(2))
    warm = Case(sizes, "bf16", "f32", bits, True, seed=6)
    warm.group.step(_hp(), max_norm=1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cap.group.step(_hp(), max_norm=1.0)
    torch.cuda.synchronize()
    rng = np.random.default_rng(0)
    for t in range(5):
        g = torch.from_numpy(rng.standard_normal(sum(sizes)).astype(np.float32)).cuda()
        if t == 2:
            g[17] = float("nan")
        eager.g_all.copy_(g)
        cap.g_all.copy_(g)
        eager.group.step(_hp(), max_norm=1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((eager.p_all, *eager.group.state(), eager.group.step_count, eager.group.skip, eager.group.norm),
                        (cap.p_all, *cap.group.state(), cap.group.step_count, cap.group.skip, cap.group.norm)):
            assert torch.equal(a, b), t


def test_two_groups_on_two_streams():
    import torch
    alone, first, second = (Case([300000, 77], "f32", "f32", 8, True, seed=8) for _ in range(3))
    for _ in range(4):
        alone.group.step(_hp())
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        first.group.step(_hp(), stream=s1)
        with torch.cuda.stream(s2):
            second.group.step(_hp())
    torch.cuda.synchronize()
    for c in (first, second):
        assert torch.equal(c.p_all, alone.p_all) and all(torch.equal(a, b) for a, b in zip(c.group.state(), alone.group.state()))


def test_moments_of_a_stream_of_their_own():
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    p, g = torch.randn(70000, device="cuda"), torch.randn(70000, device="cuda")
    group = AdamWGroup([p], [g], bits=8)
    group.step(_hp())
    want = group.moments()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for kind in (torch.bfloat16, torch.float32):
        got = group.moments(dtype=kind, stream=stream)
        stream.synchronize()
        assert all(a.dtype == kind and torch.equal(a.float(), b.float()) for a, b in zip(got, want))
    got = group.moments(stream=stream.cuda_stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n", [64, 1003, 4_300_001])
def test_moments_of_short_and_long_lists(n):
    """Against the oracle's values, of any codes and any exponents that keep them out of the subnormals."""
    import torch
    from rank_gradient_compression_powersgd_amd import binding as B
    rng = np.random.default_rng(n)
    room = (n + 63) // 64 * 64
    codes = [torch.from_numpy(rng.integers(0, 256, room, dtype=np.uint8)).cuda() for _ in range(2)]
    exps = [torch.from_numpy(rng.integers(40, 256, room // 64).astype(np.uint8)).cuda() for _ in range(2)]       # no fp32 subnormals
    ctx = B.psgd_create(0, 1)
    for dtype in (torch.float32, torch.bfloat16):
        flat = [torch.full((n + 7,), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        outs = [f[1:n + 1] for f in flat]
        B.psgd_adamw_moments(ctx, codes[0], exps[0], codes[1], exps[1], *outs)
        for i, second in ((0, False), (1, True)):
            want = torch.from_numpy(L.decode8(codes[i].cpu().numpy(), exps[i].cpu().numpy(), second)[:n].astype(np.float32)).to(dtype)
            got = outs[i].cpu()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(torch.nan_to_num(got, 0.0), torch.nan_to_num(want, 0.0))
            assert float(flat[i][0]) == 7.0 and (flat[i][n + 1:] == 7).all()
    B.psgd_destroy(ctx)


def test_neighbours_of_a_list_are_left_alone():
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    p, g = torch.full((1000,), 3.0, device="cuda").half(), torch.ones(1000, device="cuda").half()
    group = AdamWGroup([p[7:400], p[500:993]], [g[1:394], g[400:893]], bits=8)
    group.step(_hp())
    assert (p[:7] == 3).all() and (p[400:500] == 3).all() and (p[993:] == 3).all()
    assert (p[7:400] != 3).all() and (p[500:993] != 3).all() and (g == 1).all()


def test_elements_past_32_bits():
    """A tensor of 2^32 + 4101 elements: its last ones against a tensor of their own, whose bits differ only by
    the index's high half."""
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    n, tail = 2 ** 32 + 4101, 4101
    p = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    gt = torch.from_numpy(rng.standard_normal(tail)).to("cuda", torch.bfloat16)
    g[-tail:] = gt
    group = AdamWGroup([p], [g], seed=21)
    group.step(_hp())
    r = L.hash_bits(L.hash_key(21, 1, 0), np.arange(2 ** 32, n, dtype=np.uint64))
    w1, w2 = L.moments32(np.zeros(tail), np.zeros(tail), _np(gt), 1.0, 0.9, 0.999)
    for w, second, u, code, exp in ((w1, False, r >> 16, group.m1, group.e1), (w2, True, r & 0xFFFF, group.m2, group.e2)):
        c, e = L.encode8(_pad(w), second, _pad((u + 0.5) / 65536.0))
        assert np.array_equal(code[2 ** 32:].cpu().numpy(), c) and np.array_equal(exp[2 ** 26:].cpu().numpy(), e)
    assert not group.m1[:2 ** 32].any()
    assert (p[-tail:] != 0.5).float().mean() > 0.3


def test_a_refused_step_counts_nothing():
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup, binding as B
    f = torch.ones(100, device="cuda")
    group = AdamWGroup([f], [f.clone()])
    for bad in ((-1.0, 0.9, 0.999, 1e-8, 0.0), (1e-3, 1.0, 0.999, 1e-8, 0.0), (1e-3, 0.9, float("nan"), 1e-8, 0.0), (1e-3, 0.9, 0.999, float("inf"), 0.0)):
        with pytest.raises(B.PsgdError):
            group.step(_hp(bad))
    assert int(group.step_count) == 0 and (f == 1).all()


def test_refusals():
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup, binding as B

    def refused(status, fn):
        with pytest.raises(B.PsgdError) as ei:
            fn()
        assert ei.value.status == status, str(ei.value)

    f = torch.zeros(100, device="cuda")
    group = AdamWGroup([f], [f.clone()])
    word, norm = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    for bad in ((-1.0, 0.9, 0.999, 1e-8, 0.0), (1e-3, 1.0, 0.999, 1e-8, 0.0), (1e-3, 0.9, -0.1, 1e-8, 0.0), (1e-3, 0.9, 0.999, float("nan"), 0.0)):
        refused(B.PSGD_EINVAL, lambda: group.step(_hp(bad)))
    refused(B.PSGD_EINVAL, lambda: group.step(_hp(), max_norm=float("nan")))
    refused(B.PSGD_EINVAL, lambda: B.psgd_adamw_prepare(group.ctx, group.plan, 0.0, None, None, word, norm))
    refused(B.PSGD_EINVAL, lambda: B.psgd_adamw_update(group.ctx, group.plan, None, word, norm, _hp()))
    other = B.psgd_create(0, 1)
    refused(B.PSGD_EINVAL, lambda: B.psgd_adamw_update(other, group.plan, word, word, norm, _hp()))
    lib = B.load_library()
    assert lib.psgd_adamw_update(group.ctx, group.plan, word.data_ptr(), word.data_ptr(), None, B.ctypes.byref(_hp()), 2, 0, None) == B.PSGD_EINVAL
    args = [t.data_ptr() for t in (group.m1, group.e1, group.m2, group.e2)]
    assert lib.psgd_adamw_moments(group.ctx, *args, 2 ** 35 + 1, f.data_ptr(), f.data_ptr(), 3, None) == B.PSGD_EUNSUPPORTED
    assert lib.psgd_adamw_moments(group.ctx, *args, -1, f.data_ptr(), f.data_ptr(), 3, None) == B.PSGD_EINVAL
    t = B.make_adamw_tensor(f, f.clone(), group.m1, group.m2, group.e1, group.e2)
    refused(B.PSGD_EDTYPE, lambda: B.psgd_adamw_plan_create(other, [t], 7, 3, 1))
    refused(B.PSGD_EDTYPE, lambda: B.psgd_adamw_plan_create(other, [t], 3, 0, 1))
    refused(B.PSGD_EINVAL, lambda: B.psgd_adamw_plan_create(other, [t], 3, 3, 2))
    refused(B.PSGD_EINVAL, lambda: B.psgd_adamw_plan_create(other, [], 3, 3, 1))
    for field, value, status in (("param", None, B.PSGD_EINVAL), ("e2", None, B.PSGD_EINVAL), ("numel", -1, B.PSGD_EINVAL),
                                 ("m1", group.m1.data_ptr() + 4, B.PSGD_EINVAL), ("param", f.data_ptr() + 2, B.PSGD_EINVAL),
                                 ("numel", 2 ** 40, B.PSGD_EUNSUPPORTED)):
        x = B.psgd_adamw_tensor.from_buffer_copy(t)
        setattr(x, field, value)
        refused(status, lambda: B.psgd_adamw_plan_create(other, [x], 3, 3, 1))
    # two tensors that share elements, of the parameters or of the state
    g2, m = f.clone(), [torch.zeros(128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    e = [torch.zeros(2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    refused(B.PSGD_EINVAL, lambda: AdamWGroup([f, f[50:]], [g2, g2[50:]]))
    refused(B.PSGD_EINVAL, lambda: AdamWGroup([f], [f]))
    refused(B.PSGD_EINVAL, lambda: B.psgd_adamw_plan_create(other, [t, B.make_adamw_tensor(g2, g2.clone(), m[0], group.m1, *e)], 3, 3, 1))
    B.psgd_destroy(other)


class _AfterALoss(Case):
    """Reads groups of byte 255 as a step does."""

    def moments(self):
        g = self.group
        m1, m2 = L.carried8(*(x.cpu().numpy() for x in (g.m1, g.e1, g.m2, g.e2)))
        ends = [o + len(_pad(np.zeros(n))) for o, n in zip(g.offsets, self.sizes)]
        return [(m1[o:e], m2[o:e]) for o, e in zip(g.offsets, ends)]


@pytest.mark.parametrize("stochastic", [True, False])
@pytest.mark.parametrize("sizes", [[192], [4096 + 200, 70]], ids=lambda s: "_".join(map(str, s)))
def test_a_gradient_whose_square_is_past_fp32_leaves_its_neighbours_finite(sizes, stochastic):
    """The step after it and later ones: bit by bit, and every parameter stays a number."""
    import torch
    c = _AfterALoss(sizes, "f32", "f32", 8, stochastic, seed=4)
    good = c.g_all.clone()
    c.grads[0][70] = 1e25
    c.group.step(_hp())
    c.t += 1
    assert int(c.group.e2[1]) == 255 and c.group.skip.item() == 0 and torch.isfinite(c.p_all).all()
    c.g_all.copy_(good)
    for _ in range(3):
        c.step_and_check()
        assert torch.isfinite(c.p_all).all() and int(c.group.e2[1]) == 254
    c.grads[0][70] = -1e25                                         # and once more
    c.group.step(_hp())
    c.t += 1
    c.g_all.copy_(good)
    c.step_and_check()
    assert torch.isfinite(c.p_all).all()


def test_a_lost_group_moves_again_once_its_second_moment_has_decayed():
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    p, g = torch.zeros(192, device="cuda"), torch.ones(192, device="cuda")
    g[70] = 1e25
    group = AdamWGroup([p], [g])
    hp = _hp((1e-3, 0.9, 0.5, 1e-8, 0.0))
    group.step(hp)
    g[70] = 1.0
    still = p[64:128].clone()
    for _ in range(20):                                            # 1.875 2^127 halves in a step
        group.step(hp)
    assert (p[64:128] - still).abs().max() < 1e-9 and torch.isfinite(p).all()
    for _ in range(200):
        group.step(hp)
    assert torch.isfinite(p).all() and (p[64:128] < still - 0.05).all() and torch.isfinite(group.moments(torch.float32)[1]).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1.1e-38, 1.2e-38])
def test_an_eps_among_the_subnormals_leaves_parameters_without_a_gradient(bits, eps):
    """0 of any eps > 0 is 0, and of eps = 0 counts as that."""
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    p, g = torch.ones(200, device="cuda"), torch.zeros(200, device="cuda")
    g[150:] = 0.5
    group = AdamWGroup([p], [g], bits=bits)
    for t in range(1, 4):
        group.step(_hp((0.1, 0.9, 0.999, eps, 0.0)))
        assert (p[:150] == 1).all() and torch.isfinite(p).all()
        assert t > 1 or (p[150:] - 0.9).abs().max() < 1e-5         # |update| 1 in the first step


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("b1", [0.9, 0.95])
def test_a_gradient_at_the_end_of_fp32_leaves_its_parameter_a_number(bits, b1):
    """Its second moment is an infinity: no update. Its first moment, bias corrected, rounds past fp32 for these b1."""
    import torch
    from rank_gradient_compression_powersgd_amd import AdamWGroup
    top = torch.finfo(torch.float32).max
    f = np.float32
    with np.errstate(over="ignore"):
        assert np.isinf(f(top) * (f(1) - f(b1)) * f(L.bias_free(b1, 1)))
    p, g = torch.ones(200, device="cuda"), torch.full((200,), 1e-3, device="cuda")
    g[7], g[100] = top, -top
    group = AdamWGroup([p], [g], bits=bits)
    for _ in range(4):
        group.step(_hp((0.1, b1, 0.999, 1e-8, 0.0)))
        assert group.skip.item() == 0 and torch.isfinite(p).all() and (p[[7, 100]] == 1).all()


def test_moments_refuse_outputs_over_their_inputs_and_one_another():
    import torch
    from rank_gradient_compression_powersgd_amd import binding as B
    n = 1000
    flat = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    at = lambda o, size: flat[o:o + size]  # noqa: E731
    m1, m2, e1, e2 = at(0, 1024), at(1024, 1024), at(2048, 16), at(2064, 16)
    ctx = B.psgd_create(0, 1)

    def out(o, dtype):
        return at(o, n * dtype.itemsize).view(dtype)

    for dtype in (torch.float32, torch.bfloat16):
        size = n * dtype.itemsize
        free, second = 4096, 4096 + size
        B.psgd_adamw_moments(ctx, m1, e1, m2, e2, out(free, dtype), out(second, dtype))               # neighbours
        B.psgd_adamw_moments(ctx, m1, e1, m2, e2, out(2080, dtype), out(2080 + size, dtype))          # right behind the exponents
        for bad in (0, 1020, 2044, 2060, 2076):                                                        # over m1, m1 and m2, m2, e1, e2
            for outs in ((out(bad, dtype), out(second, dtype)), (out(free, dtype), out(bad, dtype))):
                with pytest.raises(B.PsgdError) as ei:
                    B.psgd_adamw_moments(ctx, m1, e1, m2, e2, *outs)
                assert ei.value.status == B.PSGD_EINVAL and "overlap the moments" in str(ei.value), bad
        with pytest.raises(B.PsgdError) as ei:
            B.psgd_adamw_moments(ctx, m1, e1, m2, e2, out(free, dtype), out(second - 4, dtype))
        assert ei.value.status == B.PSGD_EINVAL and "overlap" in str(ei.value)
    assert not flat[:2080].any()
    B.psgd_destroy(ctx)
