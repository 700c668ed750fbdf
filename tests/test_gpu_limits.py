"""Calls at the limits of memory and of sizes: what is refused leaves nothing behind, and what is
allowed goes through the whole step."""
from __future__ import annotations

import math
import resource
import time

import numpy as np
import pytest

import oracle
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu


def _muon_pair(seed=3):
    """Two groups of one state, each with its parameters and momentum."""
    import torch
    from rank_gradient_compression_powersgd_amd import PowerSGDGroup
    out = []
    for _ in range(2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shapes = [(96, 136), (200, 64)]
        err = [torch.zeros(s, device="cuda") for s in shapes]
        g = PowerSGDGroup([None] * 2, [0, 0], torch.ones(1, device="cuda"), 4, [torch.zeros(s[1], 4) for s in shapes], err)
        for o in g.out:
            o.normal_(generator=gen)
        params = [torch.randn(s, device="cuda", generator=gen) for s in shapes]
        mom = [torch.randn(s, device="cuda", generator=gen) for s in shapes]
        g.attach_muon(params, mom)
        out.append((g, params, mom))
    return out


def _refused_ns_plan(ctx, x, total):
    from rank_gradient_compression_powersgd_amd import binding as B
    side = math.isqrt(int(0.9 * total / 12))         # 8 bytes an element, 4 of s x s: less than the card, more than is free
    B.psgd_ns_plan_create(ctx, [B.psgd_ns_matrix(x.data_ptr(), side, x.data_ptr(), side, side, side)], B.PSGD_F32, B.PSGD_F32)


def _refused_plan(ctx, x, total):
    from rank_gradient_compression_powersgd_amd import binding as B
    side, p = 20000, x.data_ptr()                    # rank above 128: 4 bytes of workspace an element
    mat = B.psgd_matrix(p, side, p, side, p, p, p, 0, 0, side, side, 0, 0)
    big = B.psgd_create(0, 896)
    try:
        B.psgd_plan_create(big, [mat] * int(0.9 * total / (4 * side * side)), B.PSGD_F16, 1)
    finally:
        B.psgd_destroy(big)


@pytest.mark.parametrize("refused", [_refused_ns_plan, _refused_plan])
def test_a_refused_allocation_leaves_no_error_behind(refused):
    """A plan that does not fit is refused, and the Muon step of a group that was there before runs whole:
    momentum and parameters are those of its twin, bit for bit. The descriptors of the refused plan
    name memory that nothing reads: it is never made."""
    import torch
    from rank_gradient_compression_powersgd_amd import binding as B
    (a, pa, ma), (b, pb, mb) = _muon_pair()
    hp = B.muon_hparams(0.1)
    B.psgd_muon_update(a.ctx, a.plan, a.skip, None, hp)
    torch.cuda.synchronize()
    total = torch.cuda.mem_get_info()[1]
    hold = torch.empty(int(0.3 * total), dtype=torch.uint8, device="cuda")
    with pytest.raises(B.PsgdError) as ei:
        refused(b.ctx, hold, total)
    assert ei.value.status == B.PSGD_ENOMEM
    B.psgd_muon_update(b.ctx, b.plan, b.skip, None, hp)
    torch.cuda.synchronize()
    for x, y in zip(pa + ma, pb + mb):
        assert torch.equal(x, y)
    del hold
    torch.cuda.empty_cache()
    a.close()
    b.close()


@pytest.mark.parametrize("side,count", [(2 ** 22, 1), (2 ** 20, 3000)])
def test_groups_past_the_memory_are_refused_before_they_are_planned(side, count):
    """The largest shapes a descriptor may hold want terabytes: refused from their sizes, without host
    lists of their tiles (2^32 of them)."""
    import torch
    from rank_gradient_compression_powersgd_amd import binding as B
    x = torch.zeros(4, device="cuda")
    ctx = B.psgd_create(0, 1)
    before, t0 = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss, time.monotonic()
    with pytest.raises(B.PsgdError) as ei:
        B.psgd_ns_plan_create(ctx, [B.psgd_ns_matrix(x.data_ptr(), side, x.data_ptr(), side, side, side)] * count, B.PSGD_F32, B.PSGD_F32)
    grown = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before
    assert ei.value.status == B.PSGD_ENOMEM
    assert grown < 1 << 18 and time.monotonic() - t0 < 5.0, (grown, time.monotonic() - t0)        # KiB
    B.psgd_destroy(ctx)


def test_step_with_an_embedding_past_2_29_elements():
    """The gradient of a table of 2^29 elements and more goes through the whole Muon step: norm, clipping
    and Adam on the rows that have a gradient; the others stay as they are (no decay, zero moments)."""
    import torch
    from rank_gradient_compression_powersgd_amd import binding as B
    vocab, dim, n = 2 ** 18 + 5, 2056, 300
    assert vocab * dim > 2 ** 29
    (g, params, mom), (other, _, _) = _muon_pair()
    other.close()
    gen = torch.Generator(device="cuda").manual_seed(11)
    table = torch.randn(vocab, dim, device="cuda", generator=gen)
    m1, m2, dtable = torch.zeros_like(table), torch.zeros_like(table), torch.empty_like(table)
    ids = torch.randint(0, vocab, (n,), device="cuda", generator=gen)
    ids[0], ids[1] = vocab - 1, 0
    dx = torch.randn(n, dim, device="cuda", generator=gen)
    B.psgd_embed_grad(g.ctx, dx, ids, dtable)
    rows = torch.unique(ids)
    old = table[rows].double().cpu().numpy()
    sums = [float(table[i:i + 65536].double().sum()) for i in range(0, vocab, 65536)]
    hp, hpa = B.muon_hparams(0.01), B.psgd_adam_hparams(1e-2, 0.9, 0.999, 1e-8, 0.0)
    log(f"step_muon with a table of {vocab} x {dim}")
    g.step_muon(hp, [(table, m1, m2, dtable)], hpa, max_norm=5.0)
    torch.cuda.synchronize()
    grad = dtable[rows].double().cpu().numpy()
    norm = math.sqrt(float((grad ** 2).sum()) + sum(float((q.double() ** 2).sum()) for q in g.q_next))
    assert abs(float(g.adam_norm[0]) - norm) <= 1e-6 * norm
    clip = float(g.adam_norm[1])
    assert abs(clip - 5.0 / norm) <= 1e-6
    state = oracle.AdamState(old, np.zeros_like(old), np.zeros_like(old), "f32", "f32", "f32")
    (state,), _, _, _ = oracle.adam_group_step([state], [grad * clip], 0, False, hpa, hpa, n_mats=0, max_norm=0.0)
    got = table[rows].double().cpu().numpy()
    assert np.linalg.norm(got - state.theta) <= 1e-6 * np.linalg.norm(state.theta)
    table[rows] = torch.from_numpy(old).float().cuda()
    assert sums == [float(table[i:i + 65536].double().sum()) for i in range(0, vocab, 65536)]
    g.close()


def test_too_many_pass_through_tensors():
    """More tensors than the norm has items are refused, whatever their size."""
    import torch
    from rank_gradient_compression_powersgd_amd import binding as B
    (g, _, _), (other, _, _) = _muon_pair()
    other.close()
    x = torch.ones(4, device="cuda")
    with pytest.raises(B.PsgdError) as ei:
        B.psgd_adam_prepare(g.ctx, g.plan, [B.make_adam_tensor(x, x, x, x)] * 8193, 0.0, g.skip, g.adam_step, g.adam_norm)
    assert ei.value.status == B.PSGD_EINVAL
    g.close()
