"""Calls at the limits of memory and of sizes: what is refused leaves nothing behind."""
from __future__ import annotations

import math
import resource
import time

import pytest

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
