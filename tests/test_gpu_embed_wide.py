"""The embedding's gradient at widths that take several workgroups' columns, in chunks of 32 sorted tokens
and of 8, against the float64 oracle. The sum of a token seen k times is k fp32 terms in some grouping,
then one product and, when accumulating, one more sum: at most (k + 2) 2^-24 of what is summed."""
from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_helpers import log
from tests.test_gpu_embed import _dt, _grad_case

pytestmark = pytest.mark.gpu


@pytest.fixture()
def ctx():
    import rank_gradient_compression_powersgd_amd as psgd
    c = psgd.psgd_create(0, 1)
    yield c
    psgd.psgd_destroy(c)


def _skewed(n, vocab, seed):
    """A third of the tokens one id, the rest falling off, some outside."""
    rng = np.random.default_rng(seed)
    ids = np.minimum(rng.geometric(0.01, n) - 1, vocab - 1)
    ids[rng.random(n) < 0.3] = vocab // 3
    ids[rng.random(n) < 0.05] = -1
    return ids


# columns in one workgroup and in several, whole and with a last one in part; one element a lane, four
# and eight; fewer tokens than fill 2^22 elements (chunks of 8) and more (of 32)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dt,n,dim", [("f32", 700, 3968), ("f32", 1200, 3968), ("bf16", 1200, 3968), ("f32", 600, 1032), ("f32", 4200, 1032),
                                      ("bf16", 4200, 1032), ("bf16", 500, 2056), ("f16", 2100, 2056), ("f32", 4300, 1001), ("bf16", 700, 1001),
                                      ("f16", 4300, 1001), ("f32", 9000, 260)])
def test_wide_rows(ctx, dt, n, dim, accumulate):
    _grad_case(ctx, n, 90, dim, dt, "i64", 0.37, accumulate, _skewed(n, 90, n + dim))


@pytest.mark.parametrize("dt,dim,pad", [("f32", 3968, 0), ("bf16", 2056, 0), ("f32", 1001, 0), ("bf16", 1032, 3), ("f32", 1032, 1)])
def test_runs_at_the_borders_of_chunks_of_32(ctx, dt, dim, pad):
    """Runs of 31, 32, 33, 64, 65, 97 and 1025 tokens in chunks of 32, so that runs begin and end at, before
    and behind the borders, between fillers that shift them; sizes past 2^22 elements or 8192 tokens."""
    counts = [31, 32, 33, 64, 65, 97, 1025, 1, 32, 128, 7, 1, 96, 31]
    n0 = sum(counts)
    fill = max(0, (1 << 22) // dim + 1 - n0)
    ids = np.concatenate([np.full(c, 2 * i) for i, c in enumerate(counts)] + [np.full(fill, 60)])
    assert len(ids) * dim > 1 << 22 or len(ids) > 8192
    ids = np.random.default_rng(dim).permutation(ids)
    for accumulate in (False, True):
        _grad_case(ctx, len(ids), 64, dim, dt, "i32", 2.0, accumulate, ids, ld_pad=pad)


@pytest.mark.parametrize("n,dim", [(200, 3968), (4400, 1032)])
def test_zero_rows_in_every_column(ctx, n, dim):
    """Absent tokens' rows become zeros over their whole width, whatever stood there."""
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_grad
    vocab = 1003
    ids = torch.from_numpy(np.random.default_rng(n).integers(0, vocab // 2, n) * 2).cuda()
    dx = torch.ones(n, dim, dtype=_dt("bf16"), device="cuda")
    d = torch.full((vocab, dim), float("nan"), device="cuda")
    log(f"zero rows n={n} dim={dim}")
    psgd_embed_grad(ctx, dx, ids, d)
    torch.cuda.synchronize()
    want = torch.bincount(ids, minlength=vocab).float()[:, None].expand(vocab, dim)
    assert torch.equal(d, want)


@pytest.mark.parametrize("dim", [4, 1])
def test_most_tokens(ctx, dim):
    """2^25 tokens, the most a call takes, half of them one id: sums of whole numbers up to 2^24 are exact
    in any grouping."""
    import torch
    from rank_gradient_compression_powersgd_amd import psgd_embed_grad
    n, vocab = 2 ** 25, 1000
    gen = torch.Generator(device="cuda").manual_seed(dim)
    ids = torch.randint(-1, vocab, (n,), device="cuda", generator=gen, dtype=torch.int32)
    ids[torch.randperm(n, device="cuda", generator=gen)[:2 ** 24 - 2 ** 20]] = 7
    dx = torch.ones(n, dim, dtype=_dt("f16"), device="cuda")
    count = torch.bincount(ids[ids >= 0], minlength=vocab).float()[:, None].expand(vocab, dim)
    assert float(count.max()) <= 2.0 ** 24
    d = torch.full((vocab, dim), float("nan"), device="cuda")
    log(f"most tokens, dim={dim}")
    psgd_embed_grad(ctx, dx, ids, d)
    torch.cuda.synchronize()
    assert torch.equal(d, count)
    d.fill_(0.0)
    psgd_embed_grad(ctx, dx, ids, d, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(d, count)
