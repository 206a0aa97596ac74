"""Lengths that do not fit, in the calls of the 8-bit cache with block scales and of attention over chosen blocks."""
import pytest
import torch

import scaled_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


def cuda(*ts):
    return [t.cuda() for t in ts]


@pytest.mark.parametrize("ctx, ql, n, k", [([20], [11], 10, 0), ([20, 40], [5, 8], 12, 5), ([20, 40, 9], [5, 8, 2], 13, 13)])
def test_append_leaves_queries_out_with_their_keys(F, ctx, ql, n, k):
    """A sequence that runs past the call's rows: none of its queries is turned either."""
    d, H, Hq = 64, 2, 4
    table, nb = R.tables(ctx, 1)
    cache = cuda(*R.random_cache8(nb, H, d, 2))
    before = [t.clone() for t in cache]
    kv, q = R.normal(n, H, d, seed=3).cuda(), R.normal(n, Hq, d, seed=4).cuda()
    turns = R.normal(64, d, seed=5).float().cuda()
    out = torch.full((n, Hq, d), 7.0, dtype=torch.bfloat16).cuda()
    F.fa_cache_append_fp8_scaled(kv, kv, *cache, *cuda(table, R.i32(ctx), R.i32(ql)), q=q, cos_sin=turns, q_out=out)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    want = torch.full_like(out, 7.0)
    good = [x if sum(ql[:s + 1]) <= n else 0 for s, x in enumerate(ql)]
    assert sum(good) == k
    F.fa_cache_append_fp8_scaled(kv, kv, *before, *cuda(table, R.i32(ctx), R.i32(good)), q=q, cos_sin=turns, q_out=want)
    assert F.fa_get_error() == F.FA_OK
    assert torch.equal(out, want) and bool((out[k:] == 7.0).all())
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
