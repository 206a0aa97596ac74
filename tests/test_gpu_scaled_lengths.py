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


@pytest.mark.parametrize("ctx, ql, Hq, wide", [([40, 300], [1, 0], 4, False), ([40, 300], [1, 0], 4, True), ([40, 300], [30, 0], 4, False),
                                               ([40, 300], [30, 0], 40, False), ([300, 40], [2, 0], 40, True)])
@pytest.mark.parametrize("bad", [-3, 1 << 20, -(1 << 31)])
def test_lengths_of_sequences_without_queries_are_checked(F, ctx, ql, Hq, wide, bad):
    """A context that is negative or longer than its table is reported by every call, whatever form the sizes choose;
    the other sequence gets what it gets without."""
    d, H, n = 128, 2, sum(ql)
    table, nb = R.tables(ctx, 11, mbps=600 if wide else None)
    cache = cuda(*R.random_cache8(nb, H, d, 12))
    q, kv = R.normal(n, Hq, d, seed=13).cuda(), R.normal(n, H, d, seed=14).cuda()
    bounds = torch.zeros(nb, H, 2, d, dtype=torch.bfloat16).cuda()
    sel = torch.tensor([0, 1, -1]).int().expand(n, H, 3).contiguous().cuda()

    def run(ctx):
        got, errors = [], []

        def call(f, *a, **k):
            got.append(f(*a, **k))
            errors.append(F.fa_get_error())
        at = cuda(table, R.i32(ctx), R.i32(ql))
        mine = [t.clone() for t in cache]
        call(F.fa_cache_append_fp8_scaled, kv, kv, *mine, *at)
        call(F.fa_block_bounds, mine[0], *at, bounds.clone(), total_q=n, k_exp=mine[2])
        call(F.fa_block_select, q, got[-1], *at, 2)
        call(F.fa_paged_attn_blocks, q, mine[0], mine[1], *at, sel, k_exp=mine[2], v_exp=mine[3])
        call(F.fa_paged_attn_fp8_scaled, q, *mine, *at, max_q_len=max(ql))
        return got[1:] + mine, errors
    want, fine = run(ctx)
    got, errors = run([ctx[0], bad])
    assert fine == [F.FA_OK] * 5 and errors == [F.FA_ERR_BOUNDS] * 5
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_that_add_up_to_two_to_the_31_are_reported(F):
    """32 sequences of 2^26 rows each, every one of them consistent, in a call of ten rows."""
    n, many = 32, 1 << 26
    table = torch.zeros(n, many // 16, dtype=torch.int32, device="cuda")  # (512 MB; the first blocks of the first are done)
    lens = torch.full((n,), many, dtype=torch.int32, device="cuda")
    k = R.normal(1, 1, 16, 64, seed=1).cuda()
    bounds = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    F.fa_block_bounds(k, table, lens, lens, bounds, total_q=10)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    assert torch.equal(bounds, torch.stack([k.amin(2), k.amax(2)], 2))
