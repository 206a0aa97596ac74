"""Batches with rows behind the last sequence's (a captured step of fewer sequences than it was made for): those rows are
left as they were, and the others get what they get without them."""
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


PAD = 7


def pad(t):
    return torch.cat([t, torch.full((PAD, *t.shape[1:]), 3, dtype=t.dtype)]).cuda()


def kept(got, want):
    """The first rows as without padding, the last as they were."""
    return torch.equal(got[:-PAD], want) and bool((got[-PAD:] == 3).all())


def case(ctx, ql, H, d, seed):
    """Tables with two sequences of no queries and no tokens behind the batch, and a random cache."""
    table, nb = R.tables(ctx, seed)
    wide = torch.cat([table, torch.full((2, table.shape[1]), -1, dtype=table.dtype)]).cuda()
    return (table.cuda(), R.i32(ctx).cuda(), R.i32(ql).cuda()), (wide, R.i32(ctx + [0, 0]).cuda(), R.i32(ql + [0, 0]).cuda()), nb


@pytest.mark.parametrize("ctx, ql", [([40, 300, 17], [1, 1, 1]), ([40, 5000], [1, 1]), ([300, 170], [100, 60])])
def test_attention(F, ctx, ql):
    at, padded, nb = case(ctx, ql, 2, 128, 11)
    cache = [t.cuda() for t in R.random_cache8(nb, 2, 128, 12)]
    q = R.normal(sum(ql), 4, 128, seed=13)
    lse = torch.zeros(sum(ql), 4).cuda()
    want = F.fa_paged_attn_fp8_scaled(q.cuda(), *cache, *at, lse=lse, max_q_len=max(ql))
    out, got_lse = pad(want.cpu()), pad(lse.cpu())
    F.fa_paged_attn_fp8_scaled(pad(q), *cache, *padded, out=out, lse=got_lse, max_q_len=max(ql))
    assert F.fa_get_error() == F.FA_OK
    assert kept(out, want) and kept(got_lse, lse)


@pytest.mark.parametrize("ctx, ql", [([40, 300, 17], [1, 1, 1]), ([300, 170], [100, 60])])
def test_append_and_bounds(F, ctx, ql):
    at, padded, nb = case(ctx, ql, 2, 64, 21)
    n = sum(ql)
    k, v, q = R.normal(n, 2, 64, seed=22), R.normal(n, 2, 64, seed=23), R.normal(n, 4, 64, seed=24)
    turns = R.normal(512, 64, seed=25).float().cuda()
    a, b = ([t.cuda() for t in R.random_cache8(nb, 2, 64, 26)] for _ in range(2))
    want = F.fa_cache_append_fp8_scaled(k.cuda(), v.cuda(), *a, *at, q=q.cuda(), cos_sin=turns)
    got = pad(want.cpu())
    F.fa_cache_append_fp8_scaled(pad(k), pad(v), *b, *padded, q=pad(q), cos_sin=turns, q_out=got)
    assert F.fa_get_error() == F.FA_OK
    assert kept(got, want) and all(torch.equal(x, y) for x, y in zip(a, b))
    bounds = [torch.zeros(nb, 2, 2, 64, dtype=torch.bfloat16).cuda() for _ in range(2)]
    F.fa_block_bounds(a[0], *at, bounds[0], total_q=n, k_exp=a[2])
    F.fa_block_bounds(a[0], *padded, bounds[1], total_q=n + PAD, k_exp=a[2])
    assert F.fa_get_error() == F.FA_OK
    assert torch.equal(*bounds)


@pytest.mark.parametrize("ctx, ql", [([400, 3000, 17], [1, 1, 1]), ([900, 1700], [100, 60])])
def test_selected_blocks(F, ctx, ql):
    at, padded, nb = case(ctx, ql, 2, 128, 31)
    q, k, v = R.normal(sum(ql), 4, 128, seed=32), R.normal(nb, 2, 16, 128, seed=33).cuda(), R.normal(nb, 2, 16, 128, seed=34).cuda()
    bounds = torch.stack([k.amin(2), k.amax(2)], 2)
    want = F.fa_block_select(q.cuda(), bounds, *at, 12, max_q_len=max(ql))
    sel = pad(want.cpu())
    F.fa_block_select(pad(q), bounds, *padded, 12, sel=sel, max_q_len=max(ql))
    assert F.fa_get_error() == F.FA_OK
    assert kept(sel, want)
    lse = torch.zeros(sum(ql), 4).cuda()
    want = F.fa_paged_attn_blocks(q.cuda(), k, v, *at, want, lse=lse)
    out, got_lse = pad(want.cpu()), pad(lse.cpu())
    F.fa_paged_attn_blocks(pad(q), k, v, *padded, sel, out=out, lse=got_lse)
    assert F.fa_get_error() == F.FA_OK
    assert kept(out, want) and kept(got_lse, lse)


def test_negative_lengths_are_reported(F):
    """Also where the others add up to the rows of the call."""
    at, _, nb = case([40, 300], [-1, 2], 1, 64, 41)
    q, k = R.normal(2, 2, 64, seed=42).cuda(), R.normal(nb, 1, 16, 64, seed=43).cuda()
    bounds = torch.stack([k.amin(2), k.amax(2)], 2)
    sel = F.fa_block_select(q, bounds, *at, 4)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    F.fa_paged_attn_blocks(q, k, k, *at, sel)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    F.fa_block_bounds(k, *at, bounds, total_q=2)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
