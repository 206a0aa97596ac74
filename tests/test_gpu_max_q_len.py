"""A chunk above the caller's bound on the chunk lengths is reported by every paged call, however few rows it has and
wherever its keys lie: the bound sizes what the calls keep per row."""
import pytest
import torch

import mod_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


# (heads, contexts, chunks, bound): two and three rows, a chunk that would take the other kernel; each in contexts that
# one warp holds and in contexts cut between CTAs
CASES = [((1, 1, 64), [4000, 3000], [1, 3], 1), ((2, 2, 128), [40, 33], [2, 1], 1), ((2, 2, 64), [90, 5000], [1, 3], 2),
         ((4, 2, 64), [300, 200], [1, 60], 1), ((6, 1, 64), [16, 200], [2, 1], 1)]


@pytest.mark.parametrize("heads, ctx, ql, bound", CASES, ids=str)
def test_reported(F, heads, ctx, ql, bound):
    p = R.Paged(71, ctx, ql, *heads)
    q, kc, vc, table, c, n = p.cuda()
    acc = torch.zeros(2, heads[1], max(ctx), device="cuda")
    calls = [lambda m: F.fa_paged_attn(q, kc, vc, table, c, n, max_q_len=m),
             lambda m: F.fa_paged_attn_mod(q, kc, vc, table, c, n, softcap=30.0, max_q_len=m),
             lambda m: F.fa_paged_attn_accum(q, kc, vc, table, c, n, None, acc, max_q_len=m)]
    for call in calls:
        call(bound)
        assert F.fa_get_error() == F.FA_ERR_BOUNDS
        call(max(ql))
        assert F.fa_get_error() == F.FA_OK
        call(max(ql) + 5)  # any bound will do
        assert F.fa_get_error() == F.FA_OK
    g = heads[0] // heads[1]
    total = acc.double().sum(2).cpu()  # the last call's: every query gives each head a weight of 1 in all
    for s in range(2):
        assert (total[s] - g * ql[s]).abs().max() <= 1e-3 * g * ql[s]


def test_reported_over_the_8_bit_cache(F):
    k = torch.randn(64, 2, 128, device="cuda").bfloat16()
    kc, vc = torch.zeros(8, 2, 16, 128, dtype=torch.uint8, device="cuda"), torch.zeros(8, 2, 128, 16, dtype=torch.uint8, device="cuda")
    F.fa_cache_append_fp8(k, k, kc, vc, torch.arange(64, dtype=torch.int32, device="cuda"), 0.02, 0.02)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.randn(4, 2, 128, device="cuda").bfloat16()
    for bound, want in ((1, F.FA_ERR_BOUNDS), (2, F.FA_ERR_BOUNDS), (3, F.FA_OK)):
        F.fa_paged_attn_fp8(q, kc, vc, 0.02, 0.02, table, i32(32, 20), i32(1, 3), max_q_len=bound)
        assert F.fa_get_error() == want
