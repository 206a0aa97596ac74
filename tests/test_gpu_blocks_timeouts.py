"""Waits of the listed blocks' kernel that give up while pages are on their way (a test hook; no fault, trap or hang)."""
import time

import pytest
import torch

import scaled_ref as R

pytestmark = pytest.mark.gpu
DEFAULT_LIMIT_NS = 4_000_000_000


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    yield fattn
    fattn.fa_debug_force_timeout(False)
    fattn.fa_debug_set_wait_limit(DEFAULT_LIMIT_NS)


class gives_up_at:
    """Each warp before its n-th page, after a millisecond."""

    def __init__(self, F, n):
        self.F, self.n = F, n

    def __enter__(self):
        self.F.fa_debug_set_wait_limit(1_000_000)
        self.F.fa_debug_force_timeout(self.n)

    def __exit__(self, *exc):
        self.F.fa_debug_force_timeout(False)
        self.F.fa_debug_set_wait_limit(DEFAULT_LIMIT_NS)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def case(S, Hq, H, d, fp8, seed=1):
    table, nb = R.tables([1600], seed)
    table = table.expand(S, -1).contiguous()  # one context for all
    if fp8:
        k, v, ke, ve = R.random_cache8(nb, H, d, seed)
    else:
        k, v, ke, ve = R.normal(nb, H, 16, d, seed=seed), R.normal(nb, H, 16, d, seed=seed + 1), None, None
    q = R.normal(S, Hq, d, seed=seed + 2)
    return cuda(q, k, v, table, R.i32([1600] * S), R.i32([1] * S)), dict(zip(("k_exp", "v_exp"), cuda(ke, ve)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("page", [2, 11, 21, 32])
def test_only_copies_in_flight_are_waited_for(F, fp8, d, page):
    """A warp that gives up has at most its ring's pages on their way; a wait for an earlier one, whose place was taken
    again since, would run its whole second."""
    args, exps = case(60, 8, 8, d, fp8)  # single CTAs of three warps, 33 pages each
    sel = torch.arange(99).int().expand(60, 8, 99).contiguous().cuda()
    want = F.fa_paged_attn_blocks(*args, sel, **exps)
    out = torch.full_like(want, 7.0)
    assert F.fa_get_error() == F.FA_OK
    with gives_up_at(F, page):
        began = time.perf_counter()
        F.fa_paged_attn_blocks(*args, sel, out=out, **exps)
        assert F.fa_get_error() == F.FA_ERR_TIMEOUT
        assert time.perf_counter() - began < 0.5
    assert bool((out == 7.0).all())
    assert torch.equal(F.fa_paged_attn_blocks(*args, sel, **exps), want) and F.fa_get_error() == F.FA_OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("slow", [0, 5, 31])
def test_a_cluster_writes_whole_rows_or_none(F, fp8, d, slow):
    """One warp of a cluster gives up, the others have read their pages: nothing of that list's rows is written, and all of
    the other list's."""
    args, exps = case(1, 8, 2, d, fp8, 4)
    sel = torch.full((1, 2, 256), -1, dtype=torch.int32)
    sel[0, 0, slow::32] = torch.arange(8).int() + 20  # eight pages for one of 32 warps
    sel[0, :, 1::37] = torch.arange(60, 67).int()     # one here and there
    sel = sel.cuda()
    lse = torch.zeros(1, 8).cuda()
    want = F.fa_paged_attn_blocks(*args, sel, lse=lse, **exps)
    assert F.fa_get_error() == F.FA_OK
    out, got = torch.full_like(want, 7.0), torch.full_like(lse, 7.0)
    with gives_up_at(F, 6):
        F.fa_paged_attn_blocks(*args, sel, out=out, lse=got, **exps)
        assert F.fa_get_error() == F.FA_ERR_TIMEOUT
    assert bool((out[:, :4] == 7.0).all()) and bool((got[:, :4] == 7.0).all())
    assert torch.equal(out[:, 4:], want[:, 4:]) and torch.equal(got[:, 4:], lse[:, 4:])
