"""Tables and prompts whose lists take the last bytes of the shared memory that a kernel has without asking for more."""
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


# 4 bytes for every 8 blocks, and 8 more: 98288 blocks take 48 KB
@pytest.mark.parametrize("blocks", [97400, 98200, 98281, 98288, 98296])
def test_tables(F, blocks):
    p = R.Paged(91, [300, 40], [40, 1], 2, 1, 64)
    q, kc, vc, table, c, n = p.cuda()
    wide = torch.full((2, blocks), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    want = F.fa_paged_attn(q, kc, vc, table, c, n, max_q_len=40)
    assert torch.equal(F.fa_paged_attn(q, kc, vc, wide, c, n, max_q_len=40), want)
    acc = torch.zeros(2, 1, 300, device="cuda")
    lse = torch.empty(p.total, 2, device="cuda")
    out = F.fa_paged_attn_accum(q, kc, vc, wide, c, n, None, acc, lse=lse, max_q_len=40)
    assert F.fa_get_error() == F.FA_OK
    for s, h, at, ref in p.rows():
        R.check(out[at:at + p.ql[s], h], ref.out, ref.out_tol, f"out s{s} h{h}")
        R.check(lse[at:at + p.ql[s], h], ref.lse, ref.lse_tol, f"lse s{s} h{h}")
    assert ((acc.double().sum(2).cpu()[:, 0] - 2 * torch.tensor(p.ql)).abs() < 1e-3).all()


@pytest.mark.parametrize("blocks", [98200, 98288])
def test_tables_of_calls_that_cut_nothing(F, blocks):
    """Enough queries for every SM: the lists come from another variant."""
    p = R.Paged(92, [280], [270], 160, 160, 64)
    q, kc, vc, table, c, n = p.cuda()
    wide = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    kw = dict(window=100, max_q_len=270)
    want = F.fa_paged_attn_mod(q, kc, vc, table, c, n, **kw)
    assert torch.equal(F.fa_paged_attn_mod(q, kc, vc, wide, c, n, **kw), want)
    assert F.fa_get_error() == F.FA_OK


@pytest.mark.parametrize("T", [1568513, 1570001, 1572608])
def test_documents_of_a_long_prompt(F, T):
    d, n = 64, 100  # documents of 100 rows
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(1, T, 1, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    ids = (torch.arange(T, device="cuda") // n).to(torch.int32).view(1, T)
    out = F.fa_prefill_mod(q, k, v, doc_ids=ids)
    assert F.fa_get_error() == F.FA_OK
    for first in (0, n, 700 * n, T // n * n - n, T // n * n):
        rows = slice(first, min(T, first + n))
        m = rows.stop - rows.start
        if m:
            pos = torch.arange(m)
            ref = R.Rows(q[0, rows, 0].cpu(), k[0, rows, 0].cpu(), v[0, rows, 0].cpu(), pos, R.visible(pos, m, True), d ** -0.5)
            R.check(out[0, rows, 0], ref.out, ref.out_tol, f"rows from {first}")
