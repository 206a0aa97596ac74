"""How a chunk's keys are shared between SMs goes by the lengths: a wider table changes no bit."""
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


@pytest.mark.parametrize("heads, ctx, ql", [((2, 1, 64), [11 * 128], [24]), ((2, 1, 128), [9 * 128], [40]),
                                            ((3, 1, 64), [15 * 128], [20]), ((8, 2, 64), [19 * 128, 300], [33, 9]),
                                            ((1, 1, 64), [8 * 128 - 5], [17]), ((2, 1, 64), [23 * 128, 11 * 128], [90, 70])],
                         ids=str)
def test_same_bits_in_wider_tables(F, heads, ctx, ql):
    p = R.Paged(81, ctx, ql, *heads)
    q, kc, vc, table, c, n = p.cuda()
    table = table[:, :-(-max(ctx) // 16)].contiguous()  # the contexts fill it
    got = []
    for more in (0, 8, 40, 4000):
        wide = torch.cat([table, torch.full((len(ctx), more), -1, dtype=torch.int32, device="cuda")], 1)
        lse = torch.empty(p.total, heads[0], device="cuda")
        acc = torch.zeros(len(ctx), heads[1], max(ctx), device="cuda")
        out = F.fa_paged_attn_accum(q, kc, vc, wide, c, n, None, acc, lse=lse, max_q_len=max(ql))
        assert F.fa_get_error() == F.FA_OK
        got.append((out, lse, acc))
    for s, h, at, ref in p.rows():
        R.check(got[0][0][at:at + p.ql[s], h], ref.out, ref.out_tol, f"out s{s} h{h}")
        R.check(got[0][1][at:at + p.ql[s], h], ref.lse, ref.lse_tol, f"lse s{s} h{h}")
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)
