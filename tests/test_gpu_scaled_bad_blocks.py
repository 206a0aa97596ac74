"""Blocks outside the pool: reported, and zeros at scale 1 in every form of the calls over the 8-bit cache with block scales
and over chosen blocks."""
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


# single tokens with a CTA or a cluster for each list, the stream (a wide table), few tokens, chunks, chunks shared along their keys
@pytest.mark.parametrize("ctx, ql, mbps", [([50, 600], [1, 1], None), ([50, 600], [1, 1], 700), ([50, 600], [2, 3], None),
                                           ([50, 600], [40, 60], None), ([50, 4000], [40, 60], None)], ids=str)
@pytest.mark.parametrize("bad", [0, 9, -1, -(1 << 31)])
@pytest.mark.parametrize("d", [128, 64])
def test_zeros_at_scale_1(F, ctx, ql, mbps, bad, d):
    Hq, H = 8, 2
    table, nb = R.tables(ctx, 21, mbps=mbps)
    k, v, ke, ve = R.random_cache8(nb, H, d, 22, 2)
    q = R.normal(sum(ql), Hq, d, seed=23, std=2.0)
    table[1, 20] = nb + bad if bad >= 0 else bad
    lse = torch.zeros(sum(ql), Hq).cuda()
    out = F.fa_paged_attn_fp8_scaled(*cuda(q, k, v, ke, ve, table, R.i32(ctx), R.i32(ql)), lse=lse, max_q_len=max(ql))
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    sel = torch.full((sum(ql), H, 40), -1, dtype=torch.int32)
    sel[:, :, :-(-ctx[1] // 16)] = torch.arange(-(-ctx[1] // 16))[:40].int()
    sel[:ql[0], :, -(-ctx[0] // 16):] = -1
    by_lse = torch.zeros(sum(ql), Hq).cuda()
    at = cuda(table, R.i32(ctx), R.i32(ql))
    by_blocks = F.fa_paged_attn_blocks(*cuda(q, k, v), *at, sel.cuda(), *cuda(ke, ve), lse=by_lse)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    kk, vv = R.values(k, ke), R.values(v, ve, True)
    zeros = torch.zeros(1, *kk.shape[1:], dtype=torch.float64)
    kk, vv = torch.cat([kk, zeros]), torch.cat([vv, zeros])
    table[1, 20] = nb
    i = 0
    for s, (c, n) in enumerate(zip(ctx, ql)):
        p = table[s, :-(-c // 16)].long()
        see = torch.arange(c)[None] <= torch.arange(c - n, c)[:, None]
        for h in range(Hq):
            keys, vals = (x[p, h // 4].reshape(-1, d)[:c] for x in (kk, vv))
            R.Rows(q[i:i + n, h], keys, vals, see, d ** -0.5, R.HALF_F16).check(out.cpu()[i:i + n, h], lse.cpu()[i:i + n, h], "whole")
            m = min(c, 640)  # (the lists hold 40 blocks)
            R.Rows(q[i:i + n, h], keys[:m], vals[:m], see[:, :m], d ** -0.5, R.HALF_F16).check(
                by_blocks.cpu()[i:i + n, h], by_lse.cpu()[i:i + n, h], "by blocks")
        i += n


@pytest.mark.parametrize("d", [128, 64])
def test_zeros_in_the_bf16_lists(F, d):
    ctx, H, Hq = [600], 2, 4
    table, nb = R.tables(ctx, 31)
    k, v, q = R.normal(nb, H, 16, d, seed=32), R.normal(nb, H, 16, d, seed=33), R.normal(1, Hq, d, seed=34)
    table[0, 7] = nb
    sel = torch.arange(30).int().expand(1, H, 30).contiguous()
    lse = torch.zeros(1, Hq).cuda()
    out = F.fa_paged_attn_blocks(*cuda(q, k, v, table, R.i32(ctx), R.i32([1]), sel), lse=lse)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    zeros = torch.zeros(1, H, 16, d, dtype=torch.bfloat16)
    k, v, p = torch.cat([k, zeros]).double(), torch.cat([v, zeros]).double(), table[0, :30].long()
    for h in range(Hq):
        R.Rows(q[:, h], k[p, h // 2].reshape(-1, d), v[p, h // 2].reshape(-1, d), torch.ones(1, 480, dtype=torch.bool), d ** -0.5,
               R.HALF_BF16).check(out.cpu()[:, h], lse.cpu()[:, h])
