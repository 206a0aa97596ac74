"""Weights far below a row's largest, whose sum is all that most channels of the output hold: single tokens over the 8-bit
cache with block scales and over listed blocks of it."""
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


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("at", [0, 1500, 3999])
@pytest.mark.parametrize("H, mbps, ql", [(1, None, 1), (8, None, 1), (2, 700, 1), (2, None, 4)])
def test_their_sum_is_kept(F, d, at, H, mbps, ql):
    """One key 2^30 above 3999 others, its value 0 in all channels but the last."""
    c, Hq = 4000, 2 * H
    table, nb = R.tables([c], 41, mbps=mbps)
    k, v, ke, ve = R.random_cache8(nb, H, d, 42)
    ke[:], ve[:] = 127, 127
    k[:] = 0
    b, t = int(table[0, at // 16]), at % 16
    per = 30.0 / 1.4426950408889634 / d ** 0.5   # of q . k
    k[b, :, t] = torch.tensor(float(per)).to(R.FP8).view(torch.uint8)
    v[b, :, :, t] = 0
    v[b, :, d - 1, t] = 0x7E  # 448
    q = torch.ones(ql, Hq, d).bfloat16()
    at_ = cuda(table, R.i32([c]), R.i32([ql]))
    outs = []
    lse = torch.zeros(ql, Hq).cuda()
    outs.append((F.fa_paged_attn_fp8_scaled(*cuda(q, k, v, ke, ve), *at_, lse=lse, max_q_len=ql), lse))
    sel = torch.arange(250).int().expand(ql, H, 250).contiguous().cuda()
    lse = torch.zeros(ql, Hq).cuda()
    outs.append((F.fa_paged_attn_blocks(*cuda(q, k, v), *at_, sel, *cuda(ke, ve), lse=lse), lse))
    assert F.fa_get_error() == F.FA_OK
    p = table[0, :250].long()
    see = torch.arange(c)[None] <= torch.arange(c - ql, c)[:, None]
    for h in range(Hq):
        kk, vv = R.values(k[p, h // 2], ke[p, h // 2]).reshape(-1, d), R.values(v[p, h // 2], ve[p, h // 2], True).reshape(-1, d)
        rows = R.Rows(q[:, h], kk, vv, see, d ** -0.5, R.HALF_F16)
        # f16's smallest step is 2^-24 where the largest weight is 2^15: half of it for each key, not 2^-24 of the largest
        top = float(vv.abs().max()) * c
        rows.off = rows.off - 2.0 ** -24 * top + 2.0 ** -40 * top
        for out, l in outs:
            rows.check(out.cpu()[:, h], l.cpu()[:, h], f"head {h}")
