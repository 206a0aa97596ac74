"""Distance slopes up to the largest that fp32 holds: a query keeps its own key, at distance 0, and nothing else."""
import pytest
import torch

import mod_ref as R

pytestmark = pytest.mark.gpu
SLOPES = [3.4e38, 2.4e38, 1e38, 1e30, 60.0, 12.0]


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


def own_key(q, k, scale):
    """The score of every query with the key at its own position (rows of one head), and the bound on its error: d
    products accumulated in fp32, a few more roundings, and what lse's own logarithm and conversions add.  (From a
    slope of 1e30 on the other keys' weights are 0 in fp32.)"""
    q, k = q.double(), k.double()
    s = scale * (q * k).sum(1)
    return s, (q.shape[1] + 6) * R.F32 * scale * (q.abs() * k.abs()).sum(1) + 2.0 ** -20


def data(T, Hq, d, seed):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, Hq, d, generator=g) * 0.3).bfloat16()
    k, v = (torch.randn(T, 1, d, generator=g).bfloat16() for _ in range(2))
    return q, k, v


@pytest.mark.parametrize("cap", [0.0, 50.0])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt(F, cap, causal):
    T, Hq, d = 300, len(SLOPES), 64
    q, k, v = data(T, Hq, d, 60)
    lse = torch.empty(1, Hq, T, device="cuda")
    out = F.fa_prefill_mod(q[None].cuda(), k[None].cuda(), v[None].cuda(), causal=causal, softcap=cap, lse=lse,
                           alibi_slopes=torch.tensor(SLOPES).cuda())
    assert F.fa_get_error() == F.FA_OK
    pos = torch.arange(T)
    for h, slope in enumerate(SLOPES):
        if slope > 100.0:
            s, tol = own_key(q[:, h], k[:, 0], d ** -0.5)
            if cap:
                s, tol = cap * torch.tanh(s / cap), tol + 4e-7 * cap
            R.check(lse[0, h], s, tol, f"lse slope {slope}")
            assert torch.equal(out[0, :, h].cpu(), v[:, 0]), f"slope {slope}"  # a weight of 1
        else:
            ref = R.Rows(q[:, h], k[:, 0], v[:, 0], pos, R.visible(pos, T, causal), d ** -0.5, cap, slope)
            R.check(lse[0, h], ref.lse, ref.lse_tol, f"lse slope {slope}")
            R.check(out[0, :, h], ref.out, ref.out_tol, f"out slope {slope}")


@pytest.mark.parametrize("heads", [len(SLOPES), 16], ids=str)
def test_paged_and_sums(F, heads):
    """Single tokens and a chunk, with the group's heads in rows of their own (6) and packed into one tile (16)."""
    d, ctx, ql = 64, [200, 90, 33], [150, 1, 2]
    sl = torch.tensor((SLOPES[:4] * 4)[:heads])
    p = R.Paged(61, ctx, ql, heads, 1, d, std=0.3)
    q, kc, vc, table, c, n = p.cuda()
    lse = torch.empty(p.total, heads, device="cuda")
    acc = torch.zeros(3, 1, 200, device="cuda")
    out = F.fa_paged_attn_accum(q, kc, vc, table, c, n, None, acc, alibi_slopes=sl.cuda(), lse=lse, max_q_len=150)
    assert F.fa_get_error() == F.FA_OK
    at = 0
    for s in range(3):
        old = ctx[s] - ql[s]
        for h in range(heads):
            x, tol = own_key(p.q[at:at + ql[s], h], p.k[s][old:, 0], d ** -0.5)
            R.check(lse[at:at + ql[s], h], x, tol, f"lse s{s} h{h}")
            assert torch.equal(out[at:at + ql[s], h].cpu(), p.v[s][old:, 0]), (s, h)
        want = torch.zeros(200, dtype=torch.float64)
        want[old:ctx[s]] = heads  # every head gives a token of the chunk its whole weight
        # a weight is 2^(x - lse): both in fp32, log2 units of at most 8
        R.check(acc[s, 0], want, want * 2.0 ** -16, f"sums s{s}")
        at += ql[s]


def test_slopes_that_favour_distance(F):
    """A large negative slope within the documented range: every query reads the farthest key."""
    T, d = 260, 64
    q, k, v = data(T, 2, d, 62)
    out = F.fa_prefill_mod(q[None].cuda(), k[None].cuda(), v[None].cuda(),
                           alibi_slopes=torch.tensor([-8e35, -1e20]).cuda())
    assert F.fa_get_error() == F.FA_OK
    assert torch.equal(out[0].cpu(), v[:1].expand(T, 2, d))
