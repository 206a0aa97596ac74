"""Caps far above the scores bend next to nothing: the logits must keep a relative accuracy, whatever the cap.

Prompts, chunks and single tokens, with and without a distance bias, and the weight sums, against 64 bits.
"""
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


class Rows(R.Rows):
    """R.Rows with a bound on the cap's own error that does not grow with the cap.  c tanh(z / c): the kernels' tanh is
    off by at most 4e-7 of its value (5e-8 to 2.8e-7 where it is a polynomial, 3e-7 of 0.76 and more beyond), the factors
    z scale / c and c are each rounded twice (rounding the argument changes tanh by at most as much, relatively), and
    the product once: 4e-7 + 5 * 2^-24 of the capped score, 12 * 2^-24 in all."""

    def __init__(self, q, k, v, pos, see, scale, cap, slope=None):
        super().__init__(q, k, v, pos, see, scale, cap, slope)
        q, k, v = q.double(), k.double(), v.double()
        inside = lambda x: torch.where(see, x, torch.zeros_like(x)).amax(1)
        z = cap * torch.tanh(scale * (q @ k.T) / cap)
        x = z if slope is None else z - float(slope) * (pos[:, None] - torch.arange(k.shape[0])[None]).abs()
        self.logit_tol = ((q.shape[1] + 2) * R.F32 * inside(scale * (q.abs() @ k.abs().T)) + 12 * R.F32 * inside(z.abs()) +
                          4 * R.F32 * inside(x.abs()))
        self.lse_tol = self.logit_tol + 2.0 ** -20 + 4 * R.F32 * self.lse.abs()
        self.w_rel = 2 * (self.logit_tol + self.lse_tol)
        mass = self.w @ v.abs()
        self.out_tol = (R.HALF_BF16 + self.w_rel[:, None] + 2.0 ** -18) * mass + R.HALF_BF16 * (
            self.out.abs() + (R.HALF_BF16 + self.w_rel[:, None]) * mass) + 1e-30


CAPS = [300.0, 5e3, 1e4, 1e5, 1e7, 1e9, 1e30]


def make(T, Hq, d, seed, loud):
    """q, k, v of one kv head; with `loud` every 29th row's scores reach far beyond a cap of 300 to 5000."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(T, Hq, d, generator=g)
    if loud:
        q[::29] *= 5e3
    k, v = (torch.randn(T, 1, d, generator=g).bfloat16() for _ in range(2))
    return q.bfloat16(), k, v


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("loud", [False, True], ids=["quiet", "loud"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt(F, cap, bias, loud, d):
    T, Hq = 270, 2
    q, k, v = make(T, Hq, d, 50, loud)
    sl = R.slopes(Hq) if bias else None
    lse = torch.empty(1, Hq, T, device="cuda")
    out = F.fa_prefill_mod(q[None].cuda(), k[None].cuda(), v[None].cuda(), softcap=cap, lse=lse,
                           alibi_slopes=sl.cuda() if bias else None)
    assert F.fa_get_error() == F.FA_OK
    pos = torch.arange(T)
    for h in range(Hq):
        ref = Rows(q[:, h], k[:, 0], v[:, 0], pos, R.visible(pos, T, True), d ** -0.5, cap, sl[h] if bias else None)
        R.check(lse[0, h], ref.lse, ref.lse_tol, f"lse h{h}")
        R.check(out[0, :, h], ref.out, ref.out_tol, f"out h{h}")


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (3, 1, 128)], ids=str)
def test_paged_and_sums(F, cap, bias, heads):
    """Single tokens, a short chunk and a long one: the outputs, and every cached token's weight."""
    Hq, Hkv, d = heads
    p = R.Paged(51, [300, 77, 1, 900], [200, 9, 1, 1], *heads)
    sl = R.slopes(Hq) if bias else None
    q, kc, vc, table, ctx, ql = p.cuda()
    lse = torch.empty(p.total, Hq, device="cuda")
    acc = torch.full((4, Hkv, 900), 9.0, device="cuda")
    out = F.fa_paged_attn_accum(q, kc, vc, table, ctx, ql, None, acc, softcap=cap, lse=lse,
                                alibi_slopes=sl.cuda() if bias else None, max_q_len=200)
    assert F.fa_get_error() == F.FA_OK
    g = Hq // Hkv
    want = torch.full(acc.shape, 9.0, dtype=torch.float64)
    for s, c in enumerate(p.ctx):
        want[s, :, :c] = 0
    tol = torch.zeros_like(want)
    at = 0
    for s, (c, n) in enumerate(zip(p.ctx, p.ql)):
        pos = torch.arange(c - n, c)
        see = R.visible(pos, c, True)
        for h in range(Hq):
            ref = Rows(p.q[at:at + n, h], p.k[s][:, h // g], p.v[s][:, h // g], pos, see, d ** -0.5, cap,
                       sl[h] if bias else None)
            R.check(lse[at:at + n, h], ref.lse, ref.lse_tol, f"lse s{s} h{h}")
            R.check(out[at:at + n, h], ref.out, ref.out_tol, f"out s{s} h{h}")
            want[s, h // g, :c] += ref.w.sum(0)
            # each weight's relative error, and one fp32 rounding of at most sum-of-the-rest per add
            tol[s, h // g, :c] += ((ref.w_rel + (n * g + 4) * R.F32)[:, None] * ref.w).sum(0) + 1e-30
        at += n
    R.check(acc, want, tol, "sums")


def test_a_cap_that_bends_nothing_is_no_cap(F):
    """The weights with a cap of 1e9 are those without one within the bounds of both."""
    T, d = 300, 128
    q, k, v = make(T, 2, d, 52, False)
    got = []
    for cap in (0.0, 1e9):
        lse = torch.empty(1, 2, T, device="cuda")
        out = F.fa_prefill_mod(q[None].cuda(), k[None].cuda(), v[None].cuda(), softcap=cap, lse=lse)
        got.append((out.cpu(), lse.cpu()))
    pos = torch.arange(T)
    for h in range(2):
        ref = Rows(q[:, h], k[:, 0], v[:, 0], pos, R.visible(pos, T, True), d ** -0.5, 1e9)
        R.check(got[0][1][0, h] - got[1][1][0, h], torch.zeros(T, dtype=torch.float64), 2 * ref.lse_tol, "lse")
        R.check(got[0][0][0, :, h].float() - got[1][0][0, :, h].float(), torch.zeros_like(ref.out), 2 * ref.out_tol, "out")
