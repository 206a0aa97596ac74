"""Lengths that do not add up to the call's rows: a negative one counts as none, a sequence whose rows do not all lie in
the call is left out, both are reported, and nothing before or behind the call's rows is written."""
import pytest
import torch

import scaled_ref as R

pytestmark = pytest.mark.gpu
GUARD, MARK = 64, 7.0
HUGE = 2 ** 31 - 1


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


class Guarded:
    """A tensor of n rows within a larger one that is filled with MARK."""

    def __init__(self, n, *shape, dtype=torch.bfloat16):
        self.whole = torch.full((n + 2 * GUARD, *shape), MARK, dtype=dtype, device="cuda")
        self.t = self.whole[GUARD:GUARD + n]

    def untouched_around(self):
        return bool((self.whole[:GUARD] == MARK).all()) and bool((self.whole[GUARD + len(self.t):] == MARK).all())


# (contexts, chunks, rows of the call, the sequences that fit): single tokens and few, chunks, rows that pass 31 bits
CASES = [([40, 300], [-1, 2], 2, [1]), ([40, 300, 33], [1, 1, 1], 2, [0, 1]), ([40, 300, 33], [1, 2, 1], 3, [0, 1]), ([40, 300, 33], [1, -HUGE, 2], 2, [0]),
         ([200, 300], [-7, 60], 60, [1]), ([200, 300, 170], [100, 60, 30], 150, [0]), ([500, 300, 170], [100, 1, 60], 120, [0, 1]),
         ([300, 30, 30, 30, 170], [60, HUGE, HUGE, 2, 70], 130, [0]), ([40, 30, 30, 30, 170], [1, HUGE, HUGE, 2, 1], 4, [0])]


def run(F, kind, args, Hq, H, d, n, ql, m):
    q = R.normal(n, Hq, d, seed=9)
    rows, out, lse = Guarded(n, Hq, d), Guarded(n, Hq, d), Guarded(n, Hq, dtype=torch.float32)
    rows.t.copy_(q)
    acc = torch.full((len(ql), H, 600), MARK, device="cuda")
    bf16, fp8, (table, ctx) = args
    at = (table, ctx, R.i32(ql).cuda())
    if kind == "attn":
        F.fa_paged_attn(rows.t, *bf16, *at, out=out.t, max_q_len=m)
    elif kind == "mod":
        F.fa_paged_attn_mod(rows.t, *bf16, *at, softcap=30.0, out=out.t, lse=lse.t, max_q_len=m)
    elif kind == "accum":
        F.fa_paged_attn_accum(rows.t, *bf16, *at, None, acc, out=out.t, lse=lse.t, max_q_len=m)
    elif kind == "fp8":
        F.fa_paged_attn_fp8(rows.t, fp8[0], fp8[1], 0.01, 0.01, *at, out=out.t, max_q_len=m)
    elif kind == "scaled":
        F.fa_paged_attn_fp8_scaled(rows.t, *fp8, *at, out=out.t, lse=lse.t, max_q_len=m)
    else:
        sel = torch.arange(20).int().expand(n, H, 20).contiguous().cuda()
        sel[:, :, 2:] = -1  # (blocks that every context has)
        F.fa_paged_attn_blocks(rows.t, *bf16, *at, sel, out=out.t, lse=lse.t)
    return F.fa_get_error(), out, lse, acc


def are_few(ql, g):
    return all(x * g <= 16 or x == HUGE for x in ql)


KINDS = ["attn", "mod", "accum", "fp8", "scaled", "blocks"]  # (fp8: single tokens and few only)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ctx, ql, n, fit, kind", [(*c, k) for c in CASES for k in KINDS if k != "fp8" or are_few(c[1], 2)], ids=str)
def test_rows(F, ctx, ql, n, fit, kind, wide):
    Hq, H, d = 4, 2, 128
    few = are_few(ql, Hq // H)
    table, nb = R.tables(ctx, 3, mbps=600 if wide else None)  # (a wide table: the stream, also of the 8-bit cache)
    fp8 = R.random_cache8(nb, H, d, 4)
    bf16 = [R.normal(nb, H, 16, d, seed=s) for s in (5, 6)]
    args = ([t.cuda() for t in bf16], [t.cuda() for t in fp8], (table.cuda(), R.i32(ctx).cuda()))
    m = max([1 if few else 200] + [x for x in ql if x < HUGE])
    err, out, lse, acc = run(F, kind, args, Hq, H, d, n, ql, m)
    assert err == F.FA_ERR_BOUNDS
    assert out.untouched_around() and lse.untouched_around()
    good = [x if s in fit else 0 for s, x in enumerate(ql)]
    ok, want, want_lse, want_acc = run(F, kind, args, Hq, H, d, n, good, m)
    assert ok == F.FA_OK
    k = sum(good)
    # two correct roundings of the same rows, possibly summed in another order: outputs and weights in 16 bits (2^-8 each,
    # twice), fp32 sums beside them
    top = {"fp8": 4.48, "scaled": float(R.values(fp8[1], fp8[3]).abs().max())}.get(kind, float(bf16[1].abs().max()))
    assert float((out.t[:k].double() - want.t[:k].double()).abs().max()) <= 2.0 ** -6 * top
    assert bool((out.t[k:] == MARK).all()) and bool((want.t[k:] == MARK).all())
    if kind in ("mod", "accum", "scaled", "blocks"):
        assert float((lse.t[:k] - want_lse.t[:k]).abs().max()) <= 1e-3
        assert bool((lse.t[k:] == MARK).all())
    if kind == "accum":
        for s in range(len(ctx)):
            if s in fit:
                assert float((acc[s] - want_acc[s]).abs().max()) <= 1e-3 * Hq // H * max(1, ql[s]) + 1e-3
            elif ql[s] != 0:
                assert bool((acc[s] == MARK).all())
