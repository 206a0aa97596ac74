"""Block bounds, the choice of blocks and attention over chosen blocks, against 64 bits."""
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
    return [None if t is None else t.cuda() for t in ts]


# ------------------------------------------------------------------ bounds --
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d, H", [(128, 2), (64, 3)])
@pytest.mark.parametrize("ctx, ql", [([1, 16, 17, 100], [1, 1, 1, 1]), ([40, 300, 16], [40, 3, 0]), ([257], [256])])
def test_bounds(F, fp8, d, H, ctx, ql):
    table, nb = R.tables(ctx, 61)
    if fp8:
        k, _, e, _ = R.random_cache8(nb, H, d, 61, 30)
        vals = R.values(k, e)
    else:
        k, e = R.normal(nb, H, 16, d, seed=61), None
        vals = k.double()
    bounds = R.normal(nb, H, 2, d, seed=62)
    want = bounds.clone()
    for s, (c, n) in enumerate(zip(ctx, ql)):
        for b in range((c - n) // 16, (c - 1) // 16 + 1 if n else 0):
            page = vals[int(table[s, b]), :, :c - b * 16]
            want[int(table[s, b])] = torch.stack([page.amin(1), page.amax(1)], 1).bfloat16()
            if c % 16 and b == c // 16:  # what lies behind the last token does not count
                k[int(table[s, b]), :, c % 16:] = 0x7E if fp8 else 1e30
    got = bounds.cuda()
    F.fa_block_bounds(k.cuda(), *cuda(table, R.i32(ctx), R.i32(ql)), got, k_exp=None if e is None else e.cuda(), total_q=sum(ql))
    assert F.fa_get_error() == F.FA_OK
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 64])
def test_bounds_pass_over_nan(F, fp8, d):
    table, nb = R.tables([40], 63)
    k, _, e, _ = R.random_cache8(nb, 1, d, 63, 20) if fp8 else (R.normal(nb, 1, 16, d, seed=63), None, None, None)
    vals = R.values(k, e) if fp8 else k.double()
    lost = torch.rand(k.shape, generator=torch.Generator().manual_seed(64)) < 0.3
    lost[:, :, 0] = False  # (a channel keeps a number)
    k[lost] = 0xFF if fp8 else float("nan")
    bounds = torch.zeros(nb, 1, 2, d, dtype=torch.bfloat16)
    want = bounds.clone()
    for b in range(3):
        p, n = int(table[0, b]), min(16, 40 - 16 * b)
        page, no = vals[p, :, :n], lost[p, :, :n]
        want[p] = torch.stack([page.masked_fill(no, 1e300).amin(1), page.masked_fill(no, -1e300).amax(1)], 1).bfloat16()
    got = bounds.cuda()
    F.fa_block_bounds(k.cuda(), *cuda(table, R.i32([40]), R.i32([40])), got, k_exp=None if e is None else e.cuda(), total_q=40)
    assert F.fa_get_error() == F.FA_OK
    assert torch.equal(got.cpu(), want)


# ------------------------------------------------------------------ select --
def boxes(nb, H, d, seed):
    mid, wide = R.normal(nb, H, d, seed=seed).float(), R.normal(nb, H, d, seed=seed + 1).float().abs() + 0.5
    return torch.stack([mid - wide, mid + wide], 2).bfloat16()


def check_select(F, q, bounds, table, ctx, ql, keep, recent, sink, max_q=None):
    want = R.select(q, bounds, table, ctx, ql, keep, recent, sink)
    got = F.fa_block_select(*cuda(q, bounds, table, R.i32(ctx), R.i32(ql)), keep, recent=recent, sink=sink, max_q_len=max_q)
    assert F.fa_get_error() == F.FA_OK
    got = got.cpu()
    assert torch.equal(got, want), f"{int((got != want).any(-1).sum())} of {want.shape[0] * want.shape[1]} rows differ"


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("Hq, H", [(4, 4), (12, 2), (16, 1), (3, 1), (20, 1), (34, 1)])
@pytest.mark.parametrize("keep, recent, sink", [(8, 1, 0), (20, 7, 2), (5, 0, 0), (6, 4, 2)])
def test_select_single_tokens(F, d, Hq, H, keep, recent, sink):
    ctx = [1, 16 * keep, 16 * keep + 1, 1000, 333, 5000]
    table, nb = R.tables(ctx, 71)
    check_select(F, R.normal(6, Hq, d, seed=72, std=2.0), boxes(nb, H, d, 73), table, ctx, [1] * 6, keep, recent, sink, 1)


@pytest.mark.parametrize("d, Hq, H", [(128, 8, 2), (64, 5, 1), (64, 17, 1), (128, 1, 1)])
@pytest.mark.parametrize("max_q", [None, 1])
def test_select_chunks(F, d, Hq, H, max_q):
    ctx, ql = [700, 90, 2000, 16, 300], [140, 90, 33, 0, 1]
    table, nb = R.tables(ctx, 74)
    check_select(F, R.normal(sum(ql), Hq, d, seed=75, std=2.0), boxes(nb, H, d, 76), table, ctx, ql, 9, 2, 1, max_q)


def test_select_equal_scores_take_the_earlier_block(F):
    """All bounds alike; queries of zeros; a few kinds of blocks, each many times; zeros in the bounds."""
    d, H, ctx = 128, 2, [16 * 700, 16 * 90]
    table, nb = R.tables(ctx, 77)
    q = R.normal(2, 4, d, seed=78)
    one = boxes(1, H, d, 79).expand(nb, H, 2, d).contiguous()
    check_select(F, q, one, table, ctx, [1, 1], 33, 3, 1)
    check_select(F, q * 0, boxes(nb, H, d, 80), table, ctx, [1, 1], 33, 3, 1)
    kinds = boxes(3, H, d, 81)[torch.arange(nb) % 3].contiguous()
    check_select(F, q, kinds, table, ctx, [1, 1], 300, 0, 0)
    check_select(F, q, one * 0, table, ctx, [1, 1], 33, 0, 2)


def test_select_scores_that_fp32_cannot_tell_apart(F):
    """Blocks that differ in the last bit of one small channel, beside large ones that nearly cancel."""
    d, H, n = 64, 1, 600
    g = torch.Generator().manual_seed(5)
    mid = torch.randn(d, generator=g).mul(100).bfloat16().float()
    b = mid.expand(n, d).clone()
    b[:, 0] = 2.0 ** -10 * (1 + torch.randint(0, 100, (n,), generator=g) / 128)
    bounds = torch.stack([b, b], 1)[:, None].bfloat16().contiguous()
    q = torch.randn(1, 2, d, generator=g).mul(30).bfloat16()
    q[:, :, 0] = 1.0
    table = torch.randperm(n, generator=g).int()[None]
    check_select(F, q, bounds, table, [16 * n], [1], 100, 1, 1)


def test_select_wide_tables_and_long_contexts(F):
    ctx = [16 * 5000 + 3, 400]  # more blocks than stay in registers
    table, nb = R.tables(ctx, 82, mbps=9000)
    check_select(F, R.normal(2, 2, 64, seed=83, std=2.0), boxes(nb, 1, 64, 84), table, ctx, [1, 1], 257, 16, 4)
    table, nb = R.tables([500], 85)  # every block taken: no scores
    check_select(F, R.normal(3, 2, 64, seed=86), boxes(nb, 1, 64, 87), table, [500], [3], 64, 2, 1)


def test_select_reports_what_is_inconsistent(F):
    ctx, ql = [1000, 1000], [2, 3]
    table, nb = R.tables(ctx, 88)
    q, bounds = R.normal(5, 2, 64, seed=89), boxes(nb, 1, 64, 90)
    sel = torch.full((5, 1, 8), 77, dtype=torch.int32).cuda()
    F.fa_block_select(*cuda(q, bounds, table, R.i32([1000, 2]), R.i32(ql)), 8, sel=sel)  # a chunk longer than its context
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    assert torch.equal(sel[:2].cpu(), R.select(q[:2], bounds, table[:1], [1000], [2], 8, 1, 0)) and bool((sel[2:] == 77).all())
    table[0, 5] = nb + 1
    F.fa_block_select(*cuda(q, bounds, table, R.i32(ctx), R.i32(ql)), 8, sel=sel)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    assert bool(((sel >= 0) & (sel < 63)).all())


def test_select_time_out_is_reported_and_recoverable(F):
    for ql in ([1, 1], [60, 9]):
        table, nb = R.tables([3000, 1000], 94)
        args = cuda(R.normal(sum(ql), 4, 64, seed=95), boxes(nb, 2, 64, 96), table, R.i32([3000, 1000]), R.i32(ql))
        want = F.fa_block_select(*args, 12, max_q_len=max(ql))
        assert F.fa_get_error() == F.FA_OK
        try:
            F.fa_debug_set_wait_limit(1_000_000)
            F.fa_debug_force_timeout(True)
            F.fa_block_select(*args, 12, max_q_len=max(ql))
            assert F.fa_get_error() == F.FA_ERR_TIMEOUT
        finally:
            F.fa_debug_force_timeout(False)
            F.fa_debug_set_wait_limit(4_000_000_000)
        assert torch.equal(F.fa_block_select(*args, 12, max_q_len=max(ql)), want) and F.fa_get_error() == F.FA_OK


def test_select_infinite_and_nan_inputs_end(F):
    ctx = [3000]
    table, nb = R.tables(ctx, 91)
    for bad in (float("inf"), float("nan"), -float("inf")):
        q, bounds = R.normal(1, 2, 64, seed=92), boxes(nb, 1, 64, 93)
        bounds[3:50, 0, 0, 5] = bad
        q[0, 1, 7] = bad
        sel = F.fa_block_select(*cuda(q, bounds, table, R.i32(ctx), R.i32([1])), 40, recent=3, sink=1).cpu()[0, 0]
        assert F.fa_get_error() == F.FA_OK
        assert bool((sel[1:] > sel[:-1]).all()) and sel[0] == 0 and sel[-3:].tolist() == [185, 186, 187]


# --------------------------------------------------------------- attention --
def check_blocks(F, ctx, ql, Hq, H, d, keep, fp8, seed, shuffle=True, sel=None, spread=2):
    table, nb = R.tables(ctx, seed)
    g = torch.Generator().manual_seed(seed)
    if fp8:
        k, v, ke, ve = R.random_cache8(nb, H, d, seed, spread)
    else:
        k, v, ke, ve = R.normal(nb, H, 16, d, seed=seed), R.normal(nb, H, 16, d, seed=seed + 1), None, None
    N = sum(ql)
    q = R.normal(N, Hq, d, seed=seed + 2, std=2.0)
    rows = [(s, p) for s, (c, n) in enumerate(zip(ctx, ql)) for p in range(c - n, c)]
    if sel is None:
        sel = torch.full((N, H, keep), -1, dtype=torch.int32)
        for i, (s, p) in enumerate(rows):
            for h in range(H):
                b = torch.randperm(-(-ctx[s] // 16), generator=g)[:keep].int()  # some behind the position
                b = b if shuffle else b.sort().values
                at = torch.randperm(keep, generator=g)[:len(b)].sort().values if shuffle else torch.arange(len(b))
                sel[i, h, at] = b
    for s, c in enumerate(ctx):  # keys and values behind the last token must not matter
        if c % 16:
            b = int(table[s, c // 16])
            k[b, :, c % 16:] = 0x7F if fp8 else float("nan")
            if fp8:
                v[b, :, :, c % 16:] = 0x7F
            else:
                v[b, :, c % 16:] = float("inf")
    lse = torch.full((N, Hq), 7.0).cuda()
    out = F.fa_paged_attn_blocks(*cuda(q, k, v, table, R.i32(ctx), R.i32(ql), sel), *cuda(ke, ve), lse=lse)
    assert F.fa_get_error() == F.FA_OK
    out, lse = out.cpu(), lse.cpu()
    for i, (s, p) in enumerate(rows):
        for h in range(H):
            b = sel[i, h][sel[i, h] >= 0].long()
            ph = table[s, b].long()
            kk = (R.values(k[ph, h], ke[ph, h]) if fp8 else k[ph, h].double()).reshape(-1, d)
            vv = (R.values(v[ph, h], ve[ph, h], True) if fp8 else v[ph, h].double()).reshape(-1, d)
            see = ((b[:, None] * 16 + torch.arange(16)).reshape(1, -1) <= p).expand(Hq // H, -1)
            hs = slice(h * (Hq // H), (h + 1) * (Hq // H))
            R.Rows(q[i, hs], kk, vv, see, d ** -0.5, R.HALF_F16 if fp8 else R.HALF_BF16).check(out[i, hs], lse[i, hs], f"row {i}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("Hq, H, keep", [(4, 4, 1), (12, 2, 9), (16, 1, 70), (20, 1, 33), (3, 3, 300)])
def test_blocks_single_tokens(F, fp8, d, Hq, H, keep):
    check_blocks(F, [1, 16, 17, 1000, 3333], [1] * 5, Hq, H, d, keep, fp8, 101)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d, Hq, H", [(128, 6, 2), (64, 4, 1)])
def test_blocks_chunks(F, fp8, d, Hq, H):
    check_blocks(F, [50, 300, 16, 129], [50, 40, 0, 7], Hq, H, d, 5, fp8, 102)
    check_blocks(F, [700], [130], Hq, H, d, 40, fp8, 103, shuffle=False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("n, Hq, H", [(550, 3, 1), (275, 20, 1), (325, 4, 2)])
def test_blocks_of_several_hundred_lists(F, fp8, d, n, Hq, H):
    """About as many lists as the GPU takes at once, with three warps each and with two."""
    check_blocks(F, [n + 150], [n], Hq, H, d, 10, fp8, 108)


@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_rows_without_keys(F, fp8):
    """Lists of nothing, and of blocks behind the position only."""
    sel = torch.full((3, 2, 6), -1, dtype=torch.int32)
    sel[1, 0, 3] = 11
    sel[2, 1, :2] = R.i32([1, 0])
    check_blocks(F, [40, 200, 60], [1, 1, 1], 4, 2, 64, 6, fp8, 104, sel=torch.cat([sel[:1], sel[1:]]))
    table, nb = R.tables([200], 105)
    k = R.normal(nb, 1, 16, 64, seed=1)
    lse = torch.zeros(2, 2).cuda()
    sel = R.i32([[[12, 11, -1]], [[12, -7, 0]]])
    k[int(table[0, 11])] = float("nan")
    k[int(table[0, 12])] = float("inf")
    out = F.fa_paged_attn_blocks(*cuda(R.normal(2, 2, 64, seed=2), k, k, table, R.i32([200]), R.i32([2]) * 0 + 2, sel * 1), lse=lse)
    # position 198, 199 lie in block 12: visible; rows of a chunk earlier in the sequence below
    assert not bool(out.isfinite().all()) and F.fa_get_error() == F.FA_OK
    q = R.normal(180, 2, 64, seed=3)
    sel = torch.full((180, 1, 2), 12, dtype=torch.int32)
    sel[:, :, 1] = 11
    lse = torch.zeros(180, 2).cuda()
    out = F.fa_paged_attn_blocks(*cuda(q, k, k, table, R.i32([200]), R.i32([180]), sel), lse=lse)
    assert bool((out[:156] == 0).all()) and bool((lse[:156] == -float("inf")).all())  # positions 20 .. 175
    assert F.fa_get_error() == F.FA_OK


def test_blocks_errors_are_reported(F):
    table, nb = R.tables([100, 100], 106)
    k, q = R.normal(nb, 1, 16, 64, seed=1), R.normal(2, 2, 64, seed=2)
    sel = R.i32([[[0, 3]], [[6, 7]]])  # 7 lies behind the last block
    args = cuda(q, k, k, table, R.i32([100, 100]), R.i32([1, 1]))
    ok = F.fa_paged_attn_blocks(*args, R.i32([[[0, 3]], [[6, -1]]]).cuda())
    assert F.fa_get_error() == F.FA_OK
    got = F.fa_paged_attn_blocks(*args, sel.cuda())
    assert F.fa_get_error() == F.FA_ERR_BOUNDS and torch.equal(got, ok)
    table[1, 6] = nb
    out = torch.full_like(q, 5.0).cuda()
    F.fa_paged_attn_blocks(*args[:3], *cuda(table, R.i32([100, 100]), R.i32([1, 1]), sel), out=out)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS and torch.equal(out[0], ok[0])
    F.fa_paged_attn_blocks(*args[:4], *cuda(R.i32([100, 0]), R.i32([1, 1]), sel), out=out.fill_(5.0))
    assert F.fa_get_error() == F.FA_ERR_BOUNDS and torch.equal(out[0], ok[0]) and bool((out[1] == 5.0).all())


def test_blocks_time_out_is_reported_and_recoverable(F):
    for S, keep in ((1, 64), (30, 4)):  # clusters, and single CTAs
        table, nb = R.tables([1500] * S, 107)
        k = R.normal(nb, 2, 16, 128, seed=1)
        sel = torch.arange(keep).int().expand(S, 2, keep).contiguous()
        args = cuda(R.normal(S, 4, 128, seed=2), k, k, table, R.i32([1500] * S), R.i32([1] * S), sel)
        want = F.fa_paged_attn_blocks(*args)
        try:
            F.fa_debug_set_wait_limit(1_000_000)
            F.fa_debug_force_timeout(True)
            F.fa_paged_attn_blocks(*args)
            assert F.fa_get_error() == F.FA_ERR_TIMEOUT
        finally:
            F.fa_debug_force_timeout(False)
            F.fa_debug_set_wait_limit(4_000_000_000)
        assert torch.equal(F.fa_paged_attn_blocks(*args), want) and F.fa_get_error() == F.FA_OK


def test_offsets_past_32_bits(F):
    """Caches, bounds and scores whose elements need more than 32 bits to number; the sequence's blocks at both ends."""
    d, H, nb = 128, 8, 270_000  # 2^32 bf16 elements in 262144 blocks
    kc = torch.empty(nb, H, 16, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    bounds = torch.empty(nb, H, 2, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.cat([torch.arange(30), torch.arange(nb - 30, nb)])[torch.randperm(60, generator=torch.Generator().manual_seed(1))]
    k, v = R.normal(60, H, 16, d, seed=2), R.normal(60, H, 16, d, seed=3)
    kc[ids.cuda()], vc[ids.cuda()] = k.cuda(), v.cuda()
    table, c = ids.int()[None], 16 * 60 - 5
    q = R.normal(1, 16, d, seed=4, std=2.0)
    at = cuda(table, R.i32([c]), R.i32([c]))
    F.fa_block_bounds(kc, *at, bounds, total_q=c)
    one = cuda(table, R.i32([c]), R.i32([1]))
    sel = F.fa_block_select(q.cuda(), bounds, *one, 20, recent=2, sink=1)
    out = F.fa_paged_attn_blocks(q.cuda(), kc, vc, *one, sel)
    assert F.fa_get_error() == F.FA_OK
    want = torch.stack([k[:, :, :, :].amin(2), k.amax(2)], 2)
    want[59] = torch.stack([k[59, :, :11].amin(1), k[59, :, :11].amax(1)], 1)
    assert torch.equal(bounds[ids.cuda()].cpu(), want)
    full = torch.arange(60).int()[None]
    pick = R.select(q, want, full, [c], [1], 20, 1 + 1, 1)
    assert torch.equal(sel.cpu(), pick)
    for h in range(H):
        b = pick[0, h].long()
        see = ((b[:, None] * 16 + torch.arange(16)).reshape(1, -1) < c).expand(2, -1)
        R.Rows(q[0, 2 * h:2 * h + 2], k[b, h].double().reshape(-1, d), v[b, h].double().reshape(-1, d), see, d ** -0.5,
               R.HALF_BF16).check(out.cpu()[0, 2 * h:2 * h + 2], what=f"head {h}")


def test_two_streams_and_equal_bits(F):
    """Calls side by side on two streams, each with memory of its own, give what they give alone."""
    d, H, Hq, S = 128, 2, 8, 40
    lens = [500 + 37 * i for i in range(S)]
    table, nb = R.tables(lens, 108)
    k, v, ke, ve = R.random_cache8(nb, H, d, 108, 2)
    bounds, q = boxes(nb, H, d, 109), R.normal(S, Hq, d, seed=110)
    args = cuda(q, k, v, ke, ve, bounds, table, R.i32(lens), R.i32([1] * S))

    def step(stream=None):
        q, k, v, ke, ve, bounds, *at = args
        sel = F.fa_block_select(q, bounds, *at, 16, recent=2, max_q_len=1, stream=stream)
        return sel, F.fa_paged_attn_blocks(q, k, v, *at, sel, k_exp=ke, v_exp=ve, stream=stream), \
            F.fa_paged_attn_fp8_scaled(q, k, v, ke, ve, *at, max_q_len=1, stream=stream)
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [step(s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want)) and F.fa_get_error() == F.FA_OK


# ------------------------------------------------------------ as a user would --
def test_a_sequence_grows_and_is_read_by_its_blocks(F):
    """A pool's sequences in the 8-bit cache: prompt, then tokens; append, bounds, select, attention.  With every block
    chosen the attention is that over the whole cache, with fewer that over those blocks; a graph replays the step."""
    d, H, Hq, S, steps = 64, 2, 6, 3, 20
    pool = F.BlockPool(80, 24)
    seqs = [pool.add_seq() for _ in range(S)]
    kc, vc = torch.zeros(80, H, 16, d, dtype=torch.uint8).cuda(), torch.zeros(80, H, d, 16, dtype=torch.uint8).cuda()
    ke, ve = torch.zeros(80, H, dtype=torch.uint8).cuda(), torch.zeros(80, H, dtype=torch.uint8).cuda()
    bounds = torch.zeros(80, H, 2, d, dtype=torch.bfloat16).cuda()
    ang = torch.arange(400, dtype=torch.float64)[:, None] * torch.exp(-9.0 * torch.arange(d // 2, dtype=torch.float64) / (d // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    host = [t.cpu().clone() for t in (kc, vc, ke, ve)]
    N = None
    for step in range(steps):
        ql = [200, 37, 90] if step == 0 else [1] * S
        for s, n in zip(seqs, ql):
            pool.append(s, n)
        table, lens = (torch.from_numpy(x) for x in pool.tables(seqs))
        N = sum(ql)
        q, k, v = (R.normal(N, h, d, seed=1000 * step + i) for i, h in enumerate((Hq, H, H)))
        k[..., :4] *= 1 + step  # the scales of a block grow
        at = cuda(table, lens, R.i32(ql))
        qr = F.fa_cache_append_fp8_scaled(*cuda(k, v), kc, vc, ke, ve, *at, q=q.cuda(), cos_sin=cs)
        F.fa_block_bounds(kc, *at, bounds, k_exp=ke, total_q=N)
        everything = F.fa_block_select(qr, bounds, *at, 24, max_q_len=max(ql))
        full = F.fa_paged_attn_fp8_scaled(qr, kc, vc, ke, ve, *at, max_q_len=max(ql))
        some = F.fa_block_select(qr, bounds, *at, 5, recent=2, sink=1, max_q_len=max(ql))
        got = [F.fa_paged_attn_blocks(qr, kc, vc, *at, sel, k_exp=ke, v_exp=ve) for sel in (everything, some)]
        assert F.fa_get_error() == F.FA_OK
        pos = torch.cat([torch.arange(int(c) - n, int(c)) for c, n in zip(lens, ql)])
        R.append(*host, R.turn(k, cs.cpu(), pos), v.double(), table, lens.tolist(), ql)
        assert torch.equal(ke.cpu(), host[2]) and torch.equal(ve.cpu(), host[3]) and torch.equal(vc.cpu(), host[1])
        want = R.select(qr.cpu(), bounds.cpu(), table, lens.tolist(), ql, 5, 2, 1)
        assert torch.equal(some.cpu(), want)
        i = 0
        for s, n in enumerate(ql):
            c = int(lens[s])
            ph = table[s, :-(-c // 16)].long()
            for h in range(Hq):
                kk = R.values(kc.cpu()[ph, h // 3], ke.cpu()[ph, h // 3]).reshape(-1, d)[:c]
                vv = R.values(vc.cpu()[ph, h // 3], ve.cpu()[ph, h // 3], True).reshape(-1, d)[:c]
                see = torch.arange(c)[None] <= torch.arange(c - n, c)[:, None]
                x = qr.cpu()[i:i + n, h]
                rows = R.Rows(x, kk, vv, see, d ** -0.5, R.HALF_F16)
                rows.check(full.cpu()[i:i + n, h], what="whole cache")
                rows.check(got[0].cpu()[i:i + n, h], what="every block")
                listed = torch.zeros(n, -(-c // 16), dtype=torch.bool)
                for r in range(n):
                    b = want[i + r, h // 3]
                    listed[r, b[b >= 0].long()] = True
                few = see & listed.repeat_interleave(16, 1)[:, :c]
                R.Rows(x, kk, vv, few, d ** -0.5, R.HALF_F16).check(got[1].cpu()[i:i + n, h], what="some blocks")
            i += n
    # the step as a graph: same bits, on a stream of its own
    out, sel, q_out = torch.empty_like(qr), torch.empty_like(some), torch.empty_like(qr)
    ws = torch.empty(F.fa_block_select_workspace_size(S, 24, Hq, H, d, N), dtype=torch.uint8, device="cuda")
    args, at = cuda(k, v, q), cuda(table, lens, R.i32(ql))

    def run():
        F.fa_cache_append_fp8_scaled(args[0], args[1], kc, vc, ke, ve, *at, q=args[2], cos_sin=cs, q_out=q_out)
        F.fa_block_bounds(kc, *at, bounds, k_exp=ke, total_q=N)
        F.fa_block_select(q_out, bounds, *at, 5, recent=2, sink=1, sel=sel, max_q_len=1, ws=ws)
        F.fa_paged_attn_blocks(q_out, kc, vc, *at, sel, k_exp=ke, v_exp=ve, out=out)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    out.zero_(), sel.zero_(), q_out.zero_()
    graph.replay()
    assert F.fa_get_error() == F.FA_OK
    assert torch.equal(out, got[1]) and torch.equal(sel, some) and torch.equal(q_out, qr)
