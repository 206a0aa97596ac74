"""The 8-bit cache with block scales: the append's codes, and attention over them against 64 bits."""
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


# ------------------------------------------------------------------ append --
def setup(ctx, ql, H, d, seed, dtype=torch.bfloat16, spread=0):
    table, nb = R.tables(ctx, seed)
    cache = R.random_cache8(nb, H, d, seed, spread)
    N = sum(ql)
    k, v = R.normal(N, H, d, seed=seed + 1, dtype=dtype), R.normal(N, H, d, seed=seed + 2, dtype=dtype)
    return table, nb, cache, k, v


def same_bytes(got, want, what):
    got = got.cpu()
    assert torch.equal(got, want), f"{what}: {int((got != want).sum())} of {want.numel()} bytes differ"


@pytest.mark.parametrize("d, H, dtype", [(128, 2, torch.bfloat16), (64, 3, torch.bfloat16), (128, 1, torch.float32),
                                         (64, 2, torch.float32)])
@pytest.mark.parametrize("ctx, ql", [([1], [1]), ([16, 17, 33, 5], [1, 1, 1, 1]), ([40, 16, 70, 31], [25, 16, 3, 15]),
                                     ([100, 7, 64], [0, 7, 64]), ([300], [299])])
def test_append_codes_are_exact(F, d, H, dtype, ctx, ql):
    table, nb, cache, k, v = setup(ctx, ql, H, d, 11, dtype, spread=3)
    got = cuda(*cache)
    want = [t.clone() for t in cache]
    R.append(*want[:2], *want[2:], k.double(), v.double(), table, ctx, ql)
    F.fa_cache_append_fp8_scaled(*cuda(k, v), *got, *cuda(table, R.i32(ctx), R.i32(ql)))
    assert F.fa_get_error() == F.FA_OK
    for a, b, n in zip(got, want, ("k_cache", "v_cache", "k_exp", "v_exp")):
        same_bytes(a, b, n)


def test_scales_grow_and_stay(F):
    """Token by token into one block: magnitudes that rise, fall, are 0, at borders of the scale, not finite."""
    d, H = 64, 1
    rows = [0.0, 1e-30, 448.0 * 2.0 ** -40, 1e-3, 448.0 * 2.0 ** -7, 449.0 * 2.0 ** -7, 2.0, 1e4, 3e38, 1.0, float("inf"),
            float("nan"), -float("inf"), 0.0, -3e38, 5.0]
    x = torch.zeros(16, H, d)
    for i, a in enumerate(rows):
        x[i] = torch.linspace(-1, 1, d) * a if abs(a) < 1e39 else torch.linspace(-1, 1, d)
        x[i, 0, 3] = a
    table, nb = R.i32([[2]]), 4
    cache = R.random_cache8(nb, H, d, 5)
    got, want = cuda(*cache), [t.clone() for t in cache]
    for i in range(16):
        row = x[i:i + 1]
        R.append(*want, row.double(), row.double(), table, [i + 1], [1])
        F.fa_cache_append_fp8_scaled(*cuda(row, row), *got, *cuda(table, R.i32([i + 1]), R.i32([1])))
        for a, b, n in zip(got, want, ("k_cache", "v_cache", "k_exp", "v_exp")):
            same_bytes(a, b, f"{n} after token {i}")
    assert F.fa_get_error() == F.FA_OK


@pytest.mark.parametrize("d, Hq, H, dtype, given", [(128, 6, 2, torch.bfloat16, False), (64, 4, 4, torch.float32, True),
                                                    (128, 8, 1, torch.float32, False), (64, 20, 1, torch.bfloat16, True)])
def test_append_turns_keys_and_queries(F, d, Hq, H, dtype, given):
    ctx, ql = [40, 16, 200, 31, 9], [25, 1, 150, 15, 0]
    table, nb, cache, k, v = setup(ctx, ql, H, d, 21, dtype)
    N = sum(ql)
    q = R.normal(N, Hq, d, seed=24, dtype=dtype)
    ang = torch.arange(256, dtype=torch.float64)[:, None] * torch.exp(-9.0 * torch.arange(d // 2, dtype=torch.float64) / (d // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.cat([torch.arange(c - n, c) for c, n in zip(ctx, ql)])
    if given:
        pos = torch.randint(0, 256, (N,), generator=torch.Generator().manual_seed(3))
    k64, q64 = R.turn(k, cs, pos), R.turn(q, cs, pos)
    want = [t.clone() for t in cache]
    R.append(*want, k64, v.double(), table, ctx, ql)
    got = cuda(*cache)
    q_out = F.fa_cache_append_fp8_scaled(*cuda(k, v), *got, *cuda(table, R.i32(ctx), R.i32(ql)), q=q.cuda(), cos_sin=cs.cuda(),
                                         positions=pos.int().cuda() if given else None)
    assert F.fa_get_error() == F.FA_OK
    for i, n in ((1, "v_cache"), (2, "k_exp"), (3, "v_exp")):
        same_bytes(got[i], want[i], n)
    # a turned value is two fp32 products and a sum: 2^-22 of their magnitudes off, at most; bf16 then rounds it
    h = d // 2
    mag = (q.double().abs() + torch.cat([q[..., h:], q[..., :h]], -1).double().abs())
    err = (q_out.cpu().double() - q64).abs()
    assert bool((err <= R.HALF_BF16 * q64.abs() + 2.0 ** -21 * mag).all())
    # codes: the nearest one, or, within that error of the border, its neighbour
    a, b = R.values(got[0].cpu(), want[2]), R.values(want[0], want[2])
    near = (got[0].cpu() != want[0])
    assert float(near.double().mean()) < 1e-3
    true = torch.zeros_like(a)
    slot = 0
    for s, (c, n) in enumerate(zip(ctx, ql)):
        for p in range(c - n, c):
            true[int(table[s, p // 16]), :, p % 16] = k64[slot]
            slot += 1
    slack = 2.0 ** -20 * float(k.abs().max()) * 2
    assert bool(((a - true).abs() <= (b - true).abs() + slack)[near].all())


def test_append_skips_what_is_inconsistent(F):
    """Lengths and blocks that do not fit are reported and skipped, the other sequences written."""
    d, H = 128, 2
    ctx, ql = [20, 30, 40], [5, 30, 8]
    table, nb, cache, k, v = setup(ctx, ql, H, d, 31)
    table[1, 0] = nb + 7  # outside the pool
    bad_ctx = [20, 30, 4]  # shorter than its chunk
    want = [t.clone() for t in cache]
    R.append(*want, k.double(), v.double(), table[:1], ctx[:1], ql[:1])
    i = int(table[1, 1])
    part = [t.clone() for t in cache]
    t1 = table[1:2].clone()
    t1[0, 0] = nb - 1 if int(table[1, 1]) != nb - 1 else nb - 2
    R.append(*part, k[5:].double(), v[5:].double(), t1, ctx[1:2], ql[1:2])
    for w, p in zip(want, part):
        w[i] = p[i]  # the second block of sequence 1 is in order
    got = cuda(*cache)
    F.fa_cache_append_fp8_scaled(*cuda(k, v), *got, *cuda(table, R.i32(bad_ctx), R.i32(ql)))
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    for a, b in zip(got, want):
        same_bytes(a, b, "cache")
    # more rows than the call says: nothing is read past them
    got = cuda(*cache)
    F.fa_cache_append_fp8_scaled(*cuda(k[:10], v[:10]), *got, *cuda(table[:1], R.i32([20]), R.i32([11])))
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    for a, b in zip(got, cache):
        same_bytes(a, b, "untouched")
    F.fa_cache_append_fp8_scaled(*cuda(k[:3], v[:3]), *got, *cuda(table[:2], R.i32([20, 9]), R.i32([-5, 8])))
    assert F.fa_get_error() == F.FA_ERR_BOUNDS


# --------------------------------------------------------------- attention --
def check_attention(F, ctx, ql, Hq, H, d, seed, causal=True, spread=2, q_std=2.0, mbps=None, stale_nan=True, cache=None,
                    scale=None, max_q=None):
    table, nb = R.tables(ctx, seed, mbps=mbps)
    k, v, ke, ve = cache or R.random_cache8(nb, H, d, seed, spread)
    if stale_nan:  # behind the last token of every sequence
        for s, c in enumerate(ctx):
            if c % 16:
                b = int(table[s, c // 16])
                k[b, :, c % 16:] = 0x7F
                v[b, :, :, c % 16:] = 0x7F
    N = sum(ql)
    q = R.normal(N, Hq, d, seed=seed + 9, std=q_std)
    scale = scale or d ** -0.5 / max(1e-30, q_std / 2)
    lse = torch.full((N, Hq), 7.0).cuda()
    out = F.fa_paged_attn_fp8_scaled(*cuda(q, k, v, ke, ve, table, R.i32(ctx), R.i32(ql)), causal=causal, scale=scale, lse=lse,
                                     max_q_len=max(ql) if max_q is None else max_q)
    assert F.fa_get_error() == F.FA_OK
    out, lse = out.cpu(), lse.cpu()
    at, g = 0, Hq // H
    for s, (c, n) in enumerate(zip(ctx, ql)):
        p = table[s, :-(-c // 16)].long()
        see = torch.arange(c)[None] <= (torch.arange(c - n, c) if causal else torch.full((n,), c))[:, None]
        for h in range(Hq):
            kk = R.values(k[p, h // g], ke[p, h // g]).reshape(-1, d)[:c]
            vv = R.values(v[p, h // g], ve[p, h // g], True).reshape(-1, d)[:c]
            R.Rows(q[at:at + n, h], kk, vv, see, scale, R.HALF_F16).check(out[at:at + n, h], lse[at:at + n, h], f"seq {s} head {h}")
        at += n


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("Hq, H", [(4, 4), (12, 2), (16, 1), (5, 1)])
def test_single_tokens(F, d, Hq, H):
    check_attention(F, [1, 16, 17, 100, 1000, 33], [1] * 6, Hq, H, d, 41)


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("Hq, H, ql", [(2, 1, [3, 8, 1]), (6, 2, [2, 5, 1]), (1, 1, [16, 3, 7]), (4, 2, [0, 4, 1])])
def test_few_tokens(F, d, Hq, H, ql):
    check_attention(F, [40, 555, 16], ql, Hq, H, d, 42)


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("Hq, H", [(8, 2), (3, 1), (12, 2), (16, 1), (20, 1), (7, 7)])
def test_chunks(F, d, Hq, H):
    check_attention(F, [300, 64, 129, 700, 40], [299, 64, 100, 37, 1], Hq, H, d, 43)


@pytest.mark.parametrize("d, Hq, H, ctx, ql", [(128, 8, 2, [5000, 3], [70, 3]), (64, 4, 1, [9000], [128]),
                                               (128, 32, 8, [2500, 17, 100], [33, 17, 1])])
def test_few_queries_over_long_contexts(F, d, Hq, H, ctx, ql):
    check_attention(F, ctx, ql, Hq, H, d, 44)


def test_all_keys_visible(F):
    check_attention(F, [300, 64, 40], [200, 3, 1], 4, 2, 128, 45, causal=False)
    check_attention(F, [300, 64, 40], [2, 3, 1], 4, 2, 64, 46, causal=False)


@pytest.mark.parametrize("ctx, ql", [([200, 77], [1, 1]), ([200, 77], [120, 40])])
def test_scales_far_apart(F, ctx, ql):
    """Blocks whose scales differ by 2^50, and whole blocks of zeros with the smallest scale (their weights count)."""
    d, H = 128, 2
    table, nb = R.tables(ctx, 47)
    k, v, ke, ve = R.random_cache8(nb, H, d, 47, 0)
    ve = (127 + torch.randint(-25, 26, (nb, H), generator=torch.Generator().manual_seed(1))).to(torch.uint8)
    v[::3] = 0
    ve[::3] = R.LEAST
    check_attention(F, ctx, ql, 4, H, d, 47, cache=(k, v, ke, ve), stale_nan=False)


@pytest.mark.parametrize("std", [1e-30, 1e-6, 3e4, 1e30])
def test_queries_of_any_magnitude(F, std):
    check_attention(F, [200, 77], [1, 1], 4, 2, 128, 48, q_std=std)
    check_attention(F, [200, 77], [100, 40], 4, 2, 64, 49, q_std=std)


def test_many_sequences_short_and_wide_table(F):
    g = torch.Generator().manual_seed(2)
    ctx = torch.randint(1, 40, (300,), generator=g).tolist()
    check_attention(F, ctx, [1] * 300, 4, 2, 64, 50, mbps=700)
    check_attention(F, [30, 2, 500], [1, 2, 1], 4, 2, 128, 51, mbps=3001)


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("S, Hq, H, longest", [(1, 8, 8, 900), (1, 4, 1, 4000), (3, 40, 2, 2000), (12, 8, 4, 2000), (40, 16, 8, 1000),
                                               (60, 8, 8, 700), (40, 4, 2, 4090)])
def test_single_tokens_of_all_batch_sizes(F, d, S, Hq, H, longest):
    """Batches that take clusters, single CTAs of four and of two warps, and the stream."""
    g = torch.Generator().manual_seed(S)
    ctx = [longest] + torch.randint(1, longest + 1, (S - 1,), generator=g).tolist()
    check_attention(F, ctx, [1] * S, Hq, H, d, 53)


def test_single_tokens_and_sequences_without_queries(F):
    check_attention(F, [100, 0, 64, 900], [1, 0, 0, 1], 4, 2, 128, 54, max_q=1)


def test_long_streams_per_warp(F):
    """More pages to a warp than it looks up at a time."""
    check_attention(F, [20000, 15001, 30000], [1, 1, 1], 4, 4, 64, 52, stale_nan=True)


def test_a_bound_below_a_chunk_is_reported(F):
    for bound, wide in ((2, None), (1, None), (1, 3000)):
        table, nb = R.tables([50, 60], 3, mbps=wide)
        k, v, ke, ve = R.random_cache8(nb, 2, 64, 3)
        q = R.normal(6, 4, 64, seed=1)
        F.fa_paged_attn_fp8_scaled(*cuda(q, k, v, ke, ve, table, R.i32([50, 60]), R.i32([1, 5])), max_q_len=bound)
        assert F.fa_get_error() == F.FA_ERR_BOUNDS


def test_bad_blocks_are_reported(F):
    for ql in ([1, 1], [40, 60]):
        table, nb = R.tables([50, 600], 3)
        k, v, ke, ve = R.random_cache8(nb, 2, 64, 3)
        table[1, 20] = nb
        q = R.normal(sum(ql), 4, 64, seed=1)
        F.fa_paged_attn_fp8_scaled(*cuda(q, k, v, ke, ve, table, R.i32([50, 600]), R.i32(ql)), max_q_len=max(ql))
        assert F.fa_get_error() == F.FA_ERR_BOUNDS
        table[1, 20] = -5
        F.fa_paged_attn_fp8_scaled(*cuda(q, k, v, ke, ve, table, R.i32([50, 600]), R.i32(ql)), max_q_len=max(ql))
        assert F.fa_get_error() == F.FA_ERR_BOUNDS


def test_time_outs_are_reported_and_recoverable(F):
    for ql in ([1, 1], [40, 60]):
        table, nb = R.tables([50, 600], 3)
        k, v, ke, ve = R.random_cache8(nb, 2, 128, 3)
        args = cuda(R.normal(sum(ql), 4, 128, seed=1), k, v, ke, ve, table, R.i32([50, 600]), R.i32(ql))
        want = F.fa_paged_attn_fp8_scaled(*args, max_q_len=max(ql))
        assert F.fa_get_error() == F.FA_OK
        try:
            F.fa_debug_set_wait_limit(1_000_000)
            F.fa_debug_force_timeout(True)
            F.fa_paged_attn_fp8_scaled(*args, max_q_len=max(ql))
            assert F.fa_get_error() == F.FA_ERR_TIMEOUT
        finally:
            F.fa_debug_force_timeout(False)
            F.fa_debug_set_wait_limit(4_000_000_000)
        assert torch.equal(F.fa_paged_attn_fp8_scaled(*args, max_q_len=max(ql)), want)
        assert F.fa_get_error() == F.FA_OK


def test_a_workspace_for_larger_sizes_serves_smaller_ones(F):
    """One workspace, several shapes after one another, and two graphs that share it when replayed in turn."""
    d, H, Hq = 64, 2, 8
    ws = torch.empty(F.fa_paged_attn_fp8_scaled_workspace_size(6, 200, Hq, H, d, 700, 300), dtype=torch.uint8, device="cuda").fill_(0xFF)
    runs = []
    for i, (ctx, ql) in enumerate([([3000], [40]), ([100, 900, 33], [1, 300, 2]), ([50] * 6, [1] * 6)]):
        table, nb = R.tables(ctx, 120 + i)
        args = cuda(R.normal(sum(ql), Hq, d, seed=i), *R.random_cache8(nb, H, d, i), table, R.i32(ctx), R.i32(ql))
        want = F.fa_paged_attn_fp8_scaled(*args, max_q_len=max(ql))
        assert torch.equal(F.fa_paged_attn_fp8_scaled(*args, max_q_len=max(ql), ws=ws), want)
        runs.append((args, max(ql), want))
    graphs = []
    for args, m, want in runs:
        out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            F.fa_paged_attn_fp8_scaled(*args, max_q_len=m, ws=ws, out=out)
        graphs.append((graph, out, want))
    for _ in range(3):
        for graph, out, want in graphs:
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    assert F.fa_get_error() == F.FA_OK


def test_large_pool_offsets(F):
    """A pool whose bytes need more than 32 bits to number, the sequence's blocks at both ends of it."""
    d, H, nb = 128, 8, 270_000  # 2^32 bytes in 262144 blocks
    kc = torch.empty(nb, H, 16, d, dtype=torch.uint8, device="cuda")
    vc = torch.empty(nb, H, d, 16, dtype=torch.uint8, device="cuda")
    ke, ve = (torch.zeros(nb, H, dtype=torch.uint8, device="cuda") for _ in range(2))
    ids = torch.cat([torch.arange(10), torch.arange(nb - 10, nb)])[torch.randperm(20, generator=torch.Generator().manual_seed(1))]
    c = 20 * 16 - 3
    k, v = R.normal(c, H, d, seed=2), R.normal(c, H, d, seed=3)
    at = cuda(ids.int()[None], R.i32([c]), R.i32([c]))
    F.fa_cache_append_fp8_scaled(*cuda(k, v), kc, vc, ke, ve, *at)
    small = [torch.zeros(20, H, 16, d, dtype=torch.uint8), torch.zeros(20, H, d, 16, dtype=torch.uint8),
             torch.zeros(20, H, dtype=torch.uint8), torch.zeros(20, H, dtype=torch.uint8)]
    R.append(*small, k.double(), v.double(), torch.arange(20)[None], [c], [c])
    for got, want in zip((kc, vc, ke, ve), small):
        got = got[ids.cuda()].cpu()
        if want.dim() == 4:  # the last block's slots behind the last token are not written
            part = (slice(None), slice(None), slice(0, 13)) if want.shape[2] == 16 else (slice(None), slice(None), slice(None), slice(0, 13))
            assert torch.equal(got[:19], want[:19]) and torch.equal(got[19:][part], want[19:][part])
        else:
            assert torch.equal(got, want)
    for n in (1, 100):
        q = R.normal(n, 16, d, seed=4, std=2.0)
        out = F.fa_paged_attn_fp8_scaled(q.cuda(), kc, vc, ke, ve, *cuda(ids.int()[None], R.i32([c]), R.i32([n])), max_q_len=n)
        assert F.fa_get_error() == F.FA_OK
        see = torch.arange(c)[None] <= torch.arange(c - n, c)[:, None]
        for h in range(16):
            kk = R.values(small[0][:, h // 2], small[2][:, h // 2]).reshape(-1, d)[:c]
            vv = R.values(small[1][:, h // 2], small[3][:, h // 2], True).reshape(-1, d)[:c]
            R.Rows(q[:, h], kk, vv, see, d ** -0.5, R.HALF_F16).check(out.cpu()[:, h], what=f"head {h}")
