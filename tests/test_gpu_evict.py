"""Accumulated attention weights and the eviction that goes by them, and a
serving loop over all of it: append, attend, count, evict, go on."""
import math

import numpy as np
import pytest
import torch

import mod_ref as R
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


def run_accum(F, p, decay=1.0, give=True, inplace=False, causal=True, cap=0.0, bias=False, window=0, prefix=None,
              seed=0):
    sl = R.slopes(p.Hq) if bias else None
    q, kc, vc, table, ctx, ql = p.cuda()
    S, n = len(p.ctx), max(p.ctx) + 5
    acc = torch.rand(S, p.Hkv, n, generator=torch.Generator().manual_seed(seed)) * 3
    a_in = acc.cuda() if give else None
    a_out = a_in if inplace else torch.full((S, p.Hkv, n), 9.0, device="cuda")
    before = a_out.cpu().clone()
    lse = torch.empty(p.total, p.Hq, device="cuda")
    kw = dict(causal=causal, softcap=cap, alibi_slopes=None if sl is None else sl.cuda(), window=window,
              prefix_lens=None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda(),
              max_q_len=max(p.ql))
    out = F.fa_paged_attn_accum(q, kc, vc, table, ctx, ql, a_in, a_out, decay=decay, lse=lse, **kw)
    assert F.fa_get_error() == F.FA_OK
    # the attention is the call's without sums
    lse2 = torch.empty_like(lse)
    assert torch.equal(out, F.fa_paged_attn_mod(q, kc, vc, table, ctx, ql, lse=lse2, **kw)) and torch.equal(lse, lse2)
    g = p.Hq // p.Hkv
    want = torch.zeros(S, p.Hkv, n, dtype=torch.float64)
    tol = torch.zeros_like(want)
    for s, c in enumerate(p.ctx):
        old = c - p.ql[s]
        if give:
            want[s, :, :old] = decay * acc[s, :, :old].double()
    tol += 4 * R.F32 * want.abs()
    for s, h, at, ref in p.rows(causal, cap, sl, window, prefix):
        c = p.ctx[s]
        want[s, h // g, :c] += ref.w.sum(0)
        # each weight's relative error, and one fp32 rounding of at most sum-of-the-rest per add
        tol[s, h // g, :c] += ((ref.w_rel + (p.ql[s] * g + 4) * R.F32)[:, None] * ref.w).sum(0) + 1e-30
    for s, c in enumerate(p.ctx):
        want[s, :, c:] = before[s, :, c:].double()  # behind the context: left as it was
    R.check(a_out, want, tol, "acc")
    return a_out


CTX = [1, 16, 17, 200, 333, 4, 130, 512]


@pytest.mark.parametrize("mod", [dict(), dict(cap=30.0), dict(bias=True), dict(window=37), dict(window=1),
                                 dict(bias=True, cap=25.0, window=100), dict(causal=False, window=90),
                                 dict(prefix=[0, 40, 300, 5, 1000, 0, 17, 2])], ids=str)
@pytest.mark.parametrize("kind", ["decode", "few", "chunk", "mixed"])
@pytest.mark.parametrize("heads", [(6, 2, 128), (4, 4, 64), (3, 1, 64), (16, 2, 128)], ids=str)
def test_accum(F, heads, kind, mod):
    ql = {"decode": [1] * 8, "few": [1, 2, 1, 2, 0, 1, 2, 2], "chunk": [1, 16, 17, 150, 300, 4, 33, 129],
          "mixed": [1, 1, 0, 40, 1, 2, 130, 200]}[kind]
    p = R.Paged(17, CTX, ql, *heads, std=4.0 if mod.get("cap") else 1.0,
                window=mod.get("window", 0))
    run_accum(F, p, decay=0.75, **mod)


@pytest.mark.parametrize("ql", [[1, 1], [1, 40], [300, 2]], ids=str)
def test_accum_in_place_and_from_nothing(F, ql):
    p = R.Paged(18, [77, 400] if ql[0] == 1 else [400, 77], ql, 8, 2, 64)
    run_accum(F, p, inplace=True)
    run_accum(F, p, give=False)
    run_accum(F, p, decay=0.0)


def test_accum_wide_group(F):
    run_accum(F, R.Paged(19, [5, 140, 33], [1, 3, 33], 20, 1, 64), bias=True)


def test_accum_weights_sum_to_queries(F):
    """The new weights of a sequence sum to (queries x heads); twice the same call gives the same bits."""
    p = R.Paged(20, [600, 5000], [200, 1], 8, 2, 128)
    a = run_accum(F, p, give=False)
    assert torch.equal(a, run_accum(F, p, give=False))
    for s, c in enumerate(p.ctx):
        got = a[s, :, :c].double().sum(1).cpu()
        assert (got - 4 * p.ql[s]).abs().max() <= 1e-4 * 4 * p.ql[s]


def test_accum_reports_short_rows(F):
    p = R.Paged(21, [100, 50], [1, 40], 4, 2, 64)
    q, kc, vc, table, ctx, ql = p.cuda()
    acc = torch.full((2, 2, 60), 5.0, device="cuda")
    F.fa_paged_attn_accum(q, kc, vc, table, ctx, ql, acc, acc, max_q_len=40)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    assert (acc[0] == 5.0).all()          # too short for sequence 0: not written
    assert (acc[1, :, 50:] == 5.0).all()  # sequence 1 fits
    p = R.Paged(21, [50, 100], [1, 40], 4, 2, 64)  # the other way round: the chunk's row is too short
    q, kc, vc, table, ctx, ql = p.cuda()
    acc = torch.full((2, 2, 60), 5.0, device="cuda")
    F.fa_paged_attn_accum(q, kc, vc, table, ctx, ql, acc, acc, max_q_len=40)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    assert (acc[1] == 5.0).all() and not (acc[0, :, :50] == 5.0).any()


def test_accum_wide_tables(F):
    """Tables and rows far wider than the contexts; one sequence ends where a unit of 256 keys does."""
    p = R.Paged(22, [256, 40, 513, 100], [20, 1, 300, 2], 8, 2, 64)
    p.table = torch.cat([p.table, torch.full((4, 3000), -1, dtype=torch.int32)], 1)
    run_accum(F, p, bias=True)


def test_accum_chunks_over_long_contexts(F):
    """The sums go by the log-sum-exp that the pieces' join writes."""
    p = R.Paged(44, [3500, 60, 1800], [50, 1, 100], 8, 2, 128)
    run_accum(F, p, decay=0.5)
    run_accum(F, p, bias=True, prefix=[3480, 60, 500])


def test_accum_many_sequences(F):
    """More sequences than a warp, of all kinds, so that places and units run over many of them."""
    n = 70
    ctx = [(37 * i) % 300 + 1 for i in range(n)]
    ql = [min(c, [0, 1, 2, 9, 33][i % 5]) for i, c in enumerate(ctx)]
    run_accum(F, R.Paged(23, ctx, ql, 4, 2, 64), window=50)


@pytest.mark.parametrize("cap, std", [(1e4, 3.0), (300.0, 40.0), (60.0, 8.0), (40.0, 12.0), (30.0, 30.0), (2.0, 20.0)])
def test_accum_caps_of_all_sizes(F, cap, std):
    run_accum(F, R.Paged(25, [300, 200, 77], [200, 9, 1], 4, 2, 64, std=std), cap=cap)


def test_accum_long_chunk(F):
    """One long chunk: several units per CTA, query tiles past a full ring, both row layouts."""
    run_accum(F, R.Paged(24, [1500], [1400], 4, 2, 64), give=False)
    run_accum(F, R.Paged(24, [900], [700], 3, 1, 128), give=False, cap=15.0)


# ---------------------------------------------------------------------- evict
def pick(a, c, keep, recent, sink):
    """Positions kept, by sorting (weight down, position up)."""
    if c <= keep:
        return list(range(c))
    must = [t for t in range(c) if t < sink or t >= c - recent]
    rest = [t for t in range(c) if sink <= t < c - recent]
    key = lambda t: (-(a[t] if a[t] == a[t] else -math.inf), t)
    return sorted(must + sorted(rest, key=key)[:keep - len(must)])


def run_evict(F, ctx, Hkv, d, keep, recent, sink, values="spread", inplace=False, kept_out=True, seed=0):
    g = torch.Generator().manual_seed(seed + sum(ctx))
    S, n = len(ctx), max(ctx) + 3
    src_n = [-(-c // 16) for c in ctx]
    dst_n = [-(-min(c, keep) // 16) for c in ctx]
    nb = sum(src_n) + sum(dst_n) + 2
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((S, max(src_n + [1])), -1, dtype=torch.int32)
    dst = torch.full((S, max(dst_n + [1])), -1, dtype=torch.int32)
    at = 0
    for t, ns in ((table, src_n), (dst, dst_n)):
        for s, k in enumerate(ns):
            t[s, :k] = perm[at:at + k]
            at += k
    kc, vc = (torch.randn(nb, Hkv, 16, d, generator=g).bfloat16() for _ in range(2))
    acc = torch.rand(S, Hkv, n, generator=g)
    if values == "ties":
        acc = (acc * 4).floor() * 0.25
    elif values == "equal":
        acc = torch.zeros_like(acc)
    elif values == "odd":  # signs, infinities, NaN, both zeros, tiny values
        acc = (acc - 0.5) * 1e-39
        acc[..., ::7] = 0.0
        acc[..., 3::11] = -0.0
        acc[..., 5::13] = math.inf
        acc[..., 2::17] = math.nan
        acc[..., 4::19] = -math.inf
    k2, v2, a2 = kc.cuda(), vc.cuda(), acc.cuda()
    ao = a2 if inplace else torch.full((S, Hkv, keep + 4), 9.0, device="cuda")
    kept = torch.full((S, Hkv, keep), 77, dtype=torch.int32, device="cuda") if kept_out else None
    lens = F.fa_cache_evict(k2, v2, a2, table.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(), dst.cuda(), keep,
                            recent=recent, sink=sink, acc_out=ao, kept=kept)
    assert F.fa_get_error() == F.FA_OK
    assert lens.tolist() == [min(c, keep) for c in ctx]
    ek, ev, ea = kc.clone(), vc.clone(), acc.clone() if inplace else torch.full((S, Hkv, keep + 4), 9.0)
    for s, c in enumerate(ctx):
        for h in range(Hkv):
            got = pick(acc[s, h].tolist(), c, keep, recent, sink)
            if kept_out:
                assert kept[s, h].tolist() == got + [-1] * (keep - len(got)), (s, h)
            for i, t in enumerate(got):
                sb, db = int(table[s, t // 16]), int(dst[s, i // 16])
                ek[db, h, i % 16] = kc[sb, h, t % 16]
                ev[db, h, i % 16] = vc[sb, h, t % 16]
            ea[s, h, :len(got)] = acc[s, h, got]
    assert torch.equal(k2.cpu(), ek) and torch.equal(v2.cpu(), ev)
    assert torch.equal(ao.cpu().view(torch.int32), ea.view(torch.int32))


@pytest.mark.parametrize("values", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("shape", [([40, 1, 16, 100, 300], 2, 64, 16, 4, 1), ([500, 33], 1, 128, 100, 0, 0),
                                   ([65, 64, 63], 3, 64, 64, 60, 4), ([64], 1, 64, 1, 0, 0), ([64, 9], 1, 64, 1, 1, 0),
                                   ([200], 2, 128, 17, 0, 17), ([3000, 1500], 2, 64, 700, 100, 3)], ids=str)
def test_evict(F, shape, values):
    run_evict(F, *shape, values=values)


def test_evict_in_place_weights_and_workspace(F):
    run_evict(F, [700, 300, 20], 2, 64, 128, 30, 2, inplace=True)
    run_evict(F, [700, 300, 20], 2, 64, 128, 30, 2, values="ties", kept_out=False)


def test_evict_long_row(F):
    """More tokens than one pass of the scan holds."""
    run_evict(F, [20000], 1, 64, 9000, 10, 1, values="ties")


@pytest.mark.parametrize("ctx, keep", [([20000], 9000), ([5000, 9000, 2100], 600), ([70000], 3000)], ids=str)
@pytest.mark.parametrize("values", ["spread", "odd", "equal"])
def test_evict_rows_shared_by_ctas(F, ctx, keep, values):
    """Few long rows: several CTAs share a row, whose part fits their registers or not."""
    run_evict(F, ctx, 1, 64, keep, 40, 3, values=values)
    run_evict(F, ctx, 1, 64, keep, 0, 0, values=values, inplace=True)


def test_evict_reports_bad_lengths_and_blocks(F):
    S, Hkv, d = 3, 1, 64
    kc, vc = (torch.randn(12, Hkv, 16, d).bfloat16().cuda() for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    table = torch.tensor([[0, 1, 2], [3, 99, 5], [6, 7, 8]], dtype=torch.int32).cuda()
    dst = torch.tensor([[9], [10], [11]], dtype=torch.int32).cuda()
    acc = torch.rand(S, Hkv, 48).cuda()
    acc[1, 0, 16:32] = 5.0  # sequence 1 keeps tokens of its bad block
    ctx = torch.tensor([48, 48, 49], dtype=torch.int32).cuda()
    kept = torch.empty(S, Hkv, 16, dtype=torch.int32, device="cuda")
    lens = F.fa_cache_evict(kc, vc, acc, table, ctx, dst, 16, kept=kept)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    assert lens.tolist() == [16, 16, 0] and (kept[2] == -1).all()
    assert kept[1, 0].tolist() == list(range(16, 32))
    assert torch.equal(kc[10], k0[10]) and torch.equal(vc[11], v0[11])
    assert not torch.equal(kc[9], k0[9])


# --------------------------------------------------------------- the whole loop
def test_serving_loop(F):
    """Two sequences of a multimodal chat through the pool: the prompt's image tokens see each other, its weights
    are counted, the caches are thinned out into new blocks, the old ones are released, and decoding goes on over
    what was kept.  Every step against the same steps in 64 bits on the tokens that the GPU kept."""
    Hq, Hkv, d, keep, recent, sink = 8, 2, 64, 48, 8, 2
    g = Hq // Hkv
    gen = torch.Generator().manual_seed(5)
    pool = F.BlockPool(40, 12)
    prompts, prefix = [150, 70], [100, 33]
    axes = [j % 3 for j in range(d // 2)]
    table = W.rope_table(512, d).cuda()
    kc, vc = (torch.full((40, Hkv, 16, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    seqs = [pool.add_seq() for _ in prompts]
    rnd = lambda n, h: torch.randn(n, h, d, generator=gen).bfloat16().cuda()
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()

    def step(ql, pre, acc_in, acc, pos0):
        slots = np.concatenate([pool.append(s, n) for s, n in zip(seqs, ql)])
        n = sum(ql)
        pos = torch.cat([torch.arange(p, p + k) for p, k in zip(pos0, ql)]).to(torch.int32)
        pos = torch.stack([pos, pos // 2, pos % 7]).cuda()
        k, v = rnd(n, Hkv), rnd(n, Hkv)
        q = F.fa_cache_append_mrope(rnd(n, Hq), k, v, pos, axes, table, kc, vc, i32(slots))
        tab, lens = pool.tables(seqs)
        out = F.fa_paged_attn_accum(q, kc, vc, i32(tab), i32(lens), i32(ql), acc_in, acc, softcap=20.0,
                                    prefix_lens=i32(pre), max_q_len=max(ql))
        assert F.fa_get_error() == F.FA_OK
        at = 0
        for s in range(len(seqs)):
            c = int(lens[s])
            blocks = torch.tensor(tab[s, :-(-c // 16)]).long()
            for h in range(Hq):
                rows = lambda x: x.cpu()[blocks, h // g].reshape(-1, d)[:c]
                p = torch.arange(c - ql[s], c)
                ref = R.Rows(q[at:at + ql[s], h].cpu(), rows(kc), rows(vc), p, R.visible(p, c, True, 0, pre[s]),
                             d ** -0.5, 20.0)
                R.check(out[at:at + ql[s], h], ref.out, ref.out_tol, f"s{s} h{h}")
            at += ql[s]
        return tab, lens

    acc = torch.zeros(2, Hkv, 12 * 16, device="cuda")
    tab, lens = step(prompts, prefix, None, acc, [0, 0])
    total = acc.double().sum(2).cpu()
    for s, n in enumerate(prompts):
        assert (total[s] - g * n).abs().max() < 1e-3 * g * n
    new = [pool.add_seq() for _ in seqs]
    for s in new:
        pool.append(s, keep)
    dst, _ = pool.tables(new)
    kept = torch.empty(2, Hkv, keep, dtype=torch.int32, device="cuda")
    weights = acc.cpu().clone()
    old_k = kc.cpu().clone()
    out_lens = F.fa_cache_evict(kc, vc, acc, i32(tab), i32(lens), i32(dst), keep, recent=recent, sink=sink, acc_out=acc,
                                kept=kept)
    assert F.fa_get_error() == F.FA_OK and out_lens.tolist() == [keep, keep]
    for s in range(2):
        for h in range(Hkv):
            got = pick(weights[s, h].tolist(), int(lens[s]), keep, recent, sink)
            assert kept[s, h].tolist() == got
            for i in (0, 17, keep - 1):
                assert torch.equal(kc[dst[s, i // 16], h, i % 16].cpu(), old_k[tab[s, got[i] // 16], h, got[i] % 16])
    free = pool.num_free()
    for s in seqs:
        pool.release(s)
    assert pool.num_free() > free
    seqs = new
    for k in range(20):  # across a block boundary
        before = acc.clone()
        step([1, 1], [0, 0], acc, acc, [p + k for p in prompts])
        assert (acc[:, :, :keep + k] >= before[:, :, :keep + k]).all()
    step([30, 1], [0, 0], acc, acc, [p + 20 for p in prompts])


def test_accum_and_evict_captured(F):
    """Decode with sums and an eviction captured into one graph, replayed on new queries."""
    p = R.Paged(31, [100, 260], [1, 1], 8, 2, 64, spare=8)
    q, kc, vc, table, ctx, ql = p.cuda()
    used = set(table.flatten().tolist())
    spare = [b for b in range(kc.shape[0]) if b not in used][:8]
    dst = torch.tensor([spare[:4], spare[4:]], dtype=torch.int32).cuda()
    acc0 = torch.rand(2, 2, 300, generator=torch.Generator().manual_seed(1)).cuda()
    queries = [q.clone(), torch.randn_like(q)]
    want = []
    for x in queries:
        acc, ao, kept = torch.zeros_like(acc0), torch.zeros(2, 2, 64, device="cuda"), torch.empty(
            2, 2, 64, dtype=torch.int32, device="cuda")
        out = F.fa_paged_attn_accum(x, kc, vc, table, ctx, ql, acc0, acc, max_q_len=1)
        F.fa_cache_evict(kc, vc, acc, table, ctx, dst, 64, recent=4, acc_out=ao, kept=kept)
        want.append((out, acc, ao, kept, kc[spare].clone()))
    out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    acc, ao = torch.zeros_like(acc0), torch.zeros(2, 2, 64, device="cuda")
    kept, lens = torch.empty(2, 2, 64, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(F.fa_paged_attn_accum_workspace_size(2, table.shape[1], 8, 2, 64, 2, 1), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fa_paged_attn_accum(q, kc, vc, table, ctx, ql, acc0, acc, lse=lse, out=out, max_q_len=1, ws=ws)
        F.fa_cache_evict(kc, vc, acc, table, ctx, dst, 64, recent=4, acc_out=ao, kept=kept, new_lens=lens)
    for i in (1, 0, 1):
        q.copy_(queries[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, acc, ao, kept, kc[spare]), want[i]):
            assert torch.equal(a.nan_to_num(0.5) if a.is_floating_point() else a,
                               b.nan_to_num(0.5) if b.is_floating_point() else b)
    assert F.fa_get_error() == F.FA_OK
