"""Attention with modified scores (cap, distance bias, window, prefix, documents)
over dense prompts and over the paged cache, against 64-bit plain attention."""
import math

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


def doc_ids(B, T, seed):
    """Runs of random lengths; one document comes back under the same id later; padding inside and behind."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.empty(B, T, dtype=torch.int32)
    for b in range(B):
        t, n = 0, 0
        while t < T:
            k = int(torch.randint(1, max(2, T // 3), (1,), generator=g))
            ids[b, t:t + k] = [5, 7, -1, 5, 0, -3][n % 6]
            t, n = t + k, n + 1
    return ids


def run_prefill(F, B, T, Hq, Hkv, d, causal=True, cap=0.0, bias=False, window=0, prefix=None, docs=False, std=1.0,
                seed=0, ids=None):
    g = torch.Generator().manual_seed(seed + 1000 * T + Hq)
    q = (torch.randn(B, T, Hq, d, generator=g) * std).bfloat16()
    k, v = (torch.randn(B, T, Hkv, d, generator=g).bfloat16() for _ in range(2))
    sl = R.slopes(Hq) if bias else None
    pre = None if prefix is None else torch.tensor([(prefix * (b + 1)) % (T + 3) for b in range(B)], dtype=torch.int32)
    if docs and ids is None:
        ids = doc_ids(B, T, seed)
    dev = lambda t: None if t is None else t.cuda()
    lse = torch.full((B, Hq, T), 7.0, device="cuda")
    buf = torch.full((B * T + 64, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[32:32 + B * T].view(B, T, Hq, d)
    F.fa_prefill_mod(dev(q), dev(k), dev(v), causal=causal, softcap=cap, alibi_slopes=dev(sl), window=window,
                     prefix_lens=dev(pre), doc_ids=dev(ids), out=out, lse=lse)
    assert F.fa_get_error() == F.FA_OK
    assert (buf[:32] == 3.0).all() and (buf[32 + B * T:] == 3.0).all()
    pos = torch.arange(T)
    for b in range(B):
        see = R.visible(pos, T, causal, window, int(pre[b]) if pre is not None else 0, ids[b] if ids is not None else None)
        for h in range(Hq):
            ref = R.Rows(q[b, :, h], k[b, :, h // (Hq // Hkv)], v[b, :, h // (Hq // Hkv)], pos, see, d ** -0.5, cap,
                         sl[h] if bias else None)
            R.check(lse[b, h], ref.lse, ref.lse_tol, f"lse b{b} h{h}")
            R.check(out[b, :, h], ref.out, ref.out_tol, f"out b{b} h{h}")
    return out, lse


MODS = [
    dict(),
    dict(cap=5.0, std=6.0),
    dict(cap=50.0, std=8.0),
    dict(bias=True),
    dict(bias=True, causal=False),
    dict(bias=True, prefix=70),
    dict(bias=True, cap=20.0, std=4.0),
    dict(window=1),
    dict(window=40),
    dict(window=200, causal=False),
    dict(window=40, bias=True, causal=False),
    dict(prefix=150),
    dict(prefix=90, window=60),
    dict(docs=True),
    dict(docs=True, causal=False),
    dict(docs=True, cap=30.0, std=6.0, window=50),
    dict(docs=True, bias=True, prefix=100, causal=True),
    dict(causal=False),
    dict(causal=False, cap=10.0, std=3.0),
]


@pytest.mark.parametrize("mod", MODS, ids=lambda m: "-".join(f"{k}{v}" for k, v in m.items()) or "none")
@pytest.mark.parametrize("shape", [(2, 300, 4, 2, 128), (1, 129, 3, 1, 64)], ids=str)
def test_prefill_mod(F, shape, mod):
    run_prefill(F, *shape, **mod)


@pytest.mark.parametrize("T", [1, 2, 15, 127, 128, 257])
@pytest.mark.parametrize("mod", [dict(cap=30.0, std=4.0), dict(bias=True, window=5), dict(docs=True), dict(prefix=9)],
                         ids=str)
def test_prefill_mod_lengths(F, T, mod):
    run_prefill(F, 2, T, 2, 1, 64, **mod)


@pytest.mark.parametrize("heads", [(1, 1), (5, 1), (6, 2), (8, 8), (16, 1)], ids=str)
def test_prefill_mod_heads(F, heads):
    run_prefill(F, 1, 400, *heads, 64, bias=True, docs=True, seed=3)
    run_prefill(F, 1, 400, *heads, 128, cap=15.0, std=5.0, window=130, seed=4)


def test_prefill_mod_many_units(F):
    """More units than CTAs, so that every CTA runs several, with documents and without."""
    run_prefill(F, 3, 900, 8, 2, 64, docs=True, bias=True, seed=5)
    run_prefill(F, 4, 700, 12, 2, 64, cap=8.0, std=5.0, seed=6)


def test_prefill_mod_rows_without_keys(F):
    """A sequence of nothing but padding, a padding row at either end, and a row behind a full tile of padding."""
    ids = torch.full((3, 260), -1, dtype=torch.int32)
    ids[1, 1:259] = 4
    ids[2, 130:] = 2
    ids[2, 200] = -7
    out, lse = run_prefill(F, 3, 260, 4, 2, 128, docs=True, ids=ids)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    assert (out[2, 200] == 0).all() and (lse[2, :, 200] == -math.inf).all()


def test_prefill_mod_documents_are_runs(F):
    """Equal ids that do not touch are different documents; lengths of one."""
    T = 140
    ids = torch.arange(T, dtype=torch.int32).remainder(2).view(1, T)
    out, lse = run_prefill(F, 1, T, 2, 2, 64, docs=True, ids=ids, causal=False)


def test_prefill_mod_without_modifiers_is_prefill(F):
    """No modifier: the same tiles meet in the same order, so the bits are fa_prefill's."""
    g = torch.Generator().manual_seed(1)
    for (B, T, Hq, Hkv, d) in [(2, 517, 6, 2, 128), (1, 300, 3, 3, 64)]:
        q = torch.randn(B, T, Hq, d, generator=g).bfloat16().cuda()
        k, v = (torch.randn(B, T, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
        for causal in (True, False):
            a, b = torch.empty(B, Hq, T, device="cuda"), torch.empty(B, Hq, T, device="cuda")
            assert torch.equal(F.fa_prefill(q, k, v, causal=causal, lse=a),
                               F.fa_prefill_mod(q, k, v, causal=causal, lse=b))
            assert torch.equal(a, b)


def test_prefill_mod_side_stream_and_graph(F):
    """A call on another stream, and one captured and replayed with new inputs in the same buffers."""
    B, T, Hq, Hkv, d = 2, 260, 4, 2, 64
    g = torch.Generator().manual_seed(2)
    new = lambda: [torch.randn(B, T, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]
    ids = [doc_ids(B, T, s).cuda() for s in (1, 2)]
    first, second = new(), new()
    want = [F.fa_prefill_mod(*x, softcap=9.0, doc_ids=i) for x, i in zip((first, second), ids)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = F.fa_prefill_mod(*first, softcap=9.0, doc_ids=ids[0])
    side.synchronize()
    assert torch.equal(got, want[0])
    buf = [t.clone() for t in first]
    bid, out = ids[0].clone(), torch.empty_like(first[0])
    ws = torch.empty(F.fa_prefill_mod_workspace_size(B, T), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fa_prefill_mod(*buf, softcap=9.0, doc_ids=bid, out=out, ws=ws)
    for x, i, w in ((second, ids[1], want[1]), (first, ids[0], want[0])):
        for dst, src in zip(buf, x):
            dst.copy_(src)
        bid.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


# ---------------------------------------------------------------------- paged
def run_paged(F, p, causal=True, cap=0.0, bias=False, window=0, prefix=None, max_q_len=None):
    sl = R.slopes(p.Hq) if bias else None
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
    q, kc, vc, table, ctx, ql = p.cuda()
    buf = torch.full((p.total + 64, p.Hq, p.d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.total, p.Hq), 7.0, device="cuda")
    out = buf[32:32 + p.total]
    F.fa_paged_attn_mod(q, kc, vc, table, ctx, ql, causal=causal, softcap=cap,
                        alibi_slopes=None if sl is None else sl.cuda(), window=window,
                        prefix_lens=None if pre is None else pre.cuda(), out=out, lse=lse, max_q_len=max_q_len)
    assert F.fa_get_error() == F.FA_OK
    assert (buf[:32] == 3.0).all() and (buf[32 + p.total:] == 3.0).all()
    for s, h, at, ref in p.rows(causal, cap, sl, window, prefix):
        n = p.ql[s]
        R.check(lse[at:at + n, h], ref.lse, ref.lse_tol, f"lse s{s} h{h}")
        R.check(out[at:at + n, h], ref.out, ref.out_tol, f"out s{s} h{h}")
    return out, lse


PAGED_MODS = [
    dict(),
    dict(cap=30.0),
    dict(bias=True),
    dict(window=1),
    dict(window=37),
    dict(window=150, cap=20.0),
    dict(window=64, bias=True),
    dict(bias=True, cap=25.0),
    dict(prefix=[0, 40, 300, 5, 1000, 0, 17, 2]),
    dict(prefix=[3, 40, 300, 5, 1000, 0, 17, 2], bias=True),
    dict(causal=False, window=90),
    dict(causal=False, bias=True),
]
CTX = [1, 16, 17, 200, 333, 4, 130, 512]


@pytest.mark.parametrize("mod", PAGED_MODS, ids=lambda m: "-".join(f"{k}{v}" for k, v in m.items()) or "none")
@pytest.mark.parametrize("kind", ["decode", "few", "chunk", "mixed"])
@pytest.mark.parametrize("heads", [(6, 2, 128), (4, 4, 64), (3, 1, 64), (16, 2, 128)], ids=str)
def test_paged_mod(F, heads, kind, mod):
    ql = {"decode": [1] * 8, "few": [1, 2, 1, 2, 0, 1, 2, 2], "chunk": [1, 16, 17, 150, 300, 4, 33, 129],
          "mixed": [1, 1, 0, 40, 1, 2, 130, 200]}[kind]
    p = R.Paged(7, CTX, ql, *heads, std=4.0 if mod.get("cap") else 1.0,
                window=mod.get("window", 0))
    run_paged(F, p, max_q_len=max(ql), **mod)


def test_paged_mod_wide_group(F):
    """More than 16 query heads per kv head: every row takes the tensor-core path."""
    run_paged(F, R.Paged(8, [5, 140, 33], [1, 3, 33], 20, 1, 64, window=20), window=20, bias=True)
    run_paged(F, R.Paged(8, [5, 140, 33], [1, 3, 33], 18, 1, 128), cap=12.0)


def test_paged_mod_long_context_cut_between_ctas(F):
    """Few sequences with long contexts: segments cut between warps and CTAs, window starting inside a block."""
    p = R.Paged(9, [5000, 3333], [1, 3], 8, 2, 128)
    run_paged(F, p, bias=True)
    run_paged(F, p, cap=10.0)
    p = R.Paged(9, [5000, 3333], [1, 3], 8, 2, 128, window=2500)
    run_paged(F, p, window=2500, bias=True)


def test_paged_mod_equals_dense(F):
    """A whole prompt as one chunk gives the dense call's rows within twice the bound of one."""
    T = 290
    p = R.Paged(10, [T], [T], 4, 2, 128)
    out, lse = run_paged(F, p, cap=6.0, window=100)
    dense = F.fa_prefill_mod(p.q.view(1, T, 4, 128).cuda(), p.k[0].view(1, T, 2, 128).cuda(),
                             p.v[0].view(1, T, 2, 128).cuda(), softcap=6.0, window=100)
    for s, h, at, ref in p.rows(True, 6.0, None, 100):
        R.check(dense[0, :, h].cpu() - out[:, h].cpu().float(), torch.zeros_like(ref.out), 2 * ref.out_tol, f"h{h}")


def test_paged_mod_without_modifiers_is_paged_attn(F):
    """The same bits where every warp of the decode grid has a page (shorter streams are split differently)."""
    for ql in ([1, 1, 1], [1, 70, 140]):
        p = R.Paged(11, [12000, 200, 500], ql, 8, 2, 128)
        q, kc, vc, table, ctx, qls = p.cuda()
        a = F.fa_paged_attn(q, kc, vc, table, ctx, qls, max_q_len=max(ql))
        b = F.fa_paged_attn_mod(q, kc, vc, table, ctx, qls, max_q_len=max(ql))
        assert torch.equal(a, b)


def test_paged_mod_bad_blocks_and_lengths(F):
    """Bad ids inside the visible range and lengths past the table are reported; the call ends."""
    for ql in ([1, 1], [40, 1]):
        p = R.Paged(12, [100, 90], ql, 4, 2, 64)
        q, kc, vc, table, ctx, qls = p.cuda()
        bad = table.clone()
        bad[0, 2] = kc.shape[0] + 5
        F.fa_paged_attn_mod(q, kc, vc, bad, ctx, qls, softcap=9.0, max_q_len=max(ql))
        assert F.fa_get_error() == F.FA_ERR_BOUNDS
        long = ctx.clone()
        long[1] = table.shape[1] * 16 + 1
        F.fa_paged_attn_mod(q, kc, vc, table, long, qls, window=30, max_q_len=max(ql))
        assert F.fa_get_error() == F.FA_ERR_BOUNDS
    assert F.fa_get_error() == F.FA_OK


def test_paged_mod_graph_replay(F):
    """Decode and chunk rows captured once, replayed on longer contexts in the same buffers."""
    p = R.Paged(13, [60, 200, 400], [1, 60, 1], 8, 2, 64)
    q, kc, vc, table, ctx, ql = p.cuda()
    sl = R.slopes(8).cuda()
    kw = dict(alibi_slopes=sl, window=77, max_q_len=60)
    ctxs = [ctx.clone(), ctx - torch.tensor([7, 33, 100], dtype=torch.int32, device="cuda")]
    want = [F.fa_paged_attn_mod(q, kc, vc, table, c, ql, **kw) for c in ctxs]
    out, lse = torch.empty_like(q), torch.empty(q.shape[0], 8, device="cuda")
    ws = torch.empty(F.fa_paged_attn_mod_workspace_size(3, table.shape[1], 8, 2, 64, q.shape[0], 60), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fa_paged_attn_mod(q, kc, vc, table, ctx, ql, out=out, lse=lse, ws=ws, **kw)
    for c, w in ((ctxs[1], want[1]), (ctxs[0], want[0]), (ctxs[1], want[1])):
        ctx.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert F.fa_get_error() == F.FA_OK


def test_prefill_mod_caps_of_all_sizes(F):
    """The forms of the cap: scores far below it, around it, far above it, and rows whose every score is very low."""
    for cap, std in ((1e4, 3.0), (300.0, 40.0), (60.0, 8.0), (40.0, 12.0), (30.0, 30.0), (2.0, 20.0), (0.01, 1.0)):
        run_prefill(F, 1, 200, 2, 1, 64, cap=cap, std=std, causal=False, seed=int(cap))
    g = torch.Generator().manual_seed(9)
    T, d = 200, 64
    k = torch.randn(1, T, 1, d, generator=g).abs().bfloat16()
    q = -(torch.randn(1, T, 2, d, generator=g).abs() * 4).bfloat16()  # every score is negative
    v = torch.randn(1, T, 1, d, generator=g).bfloat16()
    for cap in (50.0, 30.0, 8.0):
        lse = torch.empty(1, 2, T, device="cuda")
        out = F.fa_prefill_mod(q.cuda(), k.cuda(), v.cuda(), softcap=cap, lse=lse)
        pos = torch.arange(T)
        for h in range(2):
            ref = R.Rows(q[0, :, h], k[0, :, 0], v[0, :, 0], pos, R.visible(pos, T, True), d ** -0.5, cap)
            R.check(lse[0, h], ref.lse, ref.lse_tol, f"lse cap {cap}")
            R.check(out[0, :, h], ref.out, ref.out_tol, f"out cap {cap}")


def test_prefill_mod_slopes_of_all_sizes(F):
    """Steep slopes, none, and slopes that favour distant keys."""
    g = torch.Generator().manual_seed(10)
    B, T, Hq, d = 1, 300, 6, 64
    q = torch.randn(B, T, Hq, d, generator=g).bfloat16()
    k, v = (torch.randn(B, T, 1, d, generator=g).bfloat16() for _ in range(2))
    sl = torch.tensor([8.0, 1.5, 0.0, 1e-4, -0.02, -0.5])
    for kw in (dict(), dict(causal=False), dict(prefix_lens=torch.tensor([150], dtype=torch.int32).cuda())):
        lse = torch.empty(B, Hq, T, device="cuda")
        out = F.fa_prefill_mod(q.cuda(), k.cuda(), v.cuda(), alibi_slopes=sl.cuda(), lse=lse, **kw)
        pos = torch.arange(T)
        see = R.visible(pos, T, kw.get("causal", True), 0, 150 if "prefix_lens" in kw else 0)
        for h in range(Hq):
            ref = R.Rows(q[0, :, h], k[0, :, 0], v[0, :, 0], pos, see, d ** -0.5, 0.0, sl[h])
            R.check(lse[0, h], ref.lse, ref.lse_tol, f"lse slope {float(sl[h])}")
            R.check(out[0, :, h], ref.out, ref.out_tol, f"out slope {float(sl[h])}")


def test_waits_run_out(F):
    """Every kernel behind these calls reports a wait that runs out, and works again afterwards."""
    p = R.Paged(14, [100, 300], [1, 60], 8, 2, 64)
    q, kc, vc, table, ctx, ql = p.cuda()
    acc = torch.zeros(2, 2, 300, device="cuda")
    x = torch.randn(1, 200, 4, 64, device="cuda").bfloat16()
    calls = [lambda: F.fa_prefill_mod(x, x, x, softcap=5.0),
             lambda: F.fa_paged_attn_mod(q, kc, vc, table, ctx, ql, window=50, max_q_len=60),
             lambda: F.fa_paged_attn_accum(q, kc, vc, table, ctx, ql, None, acc, max_q_len=60)]
    want = [c() for c in calls]
    assert F.fa_get_error() == F.FA_OK
    F.fa_debug_set_wait_limit(2_000_000)
    try:
        for c in calls:
            F.fa_debug_force_timeout(True)
            c()
            assert F.fa_get_error() == F.FA_ERR_TIMEOUT
            F.fa_debug_force_timeout(False)
            assert F.fa_get_error() == F.FA_OK
    finally:
        F.fa_debug_force_timeout(False)
        F.fa_debug_set_wait_limit(4_000_000_000)
    for c, w in zip(calls, want):
        assert torch.equal(c(), w)
    assert F.fa_get_error() == F.FA_OK


def test_two_streams_at_once(F):
    """Calls on two streams at the same time, each with buffers of its own."""
    ps = [R.Paged(15, [300, 900], [1, 70], 8, 2, 64), R.Paged(16, [700, 50], [90, 1], 8, 2, 64)]
    args = [p.cuda() for p in ps]
    want = [F.fa_paged_attn_mod(*a, softcap=20.0, max_q_len=90) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(F.fa_paged_attn_mod(*args[i], softcap=20.0, max_q_len=90))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)
    # a stream given as an argument: the call's own workspace must outlive it there
    out = [F.fa_paged_attn_mod(*args[0], softcap=20.0, max_q_len=90, stream=streams[0]) for _ in range(5)]
    streams[0].synchronize()
    assert all(torch.equal(x, want[0]) for x in out)
    assert F.fa_get_error() == F.FA_OK


def test_own_tensors_come_from_the_calls_stream(F):
    """A call on a stream given as an argument must not write into memory that the current stream's queued work may
    still use: what it allocates is that stream's."""
    q, k, v = (torch.randn(1, 300, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    want = F.fa_prefill_mod(q, k, v, window=50)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        x = torch.empty_like(q)
        freed = x.data_ptr()
        del x  # (work queued on the current stream may still be reading it)
        out = F.fa_prefill_mod(q, k, v, window=50, stream=stream)
        assert out.data_ptr() != freed
        side.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(F.fa_prefill_mod(q, k, v, window=50, stream=0), want)


def test_prefix_of_the_lowest_value(F):
    """prefix_lens below 1 change nothing, down to the type's lowest value: decode rows and chunks."""
    lowest = -(1 << 31)
    p = R.Paged(31, [100, 40, 300], [1, 3, 200], 4, 2, 64)
    q, kc, vc, table, ctx, ql = p.cuda()
    want = F.fa_paged_attn_mod(q, kc, vc, table, ctx, ql)
    got = F.fa_paged_attn_mod(q, kc, vc, table, ctx, ql, prefix_lens=torch.full((3,), lowest, dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want)
    x = [torch.randn(1, 200, h, 64, device="cuda").bfloat16() for h in (4, 2, 2)]
    pre = torch.full((1,), lowest, dtype=torch.int32, device="cuda")
    assert torch.equal(F.fa_prefill_mod(*x, prefix_lens=pre), F.fa_prefill_mod(*x, window=1 << 30))
    with pytest.raises(ValueError):
        F.fa_prefill_mod(*x, window=1 << 32)


# chunks over contexts long enough that their keys are shared by several work units
LONG_MODS = [dict(), dict(cap=30.0), dict(bias=True), dict(window=1500), dict(window=900, bias=True, cap=25.0),
             dict(prefix=[3900, 0, 90, 700]), dict(causal=False, window=1100), dict(causal=False, cap=12.0)]


@pytest.mark.parametrize("mod", LONG_MODS, ids=str)
@pytest.mark.parametrize("heads", [(4, 1, 128), (6, 1, 64), (3, 1, 128), (1, 1, 64), (16, 2, 64)], ids=str)
def test_paged_mod_chunks_over_long_contexts(F, heads, mod):
    """Cut along their keys, beside a short chunk and a single token; with a window some rows see nothing in a piece."""
    p = R.Paged(41, [4000, 1700, 90, 2500], [70, 33, 40, 1], *heads, std=4.0 if mod.get("cap") else 1.0,
                window=mod.get("window", 0))
    run_paged(F, p, max_q_len=70, **mod)


def test_paged_mod_more_pieces_than_lanes(F):
    p = R.Paged(42, [27000], [24], 2, 1, 64)
    run_paged(F, p)
    run_paged(F, p, bias=True, cap=20.0)


def test_paged_mod_long_chunks_replayed(F):
    """One captured call, replayed on contexts that are cut and on some that are not; twice the same call, the same bits."""
    p = R.Paged(43, [3000, 2000], [40, 90], 8, 2, 128)
    q, kc, vc, table, ctx, ql = p.cuda()
    ctxs = [ctx.clone(), torch.tensor([300, 100], dtype=torch.int32, device="cuda"),
            torch.tensor([1999, 1111], dtype=torch.int32, device="cuda")]
    want = [F.fa_paged_attn_mod(q, kc, vc, table, c, ql, window=2500, max_q_len=90) for c in ctxs]
    out = torch.empty_like(q)
    ws = torch.full((F.fa_paged_attn_mod_workspace_size(2, table.shape[1], 8, 2, 128, q.shape[0], 90),), 255,
                    dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fa_paged_attn_mod(q, kc, vc, table, ctx, ql, window=2500, max_q_len=90, out=out, ws=ws)
    for c, w in zip(ctxs + ctxs[::-1], want + want[::-1]):
        ctx.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert F.fa_get_error() == F.FA_OK


def test_paged_mod_long_chunks_among_many_tokens(F):
    """Cut chunks among more sequences than a block has threads: places and lists run over all of them."""
    n = 1100
    ctx, ql = [3 + i % 20 for i in range(n)], [1] * n
    for at, c, q in ((5, 2600, 30), (700, 1500, 25), (1099, 1800, 40)):
        ctx[at], ql[at] = c, q
    run_paged(F, R.Paged(45, ctx, ql, 2, 1, 64), max_q_len=40)


def test_prefill_mod_documents_of_large_batches(F):
    """More rows than one pass over the ids takes: the same bits as one sequence at a time."""
    B, T = 3, 4001
    g = torch.Generator().manual_seed(46)
    q, k, v = (torch.randn(B, T, h, 64, generator=g).bfloat16().cuda() for h in (2, 1, 1))
    ids = doc_ids(B, T, 47).cuda()
    out = F.fa_prefill_mod(q, k, v, doc_ids=ids, window=700)
    for b in range(B):
        x = slice(b, b + 1)
        assert torch.equal(out[x], F.fa_prefill_mod(q[x], k[x], v[x], doc_ids=ids[x].contiguous(), window=700))
