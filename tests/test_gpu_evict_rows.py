"""Eviction with rows of every alignment shared by several CTAs and read in several passes, and with the new lengths
written over the old ones."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


def pick(a, c, keep, recent, sink):
    """Positions kept, ascending: the forced ones, then by weight (down) and position (up)."""
    if c <= keep:
        return np.arange(c)
    forced = np.r_[0:sink, c - recent:c]
    rest = np.arange(sink, c - recent)
    order = rest[np.lexsort((rest, -a[rest].astype(np.float64)))]
    return np.sort(np.r_[forced, order[:keep - len(forced)]])


def run(F, ctx, Hkv, keep, recent, sink, row, shift=0, inplace_acc=False, inplace_lens=False, d=64, seed=0):
    """`row`: elements of a row of weights; `shift`: elements by which the first row misses its allocation's start."""
    g = torch.Generator().manual_seed(seed + sum(ctx) + row)
    S = len(ctx)
    src_n, dst_n = [-(-c // 16) for c in ctx], [-(-min(c, keep) // 16) for c in ctx]
    nb = sum(src_n) + sum(dst_n)
    perm = torch.randperm(nb, generator=g).to(torch.int32).split(src_n + dst_n)
    table, dst = torch.full((S, max(src_n)), -1, dtype=torch.int32), torch.full((S, max(dst_n)), -1, dtype=torch.int32)
    for s in range(S):
        table[s, :src_n[s]], dst[s, :dst_n[s]] = perm[s], perm[S + s]
    kc, vc = (torch.randn(nb, Hkv, 16, d, generator=g).bfloat16() for _ in range(2))
    acc = (torch.rand(S, Hkv, row, generator=g) * 512).floor() / 512  # (many ties)
    buf = torch.zeros(shift + acc.numel(), device="cuda")
    a = buf[shift:].view(S, Hkv, row)
    a.copy_(acc)
    ao = a if inplace_acc else torch.full((S, Hkv, keep), 9.0, device="cuda")
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    new = lens if inplace_lens else torch.full((S,), 77, dtype=torch.int32, device="cuda")
    kept = torch.full((S, Hkv, keep), 77, dtype=torch.int32, device="cuda")
    k2, v2 = kc.cuda(), vc.cuda()
    got = F.fa_cache_evict(k2, v2, a, table.cuda(), lens, dst.cuda(), keep, recent=recent, sink=sink, acc_out=ao, kept=kept,
                           new_lens=new)
    assert F.fa_get_error() == F.FA_OK
    assert got is new and new.tolist() == [min(c, keep) for c in ctx]
    if not inplace_lens:
        assert lens.tolist() == ctx
    ek, ev = kc.clone(), vc.clone()
    ea = acc.clone() if inplace_acc else torch.full((S, Hkv, keep), 9.0)
    for s, c in enumerate(ctx):
        for h in range(Hkv):
            t = torch.from_numpy(pick(acc[s, h].numpy(), c, keep, recent, sink))
            n, i = len(t), torch.arange(len(t))
            assert torch.equal(kept[s, h, :n].cpu(), t.to(torch.int32)) and (kept[s, h, n:] == -1).all(), (s, h)
            sb, db = table[s, t // 16].long(), dst[s, i // 16].long()
            ek[db, h, i % 16], ev[db, h, i % 16] = kc[sb, h, t % 16], vc[sb, h, t % 16]
            ea[s, h, :n] = acc[s, h, t]
    assert torch.equal(k2.cpu(), ek) and torch.equal(v2.cpu(), ev) and torch.equal(ao.cpu(), ea)


LONG = [([20000], 9000), ([5000, 9000, 2100], 600), ([70000], 3000), ([8191, 8185, 4099], 4096)]


@pytest.mark.parametrize("ctx, keep", LONG, ids=str)
@pytest.mark.parametrize("pad", [0, 4, 16, 1, 2])
@pytest.mark.parametrize("inplace", [False, True])
def test_rows_of_every_alignment(F, ctx, keep, pad, inplace):
    """Rows of a multiple of four elements are read four at a time, by clusters and in several passes too; the last
    tokens of a context that ends anywhere one at a time."""
    run(F, ctx, 1, keep, 40, 3, -(-max(ctx) // 4) * 4 + pad, inplace_acc=inplace)


@pytest.mark.parametrize("shift", [1, 4])
def test_rows_that_start_anywhere(F, shift):
    run(F, [9000, 7000], 2, 1000, 5, 0, 9004, shift=shift)


@pytest.mark.parametrize("many", [False, True], ids=["one CTA a row", "CTAs that share a row"])
def test_lengths_in_place(F, many):
    """new_lens may be ctx_lens: the heads of a sequence, and the CTAs of a row, all still see the old length."""
    ctx = [20000, 9001, 40, 600] if many else [700, 300, 20, 64, 65] * 30
    for seed in range(3):
        run(F, ctx, 4, 600 if many else 64, 7, 2, max(ctx) + 4, inplace_lens=True, inplace_acc=seed == 1, seed=seed)


def test_lengths_in_place_of_a_sequence_that_does_not_fit(F):
    kc, vc = (torch.randn(8, 2, 16, 64, device="cuda").bfloat16() for _ in range(2))
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32).cuda()
    dst = torch.tensor([[4], [5]], dtype=torch.int32).cuda()
    lens = torch.tensor([33, 30], dtype=torch.int32).cuda()
    F.fa_cache_evict(kc, vc, torch.rand(2, 2, 48).cuda(), table, lens, dst, 16, new_lens=lens)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    assert lens.tolist() == [0, 16]


def test_lengths_in_place_captured(F):
    """A loop of a serving program: append, count, evict in place, replayed as one graph."""
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randn(40, 2, 16, 64, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.arange(20, dtype=torch.int32).view(2, 10).cuda()
    dst = torch.arange(20, 28, dtype=torch.int32).view(2, 4).cuda()
    acc = torch.rand(2, 2, 160, generator=g).cuda()
    first = torch.tensor([160, 90], dtype=torch.int32).cuda()
    lens, kept = first.clone(), torch.empty(2, 2, 64, dtype=torch.int32, device="cuda")
    want = torch.empty_like(kept)
    F.fa_cache_evict(kc, vc, acc, table, first, dst, 64, recent=4, kept=want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fa_cache_evict(kc, vc, acc, table, lens, dst, 64, recent=4, kept=kept, new_lens=lens)
    for _ in range(2):
        lens.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [64, 64] and torch.equal(kept, want)
