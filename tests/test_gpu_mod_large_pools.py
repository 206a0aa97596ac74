"""Blocks whose values lie past 2^31 elements and 2^32 bytes from the start of the cache."""
import pytest
import torch

import mod_ref as R
import workloads as W

pytestmark = pytest.mark.gpu
HKV, D, BLOCKS = 2, 128, 560000  # 2.3e9 elements, 4.6 GB a cache


def test_append_attend_count_evict_at_the_far_end():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn as F
    Hq, ctx, ql, keep = 8, [300, 70], [40, 1], 32
    kc, vc = (torch.zeros(BLOCKS, HKV, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = [-(-c // 16) for c in ctx]
    blocks = (BLOCKS - 1 - torch.arange(sum(n) + 4)).to(torch.int32)  # the last ones, from the end
    table = torch.full((2, max(n)), -1, dtype=torch.int32)
    table[0, :n[0]], table[1, :n[1]] = blocks[:n[0]], blocks[n[0]:sum(n)]
    dst = blocks[sum(n):].view(2, 2)
    g = torch.Generator().manual_seed(5)
    pos = torch.cat([torch.arange(c) for c in ctx])
    seq = torch.cat([torch.full((c,), s) for s, c in enumerate(ctx)])
    slots = (table[seq, pos // 16] * 16 + pos % 16).to(torch.int32)
    q, k, v = (torch.randn(sum(ctx), h, D, generator=g).bfloat16().cuda() for h in (Hq, HKV, HKV))
    cs = W.rope_table(512, D)
    rot = F.fa_cache_append_mrope(q, k, v, torch.stack([pos, pos // 3]).to(torch.int32).cuda(), [j % 2 for j in range(D // 2)],
                                  cs.cuda(), kc, vc, slots.cuda())
    assert F.fa_get_error() == F.FA_OK
    where = table[seq, pos // 16].long().cuda()
    assert torch.equal(vc[where, :, (pos % 16).cuda()], v)
    keys = kc[where, :, (pos % 16).cuda()]
    first = [ctx[0] - ql[0], ctx[0] + ctx[1] - ql[1]]
    qs = torch.cat([rot[f:f + m] for f, m in zip(first, ql)]).contiguous()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    acc = torch.zeros(2, HKV, 320, device="cuda")
    out = F.fa_paged_attn_accum(qs, kc, vc, table.cuda(), i32(ctx), i32(ql), None, acc, max_q_len=40)
    assert F.fa_get_error() == F.FA_OK
    at = 0
    for s, (c, m) in enumerate(zip(ctx, ql)):
        rows = slice(sum(ctx[:s]), sum(ctx[:s]) + c)
        p = torch.arange(c - m, c)
        for h in range(Hq):
            ref = R.Rows(qs[at:at + m, h].cpu(), keys[rows, h // 4].cpu(), v[rows, h // 4].cpu(), p, R.visible(p, c, True), D ** -0.5)
            R.check(out[at:at + m, h], ref.out, ref.out_tol, f"s{s} h{h}")
        at += m
    kept = torch.empty(2, HKV, keep, dtype=torch.int32, device="cuda")
    F.fa_cache_evict(kc, vc, acc, table.cuda(), i32(ctx), dst.cuda(), keep, recent=4, kept=kept)
    assert F.fa_get_error() == F.FA_OK
    for s in range(2):
        base = sum(ctx[:s])
        for h in range(HKV):
            t = kept[s, h].long()
            i = torch.arange(keep)
            b = dst[s, i // 16].long().cuda()
            assert torch.equal(kc[b, h, (i % 16).cuda()], keys[base + t, h])
            assert torch.equal(vc[b, h, (i % 16).cuda()], v[base + t, h])
    # nothing else was written: the caches hold the appended and the kept rows only
    used = set(blocks.tolist())
    assert kc[:BLOCKS - len(used)].count_nonzero() == 0 and vc[:BLOCKS - len(used)].count_nonzero() == 0
