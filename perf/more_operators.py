"""Cases, inputs, plain forms and 64-bit values of five operators of long-context serving: a paged cache held in
8 bits with a power-of-two scale for each block and head, and attention over the blocks that matter to a query.

  append  new keys (rotated on the way) and values written to the 8-bit cache, each (block, kv head) with a scale
          of its own that grows with the block (fa_cache_append_fp8_scaled)
  attn8   attention over that cache: single tokens and chunks (fa_paged_attn_fp8_scaled)
  bounds  the smallest and largest value of every channel over a block's keys, kept up to date as a cache grows
          (fa_block_bounds)
  select  for each query the blocks whose bounds allow the largest scores, the first and the last ones always
          (fa_block_select)
  blocks  attention of each query over its own blocks (fa_paged_attn_blocks)

`own` selects between the plain form (elementary torch operations in 32 bits, scores that decide an order in 64,
rounded once) and the library's calls.
"""
import math
import random

import torch

own = False

BLOCK = 16
BIAS = 127  # scale code e stands for 2^(e - BIAS)
LEAST = 87  # the smallest scale code
LOG_BASE = math.log(1.0e6)  # rotary base of the shapes below
FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one token for each sequence of a serving batch
        dict(name="append_decode", op="append", S=64, ctx_lo=128, ctx_hi=2048, q_hi=1, Hq=12, Hkv=2, d=128, rope=True,
             f32=False, layout=1),
        # chunks of prompts, some ending and some starting inside a block
        dict(name="append_prompt", op="append", S=8, ctx_lo=512, ctx_hi=1500, q_hi=1024, Hq=32, Hkv=8, d=128, rope=True,
             f32=False, layout=2),
        # a step of one sequence: latency
        dict(name="attn8_decode_one", op="attn8", S=1, ctx_lo=1000, ctx_hi=1000, q_hi=1, Hq=8, Hkv=8, d=128, layout=3),
        # a serving step of a batch with long contexts
        dict(name="attn8_decode", op="attn8", S=64, ctx_lo=128, ctx_hi=8192, q_hi=1, Hq=12, Hkv=2, d=128, layout=4),
        # chunks of prompts
        dict(name="attn8_chunk", op="attn8", S=16, ctx_lo=300, ctx_hi=4600, q_hi=512, Hq=32, Hkv=8, d=128, layout=5),
        # bounds of the block that each sequence's new token went to
        dict(name="bounds_decode", op="bounds", S=64, ctx_lo=128, ctx_hi=2048, q_hi=1, Hkv=8, d=128, fp8=False, layout=6),
        # bounds of prompts just written
        dict(name="bounds_prompt", op="bounds", S=8, ctx_lo=3000, ctx_hi=4600, q_hi=4600, Hkv=8, d=128, fp8=False, layout=7),
        # a step of sequences of tens of thousands of tokens
        dict(name="select_decode", op="select", S=16, ctx_lo=8000, ctx_hi=32768, q_hi=1, Hq=32, Hkv=8, d=128, keep=128,
             recent=8, sink=1, layout=8),
        # each query of chunks picks its own blocks
        dict(name="select_chunk", op="select", S=4, ctx_lo=3000, ctx_hi=8000, q_hi=256, Hq=12, Hkv=2, d=128, keep=64,
             recent=4, sink=1, layout=9),
        # one long sequence: latency
        dict(name="blocks_decode_one", op="blocks", S=1, ctx_lo=65536, ctx_hi=65536, q_hi=1, Hq=32, Hkv=8, d=128, keep=128,
             fp8=False, layout=10),
        # a batch over the 8-bit cache
        dict(name="blocks_decode_8bit", op="blocks", S=64, ctx_lo=512, ctx_hi=8192, q_hi=1, Hq=32, Hkv=8, d=128, keep=64,
             fp8=True, layout=11),
        # chunks whose queries each read their own blocks
        dict(name="blocks_chunk", op="blocks", S=4, ctx_lo=2000, ctx_hi=6000, q_hi=128, Hq=12, Hkv=2, d=128, keep=48,
             fp8=False, layout=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn8", "attn8", "bounds", "select", "blocks", "blocks"])
    Hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
    S = _log_int(rng, 1, 48)
    hi = _log_int(rng, 16, 16000 if S <= 4 else 4000)
    q_hi = rng.choice([1, 1, 2, 5, _log_int(rng, 6, 300)])
    c = dict(op=op, S=S, q_hi=q_hi, Hkv=Hkv, d=rng.choice([64, 128]), layout=rng.randrange(1 << 30))
    if op != "bounds":
        c["Hq"] = Hkv * g
    if op == "append":
        c["q_hi"] = q_hi = rng.choice([1, 3, _log_int(rng, 6, 1000)])
        hi = min(hi, 1500)
        c.update(rope=rng.random() < 0.7, f32=rng.random() < 0.3)
    if op in ("bounds", "blocks"):
        c["fp8"] = rng.random() < 0.5
    if op in ("select", "blocks"):
        c["keep"] = _log_int(rng, 4, 200)
    if op == "select":
        c["recent"] = rng.randint(0, c["keep"] // 2)
        c["sink"] = rng.choice([0, 1, 2])
    c["ctx_lo"] = max(q_hi, hi // rng.choice([1, 4, 30]))
    c["ctx_hi"] = max(hi, c["ctx_lo"])
    if op == "select":  # contexts of more blocks than are kept, and shorter ones among them
        c["ctx_hi"] = max(c["ctx_hi"], 40 * c["keep"])
        if S <= 4:
            c["ctx_lo"] = max(c["ctx_lo"], 20 * c["keep"])

    def cost():
        pairs = c["S"] * q_hi * (c["keep"] * BLOCK if op == "blocks" else c["ctx_hi"])
        return max(pairs * c.get("Hq", Hkv) * c["d"] / 4e10, c["S"] * c["ctx_hi"] * Hkv * c["d"] / 2e8,
                   pairs * Hkv * c["d"] * (1 if c["fp8"] else 2) / (2e8 if q_hi > 5 else 1e8) if op == "blocks" else 0)
    while c["S"] > 1 and cost() > 1:
        c["S"] //= 2
    while op == "blocks" and c["keep"] > 4 and cost() > 1:
        c["keep"] //= 2
    return c


# ----------------------------------------------------------------- layouts --
# What a case fixes beside its sizes: the lengths of its sequences.  Values come from the seed.
def _lengths(case):
    r = random.Random(case["layout"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["S"])]
    return ctx, [min(c, r.randint(max(1, case["q_hi"] // 8), case["q_hi"])) for c in ctx]


# ------------------------------------------------------------------ inputs --
def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(gen, lens, mbps, num_blocks):
    """Block tables of sequences of these lengths over a shuffled pool; unused entries are -1."""
    perm = torch.randperm(num_blocks, generator=gen, device="cuda").cpu()
    table = torch.full((len(lens), mbps), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        nb = -(-n // BLOCK)
        table[s, :nb] = perm[at:at + nb].to(torch.int32)
        at += nb
    return table.cuda()


def _scale_code(amax):
    """The smallest e >= LEAST with amax <= 448 * 2^(e - BIAS)."""
    m, x = torch.frexp(amax.double() / 448.0)  # m in [0.5, 1), or 0
    e = torch.where(m == 0.5, x - 1, x).long() + BIAS
    return torch.where(amax == 0, torch.full_like(e, LEAST), e).clamp(min=LEAST)


def _pow2(e):
    """2^e of whole numbers, exactly."""
    return torch.ldexp(torch.ones((), dtype=torch.float32, device="cuda"), e.to(torch.int32))


def _cache8(gen, nb, Hkv, d, values):
    """Codes and scale codes of a cache whose blocks were written whole: K rows by token, V rows by channel."""
    x = _normal(gen, nb, Hkv, BLOCK, d).float()
    if not values:
        # some channels of the keys are larger than the others, some blocks as a whole
        x *= torch.rand(d, generator=gen, device="cuda").pow(6) * 3 + 0.7
    x *= torch.rand(nb, Hkv, 1, 1, generator=gen, device="cuda") + 0.5
    e = _scale_code(x.abs().amax((2, 3)))
    codes = (x * _pow2(BIAS - e)[..., None, None]).to(FP8)
    if values:
        codes = codes.transpose(2, 3).contiguous()
    return codes.view(torch.uint8), e.to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, S, Hkv, d = case["op"], case["S"], case["Hkv"], case["d"]
    Hq = case.get("Hq", Hkv)
    ctx, ql = _lengths(case)
    mbps, nb, N = -(-max(ctx) // BLOCK) + 1, sum(-(-n // BLOCK) for n in ctx) + 3, sum(ql)
    st = dict(case=case, table=_tables(gen, ctx, mbps, nb), ctx=_i32(ctx), ql=_i32(ql), max_q=max(ql), N=N)
    if op == "append" or (op in ("attn8", "blocks", "bounds") and case.get("fp8", True)):
        st["kc"], st["ke"] = _cache8(gen, nb, Hkv, d, False)
        st["vc"], st["ve"] = _cache8(gen, nb, Hkv, d, True)
    elif op != "select":
        st.update(kc=_normal(gen, nb, Hkv, BLOCK, d), vc=_normal(gen, nb, Hkv, BLOCK, d), ke=None, ve=None)
    if op == "append":
        dt = torch.float32 if case["f32"] else torch.bfloat16
        st.update(k=_normal(gen, N, Hkv, d, dtype=dt), v=_normal(gen, N, Hkv, d, dtype=dt), q=None, angles=None, q_out=None)
        st["k"] *= (torch.rand(d, generator=gen, device="cuda").pow(6) * 3 + 0.7).to(dt)
        if case["rope"]:
            half = d // 2
            freq = torch.exp(-LOG_BASE * torch.arange(half, dtype=torch.float64, device="cuda") / half)
            ang = torch.arange(max(ctx), dtype=torch.float64, device="cuda")[:, None] * freq
            st.update(q=_normal(gen, N, Hq, d, dtype=dt), angles=torch.cat([ang.cos(), ang.sin()], 1).float(),
                      q_out=torch.empty(N, Hq, d, dtype=torch.bfloat16, device="cuda"))
        return st
    if op == "bounds":
        st["bounds"] = _normal(gen, nb, Hkv, 2, d)  # of earlier owners of the blocks
        return st
    st["q"] = _normal(gen, N, Hq, d, std=2.0)
    if op == "select":
        # a block's keys lie about a centre of its own
        mid, wide = _normal(gen, nb, Hkv, d, std=0.7), _normal(gen, nb, Hkv, d, std=0.3).abs() + 1.2
        st["bounds"] = torch.stack([mid - wide, mid + wide], 2).contiguous()
        st["sel"] = torch.empty(N, Hkv, case["keep"], dtype=torch.int32, device="cuda")
        if own:
            from paged_kv_cache_tiled_gb300 import fattn as F
            st["ws"] = torch.empty(F.fa_block_select_workspace_size(S, mbps, Hq, Hkv, d, N), dtype=torch.uint8, device="cuda")
        return st
    st["out"] = torch.empty(N, Hq, d, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty(N, Hq, dtype=torch.float32, device="cuda")
    if op == "blocks":
        # the query's own block, and others of those before it, each once; -1 behind the last
        seq, pos = _rows(st)
        near = (pos // BLOCK)[:, None, None]
        b = torch.arange(mbps, device="cuda")
        r = torch.rand(N, Hkv, mbps, generator=gen, device="cuda").masked_fill(b == near, 2.0).masked_fill(b > near, -1.0)
        keep = case["keep"]
        best = torch.nn.functional.pad(r.topk(min(keep, mbps), -1).indices, (0, max(0, keep - mbps)), value=mbps)
        best = best.masked_fill(best > near, mbps).sort(-1).values
        st["sel"] = torch.where(best < mbps, best, torch.full_like(best, -1)).to(torch.int32)
    elif own:
        from paged_kv_cache_tiled_gb300 import fattn as F
        size = F.fa_paged_attn_fp8_scaled_workspace_size(S, mbps, Hq, Hkv, d, N, max(ql))
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- plain forms --
def _rows(st):
    """Per packed query row its sequence and its position."""
    ctx, ql = st["ctx"].long(), st["ql"].long()
    seq = torch.repeat_interleave(torch.arange(ql.numel(), device="cuda"), ql, output_size=st["N"])
    start = ql.cumsum(0) - ql
    return seq, torch.arange(st["N"], device="cuda") - start[seq] + (ctx - ql)[seq]


def _padded(st):
    """The packed rows as [S, max_q]: where each is in the pack, which are real, and their positions."""
    ctx, ql = st["ctx"].long(), st["ql"].long()
    i = torch.arange(st["max_q"], device="cuda")
    rows = ((ql.cumsum(0) - ql)[:, None] + i).clamp(max=st["N"] - 1)
    return rows, i < ql[:, None], (ctx - ql)[:, None] + i


def _values(codes, e):
    """[..., a, b] codes with a scale code for each leading index, as numbers."""
    return codes.view(FP8).float() * _pow2(e.int() - BIAS)[..., None, None]


def _softmax(x, seen):
    """Weights (0 in rows that see nothing) and the logarithm of their sum (-inf there)."""
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total)), (m + torch.log(total)).squeeze(-1)


def _plain_append(st):
    case = st["case"]
    S, d, half = case["S"], case["d"], case["d"] // 2
    seq, pos = _rows(st)
    # 64 bits: what is near a border of the 8-bit values goes to its own side
    k, v = st["k"].double(), st["v"].double()
    if case["rope"]:
        c, s = st["angles"][pos][:, None].double().split(half, -1)

        def turn(x):
            a, b = x.double().split(half, -1)
            return torch.cat([a * c - b * s, b * c + a * s], -1)
        k = turn(k)
        st["q_out"].copy_(turn(st["q"]))
    first = (st["ctx"] - st["ql"]).long()
    mbps = st["table"].shape[1]
    # the blocks written, each once, and the tokens that lie in them already
    key, row = torch.unique(seq * mbps + pos // BLOCK, return_inverse=True)
    bs, blk = key // mbps, key % mbps
    phys = st["table"][bs, blk].long()
    before = torch.arange(BLOCK, device="cuda") < (first[bs] - blk * BLOCK)[:, None]  # [blocks, 16]
    for x, cache, scales, by_channel in ((k, st["kc"], st["ke"], False), (v, st["vc"], st["ve"], True)):
        x = x.float() if not case["rope"] else x
        amax = torch.zeros(key.numel(), case["Hkv"], dtype=x.dtype, device="cuda")
        amax.scatter_reduce_(0, row[:, None].expand(-1, case["Hkv"]), x.abs().amax(-1), "amax")
        old_e = scales[phys].long()
        e = torch.maximum(_scale_code(amax), torch.where(before.any(1)[:, None], old_e, torch.zeros_like(old_e)))
        page = cache[phys].view(FP8)
        if by_channel:
            page = page.transpose(2, 3)
        moved = (page.float() * _pow2(old_e - e)[..., None, None]).to(FP8)
        page = torch.where(before[:, None, :, None], moved.view(torch.uint8), page.contiguous().view(torch.uint8))
        codes = (x * _pow2(BIAS - e)[row][..., None].to(x.dtype)).clamp(-448.0, 448.0)
        page[row, :, pos % BLOCK] = codes.to(FP8).view(torch.uint8)
        cache[phys] = page.transpose(2, 3) if by_channel else page
        scales[phys] = e.to(torch.uint8)
    return st


def _append_outputs(st):
    got = dict(kc=st["kc"].view(FP8), vc=st["vc"].view(FP8), k_exp=st["ke"], v_exp=st["ve"])
    return got if st["q"] is None else dict(got, q=st["q_out"])


def _plain_attn8(st):
    case = st["case"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    rows, real, pos = _padded(st)
    at = st["table"].clamp(min=0).long()
    k = _values(st["kc"][at], st["ke"][at]).transpose(1, 2).flatten(2, 3)  # [S, Hkv, keys, d]
    v = _values(st["vc"][at], st["ve"][at]).transpose(3, 4).transpose(1, 2).flatten(2, 3)
    q = st["q"][rows].float().unflatten(2, (Hkv, Hq // Hkv))
    x = torch.einsum("sqhgd,shkd->shgqk", q, k) * d ** -0.5
    keys = torch.arange(k.shape[2], device="cuda")
    seen = (keys <= pos[..., None]) & real[..., None]
    p, lse = _softmax(x, seen[:, None, None])
    del x
    out = torch.einsum("shgqk,shkd->sqhgd", p, v).flatten(2, 3)
    st["out"][rows[real]] = out[real].to(torch.bfloat16)
    st["lse"][rows[real]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[real]
    return dict(out=st["out"], lse=st["lse"])


def _plain_bounds(st):
    seq, pos = _rows(st)
    mbps = st["table"].shape[1]
    key = torch.unique(seq * mbps + pos // BLOCK)
    s, blk = key // mbps, key % mbps
    phys = st["table"][s, blk].long()
    k = st["kc"][phys].float() if st["ke"] is None else _values(st["kc"][phys], st["ke"][phys])
    real = (blk[:, None] * BLOCK + torch.arange(BLOCK, device="cuda") < st["ctx"][s].long()[:, None])[:, None, :, None]
    lo, hi = k.masked_fill(~real, math.inf).amin(2), k.masked_fill(~real, -math.inf).amax(2)
    st["bounds"][phys] = torch.stack([lo, hi], 2).to(torch.bfloat16)
    return dict(bounds=st["bounds"])


def _plain_select(st):
    case = st["case"]
    Hq, Hkv, keep = case["Hq"], case["Hkv"], case["keep"]
    rows, real, pos = _padded(st)
    at = st["table"].clamp(min=0).long()
    # 64 bits: the scores decide an order
    lo, hi = st["bounds"][at].double().unbind(3)  # [S, blocks, Hkv, d]
    q = st["q"][rows].double().unflatten(2, (Hkv, Hq // Hkv))
    u = torch.einsum("sqhgd,sbhd->sqhgb", q.clamp(min=0), hi) + torch.einsum("sqhgd,sbhd->sqhgb", q.clamp(max=0), lo)
    u = u.amax(3)  # a block matters as much as it does to the head that it matters most to
    b = torch.arange(u.shape[-1], device="cuda")
    count = (pos // BLOCK + 1)[:, :, None, None]  # blocks that the query sees
    u = u.masked_fill((b < case["sink"]) | (b >= count - case["recent"]), math.inf).masked_fill(b >= count, -math.inf)
    n = count.clamp(max=keep)
    best = torch.argsort(u, dim=-1, descending=True, stable=True)[..., :keep]  # equal scores: the earlier block first
    best = torch.nn.functional.pad(best, (0, keep - best.shape[-1]), value=u.shape[-1])
    r = torch.arange(keep, device="cuda")
    best = best.masked_fill(r >= n, u.shape[-1]).sort(-1).values
    best = torch.where(r < n, best, torch.full_like(best, -1)).to(torch.int32)
    st["sel"][rows[real]] = best[real]
    return dict(sel=st["sel"])


def _plain_blocks(st):
    case = st["case"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    seq, pos = _rows(st)
    sel = st["sel"].long()
    phys = st["table"][seq[:, None, None], sel.clamp(min=0)].long().clamp(min=0)
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    if st["ke"] is None:
        k, v = st["kc"][phys, h].float(), st["vc"][phys, h].float()
    else:
        k = _values(st["kc"][phys, h], st["ke"][phys, h])
        v = _values(st["vc"][phys, h], st["ve"][phys, h]).transpose(3, 4)
    k, v = k.flatten(2, 3), v.flatten(2, 3)  # [rows, Hkv, keys, d]
    at = sel[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    seen = ((sel[..., None] >= 0) & (at <= pos[:, None, None, None])).flatten(2)
    q = st["q"].float().unflatten(1, (Hkv, Hq // Hkv))
    p, lse = _softmax(torch.einsum("nhgd,nhkd->nhgk", q, k) * d ** -0.5, seen[:, :, None])
    st["out"].copy_(torch.einsum("nhgk,nhkd->nhgd", p, v).flatten(1, 2))
    st["lse"].copy_(lse.flatten(1, 2))
    return dict(out=st["out"], lse=st["lse"])


# --------------------------------------------------------------------- run --
def run(state):
    return _own(state) if own else _plain(state)


def _plain(st):
    op = st["case"]["op"]
    if op == "append":
        return _append_outputs(_plain_append(st))
    return {"attn8": _plain_attn8, "bounds": _plain_bounds, "select": _plain_select, "blocks": _plain_blocks}[op](st)


def _own(st):
    from paged_kv_cache_tiled_gb300 import fattn as F

    case = st["case"]
    op = case["op"]
    at = (st["table"], st["ctx"], st["ql"])
    if op == "append":
        F.fa_cache_append_fp8_scaled(st["k"], st["v"], st["kc"], st["vc"], st["ke"], st["ve"], *at, q=st["q"],
                                     cos_sin=st["angles"], q_out=st["q_out"])
        return _append_outputs(st)
    if op == "attn8":
        F.fa_paged_attn_fp8_scaled(st["q"], st["kc"], st["vc"], st["ke"], st["ve"], *at, causal=True, out=st["out"],
                                   lse=st["lse"], max_q_len=st["max_q"], ws=st["ws"])
        return dict(out=st["out"], lse=st["lse"])
    if op == "bounds":
        F.fa_block_bounds(st["kc"], *at, st["bounds"], k_exp=st["ke"], total_q=st["N"])
        return dict(bounds=st["bounds"])
    if op == "select":
        F.fa_block_select(st["q"], st["bounds"], *at, case["keep"], recent=case["recent"], sink=case["sink"],
                          sel=st["sel"], max_q_len=st["max_q"], ws=st["ws"])
        return dict(sel=st["sel"])
    F.fa_paged_attn_blocks(st["q"], st["kc"], st["vc"], *at, st["sel"], k_exp=st["ke"], v_exp=st["ve"], out=st["out"],
                           lse=st["lse"])
    return dict(out=st["out"], lse=st["lse"])


# -------------------------------------------------------------------- work --
def work(case):
    op, d, Hkv, S = case["op"], case["d"], case["Hkv"], case["S"]
    Hq = case.get("Hq", Hkv)
    ctx, ql = _lengths(case)
    N = sum(ql)
    table = 4 * sum(-(-c // BLOCK) for c in ctx)
    if op == "append":
        size = 4 if case["f32"] else 2
        written = sum((c - 1) // BLOCK - (c - n) // BLOCK + 1 for c, n in zip(ctx, ql))
        b = N * Hkv * d * 2 * (size + 1) + written * (2 * Hkv + 4) + 8 * S
        if case["rope"]:
            b += N * Hq * d * (size + 2) + len({p for c, n in zip(ctx, ql) for p in range(c - n, c)}) * d * 4
        return dict(bytes=b, flops=(3.0 * N * d * (Hq + Hkv) if case["rope"] else 0.0) + 4.0 * N * Hkv * d)
    if op == "attn8":
        pairs = sum(n * c - n * (n - 1) // 2 for c, n in zip(ctx, ql))
        return dict(bytes=2 * Hkv * d * sum(ctx) + table // 2 * Hkv + table + N * Hq * (4 * d + 4), flops=4.0 * d * Hq * pairs)
    if op == "bounds":
        lo = [(c - n) // BLOCK for c, n in zip(ctx, ql)]
        blocks, keys = sum(-(-c // BLOCK) - b for c, b in zip(ctx, lo)), sum(c - b * BLOCK for c, b in zip(ctx, lo))
        return dict(bytes=Hkv * d * ((1 if case["fp8"] else 2) * keys + 4 * blocks) + 4 * blocks, flops=2.0 * Hkv * d * keys)
    if op == "select":
        keep = case["keep"]
        scored = [[p // BLOCK + 1 for p in range(c - n, c) if p // BLOCK + 1 > keep] for c, n in zip(ctx, ql)]
        most = sum(max(x, default=0) for x in scored)
        return dict(bytes=4 * d * Hkv * most + 4 * most + 2 * d * Hq * sum(map(len, scored)) + 4 * N * Hkv * keep,
                    flops=4.0 * d * Hq * sum(map(sum, scored)))
    keep = case["keep"]
    rows = [[min(keep, p // BLOCK + 1) for p in range(c - n, c)] for c, n in zip(ctx, ql)]
    # a sequence's blocks are read once, however many of its queries chose them
    read = sum(min(sum(x), -(-c // BLOCK)) for x, c in zip(rows, ctx)) * BLOCK
    return dict(bytes=2 * Hkv * d * read * (1 if case["fp8"] else 2) + 4 * N * Hkv * keep + N * Hq * (4 * d + 4),
                flops=4.0 * d * Hq * BLOCK * sum(map(sum, rows)))


# ------------------------------------------------------------------- exact --
def _one_page(codes, e):
    return codes.view(FP8).double() * 2.0 ** (int(e) - BIAS)


def _head(q, k, v, seen):
    """One head in 64 bits: outputs and log sums of q [n, d] over k, v [m, d]; seen [n, m]."""
    z = (q.double() @ k.t()) / math.sqrt(q.shape[1])
    z[~seen] = -math.inf
    lse = torch.logsumexp(z, 1)
    return torch.exp(z - lse.masked_fill(lse == -math.inf, 0.0)[:, None]) @ v, lse


def _exact_append(st, case):
    """Sequence by sequence and block by block; codes as the values of their 8 bits."""
    d, half = case["d"], case["d"] // 2
    ctx, ql = _lengths(case)
    qs = None
    k = st["k"].double()
    seq, pos = _rows(st)
    if case["rope"]:
        w = torch.complex(st["angles"][pos, :half].double(), st["angles"][pos, half:].double())[:, None]

        def turn(x):
            z = torch.complex(x[..., :half].double(), x[..., half:].double()) * w
            return torch.cat([z.real, z.imag], -1)
        k, qs = turn(st["k"]), turn(st["q"])
    kc, vc = st["kc"].view(FP8).double(), st["vc"].view(FP8).double().transpose(2, 3).contiguous()
    ke, ve = st["ke"].clone(), st["ve"].clone()
    table = st["table"].tolist()
    at = 0
    for s, (c, n) in enumerate(zip(ctx, ql)):
        for b in range((c - n) // BLOCK, (c - 1) // BLOCK + 1):
            lo, hi = max(c - n, b * BLOCK), min(c, (b + 1) * BLOCK)
            i, p = at + lo - (c - n), table[s][b]
            for x, cache, es in ((k, kc, ke), (st["v"].double(), vc, ve)):
                new, kept = x[i:i + hi - lo].transpose(0, 1), cache[p, :, :lo - b * BLOCK]
                ratio = new.abs().amax((1, 2)) / 448.0
                e = (torch.ceil(torch.log2(ratio.clamp(min=1e-60))) + BIAS).clamp(min=LEAST)
                e = torch.where(ratio > 2.0 ** (e - BIAS), e + 1, e)  # (log2 rounds)
                e = torch.where((e > LEAST) & (ratio <= 2.0 ** (e - 1 - BIAS)), e - 1, e)
                if lo > b * BLOCK:
                    e = torch.maximum(e, es[p].double())
                step = 2.0 ** (es[p].double() - e)
                cache[p, :, :lo - b * BLOCK] = (kept * step[:, None, None]).to(FP8).double()
                # what is to be held in 8 bits, unrounded
                cache[p, :, lo - b * BLOCK:hi - b * BLOCK] = new * (2.0 ** (BIAS - e))[:, None, None]
                es[p] = e.to(torch.uint8)
        at += n
    got = dict(kc=kc, vc=vc.transpose(2, 3).contiguous(), k_exp=ke, v_exp=ve)
    return got if qs is None else dict(got, q=qs)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, Hkv, N = case["op"], case["Hkv"], st["N"]
    ctx, ql = _lengths(case)
    if op == "append":
        if sum(n // BLOCK + 2 for n in ql) > 4000:
            return None
        return _exact_append(st, case)
    table = st["table"].long()
    if op == "bounds":
        bounds = st["bounds"].double()
        for s, (c, n) in enumerate(zip(ctx, ql)):
            for b in range((c - n) // BLOCK, (c - 1) // BLOCK + 1):
                p = int(table[s, b])
                for h in range(Hkv if st["ke"] is not None else 1):
                    page = st["kc"][p].double() if st["ke"] is None else _one_page(st["kc"][p, h:h + 1], st["ke"][p, h])
                    page = page[:, :c - b * BLOCK]
                    which = slice(None) if st["ke"] is None else slice(h, h + 1)
                    bounds[p, which, 0], bounds[p, which, 1] = page.min(1).values, page.max(1).values
        return dict(bounds=bounds)
    Hq, g = case["Hq"], case["Hq"] // Hkv
    if op == "select":
        keep, sink, recent = case["keep"], case["sink"], case["recent"]
        sel = torch.full((N, Hkv, keep), -1, dtype=torch.int32)
        at = 0
        for s, (c, n) in enumerate(zip(ctx, ql)):
            for h in range(Hkv):
                box = st["bounds"][table[s, :-(-c // BLOCK)], h].double()  # [blocks, 2, d]
                x = st["q"][at:at + n, h * g:(h + 1) * g].double()
                best = None
                for i in range(g):  # the largest product with any corner of the box
                    corner = (x[:, i, None, None] * box).amax(2).sum(-1)
                    best = corner if best is None else torch.maximum(best, corner)
                best = best.cpu().tolist()
                for r in range(n):
                    count = (c - n + r) // BLOCK + 1
                    must = set(range(min(count, sink))) | set(range(max(0, count - recent), count))
                    rest = sorted((b for b in range(count) if b not in must), key=lambda b: (-best[r][b], b))
                    got = sorted((sorted(must) + rest)[:min(keep, count)]) if count > keep else range(count)
                    sel[at + r, h, :len(got)] = torch.tensor(list(got), dtype=torch.int32)
            at += n
        return dict(sel=sel.cuda())
    out = torch.empty(N, Hq, case["d"], dtype=torch.float64, device="cuda")
    lse = torch.empty(N, Hq, dtype=torch.float64, device="cuda")
    if op == "attn8":
        at = 0
        for s, (c, n) in enumerate(zip(ctx, ql)):
            p = table[s, :-(-c // BLOCK)]
            seen = torch.arange(c, device="cuda")[None] <= torch.arange(c - n, c, device="cuda")[:, None]
            for h in range(Hkv):
                f = [2.0 ** (e[p, h].double() - BIAS)[:, None, None] for e in (st["ke"], st["ve"])]
                k = (st["kc"][p, h].view(FP8).double() * f[0]).reshape(-1, case["d"])[:c]
                v = (st["vc"][p, h].view(FP8).double() * f[1]).transpose(1, 2).reshape(-1, case["d"])[:c]
                for i in range(h * g, (h + 1) * g):
                    out[at:at + n, i], lse[at:at + n, i] = _head(st["q"][at:at + n, i], k, v, seen)
            at += n
        return dict(out=out, lse=lse)
    seq, pos = (x.tolist() for x in _rows(st))
    sel = st["sel"].tolist()
    if N * Hkv > 2500:
        return None
    for i in range(N):
        for h in range(Hkv):
            b = torch.tensor([x for x in sel[i][h] if x >= 0], device="cuda")
            p = table[seq[i], b]
            if st["ke"] is None:
                k, v = st["kc"][p, h].double(), st["vc"][p, h].double()
            else:
                k = st["kc"][p, h].view(FP8).double() * 2.0 ** (st["ke"][p, h].double() - BIAS)[:, None, None]
                v = (st["vc"][p, h].view(FP8).double() * 2.0 ** (st["ve"][p, h].double() - BIAS)[:, None, None]).transpose(1, 2)
            seen = ((b[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(1, -1) <= pos[i]).expand(g, -1)
            out[i, h * g:(h + 1) * g], lse[i, h * g:(h + 1) * g] = _head(
                st["q"][i, h * g:(h + 1) * g], k.reshape(-1, case["d"]), v.reshape(-1, case["d"]), seen)
    return dict(out=out, lse=lse)
