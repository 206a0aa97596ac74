"""Cases, inputs, plain forms and 64-bit values of five serving operators.

  prefill   attention over [B, T, H, d] whose scores are capped by a tanh, get a
            bias that falls with distance, or see only a window, a prefix or
            their own document (fa_prefill_mod)
  paged     the same over the paged cache: single tokens and chunks
            (fa_paged_attn_mod)
  mrope     rotary positions with several axes (time, height, width), fused with
            the cache append (fa_cache_append_mrope)
  accum     paged attention that also adds up how much weight every cached token
            received (fa_paged_attn_accum)
  evict     the cache tokens with the largest accumulated weight, and the most
            recent ones, moved into fewer blocks (fa_cache_evict)

`own` selects between the plain form (elementary torch operations in 32 bits,
rounded once) and the library's calls.
"""
import math
import random

import torch

own = False

BLOCK = 16
LOG_BASE = math.log(1.0e6)  # rotary base of the shapes below


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # a short prompt of a small model with capped scores: launch latency
        dict(name="prefill_short_capped", op="prefill", B=2, T=130, Hq=4, Hkv=2, d=64, causal=True, cap=30.0,
             bias=False, window=0, docs=0, prefix=False, layout=1),
        # prompts of a model with a linear distance bias, an odd length
        dict(name="prefill_bias", op="prefill", B=4, T=2041, Hq=12, Hkv=2, d=128, causal=True, cap=0.0, bias=True,
             window=0, docs=0, prefix=False, layout=2),
        # one long row of packed documents, the last part of it padding
        dict(name="prefill_documents_capped", op="prefill", B=1, T=8192, Hq=32, Hkv=8, d=128, causal=True, cap=50.0,
             bias=False, window=0, docs=6, prefix=False, layout=3),
        # a serving step of one sequence: latency
        dict(name="decode_one_bias", op="paged", S=1, ctx_lo=1000, ctx_hi=1000, q_hi=1, Hq=8, Hkv=8, d=128, cap=0.0,
             bias=True, window=0, prefix=False, layout=4),
        # a serving step of a batch, a layer with capped scores and a sliding window
        dict(name="decode_capped_window", op="paged", S=64, ctx_lo=128, ctx_hi=8192, q_hi=1, Hq=12, Hkv=2, d=128,
             cap=50.0, bias=False, window=4096, prefix=False, layout=5),
        # chunks of prompts that begin with an image whose tokens all see each other
        dict(name="chunk_prefix", op="paged", S=16, ctx_lo=300, ctx_hi=4600, q_hi=512, Hq=32, Hkv=8, d=128, cap=0.0,
             bias=False, window=0, prefix=True, layout=6),
        # one token for each sequence of a batch of video chats
        dict(name="mrope_decode", op="mrope", N=64, Hq=12, Hkv=2, d=128, axes=3, interleaved=False, f32=False,
             layout=7),
        # a chunk of an image or video prompt
        dict(name="mrope_prompt", op="mrope", N=4096, Hq=32, Hkv=8, d=128, axes=3, interleaved=True, f32=False,
             layout=8),
        # a serving step that keeps count of the attention weights
        dict(name="accum_decode", op="accum", S=64, ctx_lo=128, ctx_hi=4096, q_hi=1, Hq=12, Hkv=2, d=128, cap=0.0,
             bias=False, window=0, prefix=False, decay=1.0, layout=9),
        # chunks of prompts whose weights are counted before the cache is thinned out
        dict(name="accum_chunk", op="accum", S=8, ctx_lo=300, ctx_hi=4600, q_hi=512, Hq=32, Hkv=8, d=128, cap=0.0,
             bias=False, window=0, prefix=False, decay=1.0, layout=10),
        # a batch of sequences brought down to 512 tokens each
        dict(name="evict_batch", op="evict", S=64, ctx_lo=513, ctx_hi=4096, Hkv=2, d=128, keep=512, recent=64, sink=4,
             layout=11),
        # two long sequences brought down to a quarter
        dict(name="evict_long", op="evict", S=2, ctx_lo=32000, ctx_hi=32768, Hkv=8, d=128, keep=8192, recent=256,
             sink=0, layout=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "paged", "paged", "mrope", "accum", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8])
    c = dict(op=op, d=d, Hkv=Hkv, layout=rng.randrange(1 << 30))
    if op == "prefill":
        c.update(Hq=Hkv * g, B=rng.choice([1, 1, 2, 3]), T=_log_int(rng, 16, 4096), causal=rng.random() < 0.8,
                 cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.4, window=0,
                 docs=rng.choice([0, 0, 1, 5, 20]), prefix=rng.random() < 0.3)
        while c["B"] * c["Hq"] * c["T"] ** 2 * d > 2.5e10:
            c["T"] = c["T"] * 2 // 3
        if rng.random() < 0.3:
            c["window"] = _log_int(rng, 1, 2 * c["T"])
        return c
    if op in ("paged", "accum"):
        S = _log_int(rng, 1, 48)
        hi = _log_int(rng, 16, 8000 if S <= 16 else 4000)
        q_hi = rng.choice([1, 1, 2, 5, _log_int(rng, 6, 300)])
        c.update(Hq=Hkv * g, S=S, ctx_lo=max(q_hi, hi // rng.choice([1, 4, 30])), q_hi=q_hi, cap=rng.choice([0.0, 0.0, 30.0]),
                 bias=rng.random() < 0.3, window=rng.choice([0, 0, _log_int(rng, 4, 4096)]), prefix=rng.random() < 0.2)
        c["ctx_hi"] = max(hi, c["ctx_lo"])
        while c["S"] > 1 and (S * q_hi * hi * c["Hq"] * d > 6e10 or S * hi * Hkv * d > 2e8):
            S = c["S"] = c["S"] // 2
        if op == "accum":
            c["decay"] = rng.choice([1.0, 1.0, 0.9])
        return c
    if op == "mrope":
        c.update(Hq=Hkv * g, N=_log_int(rng, 1, 1800), axes=rng.choice([1, 2, 3, 4]), interleaved=rng.random() < 0.5,
                 f32=rng.random() < 0.3)
        return c
    hi = _log_int(rng, 64, 16000)
    S = _log_int(rng, 1, max(1, min(64, 120000 // hi)))
    keep = _log_int(rng, 16, max(17, hi // 2))
    c.update(S=S, ctx_lo=max(1, hi // rng.choice([1, 2, 20])), ctx_hi=hi, keep=keep, recent=rng.randrange(0, keep // 2 + 1),
             sink=rng.choice([0, 1, 4]))
    return c


# ----------------------------------------------------------------- layouts --
# What a case fixes beside its sizes: the lengths of its sequences, documents
# and prefixes.  Values come from the seed.
def _paged_lengths(case):
    r = random.Random(case["layout"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["S"])]
    ql = [min(c, r.randint(max(1, case["q_hi"] // 8), case["q_hi"])) for c in ctx]
    pre = [r.randint(0, c) if r.random() < 0.8 else 0 for c in ctx]
    return ctx, ql, pre


def _documents(case):
    """Per row of the batch: the documents' lengths, and the length of the padding behind them."""
    r = random.Random(case["layout"])
    rows = []
    for _ in range(case["B"]):
        T = case["T"]
        pad = r.randint(0, T // 16)
        cuts = sorted(r.randint(0, T - pad) for _ in range(case["docs"] - 1))
        ends = [0] + cuts + [T - pad]
        rows.append(([b - a for a, b in zip(ends, ends[1:]) if b > a], pad))
    return rows


def _prefixes(case):
    r = random.Random(case["layout"] + 1)
    return [r.randint(0, case["T"]) for _ in range(case["B"])]


# ------------------------------------------------------------------ inputs --
def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _slopes(Hq):
    """2^(-8 (h + 1) / Hq): a geometric series over the heads."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(gen, lens, mbps, num_blocks, perm=None, at=0):
    """Block tables of sequences of these lengths over a shuffled pool; unused entries are -1."""
    if perm is None:
        perm = torch.randperm(num_blocks, generator=gen, device="cuda").cpu()
    table = torch.full((len(lens), mbps), -1, dtype=torch.int32)
    for s, n in enumerate(lens):
        nb = -(-n // BLOCK)
        table[s, :nb] = perm[at:at + nb].to(torch.int32)
        at += nb
    return table.cuda(), perm, at


def _blocks(lens):
    return sum(-(-n // BLOCK) for n in lens)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    st = dict(case=case)
    if op == "prefill":
        B, T, Hq = case["B"], case["T"], case["Hq"]
        # score deviations of about 2 (8 where they are capped, so that the cap bends them)
        std = 8.0 if case["cap"] else 2.0
        st.update(q=_normal(gen, B, T, Hq, d, std=std), k=_normal(gen, B, T, Hkv, d), v=_normal(gen, B, T, Hkv, d),
                  slopes=_slopes(Hq) if case["bias"] else None, docs=None, prefix=None,
                  out=torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.empty(B, Hq, T, dtype=torch.float32, device="cuda"))
        if case["docs"]:
            ids = []
            for lens, pad in _documents(case):
                ids.append([i for i, n in enumerate(lens) for _ in range(n)] + [-1] * pad)
            st["docs"] = _i32(ids)
        if case["prefix"]:
            st["prefix"] = _i32(_prefixes(case))
        if own:
            from paged_kv_cache_tiled_gb300 import fattn as F
            st["ws"] = torch.empty(max(1, F.fa_prefill_mod_workspace_size(B, T)), dtype=torch.uint8, device="cuda")
        return st
    if op in ("paged", "accum"):
        Hq = case["Hq"]
        ctx, ql, pre = _paged_lengths(case)
        mbps = -(-max(ctx) // BLOCK) + 1
        nb = _blocks(ctx) + 3
        table, _, _ = _tables(gen, ctx, mbps, nb)
        total = sum(ql)
        st.update(q=_normal(gen, total, Hq, d, std=8.0 if case["cap"] else 2.0), kc=_normal(gen, nb, Hkv, BLOCK, d),
                  vc=_normal(gen, nb, Hkv, BLOCK, d), table=table, ctx=_i32(ctx), ql=_i32(ql), max_q=max(ql),
                  slopes=_slopes(Hq) if case["bias"] else None, prefix=_i32(pre) if case["prefix"] else None,
                  out=torch.empty(total, Hq, d, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.empty(total, Hq, dtype=torch.float32, device="cuda"))
        if op == "accum":
            # weights counted by earlier steps: most tokens next to nothing, a few a lot
            st["acc"] = torch.rand(case["S"], Hkv, mbps * BLOCK, generator=gen, device="cuda").pow(8).mul_(20)
            st["acc_out"] = torch.zeros_like(st["acc"])
        if own:
            from paged_kv_cache_tiled_gb300 import fattn as F
            size = F.fa_paged_attn_accum_workspace_size if op == "accum" else F.fa_paged_attn_mod_workspace_size
            st["ws"] = torch.empty(size(case["S"], mbps, Hq, Hkv, d, total, max(ql)), dtype=torch.uint8, device="cuda")
        return st
    if op == "mrope":
        N, Hq, A = case["N"], case["Hq"], case["axes"]
        nb = -(-N // BLOCK) + 2
        max_pos = 4096
        dt = torch.float32 if case["f32"] else torch.bfloat16
        half = d // 2
        freq = torch.exp(-LOG_BASE * torch.arange(half, dtype=torch.float64, device="cuda") / half)
        ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq
        axes = [j % A for j in range(half)] if case["interleaved"] else [min(A - 1, j * A // half) for j in range(half)]
        slots = torch.randperm(nb * BLOCK, generator=gen, device="cuda")[:N].to(torch.int32)
        slots[3::97] = -1  # tokens that are not cached
        st.update(q=_normal(gen, N, Hq, d, dtype=dt), k=_normal(gen, N, Hkv, d, dtype=dt),
                  v=_normal(gen, N, Hkv, d, dtype=dt), axes=axes, axes_dev=_i32(axes).long(),
                  positions=torch.randint(0, max_pos, (A, N), generator=gen, device="cuda", dtype=torch.int32),
                  table=torch.cat([ang.cos(), ang.sin()], 1).float(), slots=slots,
                  q_out=torch.empty(N, Hq, d, dtype=torch.bfloat16, device="cuda"),
                  kc=torch.zeros(nb, Hkv, BLOCK, d, dtype=torch.bfloat16, device="cuda"),
                  vc=torch.zeros(nb, Hkv, BLOCK, d, dtype=torch.bfloat16, device="cuda"))
        return st
    ctx, _, _ = _paged_lengths(dict(case, q_hi=1))
    new = [min(c, case["keep"]) for c in ctx]
    nb = _blocks(ctx) + _blocks(new) + 2
    mbps, dmbps = -(-max(ctx) // BLOCK), -(-max(new) // BLOCK)
    table, perm, at = _tables(gen, ctx, mbps, nb)
    dst, _, _ = _tables(gen, new, dmbps, nb, perm, at)
    acc = torch.rand(case["S"], Hkv, mbps * BLOCK, generator=gen, device="cuda").pow(8).mul_(20)
    acc[acc < 1e-3] = 0.0  # tokens that no query looked at: many equal values
    st.update(kc=_normal(gen, nb, Hkv, BLOCK, d), vc=_normal(gen, nb, Hkv, BLOCK, d), acc=acc, table=table, dst=dst,
              ctx=_i32(ctx), new_lens=torch.empty(case["S"], dtype=torch.int32, device="cuda"),
              kept=torch.empty(case["S"], Hkv, case["keep"], dtype=torch.int32, device="cuda"),
              acc_out=torch.zeros(case["S"], Hkv, case["keep"], device="cuda"))
    if own:
        from paged_kv_cache_tiled_gb300 import fattn as F
        st["ws"] = torch.empty(F.fa_cache_evict_workspace_size(case["S"], mbps, Hkv, case["keep"]), dtype=torch.uint8,
                               device="cuda")
    return st


# ------------------------------------------------------------- plain forms --
def _seen(pos, keys, end, causal, window, prefix):
    """Truth values of key `keys` for a query at `pos` (tensors that broadcast); `end`: the sequence's length."""
    ahead = keys <= pos if causal else keys < end
    if causal and prefix is not None:
        ahead = ahead | (keys < prefix)
    if window:
        ahead = ahead & (keys > pos - window)
        if not causal:
            ahead = ahead & (keys < pos + window)
    return ahead & (keys < end)


def _scores(dots, scale, cap, slopes, pos, keys):
    x = dots * scale
    if cap:
        x = cap * torch.tanh(x / cap)
    if slopes is not None:
        x = x - slopes * (keys - pos).abs()
    return x


def _softmax(x, seen):
    """Weights (0 in rows that see nothing) and the logarithm of their sum (-inf there)."""
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total)), (m + torch.log(total)).squeeze(-1)


def _plain_prefill(st):
    case = st["case"]
    B, T, Hq, Hkv, d = (case[n] for n in ("B", "T", "Hq", "Hkv", "d"))
    g = Hq // Hkv
    q = st["q"].float().view(B, T, Hkv, g, d)
    x = torch.einsum("bthgd,bshd->bhgts", q, st["k"].float())
    at = torch.arange(T, device="cuda")
    pos, keys = at[:, None], at[None, :]
    prefix = st["prefix"][:, None, None, None, None] if st["prefix"] is not None else None
    seen = _seen(pos, keys, T, case["causal"], case["window"], prefix)
    if st["docs"] is not None:
        ids = st["docs"]
        same = (ids[:, :, None] == ids[:, None, :]) & (ids[:, :, None] >= 0)
        seen = seen & same[:, None, None]
    slopes = st["slopes"].view(Hkv, g, 1, 1) if st["slopes"] is not None else None
    p, lse = _softmax(_scores(x, d ** -0.5, case["cap"], slopes, pos, keys), seen)
    del x
    out = torch.einsum("bhgts,bshd->bthgd", p, st["v"].float()).reshape(B, T, Hq, d)
    return dict(out=out.to(torch.bfloat16), lse=lse.reshape(B, Hq, T))


def _gathered(cache, table):
    """[S, tokens, Hkv, ...] of a paged array [blocks, Hkv, 16, ...]."""
    x = cache[table.clamp(min=0).long()].transpose(2, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:])


def _paged_weights(st):
    """Weights [S, Hkv, g, queries, keys], log sums, and the padded rows' places and which of them are real."""
    case = st["case"]
    S, Hq, Hkv, d = case["S"], case["Hq"], case["Hkv"], case["d"]
    g = Hq // Hkv
    ctx, ql = st["ctx"].long(), st["ql"].long()
    i = torch.arange(st["max_q"], device="cuda")
    real = i < ql[:, None]
    rows = ((ql.cumsum(0) - ql)[:, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().view(S, -1, Hkv, g, d)
    k = _gathered(st["kc"], st["table"]).float()
    x = torch.einsum("sqhgd,skhd->shgqk", q, k)
    pos = ((ctx - ql)[:, None] + i)[:, None, None, :, None]
    keys = torch.arange(k.shape[1], device="cuda")
    prefix = st["prefix"][:, None, None, None, None] if st["prefix"] is not None else None
    seen = _seen(pos, keys, ctx[:, None, None, None, None], True, case["window"], prefix) & real[:, None, None, :, None]
    slopes = st["slopes"].view(Hkv, g, 1, 1) if st["slopes"] is not None else None
    p, lse = _softmax(_scores(x, d ** -0.5, case["cap"], slopes, pos, keys), seen)
    return p, lse, rows, real


def _plain_paged(st):
    p, lse, rows, real = _paged_weights(st)
    v = _gathered(st["vc"], st["table"]).float()
    out = torch.einsum("shgqk,skhd->sqhgd", p, v).flatten(2, 3)
    st["out"][rows[real]] = out[real].to(torch.bfloat16)
    st["lse"][rows[real]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[real]
    return p, dict(out=st["out"], lse=st["lse"])


def _plain_accum(st):
    p, got = _plain_paged(st)
    w = p.sum((2, 3))  # [S, Hkv, keys]
    ctx, old = st["ctx"].long(), st["acc"]
    keys = torch.arange(w.shape[2], device="cuda")
    before = keys < (ctx - st["ql"].long())[:, None, None]
    new = torch.where(before, old * st["case"]["decay"], torch.zeros_like(old)) + w
    st["acc_out"].copy_(torch.where(keys < ctx[:, None, None], new, st["acc_out"]))
    return dict(got, acc=st["acc_out"])


def _plain_mrope(st):
    case = st["case"]
    half = case["d"] // 2
    j = torch.arange(half, device="cuda")
    row = st["positions"][st["axes_dev"]].long().t()  # [N, d / 2]
    c, s = st["table"][row, j][:, None], st["table"][row, j + half][:, None]

    def turn(x):
        x = x.float()
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * c - b * s, b * c + a * s], -1).to(torch.bfloat16)

    st["q_out"].copy_(turn(st["q"]))
    put = st["slots"] >= 0
    at = st["slots"][put].long()
    st["kc"][at // BLOCK, :, at % BLOCK] = turn(st["k"])[put]
    st["vc"][at // BLOCK, :, at % BLOCK] = st["v"][put].to(torch.bfloat16)
    return dict(q=st["q_out"], kc=st["kc"], vc=st["vc"])


def _plain_evict(st):
    case = st["case"]
    keep = case["keep"]
    ctx = st["ctx"].long()
    a = st["acc"]
    t = torch.arange(a.shape[2], device="cuda")
    end = ctx[:, None, None]
    a = a.masked_fill((t < case["sink"]) | (t >= end - case["recent"]), math.inf).masked_fill(t >= end, -math.inf)
    n = torch.minimum(ctx, torch.full_like(ctx, keep))
    first = torch.argsort(a, dim=-1, descending=True, stable=True)[..., :keep]  # equal weights: the earlier token first
    first = torch.nn.functional.pad(first, (0, keep - first.shape[-1]), value=t.numel())
    r = torch.arange(keep, device="cuda")
    first = first.masked_fill(r >= n[:, None, None], t.numel()).sort(-1).values
    real = r < n[:, None, None].expand_as(first)
    st["kept"].copy_(torch.where(real, first, torch.full_like(first, -1)))
    st["new_lens"].copy_(n)
    h = torch.arange(case["Hkv"], device="cuda")[None, :, None].expand_as(first)[real]
    s = torch.arange(case["S"], device="cuda")[:, None, None].expand_as(first)[real]
    src, to = first[real], r.expand_as(first)[real]
    sb, db = st["table"][s, src // BLOCK].long(), st["dst"][s, to // BLOCK].long()
    for x in (st["kc"], st["vc"]):
        x[db, h, to % BLOCK] = x[sb, h, src % BLOCK]
    st["acc_out"][s, h, to] = st["acc"][s, h, src]
    return dict(kc=st["kc"], vc=st["vc"], acc=st["acc_out"], kept=st["kept"], new_lens=st["new_lens"])


# --------------------------------------------------------------------- run --
def run(state):
    return _own(state) if own else _plain(state)


def _plain(st):
    op = st["case"]["op"]
    if op == "prefill":
        return _plain_prefill(st)
    if op == "paged":
        return _plain_paged(st)[1]
    return {"accum": _plain_accum, "mrope": _plain_mrope, "evict": _plain_evict}[op](st)


def _own(st):
    from paged_kv_cache_tiled_gb300 import fattn as F

    case = st["case"]
    op = case["op"]
    if op == "prefill":
        F.fa_prefill_mod(st["q"], st["k"], st["v"], causal=case["causal"], softcap=case["cap"],
                         alibi_slopes=st["slopes"], window=case["window"], prefix_lens=st["prefix"],
                         doc_ids=st["docs"], out=st["out"], lse=st["lse"], ws=st["ws"])
        return dict(out=st["out"], lse=st["lse"])
    if op == "paged":
        F.fa_paged_attn_mod(st["q"], st["kc"], st["vc"], st["table"], st["ctx"], st["ql"], causal=True,
                            softcap=case["cap"], alibi_slopes=st["slopes"], window=case["window"],
                            prefix_lens=st["prefix"], out=st["out"], lse=st["lse"], max_q_len=st["max_q"],
                            ws=st["ws"])
        return dict(out=st["out"], lse=st["lse"])
    if op == "accum":
        F.fa_paged_attn_accum(st["q"], st["kc"], st["vc"], st["table"], st["ctx"], st["ql"], st["acc"],
                              st["acc_out"], decay=case["decay"], causal=True, softcap=case["cap"],
                              alibi_slopes=st["slopes"], window=case["window"], prefix_lens=st["prefix"],
                              out=st["out"], lse=st["lse"], max_q_len=st["max_q"], ws=st["ws"])
        return dict(out=st["out"], lse=st["lse"], acc=st["acc_out"])
    if op == "mrope":
        F.fa_cache_append_mrope(st["q"], st["k"], st["v"], st["positions"], st["axes"], st["table"], st["kc"],
                                st["vc"], st["slots"], q_out=st["q_out"])
        return dict(q=st["q_out"], kc=st["kc"], vc=st["vc"])
    F.fa_cache_evict(st["kc"], st["vc"], st["acc"], st["table"], st["ctx"], st["dst"], case["keep"],
                     recent=case["recent"], sink=case["sink"], acc_out=st["acc_out"], new_lens=st["new_lens"],
                     kept=st["kept"], ws=st["ws"])
    return dict(kc=st["kc"], vc=st["vc"], acc=st["acc_out"], kept=st["kept"], new_lens=st["new_lens"])


# -------------------------------------------------------------------- work --
def _pairs(lo_pos, n, end, causal, window, prefix):
    """(query, key) pairs of the queries at lo_pos .. lo_pos + n - 1 of a sequence of `end` keys."""
    pairs = 0
    for p in range(lo_pos, lo_pos + n):
        hi = max(p + 1, min(prefix, end)) if causal else (min(end, p + window) if window else end)
        lo = max(0, p - window + 1) if window else 0
        pairs += max(0, hi - lo)
    return pairs


def work(case):
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "prefill":
        B, T, Hq = case["B"], case["T"], case["Hq"]
        pre = _prefixes(case) if case["prefix"] else [0] * B
        pairs = 0
        for b in range(B):
            spans, at = [(0, T)], 0
            if case["docs"]:
                spans = []
                for n in _documents(case)[b][0]:
                    spans.append((at, n))
                    at += n
            for start, n in spans:  # positions count from the start of the row, and so does the prefix
                pairs += _pairs(0, n, n, case["causal"], case["window"], max(0, pre[b] - start))
        extra = 4 * B * T if case["docs"] else 0
        return dict(bytes=2 * B * T * d * (2 * Hq + 2 * Hkv) + 4 * B * T * Hq + extra, flops=4.0 * d * Hq * pairs)
    if op in ("paged", "accum"):
        Hq = case["Hq"]
        ctx, ql, pre = _paged_lengths(case)
        pairs = keys = 0
        for c, n, p in zip(ctx, ql, pre):
            pairs += _pairs(c - n, n, c, True, case["window"], p if case["prefix"] else 0)
            keys += c - (max(0, c - n - case["window"] + 1) if case["window"] else 0)
        total = sum(ql)
        b = 2 * 2 * Hkv * d * keys + total * Hq * (4 * d + 4) + 4 * (keys // BLOCK)
        if op == "accum":
            b += 8 * Hkv * sum(ctx)
        return dict(bytes=b, flops=4.0 * d * Hq * pairs)
    if op == "mrope":
        N, Hq, size = case["N"], case["Hq"], 4 if case["f32"] else 2
        return dict(bytes=N * d * ((size + 2) * (Hq + 2 * Hkv) + 4) + 4 * N * (case["axes"] + 1),
                    flops=3.0 * N * d * (Hq + Hkv))
    ctx, _, _ = _paged_lengths(dict(case, q_hi=1))
    kept = sum(min(c, case["keep"]) for c in ctx)
    return dict(bytes=Hkv * (4 * sum(ctx) + kept * (2 * 2 * 2 * d + 4) + 4 * case["S"] * case["keep"]), flops=0.0)


# ------------------------------------------------------------------- exact --
def _exact_rows(q, k, v, scale, cap, slope, pos, visible):
    """One head in 64 bits: outputs, log sums and weights of q [n, d] over k, v [m, d]; visible [n, m]."""
    z = (q.double() @ k.double().t()) * scale
    if cap:
        e = torch.exp(-2.0 * z.abs() / cap)
        z = torch.sign(z) * cap * ((1.0 - e) / (1.0 + e))
    if slope is not None:
        z -= float(slope) * (pos[:, None] - torch.arange(k.shape[0], device=k.device)[None]).abs().double()
    z[~visible] = -math.inf
    lse = torch.logsumexp(z, 1)
    w = torch.exp(z - lse.masked_fill(lse == -math.inf, 0.0)[:, None])
    return w @ v.double(), lse, w


def _visible(pos, m, causal, window, prefix):
    k = torch.arange(m, device="cuda")[None]
    p = pos[:, None]
    v = torch.ones(pos.numel(), m, dtype=torch.bool, device="cuda")
    if causal:
        v &= (k <= p) | (k < prefix)
    if window:
        v &= (p - k < window) & ((k - p < window) | torch.tensor(causal, device="cuda"))
    return v


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "mrope":
        half = d // 2
        turned = []
        for x in (st["q"], st["k"]):
            z = torch.complex(x[..., :half].double(), x[..., half:].double())
            ang = torch.empty(case["N"], half, dtype=torch.complex128, device="cuda")
            for j, a in enumerate(st["axes"]):
                rows = st["table"][st["positions"][a].long()].double()
                ang[:, j] = torch.complex(rows[:, j], rows[:, j + half])
            z = z * ang[:, None]
            turned.append(torch.cat([z.real, z.imag], -1))
        kc, vc = st["kc"].double(), st["vc"].double()
        for i, slot in enumerate(st["slots"].tolist()):
            if slot >= 0:
                kc[slot // BLOCK, :, slot % BLOCK] = turned[1][i]
                vc[slot // BLOCK, :, slot % BLOCK] = st["v"][i].double()
        return dict(q=turned[0], kc=kc, vc=vc)
    if op == "evict":
        keep, S = case["keep"], case["S"]
        kc, vc, acc = st["kc"].double(), st["vc"].double(), st["acc_out"].double()
        for s, c in enumerate(st["ctx"].tolist()):
            src, dst = st["table"][s].long(), st["dst"][s].long()
            for h in range(Hkv):
                a = st["acc"][s, h, :c].tolist()
                must = set(range(min(c, case["sink"]))) | set(range(max(0, c - case["recent"]), c))
                best = sorted((t for t in range(c) if t not in must), key=lambda t: (-a[t], t))
                got = sorted((sorted(must) + best)[:keep])
                f, t = torch.tensor(got, device="cuda"), torch.arange(len(got), device="cuda")
                for x, y in ((kc, st["kc"]), (vc, st["vc"])):
                    x[dst[t // BLOCK], h, t % BLOCK] = y[src[f // BLOCK], h, f % BLOCK].double()
                acc[s, h, :len(got)] = st["acc"][s, h, f].double()
        return dict(kc=kc, vc=vc, acc=acc, kept=None, new_lens=None)
    Hq, scale = case["Hq"], 1.0 / math.sqrt(d)
    g = Hq // Hkv
    if op == "prefill":
        B, T = case["B"], case["T"]
        pos = torch.arange(T, device="cuda")
        out = torch.empty(B, T, Hq, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(B, Hq, T, dtype=torch.float64, device="cuda")
        pre = _prefixes(case) if case["prefix"] else [0] * B
        for b in range(B):
            vis = _visible(pos, T, case["causal"], case["window"], pre[b])
            if case["docs"]:
                block = torch.zeros_like(vis)
                at = 0
                for n in _documents(case)[b][0]:
                    block[at:at + n, at:at + n] = True
                    at += n
                vis &= block
            for h in range(Hq):
                out[b, :, h], lse[b, h], _ = _exact_rows(
                    st["q"][b, :, h], st["k"][b, :, h // g], st["v"][b, :, h // g], scale, case["cap"],
                    st["slopes"][h] if case["bias"] else None, pos, vis)
        return dict(out=out, lse=lse)
    ctx, ql, pre = _paged_lengths(case)
    total = sum(ql)
    out = torch.empty(total, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(total, Hq, dtype=torch.float64, device="cuda")
    acc = st["acc_out"].double() if op == "accum" else None
    at = 0
    for s, (c, n, p) in enumerate(zip(ctx, ql, pre)):
        blocks = st["table"][s, :-(-c // BLOCK)].long()
        pos = torch.arange(c - n, c, device="cuda")
        vis = _visible(pos, c, True, case["window"], p if case["prefix"] else 0)
        for h in range(Hkv):
            k = st["kc"][blocks, h].reshape(-1, d)[:c]
            v = st["vc"][blocks, h].reshape(-1, d)[:c]
            counted = torch.zeros(c, dtype=torch.float64, device="cuda")
            for i in range(h * g, (h + 1) * g):
                out[at:at + n, i], lse[at:at + n, i], w = _exact_rows(
                    st["q"][at:at + n, i], k, v, scale, case["cap"], st["slopes"][i] if case["bias"] else None, pos, vis)
                counted += w.sum(0)
            if acc is not None:
                old = st["acc"][s, h, :c].double() * case["decay"]
                old[c - n:] = 0.0
                acc[s, h, :c] = old + counted
        at += n
    got = dict(out=out, lse=lse)
    return got if acc is None else dict(got, acc=acc)
