"""64-bit plain attention with modified scores, and the bounds its GPU forms are held to.

Everything here is written from the formulas (logits, masks, softmax), with the
whole weight matrix of a head materialised on the CPU.
"""
import math

import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2  # 2^-8, the largest relative error of one rounding
F32 = torch.finfo(torch.float32).eps / 2         # 2^-24


def visible(pos, n_keys, causal, window=0, prefix=0, ids=None):
    """Truth values [len(pos), n_keys]."""
    i, j = pos[:, None], torch.arange(n_keys)[None]
    see = torch.ones(len(pos), n_keys, dtype=torch.bool)
    if causal:
        see &= (j <= i) | (j < prefix)
    if window:
        see &= j > i - window
        if not causal:
            see &= j < i + window
    if ids is not None:
        edge = torch.cat([torch.ones(1, dtype=torch.bool), ids[1:] != ids[:-1]])
        run = edge.cumsum(0)
        see &= (run[pos][:, None] == run[None]) & (ids[pos] >= 0)[:, None]
    return see


class Rows:
    """One head's rows: out, lse, weights, and the bounds on the GPU's errors."""

    def __init__(self, q, k, v, pos, see, scale, cap=0.0, slope=None):
        q, k, v = q.double(), k.double(), v.double()
        z = scale * (q @ k.T)
        x = cap * torch.tanh(z / cap) if cap else z
        if slope is not None:
            x = x - float(slope) * (pos[:, None] - torch.arange(k.shape[0])[None]).abs()
        x = x.masked_fill(~see, -math.inf)
        self.lse = torch.logsumexp(x, 1)
        self.w = torch.exp(x - self.lse.masked_fill(self.lse == -math.inf, 0.0)[:, None])
        self.out = self.w @ v
        # A logit is a sum of d products (exact in fp32) accumulated in fp32, with a few more fp32
        # operations; tanh is off by at most 3e-7, of a cap's size; the bias is one product.
        dots = scale * (q.abs() @ k.abs().T)
        dots = torch.where(see, dots, torch.zeros_like(dots)).amax(1)
        size = torch.where(see, x.abs(), torch.zeros_like(x)).amax(1)
        self.logit_tol = (q.shape[1] + 2) * F32 * dots + 4 * F32 * size + 3e-7 * cap
        # lse: the logits' error, 2^-22 of the exponentials and the logarithm, the sum's fp32 roundings
        self.lse_tol = self.logit_tol + 2.0 ** -20 + 4 * F32 * self.lse.abs().nan_to_num(0.0, 0.0, 0.0)
        # weights relative: both the logit's and the lse's error
        self.w_rel = 2 * (self.logit_tol + self.lse_tol)
        # out: every weight rounded to bf16 once (2^-8 of its size), the result once more
        mass = self.w @ v.abs()
        self.out_tol = (HALF_BF16 + self.w_rel[:, None] + 2.0 ** -18) * mass + HALF_BF16 * (
            self.out.abs() + (HALF_BF16 + self.w_rel[:, None]) * mass) + 1e-30


def check(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), f"{what}: non-finite values differ"
    assert torch.isfinite(got[fine]).all(), f"{what}: non-finite output"
    over = (got - want).abs()[fine] - tol.expand_as(want)[fine]
    if over.numel():
        i = int(over.argmax())
        assert over.max() <= 0, f"{what}: off by {float((got - want).abs()[fine][i]):.3e}, bound {float(tol.expand_as(want)[fine][i]):.3e}"


def slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32)


class Paged:
    """A paged problem: contexts, chunks, a shuffled pool whose unused blocks and unused rows hold NaN."""

    def __init__(self, seed, ctx, ql, Hq, Hkv, d, std=1.0, window=0, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.ql, self.Hq, self.Hkv, self.d = ctx, ql, Hq, Hkv, d
        S, self.total = len(ctx), sum(ql)
        mbps = max(1, -(-max(ctx) // 16)) + 1
        nb = sum(-(-c // 16) for c in ctx) + spare
        perm = torch.randperm(nb, generator=g).to(torch.int32)
        self.q = (torch.randn(self.total, Hq, d, generator=g) * std).bfloat16()
        self.kc = torch.full((nb, Hkv, 16, d), math.nan, dtype=torch.bfloat16)
        self.vc = self.kc.clone()
        self.table = torch.full((S, mbps), -1, dtype=torch.int32)
        self.k, self.v = [], []
        at = 0
        for s, c in enumerate(ctx):
            k = torch.randn(c, Hkv, d, generator=g).bfloat16()
            v = torch.randn(c, Hkv, d, generator=g).bfloat16()
            self.k.append(k)
            self.v.append(v)
            first = max(0, c - ql[s] - window + 1) // 16 if window and ql[s] else 0
            for b in range(-(-c // 16)):
                n = min(16, c - 16 * b)
                blk = int(perm[at])
                at += 1
                if b < first:
                    continue  # out of every query's sight: no table entry, NaN in the block
                self.table[s, b] = blk
                self.kc[blk, :, :n] = k[16 * b:16 * b + n].transpose(0, 1)
                self.vc[blk, :, :n] = v[16 * b:16 * b + n].transpose(0, 1)

    def cuda(self):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
        return self.q.cuda(), self.kc.cuda(), self.vc.cuda(), self.table.cuda(), i32(self.ctx), i32(self.ql)

    def rows(self, causal=True, cap=0.0, bias=None, window=0, prefix=None, scale=None):
        """[(sequence, head, first row, Rows)]"""
        scale = self.d ** -0.5 if scale is None else scale
        got, at = [], 0
        for s, (c, n) in enumerate(zip(self.ctx, self.ql)):
            pos = torch.arange(c - n, c)
            see = visible(pos, c, causal, window, int(prefix[s]) if prefix is not None else 0)
            for h in range(self.Hq):
                if n:
                    kv = h // (self.Hq // self.Hkv)
                    got.append((s, h, at, Rows(self.q[at:at + n, h], self.k[s][:, kv], self.v[s][:, kv], pos, see,
                                               scale, cap, None if bias is None else bias[h])))
            at += n
        return got
