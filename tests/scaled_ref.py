"""64-bit plain forms of the 8-bit cache with block scales and of attention over chosen blocks, written from the
formulas, on the CPU, and the bounds that their GPU forms are held to."""
import math

import torch

B = 16
FP8 = torch.float8_e4m3fn
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2  # 2^-8, the largest relative error of one rounding
HALF_F16 = torch.finfo(torch.float16).eps / 2    # 2^-11
LEAST, BIAS = 87, 127


def values(codes, e, by_channel=False):
    """Codes [..., a, b] with scale codes [...] as numbers; by_channel: [..., d, 16] turned to [..., 16, d]."""
    x = codes.view(FP8).double() * 2.0 ** (e.double() - BIAS)[..., None, None]
    return x.transpose(-1, -2) if by_channel else x


def scale_code(amax: float) -> int:
    e = LEAST
    while amax > 448.0 * 2.0 ** (e - BIAS):
        e += 1
    return e


def to_code(x):
    """E4M3 codes of 64-bit numbers: round to nearest even, saturating, NaN kept.  (fp32 in between would round twice.)"""
    a = x.abs().clamp(max=448.0)
    m, p = torch.frexp(a)                      # a = m 2^p, m in [0.5, 1)
    step = 2.0 ** (p.clamp(min=-5) - 4).double()  # 3 mantissa bits behind the first; 2^-9 below 2^-6
    return torch.copysign(torch.round(a / step) * step, x).float().to(FP8).view(torch.uint8)


def turn(x, table, pos):
    """Rotate-half by the table's rows."""
    h = x.shape[-1] // 2
    c, s = table[pos, :h].double()[:, None], table[pos, h:].double()[:, None]
    a, b = x[..., :h].double(), x[..., h:].double()
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def append(kc, vc, ke, ve, k, v, table, ctx, ql):
    """The append on host tensors, in place; k and v in 64 bits, k turned already."""
    at = 0
    for s, (c, n) in enumerate(zip(ctx, ql)):
        for b in range((c - n) // B, (c - 1) // B + 1 if n else 0):
            lo, hi = max(c - n, b * B), min(c, (b + 1) * B)
            p, i = int(table[s, b]), at + lo - (c - n)
            for x, cache, exps, turned in ((k, kc, ke, False), (v, vc, ve, True)):
                for h in range(x.shape[1]):
                    page = cache[p, h].T.clone() if turned else cache[p, h].clone()
                    new = x[i:i + hi - lo, h]
                    finite = new[new.isfinite()].abs()
                    e, old = scale_code(float(finite.max()) if finite.numel() else 0.0), int(exps[p, h])
                    if lo > b * B:
                        e = max(e, old)
                        if e != old:
                            page[:lo - b * B] = to_code(page[:lo - b * B].view(FP8).double() * 2.0 ** (old - e))
                    page[lo - b * B:hi - b * B] = to_code(new * 2.0 ** (BIAS - e))
                    cache[p, h] = page.T if turned else page
                    exps[p, h] = e
        at += n


class Rows:
    """One head's rows over keys k, v [m, d], `see` [n, m]: out and lse in 64 bits, and what the GPU's may be off by."""

    def __init__(self, q, k, v, see, scale, p_half):
        q, k, v = q.double(), k.double(), v.double()
        v = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))
        k = torch.where(see.any(0)[:, None], k, torch.zeros_like(k))
        x = (scale * (q @ k.T)).masked_fill(~see, -math.inf)
        self.lse = torch.logsumexp(x, 1) if k.shape[0] else torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
        w = torch.exp(x - self.lse.masked_fill(self.lse == -math.inf, 0.0)[:, None])
        self.out = w @ v
        # logits: products added in fp32, d / 16 steps of 2^-18 of the magnitudes that meet, then the scale and
        # the subtraction of the maximum (2^-22 of a logit); ex2's own 2^-22
        big = scale * (q.abs() @ k.abs().T)
        big = torch.where(see, big, torch.zeros_like(big)).amax(1) if k.shape[0] else torch.zeros(q.shape[0], dtype=torch.float64)
        dx = big * (q.shape[1] / 16 * 2.0 ** -18 + 2.0 ** -21) + 2.0 ** -20
        mass = w @ v.abs()
        # a weight: its logit's error twice (its own, and the sum's), its rounding for the MMA (relative p_half, or
        # 2^-25 of the largest weight times value scale), sums in fp32; the output's rounding
        top = v.abs().amax() if v.numel() else torch.zeros((), dtype=torch.float64)
        floor = (2.0 ** -24) * top * k.shape[0] * (p_half == HALF_F16)
        self.off = HALF_BF16 * self.out.abs() + mass * (p_half + 2 * dx[:, None] + 2.0 ** -16) * (1 + HALF_BF16) + floor + 1e-38
        self.lse_off = 2 * dx + self.lse.abs().nan_to_num(posinf=0.0, neginf=0.0) * 2.0 ** -22

    def check(self, out, lse=None, what=""):
        out = out.double()
        assert bool(((out - self.out).abs() <= self.off).all()), \
            f"{what}: out off by {float(((out - self.out).abs() / self.off).max()):.2f} of what it may"
        if lse is not None:
            lse, none = lse.double(), self.lse == -math.inf
            assert bool((lse[none] == -math.inf).all()), f"{what}: lse of a row without keys"
            assert bool(((lse - self.lse).abs()[~none] <= self.lse_off[~none]).all()), f"{what}: lse"


def tables(lens, seed, extra=3, mbps=None):
    """Block tables over a shuffled pool: (table, num_blocks)."""
    nb = sum(-(-n // B) for n in lens) + extra
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed))
    t = torch.full((len(lens), mbps or max(1, -(-max(lens) // B)) + 1), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        k = -(-n // B)
        t[s, :k] = perm[at:at + k].int()
        at += k
    return t, nb


def random_cache8(nb, H, d, seed, spread=0):
    """Codes and scale codes; `spread`: the scale codes lie up to that far apart."""
    g = torch.Generator().manual_seed(seed)
    e = [(120 + torch.randint(-spread, spread + 1, (nb, H), generator=g)).to(torch.uint8) for _ in range(2)]
    k = (torch.randn(nb, H, B, d, generator=g) * 120).clamp(-448, 448).to(FP8).view(torch.uint8)
    v = (torch.randn(nb, H, d, B, generator=g) * 120).clamp(-448, 448).to(FP8).view(torch.uint8)
    return k, v, e[0], e[1]


def normal(*shape, seed, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def select(q, bounds, table, ctx, ql, keep, recent, sink):
    """The choice in 64 bits, q [N, Hq, d] and bounds [nb, H, 2, d]."""
    N, Hq, d = q.shape
    H = bounds.shape[1]
    g = Hq // H
    sel = torch.full((N, H, keep), -1, dtype=torch.int32)
    at = 0
    for s, (c, n) in enumerate(zip(ctx, ql)):
        blocks = table[s, :-(-c // B)].long()
        for h in range(H):
            box = bounds[blocks, h].double()  # [blocks, 2, d]
            x = q[at:at + n, h * g:(h + 1) * g].double()
            u = torch.maximum(x[..., None, :] * box[:, 0], x[..., None, :] * box[:, 1]).sum(-1).amax(1)  # [n, blocks]
            for r in range(n):
                count = (c - n + r) // B + 1
                got = list(range(count))
                if count > keep:
                    must = set(range(sink)) | set(range(count - recent, count))
                    rest = sorted((b for b in got if b not in must), key=lambda b: (-float(u[r, b]), b))
                    got = sorted((sorted(must) + rest)[:keep])
                sel[at + r, h, :len(got)] = i32(got)
        at += n
    return sel
