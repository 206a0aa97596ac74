"""Rotary positions with several axes, fused with the cache append, against the
rotation in 64 bits."""
import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu
CANARY = 0x7E7E


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


def case(N, Hq, Hkv, d, A, seed=0, dtype=torch.bfloat16, max_pos=700):
    g = torch.Generator().manual_seed(seed)
    nb = -(-N // 16) + 1
    q, k, v = (torch.randn(N, h, d, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    pos = torch.randint(0, max_pos, (A, N), generator=g, dtype=torch.int32)
    slots = torch.randperm(nb * 16, generator=g)[:N].to(torch.int32)
    if N > 4:
        slots[4] = -1
    return q, k, v, pos, W.rope_table(max_pos, d), slots, nb


def run(F, q, k, v, pos, axes, table, slots, nb):
    Hkv, d = k.shape[1:]
    can = lambda *s: torch.full(s, CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    kc, vc, qo = can(nb, Hkv, 16, d), can(nb, Hkv, 16, d), can(*q.shape)
    F.fa_cache_append_mrope(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), axes, table.cuda(), kc, vc, slots.cuda(), q_out=qo)
    return qo.cpu(), kc.cpu(), vc.cpu()


def check_turned(got, x, pos, axes, table, what):
    """One bf16 rounding (2^-8 of the value) and the fp32 rounding of the two products and their sum
    (3 * 2^-24 of the terms' sizes)."""
    d = x.shape[-1]
    h = d // 2
    row = pos[torch.tensor(axes)].T.long()  # [N, d/2]
    j = torch.arange(h)
    c, s = table.double()[row, j][:, None], table.double()[row, j + h][:, None]
    a, b = x.double()[..., :h], x.double()[..., h:]
    want = torch.cat([a * c - b * s, b * c + a * s], -1)
    size = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    tol = 2.0 ** -8 * want.abs() + 3 * 2.0 ** -24 * (1 + 2.0 ** -7) * size
    over = (got.double() - want).abs() - tol
    assert over.max() <= 0, f"{what}: over by {float(over.max()):.3e}"


SECTIONS = {1: lambda h: [0] * h, 2: lambda h: [0] * (h // 2) + [1] * (h // 2),
            3: lambda h: [0] * (h // 4) + [1] * (3 * h // 8) + [2] * (h - h // 4 - 3 * h // 8),
            4: lambda h: [(3 * j + 1) % 4 for j in range(h)]}


@pytest.mark.parametrize("A", [1, 2, 3, 4])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64), (7, 6, 2, 128), (65, 5, 1, 64), (300, 32, 8, 128)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_mrope_append(F, shape, A, dtype):
    N, Hq, Hkv, d = shape
    q, k, v, pos, table, slots, nb = case(N, Hq, Hkv, d, A, dtype=dtype)
    axes = SECTIONS[A](d // 2)
    qo, kc, vc = run(F, q, k, v, pos, axes, table, slots, nb)
    assert F.fa_get_error() == F.FA_OK
    check_turned(qo, q, pos, axes, table, "q")
    put = slots >= 0
    s = slots[put].long()
    check_turned(kc[s // 16, :, s % 16], k[put], pos[:, put], axes, table, "k")
    assert torch.equal(vc[s // 16, :, s % 16], v[put].bfloat16())
    rest = torch.ones(nb * 16, dtype=torch.bool)
    rest[s] = False
    for c in (kc, vc):
        rows = c.view(torch.int16).transpose(1, 2).reshape(nb * 16, Hkv, d)
        assert (rows[rest] == CANARY).all()


def test_mrope_one_axis_is_rope(F):
    """Equal positions on every axis, or one axis: the bits of fa_cache_append_rope."""
    q, k, v, pos, table, slots, nb = case(100, 8, 2, 128, 1)
    kc, vc = (torch.zeros(nb, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = F.fa_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), pos[0].cuda(), table.cuda(), kc, vc, slots.cuda())
    for A in (1, 3):
        k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
        q2 = F.fa_cache_append_mrope(q.cuda(), k.cuda(), v.cuda(), pos.expand(A, -1).contiguous().cuda(),
                                     [j % A for j in range(64)], table.cuda(), k2, v2, slots.cuda())
        assert torch.equal(qo, q2) and torch.equal(kc, k2) and torch.equal(vc, v2)


def test_mrope_bad_positions_and_slots(F):
    q, k, v, pos, table, slots, nb = case(40, 5, 2, 64, 3)
    axes = SECTIONS[3](32)
    good = run(F, q, k, v, pos, axes, table, slots, nb)
    assert F.fa_get_error() == F.FA_OK
    pos2, slots2 = pos.clone(), slots.clone()
    pos2[2, 9] = 700
    pos2[0, 11] = -1
    slots2[20] = nb * 16
    qo, kc, vc = run(F, q, k, v, pos2, axes, table, slots2, nb)
    assert F.fa_get_error() == F.FA_ERR_BOUNDS
    skipped = [9, 11]
    assert (qo[skipped].view(torch.int16) == CANARY).all()
    for i in skipped + [20]:
        s = int(slots[i])
        assert (kc[s // 16, :, s % 16].view(torch.int16) == CANARY).all()
        assert (vc[s // 16, :, s % 16].view(torch.int16) == CANARY).all()
    rest = [i for i in range(40) if i not in skipped]
    assert torch.equal(qo[rest].view(torch.int16), good[0][rest].view(torch.int16))
