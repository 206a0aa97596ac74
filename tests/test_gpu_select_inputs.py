"""fa_block_select at the edges of what it takes: workspaces of exactly the size asked for, bounds of blocks with NaN keys,
magnitudes near fp32's largest."""
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
    return [t.cuda() for t in ts]


def boxes(nb, H, d, seed):
    mid, wide = R.normal(nb, H, d, seed=seed).float(), R.normal(nb, H, d, seed=seed + 1).float().abs() + 0.5
    return torch.stack([mid - wide, mid + wide], 2).bfloat16()


@pytest.mark.parametrize("ql, H", [([1], 1), ([1, 1, 1], 2), ([700, 1, 20], 2)])
def test_nothing_is_written_behind_the_workspace(F, ql, H):
    """All blocks alike, so that every one of them is listed as near the border."""
    d, ctx = 64, [16 * 600 + 5] + [16 * 400] * (len(ql) - 1)
    table, nb = R.tables(ctx, 1)
    q, bounds = R.normal(sum(ql), 2 * H, d, seed=2), boxes(1, H, d, 3).expand(nb, H, 2, d).contiguous()
    size = F.fa_block_select_workspace_size(len(ql), table.shape[1], 2 * H, H, d, sum(ql))
    whole = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    sel = F.fa_block_select(*cuda(q, bounds, table, R.i32(ctx), R.i32(ql)), 40, recent=2, sink=1, max_q_len=max(ql), ws=whole[:size])
    assert F.fa_get_error() == F.FA_OK
    assert bool((whole[size:] == 77).all())
    assert torch.equal(sel.cpu(), R.select(q, bounds, table, ctx, ql, 40, 2, 1))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("ctx", [33, 48, 17])
def test_bounds_of_channels_without_a_number(F, fp8, d, ctx):
    """All keys of a channel NaN, in a block of one key and in a full one: bounds of 0, the other channels' as they are."""
    table, nb = R.tables([ctx], 11)
    k, _, e, _ = R.random_cache8(nb, 2, d, 12, 5) if fp8 else (R.normal(nb, 2, 16, d, seed=12), None, None, None)
    vals = R.values(k, e) if fp8 else k.double()
    lost = torch.rand(nb, 2, 1, d, generator=torch.Generator().manual_seed(13)) < 0.3
    k[lost.expand(k.shape)] = 0x7F if fp8 else float("nan")
    bounds = torch.full((nb, 2, 2, d), 3.0, dtype=torch.bfloat16)
    want = bounds.clone()
    for b in range(-(-ctx // 16)):
        p = int(table[0, b])
        page = vals[p, :, :ctx - 16 * b]
        want[p] = torch.stack([page.amin(1), page.amax(1)], 1).masked_fill(lost[p], 0.0).bfloat16()
    got = bounds.cuda()
    F.fa_block_bounds(k.cuda(), *cuda(table, R.i32([ctx]), R.i32([ctx])), got, k_exp=None if e is None else e.cuda(), total_q=ctx)
    assert F.fa_get_error() == F.FA_OK
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("d", [128, 64])
def test_blocks_with_nan_keys_leave_the_choice_exact(F, d):
    """From the keys on: scores closer than fp32 tells apart beside blocks that hold channels of NaN."""
    n, g = 600, torch.Generator().manual_seed(14)
    mid = torch.randn(d, generator=g).mul(100).bfloat16().float()
    k = mid.expand(n, 1, 16, d).clone()
    k[:, :, :, 0] = 2.0 ** -10 * (1 + torch.randint(0, 100, (n, 1, 1), generator=g) / 128)
    k = k.bfloat16()
    k[5::50, :, :, 3] = float("nan")
    k[7, :, 1:] = float("nan")
    q = torch.randn(1, 2, d, generator=g).mul(30).bfloat16()
    q[:, :, 0] = 1.0
    table, lens = torch.randperm(n, generator=g).int()[None], R.i32([16 * n])
    bounds = torch.zeros(n, 1, 2, d, dtype=torch.bfloat16).cuda()
    F.fa_block_bounds(k.cuda(), *cuda(table, lens, lens), bounds, total_q=16 * n)
    sel = F.fa_block_select(*cuda(q, bounds, table, lens, R.i32([1])), 100, recent=1, sink=1)
    assert F.fa_get_error() == F.FA_OK
    assert bool(bounds.isfinite().all())
    assert torch.equal(sel.cpu(), R.select(q, bounds.cpu(), table, [16 * n], [1], 100, 1, 1))


@pytest.mark.parametrize("bad", [(-float("inf"), float("inf")), (float("nan"), float("nan"))])
def test_a_block_with_infinite_bounds_leaves_the_others_order(F, bad):
    d, n, g = 64, 600, torch.Generator().manual_seed(15)
    mid = torch.randn(d, generator=g).mul(100).bfloat16().float()
    b = mid.expand(n, d).clone()
    b[:, 0] = 2.0 ** -10 * (1 + torch.randint(0, 100, (n,), generator=g) / 128)
    bounds = torch.stack([b, b], 1)[:, None].bfloat16().contiguous()
    q = torch.randn(1, 2, d, generator=g).mul(30).bfloat16()
    q[:, :, 0] = 1.0
    table = torch.randperm(n, generator=g).int()[None]
    at = int(table[0, 300])
    first, last = bounds.clone(), bounds.clone()
    bounds[at, 0, 0, 9], bounds[at, 0, 1, 9] = bad
    first[at, 0, :, 9] = torch.tensor([-1e30, 1e30])
    if bad[1] != float("inf"):
        q[0, :, 9] = q[0, :, 9].abs()
    last[at, 0] = -1e20 * q[0].float().sum(0)  # (a point that both heads score far below 0)
    assert bool((q[0].double() @ last[at, 0, 0].double() < -1e20).all())
    sel = F.fa_block_select(*cuda(q, bounds, table, R.i32([16 * n]), R.i32([1])), 100, recent=1, sink=1)
    assert F.fa_get_error() == F.FA_OK
    # (+inf stands beside 0 * inf, which is NaN: before or after all others is what the call says of such a block)
    assert any(torch.equal(sel.cpu(), R.select(q, b, table, [16 * n], [1], 100, 1, 1)) for b in (first, last))


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("top", [2.0 ** 40, 2.0 ** 60, 2.0 ** -40])
def test_magnitudes_up_to_the_stated_range(F, d, top):
    """Largest |bound| times the sum of |q| just below 2^126 (and small ones), scores that fp32 cannot tell apart."""
    n, g = 500, torch.Generator().manual_seed(16)
    mid = torch.randn(d, generator=g).clamp(-2, 2)
    b = mid.expand(n, d).clone()
    b[:, 0] = 2.0 ** -17 * (1 + torch.randint(0, 100, (n,), generator=g) / 128)
    b *= top / 2
    bounds = torch.stack([b, b], 1)[:, None].bfloat16().contiguous()
    q = torch.randn(1, 2, d, generator=g)
    q[:, :, 0] = 1.0
    q = (q / q.abs().sum(-1, keepdim=True) * (2.0 ** 125.5 / top if top > 1 else 1e-3)).bfloat16()
    assert top < 1 or float(bounds.abs().max()) * float(q.double().abs().sum(-1).max()) < 2.0 ** 126
    table = torch.randperm(n, generator=g).int()[None]
    sel = F.fa_block_select(*cuda(q, bounds, table, R.i32([16 * n]), R.i32([1])), 100, recent=1, sink=1)
    assert F.fa_get_error() == F.FA_OK
    assert torch.equal(sel.cpu(), R.select(q, bounds, table, [16 * n], [1], 100, 1, 1))
