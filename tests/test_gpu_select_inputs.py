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
