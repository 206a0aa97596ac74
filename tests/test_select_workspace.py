"""The workspace of fa_block_select goes by the rows of the call."""
import pytest


@pytest.fixture(scope="module")
def size():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn as F
    return F.fa_block_select_workspace_size


@pytest.mark.parametrize("rows, Hkv", [(1, 1), (1, 8), (7, 2), (159, 8), (160, 8), (161, 8), (5000, 1)])
@pytest.mark.parametrize("entries", [1, 500, 131072])
def test_bytes_a_table_entry(size, rows, Hkv, entries):
    """Scores, largest bounds, and a row of near blocks for each CTA; four arrays, each rounded up to 256 bytes."""
    need = entries * (4 * rows * Hkv + 4 * 3 * Hkv + 12 * min(rows * Hkv, 1280))
    assert need <= size(3, entries, 4 * Hkv, Hkv, 128, rows) <= need + 4 * 256


def test_larger_calls_need_no_less(size):
    last = 0
    for S, entries, rows in ((1, 10, 1), (1, 10, 100), (4, 10, 100), (4, 90, 100), (4, 90, 1000), (4, 5000, 1000), (300, 5000, 9000)):
        now = size(S, entries, 16, 4, 64, rows)
        assert now >= last
        last = now
