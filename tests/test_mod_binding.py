"""Sizes and arguments of the calls with modified scores and of the several-axes append, on the host."""
import itertools

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


SIZES = list(itertools.product((1, 3, 40), (1, 64, 100, 4096), (1, 9, 700, 9000), (1, 5, 700, 9000)))  # S, blocks, total, max


@pytest.mark.parametrize("heads", [(1, 1), (8, 2), (6, 2), (32, 8), (20, 1), (160, 160)], ids=str)
@pytest.mark.parametrize("what", ["fa_paged_attn_mod", "fa_paged_attn_accum"])
def test_a_workspace_serves_smaller_problems(F, what, heads):
    """The size never falls when a size of the problem grows: a program that lays one workspace out for its largest step
    may use it for all."""
    size = {x: getattr(F, what + "_workspace_size")(x[0], x[1], *heads, 64, x[2], x[3]) for x in SIZES}
    for a in SIZES:
        for b in SIZES:
            if all(p <= q for p, q in zip(a, b)):
                assert size[a] <= size[b], (a, b)


def test_a_call_takes_the_workspace_of_a_larger_one(F):
    """64 queries over long contexts need room that 9000 queries would not; checked before anything is launched."""
    lib, D = F.library(), 4096  # (an address that is never read)
    size = lib.fa_paged_attn_mod_workspace_size(8, 4096, 32, 8, 128, 9000, 9000)
    call = lambda n: lib.fa_paged_attn_mod(D, D, D, D, D, D, D, None, 1, 4096, 8, 32, 8, 128, 16, 1, 0.1, 0.0, None, 0, None,
                                           64, 64, D, n, None)
    assert call(1000) == F.FA_ERR_WORKSPACE
    if not torch.cuda.is_available():  # (with a device it would go on to read its inputs)
        assert call(size) != F.FA_ERR_WORKSPACE


@pytest.mark.parametrize("axes", [[0, 1, 2, 1] * 8, (0, 1, 2, 1) * 8, bytes([0, 1, 2, 1] * 8), np.array([0, 1, 2, 1] * 8),
                                  np.array([0, 1, 2, 1] * 8, np.uint8), torch.tensor([0, 1, 2, 1] * 8),
                                  (a for a in [0, 1, 2, 1] * 8), bytearray([0, 1, 2, 1] * 8)], ids=lambda a: type(a).__name__)
def test_pair_axes(F, axes):
    assert F._pair_axes(axes, 32) == bytes([0, 1, 2, 1] * 8)


@pytest.mark.parametrize("axes", [32, [0] * 31, [0] * 33, [-1] * 32, [256] * 32, [0.0] * 32, np.zeros(4, np.int64), None, "0" * 32,
                                  np.zeros(32, np.float32), np.zeros((4, 8), np.int64)], ids=str)
def test_pair_axes_refused(F, axes):
    with pytest.raises(ValueError):
        F._pair_axes(axes, 32)
