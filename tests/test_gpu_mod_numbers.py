"""Numbers as every other call takes them: Python's, numpy's and tensors of one element."""
import numpy as np
import pytest
import torch

import mod_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("number", [float, np.float32, np.float64, torch.tensor, lambda x: torch.tensor(x, dtype=torch.float64)],
                         ids=["float", "float32", "float64", "tensor", "tensor64"])
def test_numbers(number):
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn as F
    q, k, v = (torch.randn(1, 40, h, 64, device="cuda").bfloat16() for h in (2, 1, 1))
    want = F.fa_prefill_mod(q, k, v, scale=0.125, softcap=20.0)
    assert torch.equal(F.fa_prefill_mod(q, k, v, scale=number(0.125), softcap=number(20.0)), want)
    p = R.Paged(95, [40, 9], [20, 1], 2, 1, 64)
    args = p.cuda()
    acc = torch.ones(2, 1, 40, device="cuda"), torch.zeros(2, 1, 40, device="cuda"), torch.zeros(2, 1, 40, device="cuda")
    want = F.fa_paged_attn_accum(*args, acc[0], acc[1], decay=0.5, scale=0.125, softcap=20.0)
    got = F.fa_paged_attn_accum(*args, acc[0], acc[2], decay=number(0.5), scale=number(0.125), softcap=number(20.0))
    assert torch.equal(got, want) and torch.equal(acc[1], acc[2])
    assert torch.equal(F.fa_paged_attn_mod(*args, scale=number(0.125), softcap=number(20.0)), want)
    assert F.fa_get_error() == F.FA_OK
