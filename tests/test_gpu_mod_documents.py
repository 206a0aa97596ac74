"""Documents in batches larger than one pass over the ids takes, against 64 bits, and batches of very short rows."""
import pytest
import torch

import mod_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn
    return fattn


def doc_ids(B, T, longest, seed):
    """Runs of 1 to `longest` rows; the ids come back, and some are padding."""
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(1, longest + 1, (B * T,), generator=g)
    edge = torch.zeros(B * T + 1, dtype=torch.int64)
    ends = n.cumsum(0)
    edge[ends[ends <= B * T]] = 1
    return (edge[:-1].cumsum(0) % 7 - 1).view(B, T).to(torch.int32)


def data(B, T, Hq, Hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, T, h, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv)]


@pytest.mark.parametrize("kw", [dict(window=700), dict(cap=20.0), dict(bias=True, causal=False)], ids=str)
def test_large_batches(F, kw):
    """12003 rows: the ids take two passes, and a sequence's rows begin anywhere in one."""
    B, T, Hq, Hkv, d = 3, 4001, 2, 1, 64
    q, k, v = data(B, T, Hq, Hkv, d, 46)
    ids = doc_ids(B, T, 1500, 47)
    sl = R.slopes(Hq) if kw.get("bias") else None
    causal, cap, window = kw.get("causal", True), kw.get("cap", 0.0), kw.get("window", 0)
    lse = torch.empty(B, Hq, T, device="cuda")
    out = F.fa_prefill_mod(q.cuda(), k.cuda(), v.cuda(), causal=causal, softcap=cap, window=window, lse=lse,
                           alibi_slopes=None if sl is None else sl.cuda(), doc_ids=ids.cuda())
    assert F.fa_get_error() == F.FA_OK
    pos = torch.arange(T)
    for b in range(B):
        see = R.visible(pos, T, causal, window, 0, ids[b])
        for h in range(Hq):
            ref = R.Rows(q[b, :, h], k[b, :, 0], v[b, :, 0], pos, see, d ** -0.5, cap, None if sl is None else sl[h])
            R.check(lse[b, h], ref.lse, ref.lse_tol, f"lse b{b} h{h}")
            R.check(out[b, :, h], ref.out, ref.out_tol, f"out b{b} h{h}")


@pytest.mark.parametrize("B, T", [(9000, 1), (5000, 3), (70, 128), (1, 8192), (1, 8193)], ids=str)
def test_many_rows_of_any_length(F, B, T):
    """Many sequences of few rows, and row counts at the limit of one pass."""
    q, k, v = data(B, T, 2, 2, 64, 48)
    ids = doc_ids(B, T, 90, 49)
    out = F.fa_prefill_mod(q.cuda(), k.cuda(), v.cuda(), doc_ids=ids.cuda()).cpu()
    assert F.fa_get_error() == F.FA_OK
    assert (out[ids < 0] == 0).all()
    pos = torch.arange(T)
    for b in range(0, B, max(1, B // 40)):
        see = R.visible(pos, T, True, 0, 0, ids[b])
        for h in range(2):
            ref = R.Rows(q[b, :, h], k[b, :, h], v[b, :, h], pos, see, 0.125)
            R.check(out[b, :, h], ref.out, ref.out_tol, f"out b{b} h{h}")
