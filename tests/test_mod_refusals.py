"""Arguments that the calls with modified scores, the several-axes rotary append,
the weight sums and the eviction refuse on the host, before any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def fattn():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn as F
    return F


D = 4096  # an address that is never read


def call(lib, name, order, defaults, **kw):
    args = dict(defaults, **kw)
    return getattr(lib, name)(*[args[n] for n in order])


PREFILL = "q k v out lse B T Hq Hkv d causal scale cap slopes window prefix docs ws ws_bytes stream".split()
PREFILL_OK = dict(q=D, k=D, v=D, out=D, lse=None, B=1, T=16, Hq=4, Hkv=2, d=64, causal=1, scale=0.1, cap=0.0, slopes=None,
                  window=0, prefix=None, docs=None, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw, want", [
    (dict(B=-1), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(d=96), "UNSUPPORTED"), (dict(Hq=5), "UNSUPPORTED"),
    (dict(scale=0.0), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"), (dict(cap=-1.0), "INVALID_ARG"),
    (dict(cap=float("inf")), "INVALID_ARG"), (dict(cap=float("nan")), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"),
    (dict(cap=3e38), "INVALID_ARG"), (dict(cap=1e-40), "INVALID_ARG"), (dict(cap=1e37, scale=1e-3), "INVALID_ARG"),
    (dict(q=None), "INVALID_ARG"), (dict(out=D + 16), "INVALID_ARG"), (dict(k=D + 2), "INVALID_ARG"),
    (dict(docs=D), "WORKSPACE"), (dict(docs=D, ws=D + 8, ws_bytes=1 << 30), "WORKSPACE"),
    (dict(docs=D, ws=D, ws_bytes=10), "WORKSPACE"), (dict(B=70000, T=70000), "UNSUPPORTED"),
    (dict(B=0), "OK"), (dict(T=0, q=None, k=None), "OK"), (dict(B=0, cap=-1.0), "INVALID_ARG"),
], ids=str)
def test_prefill_mod(fattn, kw, want):
    names = {"OK": 0, "INVALID_ARG": 1, "UNSUPPORTED": 2, "WORKSPACE": 6}
    assert call(fattn.library(), "fa_prefill_mod", PREFILL, PREFILL_OK, **kw) == names[want]


PAGED = ("q kc vc bt ctx ql out lse S mbps nb Hq Hkv d bs causal scale cap slopes window prefix total max_q ws ws_bytes "
         "stream").split()
PAGED_OK = dict(q=D, kc=D, vc=D, bt=D, ctx=D, ql=D, out=D, lse=D, S=2, mbps=4, nb=8, Hq=4, Hkv=2, d=64, bs=16, causal=1,
                scale=0.1, cap=0.0, slopes=None, window=0, prefix=None, total=2, max_q=1, ws=D, ws_bytes=0, stream=None)
ACCUM = PAGED[:8] + "acc_in acc_out acc_len decay".split() + PAGED[8:]
ACCUM_OK = dict(PAGED_OK, acc_in=D, acc_out=D, acc_len=64, decay=1.0)


@pytest.mark.parametrize("kw, want", [
    (dict(S=-1), 1), (dict(bs=32), 2), (dict(d=80), 2), (dict(Hq=3), 2), (dict(scale=-1.0), 1), (dict(cap=-0.5), 1),
    (dict(cap=float("nan")), 1), (dict(window=-3), 1), (dict(bt=None), 1), (dict(out=D + 16), 1), (dict(q=D + 4), 1),
    (dict(nb=0), 1), (dict(ws=None), 6), (dict(ws_bytes=-1), 6), (dict(ws=D + 16), 6), (dict(S=0), 0), (dict(total=0), 0),
    (dict(max_q=0), 0), (dict(max_q=-1), 1),
], ids=str)
def test_paged_mod_and_accum(fattn, kw, want):
    lib = fattn.library()
    for name, order, ok in (("fa_paged_attn_mod", PAGED, PAGED_OK), ("fa_paged_attn_accum", ACCUM, ACCUM_OK)):
        size = getattr(lib, name + "_workspace_size")(2, 4, 4, 2, 64, 2, 1)
        assert size > 0
        a = dict(kw)
        a["ws_bytes"] = size + a.get("ws_bytes", 0)
        assert call(lib, name, order, ok, **a) == want, name


@pytest.mark.parametrize("kw", [dict(lse=None), dict(acc_out=None), dict(acc_len=-1), dict(decay=-0.1),
                                dict(decay=float("inf")), dict(decay=float("nan"))], ids=str)
def test_accum_arguments(fattn, kw):
    lib = fattn.library()
    size = lib.fa_paged_attn_accum_workspace_size(2, 4, 4, 2, 64, 2, 1)
    assert call(lib, "fa_paged_attn_accum", ACCUM, ACCUM_OK, ws_bytes=size, **kw) == fattn.FA_ERR_INVALID_ARG


def test_accum_workspace_grows_with_the_decode_rows(fattn):
    size = lambda max_q, g=2: fattn.fa_paged_attn_accum_workspace_size(2, 4, 2 * g, 2, 64, 40, max_q)
    base = fattn.fa_paged_attn_mod_workspace_size(2, 4, 4, 2, 64, 40, 1)
    row = 2 * 4 * 2 * 16 * 4  # bytes of a decode row's logits over the pages that the tables hold
    assert size(1) >= base + 2 * row
    assert size(2) == size(1) + 2 * row and size(3) == size(1) + 4 * row
    assert size(8) == size(30) == size(1) + 14 * row  # 16 rows at most
    assert base < size(3, g=20) < size(1)  # no decode rows in so wide a group
    assert fattn.fa_paged_attn_mod_workspace_size(2, 4, 4, 2, 64, 40, -1) == 0


MROPE = "q k v pos A axes cs max_pos qo kc vc sm N Hq Hkv d nb dt stream".split()
MROPE_OK = dict(q=D, k=D, v=D, pos=D, A=3, axes=bytes(32), cs=D, max_pos=8, qo=D, kc=D, vc=D, sm=D, N=4, Hq=4, Hkv=2, d=64,
                nb=8, dt=0, stream=None)


@pytest.mark.parametrize("kw, want", [
    (dict(N=-1), 1), (dict(dt=7), 1), (dict(max_pos=0), 1), (dict(d=80), 2), (dict(A=5), 2), (dict(A=0), 1),
    (dict(axes=None), 1), (dict(axes=bytes([0] * 31 + [3])), 1), (dict(cs=None), 1), (dict(qo=D + 8), 1),
    (dict(pos=None), 1), (dict(N=0, q=None, pos=None), 0), (dict(N=0, axes=bytes([9] * 32)), 1),
], ids=str)
def test_mrope(fattn, kw, want):
    assert call(fattn.library(), "fa_cache_append_mrope", MROPE, MROPE_OK, **kw) == want


EVICT = ("kc vc acc acc_len bt ctx dst acc_out out_len new_lens kept S mbps dmbps nb Hkv d bs keep recent sink ws ws_bytes "
         "stream").split()
EVICT_OK = dict(kc=D, vc=D, acc=D, acc_len=64, bt=D, ctx=D, dst=2 * D, acc_out=2 * D, out_len=32, new_lens=D, kept=D, S=2,
                mbps=4, dmbps=2, nb=8, Hkv=2, d=64, bs=16, keep=32, recent=4, sink=2, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw, want", [
    (dict(S=-1), 1), (dict(keep=0), 1), (dict(recent=-1), 1), (dict(recent=33), 1), (dict(recent=20, sink=13), 1),
    (dict(sink=2 ** 31 - 1, recent=32), 1), (dict(d=96), 2), (dict(bs=8), 2), (dict(kc=None), 1), (dict(acc=None), 1),
    (dict(dst=None), 1), (dict(dst=D), 1), (dict(kc=D + 2), 1), (dict(out_len=31), 1), (dict(acc_out=D, out_len=63), 1),
    (dict(kept=None), 6), (dict(kept=None, ws=D, ws_bytes=16), 6), (dict(new_lens=None), 1), (dict(dmbps=0), 1),
    (dict(S=0), 0), (dict(acc_len=-1), 1), (dict(keep=1 << 20, out_len=1 << 20), 2),
], ids=str)
def test_evict(fattn, kw, want):
    assert call(fattn.library(), "fa_cache_evict", EVICT, EVICT_OK, **kw) == want


def test_binding_refuses_host_tensors(fattn):
    torch = pytest.importorskip("torch")
    z = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fattn.fa_prefill_mod(z, z, z)
    with pytest.raises(ValueError):
        fattn.fa_cache_append_mrope(z[0], z[0], z[0], torch.zeros(1, 4, dtype=torch.int32), [0] * 32, torch.zeros(8, 64),
                                    z, z, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        fattn.fa_cache_evict(z, z, torch.zeros(1, 2, 8), torch.zeros(1, 1, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32), 4)
