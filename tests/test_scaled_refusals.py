"""Arguments that the calls of the 8-bit cache with block scales and of attention over chosen blocks refuse on the host,
before any CUDA call."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_tiled_gb300 import build
    build.build()
    from paged_kv_cache_tiled_gb300 import fattn as F
    return F.library()


D = 4096  # an address that is never read
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 6


def call(lib, name, order, defaults, kw):
    args = dict(defaults, **kw)
    return getattr(lib, name)(*[args[n] for n in order.split()])


BATCH = dict(bt=D, ctx=D, ql=D, S=2, mbps=4, nb=8, Hq=4, Hkv=2, d=64, bs=16, total=2, stream=None)
APPEND = "q k v pos cs max_pos q_out kc vc ke ve bt ctx ql S mbps nb total Hq Hkv d bs dtype stream"
APPEND_OK = dict(BATCH, q=D, k=D, v=D, pos=D, cs=D, max_pos=9, q_out=D, kc=D, vc=D, ke=D, ve=D, dtype=0)


@pytest.mark.parametrize("kw, want", [
    (dict(S=-1), INVALID), (dict(total=-1), INVALID), (dict(nb=0), INVALID), (dict(mbps=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(bs=32), UNSUPPORTED), (dict(Hkv=0), INVALID), (dict(Hq=0), INVALID), (dict(dtype=7), INVALID), (dict(k=None), INVALID),
    (dict(ke=None), INVALID), (dict(ve=None), INVALID), (dict(cs=None), INVALID), (dict(cs=None, q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(kc=D + 8), INVALID), (dict(vc=D + 4), INVALID), (dict(q=D + 2), INVALID),
    (dict(cs=D + 4), INVALID), (dict(max_pos=-1), INVALID), (dict(bt=None), INVALID), (dict(S=0), OK), (dict(total=0), OK),
], ids=str)
def test_append(lib, kw, want):
    assert call(lib, "fa_cache_append_fp8_scaled", APPEND, APPEND_OK, kw) == want


ATTN = "q kc vc ke ve bt ctx ql out lse S mbps nb Hq Hkv d bs causal scale total max_q ws ws_bytes stream"
ATTN_OK = dict(BATCH, q=D, kc=D, vc=D, ke=D, ve=D, out=D, lse=None, causal=1, scale=0.1, max_q=1, ws=D, ws_bytes=0)


@pytest.mark.parametrize("kw, want", [
    (dict(S=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(d=80), UNSUPPORTED),
    (dict(Hq=3), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(ke=None), INVALID), (dict(ve=None), INVALID),
    (dict(out=D + 16), INVALID), (dict(q=D + 4), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(ws=D + 16), WORKSPACE), (dict(max_q=-1), INVALID), (dict(S=0), OK), (dict(total=0), OK), (dict(max_q=0), OK),
    (dict(Hq=1 << 17, Hkv=1 << 17), UNSUPPORTED),
], ids=str)
def test_attention(lib, kw, want):
    assert call(lib, "fa_paged_attn_fp8_scaled", ATTN, ATTN_OK, kw) == want


BOUNDS = "kc ke bt ctx ql bounds S mbps nb total Hkv d bs stream"
BOUNDS_OK = dict(BATCH, kc=D, ke=None, bounds=D)


@pytest.mark.parametrize("kw, want", [
    (dict(S=-1), INVALID), (dict(d=32), UNSUPPORTED), (dict(bs=1), UNSUPPORTED), (dict(kc=None), INVALID),
    (dict(bounds=None), INVALID), (dict(bounds=D + 2), INVALID), (dict(nb=0), INVALID), (dict(Hkv=-1), INVALID),
    (dict(total=0), OK), (dict(S=0), OK),
], ids=str)
def test_bounds(lib, kw, want):
    assert call(lib, "fa_block_bounds", BOUNDS, BOUNDS_OK, kw) == want


SELECT = "q bounds bt ctx ql sel S mbps nb Hq Hkv d bs keep recent sink total max_q ws ws_bytes stream"
SELECT_OK = dict(BATCH, q=D, bounds=D, sel=D, keep=4, recent=1, sink=1, max_q=1, ws=D, ws_bytes=0)


@pytest.mark.parametrize("kw, want", [
    (dict(keep=0), INVALID), (dict(recent=-1), INVALID), (dict(sink=-1), INVALID), (dict(recent=3, sink=2), INVALID),
    (dict(recent=5, sink=0), INVALID), (dict(sink=2 ** 31 - 1, recent=2), INVALID), (dict(d=16), UNSUPPORTED),
    (dict(Hq=5), UNSUPPORTED), (dict(sel=None), INVALID), (dict(bounds=D + 8), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=100), WORKSPACE), (dict(ws=D + 1), WORKSPACE), (dict(total=0), OK), (dict(max_q=0), OK),
    (dict(max_q=-1), INVALID),
], ids=str)
def test_select(lib, kw, want):
    assert call(lib, "fa_block_select", SELECT, SELECT_OK, kw) == want


BLOCKS = "q kc vc ke ve bt ctx ql sel keep out lse S mbps nb Hq Hkv d bs scale total stream"
BLOCKS_OK = dict(BATCH, q=D, kc=D, vc=D, ke=None, ve=None, sel=D, keep=4, out=D, lse=None, scale=0.1)


@pytest.mark.parametrize("kw, want", [
    (dict(keep=-1), INVALID), (dict(ke=D), INVALID), (dict(ve=D), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(sel=None), INVALID), (dict(out=None), INVALID), (dict(out=D + 8), INVALID),
    (dict(d=256), UNSUPPORTED), (dict(Hq=7), UNSUPPORTED), (dict(nb=0), INVALID), (dict(total=0), OK), (dict(S=0), OK),
], ids=str)
def test_blocks(lib, kw, want):
    assert call(lib, "fa_paged_attn_blocks", BLOCKS, BLOCKS_OK, kw) == want


def test_workspace_sizes_of_nothing(lib):
    assert lib.fa_block_select_workspace_size(0, 4, 4, 2, 64, 2) == 0
    assert lib.fa_block_select_workspace_size(2, 4, 4, 2, 64, -2) == 0
    assert lib.fa_paged_attn_fp8_scaled_workspace_size(-1, 4, 4, 2, 64, 2, 1) == 0
    small, large = (lib.fa_paged_attn_fp8_scaled_workspace_size(*x) for x in ((2, 4, 4, 2, 64, 2, 1), (9, 90, 4, 2, 64, 500, 300)))
    assert 0 < small <= large
