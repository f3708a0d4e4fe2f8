"""The key/value cache's entry points without a GPU: argument checks happen on the host before any launch, empty calls
return at once, and the sizes are host arithmetic."""
import pytest

from quantized_weight_matvec_hq_gb300 import build as hq_build

FAKE = 1 << 40                                  # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def hq():
    hq_build.build()
    import quantized_weight_matvec_hq_gb300 as hq
    hq.lib()
    return hq


def rows(hq, fn, fmt=8, k=FAKE, ks=256, v=FAKE, vs=256, pool=FAKE, pages=9, page=64, table=FAKE, width=4, off=FAKE, lens=FAKE,
         R=3, T=5, kv=2, dim=128, dt=2):
    return getattr(hq.lib(), fn)(fmt, k, ks, v, vs, pool, pages, page, table, width, off, lens, R, T, kv, dim, dt, 0)


def attend(hq, fmt=8, q=FAKE, qs=1024, pool=FAKE, pages=9, page=64, table=FAKE, width=4, off=FAKE, lens=FAKE, R=3, T=5,
           heads=8, kv=2, dim=128, scale=0.1, causal=1, window=0, out=FAKE, os=1024, dt=2, ws=FAKE, ws_bytes=1 << 40):
    return hq.lib().hq_cache_attention(fmt, q, qs, pool, pages, page, table, width, off, lens, R, T, heads, kv, dim, scale,
                                       causal, window, out, os, dt, ws, ws_bytes, 0)


SHARED_SHAPES = [dict(pages=0), dict(pages=1 << 31), dict(page=0), dict(page=8), dict(page=48), dict(page=2048), dict(width=0),
                 dict(width=(1 << 24) + 1), dict(R=-1), dict(R=(1 << 20) + 1), dict(T=-1), dict(T=(1 << 27) + 1), dict(kv=0),
                 dict(kv=1025), dict(dim=32), dict(dim=96), dict(dim=512)]


@pytest.mark.parametrize("fn", ["hq_cache_write", "hq_cache_read"])
def test_rows_refusals(hq, fn):
    for name in ("k", "v", "pool", "table", "off", "lens"):
        assert rows(hq, fn, **{name: 0}) == hq.HQ_ERR_NULL, name
    for bad in SHARED_SHAPES + [dict(ks=255), dict(vs=248), dict(ks=(1 << 31) + 8)]:
        assert rows(hq, fn, **bad) == hq.HQ_ERR_SHAPE, bad
    assert rows(hq, fn, fmt=75) == rows(hq, fn, fmt=1) == rows(hq, fn, dt=3) == rows(hq, fn, dt=-1) == hq.HQ_ERR_UNSUPPORTED
    for bad in (dict(k=FAKE + 8), dict(v=FAKE + 2), dict(pool=FAKE + 8), dict(table=FAKE + 2), dict(off=FAKE + 1),
                dict(lens=FAKE + 2), dict(ks=260), dict(vs=258, dt=0)):
        assert rows(hq, fn, **bad) == hq.HQ_ERR_ALIGN, bad
    assert rows(hq, fn, T=0, k=0, v=0, pool=0, table=0, off=0, lens=0) == hq.HQ_OK
    assert rows(hq, fn, R=0, k=0, v=0, pool=0, table=0, off=0, lens=0) == hq.HQ_OK


def test_attention_refusals(hq):
    for name in ("q", "out", "pool", "table", "off", "lens"):
        assert attend(hq, **{name: 0}) == hq.HQ_ERR_NULL, name
    for bad in SHARED_SHAPES + [dict(qs=1016), dict(os=0), dict(heads=0), dict(heads=7), dict(heads=4098), dict(window=-1),
                                dict(window=5, causal=0), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=2.0 ** 101)]:
        assert attend(hq, **bad) == hq.HQ_ERR_SHAPE, bad
    for bad in (dict(fmt=75), dict(dt=3), dict(causal=2), dict(causal=-1)):
        assert attend(hq, **bad) == hq.HQ_ERR_UNSUPPORTED, bad
    for bad in (dict(q=FAKE + 8), dict(out=FAKE + 8), dict(pool=FAKE + 8), dict(table=FAKE + 2), dict(off=FAKE + 1),
                dict(lens=FAKE + 2), dict(qs=1028), dict(os=1026, dt=0)):
        assert attend(hq, **bad) == hq.HQ_ERR_ALIGN, bad
    assert attend(hq, T=0, q=0, out=0, pool=0, table=0, off=0, lens=0, ws=0, ws_bytes=0) == hq.HQ_OK
    assert attend(hq, R=0, q=0, out=0, pool=0, table=0, off=0, lens=0, ws=0, ws_bytes=0) == hq.HQ_OK
    need = hq.hq_cache_attention_workspace(8, 64, 4, 3, 5, 8, 2, 128, 2)
    if need:
        assert attend(hq, ws_bytes=need - 1) == hq.HQ_ERR_SHAPE
        assert attend(hq, ws=0, ws_bytes=need) == hq.HQ_ERR_NULL
        assert attend(hq, ws=FAKE + 16, ws_bytes=need) == hq.HQ_ERR_ALIGN


def test_sizes(hq):
    """A page: 34 or 18 bytes per block of 32, keys and values."""
    for fmt, block in ((8, 34), (4, 18)):
        for kv in (1, 5, 8):
            for dim in (64, 128, 256):
                for page in (16, 64, 1024):
                    assert hq.hq_cache_page_bytes(fmt, kv, dim, page) == 2 * kv * page * dim // 32 * block
    for bad in ((75, 1, 128, 64), (8, 0, 128, 64), (8, 1, 100, 64), (8, 1, 128, 24)):
        with pytest.raises(hq.HQError):
            hq.hq_cache_page_bytes(*bad)
    for bad in ((8, 64, 4, 3, 5, 7, 2, 128, 2), (8, 64, 4, 3, 5, 8, 2, 128, 5), (8, 64, 0, 3, 5, 8, 2, 128, 2)):
        with pytest.raises(hq.HQError):
            hq.hq_cache_attention_workspace(*bad)
    assert hq.hq_cache_attention_workspace(8, 64, 4, 0, 5, 8, 2, 128, 2) == 0
    assert hq.hq_cache_attention_workspace(8, 64, 4, 3, 0, 8, 2, 128, 2) == 0
    for dt in (0, 1, 2):                        # what a larger batch needs is bounded, and a smaller one's fits a larger's
        last = 0
        for R, T in ((1, 1), (4, 9), (64, 64), (64, 4000), (1 << 20, 1 << 27)):
            n = hq.hq_cache_attention_workspace(4, 64, 1 << 12, R, T, 32, 8, 128, dt)
            assert 0 <= n < 1 << 29
