"""Argument errors of the key/value cache calls: found on the host, before anything is enqueued (no call
here reaches a kernel)."""
import ctypes
import os

import pytest

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "block_scale_search_amd", "libnvfp4.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libnvfp4.so not built")

FAKE, ODD = 1 << 20, (1 << 20) + 4           # never dereferenced


@pytest.fixture(scope="module")
def n():
    from block_scale_search_amd import nvfp4
    return nvfp4


def _cache(n, **kw):
    a = dict(pages=FAKE, layers=2, layer_stride=10 * 4608, num_pages=10, page_stride=4608, heads=2,
             head_dim=128, page_size=16, max_pages=4, max_slots=3, table=FAKE, lens=FAKE, refs=FAKE,
             S_k=FAKE, S_v=FAKE)
    a.update(kw)
    return ctypes.byref(n.KVCacheStruct(**a))


BAD_CACHES = [
    (dict(heads=0), "SHAPE"), (dict(head_dim=96), "SHAPE"), (dict(page_size=24), "SHAPE"),
    (dict(page_size=0), "SHAPE"), (dict(layers=0), "SHAPE"), (dict(num_pages=-1), "SHAPE"),
    (dict(page_stride=4592), "SHAPE"), (dict(layer_stride=9 * 4608), "SHAPE"),
    (dict(page_stride=1 << 60), "SHAPE"), (dict(max_slots=65537), "SHAPE"), (dict(max_pages=-1), "SHAPE"),
    (dict(max_pages=1 << 27), "SHAPE"), (dict(max_slots=65536, max_pages=1 << 15), "SHAPE"),
    (dict(pages=None), "NULL"), (dict(lens=None), "NULL"), (dict(table=None), "NULL"),
    (dict(pages=ODD), "ALIGN"), (dict(page_stride=4616, layer_stride=46160), "ALIGN"),
    (dict(table=FAKE + 2), "ALIGN"), (dict(lens=FAKE + 1), "ALIGN")]


def _append(n, cache=None, **kw):
    a = dict(layer=0, K=FAKE, V=FAKE, dt=1, tokens=4, skt=256, skh=128, svt=256, svh=128, cu=FAKE,
             slots=None, seqs=2, lo=-3, hi=7)
    a.update(kw)
    return n._lib.nvfp4_kv_append(_cache(n) if cache is None else cache, *a.values(), None)


def _read(n, cache=None, **kw):
    a = dict(layer=0, K=FAKE, V=FAKE, dt=1, tokens=4, cu=FAKE, slots=None, seqs=2)
    a.update(kw)
    return n._lib.nvfp4_kv_read(_cache(n) if cache is None else cache, *a.values(), None)


def _attend(n, cache=None, **kw):
    a = dict(layer=0, Q=FAKE, dt=1, tokens=4, heads=8, sqt=1024, sqh=128, cu=FAKE, slots=None, seqs=2,
             max_q=4, max_kv=64, scale=0.1, causal=1, window=0, O=FAKE, sot=1024, soh=128, lse=None,
             ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return n._lib.nvfp4_kv_attention(_cache(n) if cache is None else cache, *a.values(), None)


def _reserve(n, cache=None, **kw):
    a = dict(slots=FAKE, counts=FAKE, count=3, status=FAKE, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return n._lib.nvfp4_kv_reserve(_cache(n) if cache is None else cache, *a.values(), None)


def _fork(n, cache=None, **kw):
    a = dict(parents=FAKE, children=FAKE, count=3, status=FAKE, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return n._lib.nvfp4_kv_fork(_cache(n) if cache is None else cache, *a.values(), None)


def _free(n, cache=None, **kw):
    a = dict(slots=FAKE, count=3, status=FAKE)
    a.update(kw)
    return n._lib.nvfp4_kv_free(_cache(n) if cache is None else cache, *a.values(), None)


def _compact(n, cache=None, **kw):
    a = dict(used=FAKE, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return n._lib.nvfp4_kv_compact(_cache(n) if cache is None else cache, *a.values(), None)


@pytest.mark.parametrize("call", [_append, _read, _attend, _reserve, _fork, _free, _compact])
def test_caches_that_are_refused(n, call):
    for kw, want in BAD_CACHES:
        assert call(n, _cache(n, **kw)) == getattr(n, "ERR_" + want), kw
    assert call(n, ctypes.c_void_p(None)) == n.ERR_NULL
    if call in (_append, _read, _attend):
        assert call(n, _cache(n, S_k=None)) == n.ERR_NULL
        assert call(n, _cache(n, S_v=ODD + 1)) == n.ERR_ALIGN
    else:
        assert call(n, _cache(n, refs=None)) == n.ERR_NULL
        assert call(n, _cache(n, refs=FAKE + 2)) == n.ERR_ALIGN


def test_page_bytes(n):
    assert n.nvfp4_kv_page_bytes(2, 128, 16) == 4608
    for bad in ((0, 128, 16), (1, 32, 16), (1, 128, 8), (1, 128, 17), (70000, 128, 16)):
        assert n.nvfp4_kv_page_bytes(*bad) == 0


def test_token_call_arguments(n):
    for call in (_append, _read, _attend):
        assert call(n, dt=7) == n.ERR_DTYPE
        assert call(n, layer=2) == n.ERR_ARG and call(n, layer=-1) == n.ERR_ARG
        assert call(n, tokens=-1) == n.ERR_SHAPE and call(n, seqs=-1) == n.ERR_SHAPE
        assert call(n, seqs=65536) == n.ERR_SHAPE and call(n, tokens=1 << 31) == n.ERR_SHAPE
        assert call(n, cu=None) == n.ERR_NULL
        assert call(n, cu=FAKE + 2) == n.ERR_ALIGN and call(n, slots=FAKE + 2) == n.ERR_ALIGN
        assert call(n, tokens=0) == n.OK and call(n, seqs=0) == n.OK
    assert _append(n, tokens=1 << 28) == n.ERR_SHAPE
    assert _append(n, lo=1) == n.ERR_WINDOW and _append(n, hi=126) == n.ERR_WINDOW
    for k in ("K", "V"):
        assert _append(n, **{k: None}) == n.ERR_NULL and _append(n, **{k: ODD}) == n.ERR_ALIGN
        assert _read(n, **{k: None}) == n.ERR_NULL and _read(n, **{k: ODD}) == n.ERR_ALIGN
    for k in ("skt", "skh", "svt", "svh"):
        assert _append(n, **{k: -8}) == n.ERR_SHAPE and _append(n, **{k: 1 << 60}) == n.ERR_SHAPE
        assert _append(n, **{k: 132}) == n.ERR_ALIGN
    # a cache without pages or slots: nothing to write
    assert _append(n, _cache(n, num_pages=0, pages=None)) == n.OK
    assert _append(n, _cache(n, max_slots=0)) == n.OK


def test_attention_arguments(n):
    assert _attend(n, heads=3) == n.ERR_SHAPE and _attend(n, heads=0) == n.ERR_SHAPE
    assert _attend(n, max_q=-1) == n.ERR_SHAPE and _attend(n, max_kv=-1) == n.ERR_SHAPE
    assert _attend(n, max_q=1 << 23) == n.ERR_SHAPE
    assert _attend(n, tokens=1 << 28) == n.ERR_SHAPE                     # tokens * q_heads
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert _attend(n, scale=s) == n.ERR_ARG
    assert _attend(n, window=-1) == n.ERR_ARG and _attend(n, window=2, causal=0) == n.ERR_ARG
    for k in ("Q", "O"):
        assert _attend(n, **{k: None}) == n.ERR_NULL and _attend(n, **{k: ODD}) == n.ERR_ALIGN
    assert _attend(n, sqh=132) == n.ERR_ALIGN and _attend(n, sqt=-1) == n.ERR_SHAPE
    assert _attend(n, soh=64) == n.ERR_SHAPE and _attend(n, sot=1016) == n.ERR_SHAPE
    assert _attend(n, sot=128, soh=3 * 128) == n.ERR_SHAPE               # by head, rows overlap
    assert _attend(n, lse=FAKE + 2) == n.ERR_ALIGN
    assert _attend(n, max_q=0) == n.OK
    size = lambda **kw: n._lib.nvfp4_kv_attention_workspace_size(  # noqa: E731
        _cache(n), *{**dict(dt=1, tokens=4, heads=8, seqs=2, max_q=4, max_kv=64), **kw}.values())
    for bad in (dict(dt=9), dict(tokens=-1), dict(heads=3), dict(seqs=-1), dict(max_q=-1), dict(max_kv=-1)):
        assert size(**bad) == 0
    need = size()
    if need:
        assert _attend(n, ws_bytes=need - 1) == n.ERR_WORKSPACE and _attend(n, ws=None) == n.ERR_WORKSPACE
        assert _attend(n, ws=ODD) == n.ERR_ALIGN


def test_page_call_arguments(n):
    for call in (_reserve, _fork, _free):
        assert call(n, count=-1) == n.ERR_SHAPE and call(n, count=65537) == n.ERR_SHAPE
        assert call(n, status=None) == n.ERR_NULL and call(n, status=FAKE + 2) == n.ERR_ALIGN
    for k in ("slots", "counts"):
        assert _reserve(n, **{k: None}) == n.ERR_NULL and _reserve(n, **{k: FAKE + 1}) == n.ERR_ALIGN
    for k in ("parents", "children"):
        assert _fork(n, **{k: None}) == n.ERR_NULL
    assert _free(n, slots=None) == n.ERR_NULL
    for call in (_reserve, _fork, _compact):
        assert call(n, ws=None) == n.ERR_WORKSPACE and call(n, ws_bytes=16) == n.ERR_WORKSPACE
        assert call(n, ws=ODD) == n.ERR_ALIGN
    assert _compact(n, used=None) == n.ERR_NULL
    size = n._lib.nvfp4_kv_pages_workspace_size
    assert size(_cache(n), 3) > 0 and size(_cache(n), -1) == 0 and size(_cache(n), 65537) == 0
