"""Sizes at which the key/value cache's calls begin to refuse: found on the host, before anything is enqueued
(no call here reaches a kernel: a call whose sizes are accepted is refused for its misaligned lse)."""
import ctypes
import os

import pytest

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "block_scale_search_amd", "libnvfp4.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libnvfp4.so not built")

FAKE = 1 << 20                               # never dereferenced


@pytest.fixture(scope="module")
def n():
    from block_scale_search_amd import nvfp4
    return nvfp4


def _cache(n, heads, dim, max_pages):
    rec = n.nvfp4_kv_page_bytes(heads, dim, 16)
    return ctypes.byref(n.KVCacheStruct(
        pages=FAKE, layers=1, layer_stride=0, num_pages=10, page_stride=rec, heads=heads, head_dim=dim,
        page_size=16, max_pages=max_pages, max_slots=60000, table=FAKE, lens=FAKE, refs=FAKE, S_k=FAKE, S_v=FAKE))


def _attend(n, cache, tokens, q_heads, dim, seqs, max_q, max_kv, lse=FAKE + 2, ws=FAKE, ws_bytes=1 << 40):
    return n._lib.nvfp4_kv_attention(cache, 0, FAKE, 1, tokens, q_heads, q_heads * dim, dim, FAKE, None, seqs,
                                     max_q, max_kv, 0.1, 1, 0, FAKE, q_heads * dim, dim, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("heads,group,seqs,tokens,max_q,accepted", [
    # 2^24 / 128 = 131072 workgroups a head; tiles of 128 rows
    (128, 1, 2, 12500000, 11250000, True),
    (128, 1, 2, 128 * 131069, 16000000, True), (128, 1, 2, 128 * 131069 + 1, 16000000, False),
    (128, 1, 2, 128 * 131069 + 1, 8000000, True),            # 2 x 62500 numbered by item and tile
    # more items than are scanned to share their work out: the bounds' default is every row
    (8, 8, 6000, 6000, 6000, True), (8, 8, 6000, 6000, 1, True), (8, 1, 60000, 60000, 60000, True),
    # 2^24 / 8 = 2097152: 65535 items and 128-row tiles of 8 query heads
    (8, 8, 59000, 16 * (2097151 - 59000), 1 << 20, True), (8, 8, 59000, 16 * (2097151 - 59000) + 1, 1 << 20, False),
])
def test_the_largest_batches(n, heads, group, seqs, tokens, max_q, accepted):
    """Every batch that fits 2^24 workgroups by its rows, or by its items and bounds, is accepted."""
    got = _attend(n, _cache(n, heads, 64, 4), tokens, heads * group, 64, seqs, max_q, 64)
    assert got == (n.ERR_ALIGN if accepted else n.ERR_SHAPE)


@pytest.mark.parametrize("tokens,max_q,heads,dim", [(4, 4, 2, 128), (1, 1, 8, 64), (300, 200, 2, 256)])
def test_a_split_batch_needs_its_workspace(n, tokens, max_q, heads, dim):
    """Batches that are split along the positions have a workspace, and a call without all of it is refused."""
    cache = _cache(n, heads, dim, 1024)
    need = n._lib.nvfp4_kv_attention_workspace_size(cache, 1, tokens, 4 * heads, 2, max_q, 16384)
    assert need > 0
    call = lambda **kw: _attend(n, cache, tokens, 4 * heads, dim, 2, max_q, 16384, lse=None, **kw)  # noqa: E731
    assert call(ws_bytes=need - 1) == n.ERR_WORKSPACE
    assert call(ws_bytes=0) == n.ERR_WORKSPACE
    assert call(ws=None, ws_bytes=need) == n.ERR_WORKSPACE
    assert call(ws=FAKE + 4, ws_bytes=need) == n.ERR_ALIGN


def test_the_workspace_covers_smaller_plans(n):
    """No bound on positions below the one a workspace was asked for needs more of it (a window shortens what a
    call plans for)."""
    size = n._lib.nvfp4_kv_attention_workspace_size
    for heads, dim, group in ((1, 64, 1), (2, 128, 4), (8, 128, 4), (4, 256, 4), (3, 64, 7), (40, 128, 1)):
        cache = _cache(n, heads, dim, 8192)
        for seqs, new in ((1, 1), (4, 1), (16, 5), (60, 1), (3, 40), (2, 1000), (100, 2), (1024, 1), (1025, 1)):
            last = 0
            for span in (1, 31, 128, 129, 500, 641, 769, 1281, 1409, 2000, 5505, 9000, 40000, 131072):
                need = size(cache, 1, seqs * new, heads * group, seqs, new, span)
                assert need >= last, (heads, dim, group, seqs, new, span)
                last = need
