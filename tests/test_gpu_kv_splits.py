"""Attention over the key/value cache where positions are split: windows that begin inside a slot, every kernel
and its join, and what lies around the buffers of a call."""
import math

import pytest
import torch

from kv_helpers import (DEV, Pool, attention, check_attention, fill_cache, i32, make_cache,
                        plain_codes)

pytestmark = pytest.mark.gpu


def _q(T, heads, dim, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (2 * torch.randn((T, heads, dim), generator=g, device=DEV)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [5, 1, 3, 2], [300, 1, 40, 64]])
def test_windows_over_long_slots(nv, new, dim, dtype):
    """Rows of one tile, of 32 and of 128, over windows that start off a tile's border deep in the slot: one
    chunk (a compute unit's whole LDS up to 128 wide) and many, some of them empty, and their join."""
    lens = [7000, 1, 300, 2049]
    c = make_cache(nv, lens, 2, dim, 64, seed=dim)
    fill_cache(nv, c, lens, dim)
    cu = [0] + torch.tensor(new).cumsum(0).tolist()
    Q = _q(cu[-1], 8, dim, dtype, 3)
    split = []
    for window in (700, 1501, 4003, 1 << 20):
        out, lse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new), window=window)
        torch.cuda.synchronize()
        check_attention(out, lse, attention(c, 0, Q, cu, range(4), dim ** -0.5, True, window), f"{window}")
        split.append(nv.nvfp4_kv_attention_workspace_size(c, dtype, cu[-1], 8, 4, max(new),
                                                          min(7040, window + max(new) + 31)) > 0)
    assert split[-2:] == [True, True]
    assert split[0] == (new[0] > 5 or dim == 256)         # so short a window splits these alone


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (1, 16), (3, 1), (2, 5), (1, 40), (1, 17)])
def test_one_row_an_item_by_its_bound(nv, dtype, dim, heads, group):
    """Single tokens as a decode step passes them (max_q 1): 16, 32 and 128 rows a tile, lengths around pages
    and tiles."""
    lens = [1, 0, 15, 16, 17, 31, 32, 33, 64, 100, 129, 700]
    c = make_cache(nv, lens, heads, dim, 16, seed=dim + group)
    fill_cache(nv, c, lens, dim)
    cu = list(range(len(lens) + 1))
    Q = _q(len(lens), heads * group, dim, dtype, 5)
    out, lse = nv.kv_attention(c, 0, Q, i32(cu), max_q=1)
    torch.cuda.synchronize()
    check_attention(out, lse, attention(c, 0, Q, cu, range(len(lens)), dim ** -0.5, True, 0))


@pytest.mark.parametrize("window", [1, 2, 16, 33, 100])
def test_windows_by_their_bound(nv, window):
    for new in ([1, 1, 1], [6, 3, 5], [6, 3, 10]):
        for heads, group, dim, page, dtype in ((2, 4, 128, 16, torch.bfloat16), (1, 3, 64, 32, torch.float32),
                                               (2, 2, 256, 16, torch.bfloat16)):
            lens = [300, 5, 90]
            c = make_cache(nv, lens, heads, dim, page, seed=window)
            fill_cache(nv, c, lens, window)
            cu = [0] + torch.tensor(new).cumsum(0).tolist()
            Q = _q(cu[-1], heads * group, dim, dtype, 7)
            out, lse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new), window=window)
            torch.cuda.synchronize()
            check_attention(out, lse, attention(c, 0, Q, cu, range(3), dim ** -0.5, True, window))


OFFSETS = [[0, -(1 << 31), 20, 40], [3, 1, 60, 7], [0, 40, 0, 40], [-5, 9, 1 << 30, 40],
           [0, 10, 20, (1 << 31) - 1], [0, 10, 20, -1], [40, 40, 40, 40]]


@pytest.mark.parametrize("offsets", OFFSETS)
def test_bad_offsets_leave_workspace_neighbours_and_cache(nv, offsets):
    """Attention over offsets that are no partition: the bytes around its workspace, which takes the parts of a
    split batch, and the cache stay as they were."""
    lens = [3000, 90, 40]
    c = make_cache(nv, lens, 2, 128, 16)
    fill_cache(nv, c, lens)
    held = [t.clone() for t in (c.pages, c.table, c.lens, c.refs)]
    T, cu, pad = 40, i32(offsets), 1 << 16
    for dtype in (torch.bfloat16, torch.float32):
        Q = _q(T, 8, 128, dtype, 1)
        for max_q in (1, 8, T):
            O = torch.empty((T, 8, 128), dtype=dtype, device=DEV)
            lse = torch.empty((T, 8), device=DEV)
            need = nv.nvfp4_kv_attention_workspace_size(c, dtype, T, 8, 3, max_q, 3000)
            assert need > 0
            space = torch.full((need + 2 * pad,), 0xA5, dtype=torch.uint8, device=DEV)
            nv.nvfp4_kv_attention(c, 0, Q, cu, None, 3, max_q, 3000, 0.1, True, 0, O, lse,
                                  space[pad:pad + need])
            torch.cuda.synchronize()
            assert bool((space[:pad] == 0xA5).all()) and bool((space[pad + need:] == 0xA5).all())
            for t, before in zip((c.pages, c.table, c.lens, c.refs), held):
                assert torch.equal(t, before)


@pytest.mark.parametrize("offsets", OFFSETS)
def test_bad_offsets_of_append_and_read(nv, offsets):
    """Append and read over offsets that are no partition: append writes rows of the named slots only, read
    only its outputs' rows."""
    lens = [3000, 90, 40]
    c = make_cache(nv, lens, 2, 128, 16, extra_pages=9)
    T, cu = 40, i32(offsets)
    spare = (c.refs == 0).nonzero()[:, 0]
    rows = torch.zeros((c.num_pages, 16), dtype=torch.bool)         # positions of the slots
    for s, n in enumerate(lens):
        t = torch.arange(n)
        rows[c.table.cpu()[s, t // 16].long(), t % 16] = True
    assert len(spare) == 9
    for dtype in (torch.bfloat16, torch.float32):
        x = _q(T, 2, 128, dtype, 2)
        c.pages.fill_(255)
        nv.kv_append(c, 0, x, x, cu)
        torch.cuda.synchronize()
        for codes in plain_codes(c, 0):
            assert bool((codes.transpose(1, 2)[~rows] == 255).all())
        out = [torch.full((T + 16, 2, 128), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
        nv.nvfp4_kv_read(c, 0, out[0][8:-8], out[1][8:-8], T, cu, None, 3)
        torch.cuda.synchronize()
        for o in out:
            assert bool((o[:8] == 7).all()) and bool((o[-8:] == 7).all())


@pytest.mark.parametrize("n", [1, 1024, 1025, 3000])
def test_forks_of_many(nv, n):
    """Children of more than one round of the bookkeeping, of full, partly filled and empty parents."""
    c = nv.KVCache.empty(2, 3 * n + 200, 1, 64, 16, n + 40, 3, None, None)
    g = torch.Generator(device=DEV).manual_seed(n)
    c.pages.copy_(torch.randint(0, 256, c.pages.shape, generator=g, device=DEV, dtype=torch.uint8))
    pool = Pool(c.num_pages, 16, n + 40, 3)
    counts = [(7 * i) % 49 for i in range(40)]
    assert nv.kv_reserve(c, i32(range(40)), i32(counts)).item() == pool.reserve(list(range(40)), counts) == 0
    before = c.pages.clone()
    parents, children = [(11 * i) % 40 for i in range(n)], [40 + (i * 7919) % n for i in range(n)]
    assert math.gcd(7919, n) == 1
    want, copies = pool.fork(parents, children)
    assert nv.kv_fork(c, i32(parents), i32(children)).item() == want == 0
    pool.check(c, f"{n} children")
    for a, b in copies:
        before[:, b] = before[:, a]
    assert torch.equal(c.pages, before)


def test_thousands_of_items_with_no_bound(nv):
    """6000 one-row items with max_q left at every row: too many workgroups by items and bounds, few enough
    by rows. The bytes are those of the same items a thousand a call."""
    H, G, D, n = 8, 8, 64, 6000
    lens = [(i * 37) % 30 for i in range(n)]
    c = make_cache(nv, lens, H, D, 16, seed=77)
    fill_cache(nv, c, lens, 77)
    new = [min(t, 1) if i % 10 else min(t, 3) for i, t in enumerate(lens)]
    cu = [0] + torch.tensor(new).cumsum(0).tolist()
    Q = _q(cu[-1], H * G, D, torch.bfloat16, 8)
    out, lse = nv.kv_attention(c, 0, Q, i32(cu))
    slots = i32(range(n))
    for a in range(0, n, 1000):
        t0, t1 = cu[a], cu[a + 1000]
        part = nv.kv_attention(c, 0, Q[t0:t1], i32(x - t0 for x in cu[a:a + 1001]), slots[a:a + 1000])
        assert torch.equal(out[t0:t1], part[0]) and torch.equal(lse[t0:t1], part[1]), a
