"""Rows into and out of the paged NVFP4 key/value cache.

Bars: the appended codes and scale bytes are the CPU oracle's scale search's, bit for bit, at every
head layout, page size, element type and row order; nothing else in the pages changes; the values read
back are one rounding from level * E4M3 * S."""
import numpy as np
import pytest
import torch

from gpu_helpers import oracle_search
from kv_helpers import DEV, i32, make_cache, plain_codes, values

pytestmark = pytest.mark.gpu


def _rows(T, H, D, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, H, D), generator=g, device=DEV)
    x[torch.rand((T, H, D), generator=g, device=DEV) < 0.01] *= 30
    x[:, :, 16:32] *= (torch.rand((T, H, 1), generator=g, device=DEV) < 0.5)   # whole groups of zero
    x[0, :, :16] *= 1e-4                                                       # subnormal scale codes
    return x.to(dtype)


def _expect(x, S, lo, hi):
    W = x.transpose(0, 1).contiguous()                                         # [H, T, D]
    o = oracle_search(W, None, S.tolist(), "mse", lo, hi, False)
    return (torch.from_numpy(o["packed"]).transpose(0, 1),
            torch.from_numpy(o["scales"]).transpose(0, 1))


@pytest.mark.parametrize("heads,dim,page,dtype,lo,hi", [
    (1, 64, 16, torch.bfloat16, -3, 7), (3, 128, 16, torch.float32, -3, 7),
    (8, 128, 64, torch.bfloat16, -3, 7), (2, 256, 48, torch.bfloat16, 0, 0),
    (5, 64, 32, torch.float32, -8, 7), (1, 256, 16, torch.float32, -3, 7)])
def test_append_and_read(nv, heads, dim, page, dtype, lo, hi):
    lens = [1, 70, 0, page, page + 1, 2 * page - 1, 150]
    new = [1, 65, 0, page, 1, 17, 100]
    c = make_cache(nv, lens, heads, dim, page, layers=2, seed=dim + heads)
    before = c.pages.clone()
    cu = [0] + np.cumsum(new).tolist()
    K, V = (_rows(cu[-1], heads, dim, dtype, s) for s in (1, 2))
    nv.kv_append(c, 1, K, V, i32(cu), lo=lo, hi=hi)
    torch.cuda.synchronize()
    kc, ks, vc, vs = plain_codes(c, 1)
    touched = torch.zeros((c.num_pages, page), dtype=torch.bool)
    table = c.table.cpu()
    for x, codes, scales, S in ((K, kc, ks, c.S_k[1]), (V, vc, vs, c.S_v[1])):
        want_c, want_s = _expect(x, S, lo, hi)
        for i, (n, t) in enumerate(zip(new, lens)):
            pos = torch.arange(t - n, t)
            pg, row = table[i, pos // page].long(), pos % page
            touched[pg, row] = True
            assert torch.equal(codes[pg, :, row], want_c[cu[i]:cu[i + 1]]), f"item {i} codes"
            assert torch.equal(scales[pg, :, row], want_s[cu[i]:cu[i + 1]]), f"item {i} scales"
    assert torch.equal(c.pages[0], before[0])                                  # the other layer
    for a in (kc, ks, vc, vs):                                                 # every other row
        assert bool((a.transpose(1, 2)[~touched] == 255).all())
    k, v = nv.kv_read(c, 1, cu[-1], i32(cu), dtype=dtype)
    step = torch.finfo(dtype).eps / 2
    for got, x, codes, scales, S in ((k, K, kc, ks, c.S_k[1]), (v, V, vc, vs, c.S_v[1])):
        full = values(codes, scales, S)                                        # [N, H, P, D]
        for i, (n, t) in enumerate(zip(new, lens)):
            pos = torch.arange(t - n, t)
            want = full[table[i, pos // page].long(), :, pos % page]
            err = (got[cu[i]:cu[i + 1]].double().cpu() - want).abs()
            # one rounding to the type (two for bf16: binary32 first)
            assert bool((err <= want.abs() * (step + 2.0 ** -24)).all()), f"item {i}"


def test_strided_rows_slots_and_rows_behind_the_last(nv):
    """K and V as views of one projection, items in another order than the slots, a batch padded
    behind cu[-1], and a token tensor whose heads lie outside the tokens."""
    H, D, P = 4, 128, 32
    lens, slots, new = [40, 10, 33], [2, 0], [33, 5]
    c = make_cache(nv, lens, H, D, P, seed=3)
    T = sum(new)
    qkv = _rows(T + 6, 3 * H, D, torch.bfloat16, 5)
    K = qkv[:, H:2 * H]
    V = _rows(H, T + 6, D, torch.bfloat16, 6).transpose(0, 1)
    cu = i32([0, 33, 38])
    nv.kv_append(c, 0, K, V, cu, i32(slots))
    out = [torch.full((T + 6, H, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    nv.nvfp4_kv_read(c, 0, out[0], out[1], T + 6, cu, i32(slots), 2)
    torch.cuda.synchronize()
    kc, ks, vc, vs = plain_codes(c, 0)
    table = c.table.cpu()
    for x, codes, scales, S in ((K, kc, ks, c.S_k[0]), (V, vc, vs, c.S_v[0])):
        want_c, want_s = _expect(x[:T].contiguous(), S, -3, 7)
        for s, a, b in ((2, 0, 33), (0, 33, 38)):
            pos = torch.arange(lens[s] - (b - a), lens[s])
            pg = table[s, pos // P].long()
            assert torch.equal(codes[pg, :, pos % P], want_c[a:b])
            assert torch.equal(scales[pg, :, pos % P], want_s[a:b])
    for o in out:
        assert bool((o[T:] == 7).all()) and not bool((o[:T] == 7).all())


def test_positions_outside_the_cache(nv):
    """More rows than the slot is long, page entries of -1 and beyond the pages, slots outside the table,
    a length beyond the table: those rows are skipped, and read back as zeros."""
    H, D, P = 2, 64, 16
    c = make_cache(nv, [40, 8, 20, 30], H, D, P, seed=4)
    c.table[0, 1] = -1
    c.table[0, 2] = c.num_pages
    c.lens[3] = 1 << 30                                   # clamped to the table's 48 positions
    c.table[3, 2] = 1 << 30
    new, slots = [40, 20, 5, 5, 16], [0, 1, -1, 1 << 20, 3]
    cu = [0] + np.cumsum(new).tolist()
    K, V = (_rows(cu[-1], H, D, torch.bfloat16, s) for s in (7, 8))
    untouched = int(c.table[2, 0])
    nv.kv_append(c, 0, K, V, i32(cu), i32(slots))
    k, v = nv.kv_read(c, 0, cu[-1], i32(cu), i32(slots))
    torch.cuda.synchronize()
    there = torch.zeros(cu[-1], dtype=torch.bool)
    there[:16] = True                                     # slot 0: its first page
    there[40 + 12:60] = True                              # slot 1: the last 8 of 20 rows
    for x in (k, v):
        assert bool((x.cpu()[~there] == 0).all())
        assert bool((x.cpu()[there] != 0).any(-1).any(-1).all())
    assert bool((c.pages[0, untouched] == 255).all())


@pytest.mark.parametrize("seqs", [1, 64, 65, 300, 5000])
def test_many_items_of_one_row(nv, seqs):
    """One row an item, some items empty: every row finds its item."""
    H, D, P = 1, 64, 16
    lens = [1 + i % 5 for i in range(seqs)]
    c = make_cache(nv, lens, H, D, P, seed=seqs)
    new = [i % 3 != 1 for i in range(seqs)]
    cu = [0] + np.cumsum(new).tolist()
    K, V = (_rows(cu[-1], H, D, torch.float32, s) for s in (9, 10))
    nv.kv_append(c, 0, K, V, i32(cu))
    k, v = nv.kv_read(c, 0, cu[-1], i32(cu), dtype=torch.float32)
    torch.cuda.synchronize()
    kc, ks, vc, vs = plain_codes(c, 0)
    slot = torch.tensor([i for i in range(seqs) if new[i]])
    pos = torch.tensor(lens)[slot] - 1
    pg = c.table.cpu()[slot, 0].long()
    for x, got, codes, scales, S in ((K, k, kc, ks, c.S_k[0]), (V, v, vc, vs, c.S_v[0])):
        want_c, want_s = _expect(x, S, -3, 7)
        assert torch.equal(codes[pg, :, pos], want_c) and torch.equal(scales[pg, :, pos], want_s)


def test_refusals(nv):
    c = make_cache(nv, [20], 2, 64, 16)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=DEV)
    cu = i32([0, 4])
    with pytest.raises(ValueError):
        nv.kv_append(c, 0, x[:, :1], x[:, :1], cu)                    # heads
    with pytest.raises(ValueError):
        nv.kv_append(c, 0, x, x[:3], cu)
    with pytest.raises(TypeError):
        nv.kv_append(c, 0, x.half(), x.half(), cu)
    with pytest.raises(TypeError):
        nv.kv_append(c, 0, x.cpu(), x.cpu(), cu)
    with pytest.raises(TypeError):
        nv.kv_append(c, 0, x, x, cu.long())
    with pytest.raises(ValueError):
        nv.nvfp4_kv_append(c, 0, x, x, cu, None, 2, -3, 7)            # cu too short
    for kw in (dict(layer=1), dict(layer=-1)):
        with pytest.raises(nv.Nvfp4Error):
            nv.kv_append(c, K=x, V=x, cu_tokens=cu, **kw)
    with pytest.raises(nv.Nvfp4Error):
        nv.kv_append(c, 0, x, x, cu, lo=1)
    with pytest.raises(nv.Nvfp4Error):                                # rows off 16 bytes
        y = torch.zeros((4, 2, 72), dtype=torch.bfloat16, device=DEV)[:, :, 4:68]
        nv.kv_append(c, 0, y, y, cu)
    with pytest.raises(nv.Nvfp4Error):
        nv.KVCache.empty(1, 4, 2, 96, 16, 1, 1, None, None)
