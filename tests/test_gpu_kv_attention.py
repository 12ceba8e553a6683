"""Attention over the paged NVFP4 key/value cache against a 64-bit model of the cached values, with the
tolerance derived in kv_helpers.check_attention."""
import pytest
import torch

from kv_helpers import DEV, attention, check_attention, fill_cache, i32, make_cache

pytestmark = pytest.mark.gpu


def _q(T, heads, dim, dtype, seed, scale=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn((T, heads, dim), generator=g, device=DEV)).to(dtype)


def _run(nv, lens, new, heads, group, dim, page, dtype, causal=True, window=0, slots=None, scale=None,
         seed=0, change=None, **kw):
    c = make_cache(nv, lens, heads, dim, page, seed=seed)
    fill_cache(nv, c, lens, seed)
    if change:
        change(c)
    cu = [0] + torch.tensor(new).cumsum(0).tolist()
    Q = _q(cu[-1], heads * group, dim, dtype, seed + 2)
    out, lse = nv.kv_attention(c, 0, Q, i32(cu), None if slots is None else i32(slots), scale=scale,
                               causal=causal, window=window, **kw)
    torch.cuda.synchronize()
    want = attention(c, 0, Q, cu, range(len(new)) if slots is None else slots,
                     dim ** -0.5 if scale is None else scale, causal, window)
    check_attention(out, lse, want)
    return c, Q, cu, out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (1, 16), (3, 1), (2, 5), (1, 40)])
def test_single_tokens(nv, dtype, dim, heads, group):
    """One row an item: lengths of 0, 1, around pages and tiles, and many."""
    lens = [1, 0, 15, 16, 17, 31, 32, 33, 64, 100, 129, 700]
    _run(nv, lens, [1] * len(lens), heads, group, dim, 16, dtype, seed=dim + group)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,page", [(1, 16), (4, 48), (7, 32), (8, 64)])
def test_ragged_rows(nv, dtype, dim, group, page):
    """Rows of several tokens, items without rows, items whose rows are the whole slot."""
    lens = [150, 40, 5, 260, 1, 64]
    new = [3, 40, 0, 131, 1, 17]
    _run(nv, lens, new, 2, group, dim, page, dtype, seed=group)
    _run(nv, lens, new, 2, group, dim, page, dtype, causal=False, seed=group + 1)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 5000])
@pytest.mark.parametrize("new", [[1, 1, 1], [6, 3, 10], [200, 3, 90]])
def test_windows(nv, window, new):
    _run(nv, [300, 5, 90], new, 2, 4, 128, 16, torch.bfloat16, window=window, seed=window)
    _run(nv, [300, 5, 90], new, 1, 3, 64, 32, torch.float32, window=window, seed=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_long_slot_beside_short_ones(nv, dim, dtype):
    lens = [7000, 1, 300, 2049]
    for new in ([1, 1, 1, 1], [5, 1, 3, 2], [70, 1, 64, 33]):
        _run(nv, lens, new, 2, 4, dim, 64, dtype, seed=len(new) + new[0], max_q=max(new))


@pytest.mark.parametrize("seqs", [65, 200, 1030])
def test_many_items(nv, seqs):
    """More items than a wave has lanes, and more than are scanned: short ones, empty ones, a long one."""
    lens = [0 if i % 11 == 5 else 1 + (i * 37) % 50 for i in range(seqs)]
    lens[seqs - 3] = 2600 if seqs < 1000 else 300
    lens[70 % seqs] = 1500 if seqs < 1000 else 90
    _run(nv, lens, [1] * seqs, 1, 4, 64, 16, torch.bfloat16, seed=seqs, max_q=1)
    new = [min(i % 4, t) for i, t in enumerate(lens)]
    _run(nv, lens, new, 1, 6, 64, 16, torch.float32, seed=seqs, max_q=3)       # two tiles of 16 rows
    if seqs < 1000:
        new[seqs - 3], new[2] = 150, min(30, lens[2])
        _run(nv, lens, new, 1, 2, 64, 16, torch.bfloat16, seed=seqs, max_q=150)
        _run(nv, lens, new, 1, 2, 64, 16, torch.bfloat16, seed=seqs)            # bounds far too wide


def test_windows_beyond_every_length(nv):
    """Windows as large as int32 and int64, rows before the first position among those that see some."""
    for window in ((1 << 31) - 1, (1 << 31) - 70000, 1 << 40):
        for new in ([9, 1], [60, 40]):
            _run(nv, [5, 40], new, 1, 4, 64, 16, torch.bfloat16, window=window, seed=3)


def test_rows_that_see_nothing(nv):
    """Rows before the slot's first position, slots outside the table, an item of length 0."""
    lens, new, slots = [3, 0, 40], [5, 4, 2, 2, 3], [0, 1, 2, -1, 77]
    for dim in (64, 128, 256):
        for dtype in (torch.bfloat16, torch.float32):
            c, Q, cu, out, lse = _run(nv, lens, new, 2, 2, dim, 16, dtype, slots=slots, seed=dim)
            dark = torch.isinf(lse).all(1).cpu()
            assert dark.tolist() == [True] * 2 + [False] * 3 + [True] * 4 + [False] * 2 + [True] * 5
            assert bool((out[dark.to(DEV)] == 0).all())


@pytest.mark.parametrize("new", [[1, 1], [9, 4], [80, 45]])
def test_entries_that_name_no_page(nv, new):
    def change(c):
        c.table[0, 1] = -1
        c.table[0, 3] = c.num_pages
        c.table[1, 0] = -7
        c.table[1, 2] = 1 << 30
    for dtype in (torch.bfloat16, torch.float32):
        _run(nv, [130, 45], new, 2, 4, 128, 16, dtype, seed=5, change=change)
        _run(nv, [130, 45], new, 2, 4, 64, 16, dtype, causal=False, seed=6, change=change)


@pytest.mark.parametrize("new", [[1, 1, 1], [9, 4, 1], [80, 45, 2]])
def test_bytes_behind_the_last_position_do_not_matter(nv, new):
    """Rows of a page that were never written hold 255 (no scale, a NaN as E4M3) or any other byte."""
    lens = [130, 45, 3]
    for dim in (64, 128, 256):
        first = None
        for junk in (255, 127, 0x7E, 0):
            c = make_cache(nv, lens, 2, dim, 16, seed=9)
            c.pages.fill_(junk)
            fill_cache(nv, c, lens, 9)
            cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
            Q = _q(int(cu[-1]), 8, dim, torch.bfloat16, 3)
            for causal in (True, False):
                got = nv.kv_attention(c, 0, Q, cu, causal=causal)
                torch.cuda.synchronize()
                if first is None:
                    first = {}
                if causal in first:
                    assert all(torch.equal(a, b) for a, b in zip(got, first[causal])), (dim, junk)
                first.setdefault(causal, got)


def test_queries_of_every_size(nv):
    """Rows scaled over the range of bf16 and binary32 (a power of two a row keeps them in f16), a row of
    zeros, and rows with one large entry."""
    lens = [200]
    c = make_cache(nv, lens, 1, 128, 32, seed=11)
    fill_cache(nv, c, lens, 11)
    for dtype in (torch.bfloat16, torch.float32):
        Q = _q(40, 4, 128, torch.float32, 12)
        Q *= torch.logspace(-30, 1, 40, device=DEV)[:, None, None]
        Q[3] = 0
        Q[5, :, 7] = 40.0
        Q = Q.to(dtype)
        for rows in (Q, Q[-1:], Q[-4:]):
            out, lse = nv.kv_attention(c, 0, rows, i32([0, len(rows)]))
            torch.cuda.synchronize()
            check_attention(out, lse, attention(c, 0, rows, [0, len(rows)], [0], 128 ** -0.5, True, 0))
    # huge queries: a scale that brings the logits back
    Q = (_q(4, 4, 128, torch.float32, 13) * 1e30).to(torch.bfloat16)
    out, lse = nv.kv_attention(c, 0, Q, i32([0, 4]), scale=1e-30)
    check_attention(out, lse, attention(c, 0, Q, [0, 4], [0], 1e-30, True, 0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,new", [([90, 40], [1, 1]), ([90, 40], [6, 3]), ([90, 40], [60, 40]),
                                      ([5000, 40], [1, 1]), ([5000, 2000], [5, 2]), ([5000, 2000], [300, 80])])
def test_nan_queries_stay_in_their_rows(nv, lens, new, dtype):
    """A row with a NaN, of any bits, is NaN throughout and its lse too; every other row keeps its bytes."""
    c, Q, cu, out, lse = _run(nv, lens, new, 2, 4, 128, 32, dtype, max_q=max(new))
    bad = torch.zeros(Q.shape[:2], dtype=torch.bool)
    for k, (t, h) in enumerate([(0, 1), (cu[1] - 1, 6), (cu[-1] - 1, 3), (cu[-1] // 2, 0)]):
        bits = Q[t, h].view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
        bits[(37 * k) % 128] = [0x7FFF, -1, 0x7FC0, 0x7F81][k] if dtype == torch.bfloat16 else \
            [0x7FFFFFFF, -1, 0x7FC00000, 0x7F800001][k]
        bad[t, h] = True
    got, glse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    assert torch.isnan(got[bad]).all() and torch.isnan(glse[bad]).all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(glse[~bad], lse[~bad])


def test_sharp_and_flat_rows(nv):
    """Logits of hundreds (one position takes all), and of nothing (every position the same)."""
    for scale in (30.0, 1e-20):
        for new in ([1, 1], [5, 2], [90, 64]):
            _run(nv, [500, 64], new, 1, 4, 128, 16, torch.bfloat16, scale=scale, seed=21)
            _run(nv, [500, 64], new, 1, 4, 64, 16, torch.float32, scale=scale, seed=22)


def test_strides_streams_and_rows_behind_the_last(nv):
    """Q inside a projection, O by head, a batch padded behind cu[-1], a side stream, and bounds larger
    than needed."""
    lens, new, H, G, D = [90, 33], [20, 7], 2, 4, 128
    c = make_cache(nv, lens, H, D, 32, seed=31)
    fill_cache(nv, c, lens, 31)
    cu = [0, 20, 27]
    proj = _q(30, 3 * H * G, D, torch.bfloat16, 32)
    Q = proj[:, H * G:2 * H * G]
    O = torch.full((H * G, 30, D), 7.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    lse = torch.full((30, H * G), 7.0, device=DEV)
    side = torch.cuda.Stream()
    for max_q, max_kv in ((20, 90), (30, 4096), (1 << 20, (1 << 31) - 1)):
        O.fill_(7.0)
        lse.fill_(7.0)
        n = nv.nvfp4_kv_attention_workspace_size(c, Q.dtype, 30, H * G, 2, max_q, max_kv)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        side.wait_stream(torch.cuda.current_stream())
        nv.nvfp4_kv_attention(c, 0, Q, i32(cu), None, 2, max_q, max_kv, D ** -0.5, True, 0, O, lse, ws,
                              stream=side)
        torch.cuda.synchronize()
        check_attention(O[:27], lse[:27], attention(c, 0, Q[:27], cu, [0, 1], D ** -0.5, True, 0))
        assert bool((O[27:] == 7).all()) and bool((lse[27:] == 7).all())


@pytest.mark.parametrize("offsets", [[0, -(1 << 31), 20, 40], [3, 1, 60, 7], [0, 40, 0, 40],
                                     [-5, 9, 1 << 30, 40], [0, 10, 20, (1 << 31) - 1],
                                     [0, 10, 20, -1], [40, 40, 40, 40]])
def test_offsets_that_are_no_partition(nv, offsets):
    """Nothing outside the batch's rows and the cache is written, whatever the offsets hold."""
    c = make_cache(nv, [3000, 90, 40], 2, 128, 16)
    fill_cache(nv, c, [3000, 90, 40])
    T, cu = 40, i32(offsets)
    for dtype in (torch.bfloat16, torch.float32):
        Q = _q(T, 8, 128, dtype, 1)
        for max_q in (1, 8, T):
            O = torch.full((T + 16, 8, 128), 7.0, dtype=dtype, device=DEV)
            lse = torch.full((T + 16, 8), 7.0, device=DEV)
            ws = torch.full((max(16, nv.nvfp4_kv_attention_workspace_size(c, dtype, T, 8, 3, max_q, 3000)),),
                            0xFF, dtype=torch.uint8, device=DEV)
            nv.nvfp4_kv_attention(c, 0, Q, cu, None, 3, max_q, 3000, 0.1, True, 0, O[8:-8], lse[8:-8], ws)
            torch.cuda.synchronize()
            for t in (O, lse):
                assert bool((t[:8] == 7.0).all()) and bool((t[-8:] == 7.0).all())


def test_bounds_below_the_need(nv):
    """Rows at or beyond max_q are not written, positions at or beyond max_kv are left out."""
    lens, new = [90, 33], [20, 7]
    c = make_cache(nv, lens, 1, 128, 16, seed=41)
    fill_cache(nv, c, lens, 41)
    Q = _q(27, 4, 128, torch.bfloat16, 42)
    O = torch.full((27, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    nv.nvfp4_kv_attention(c, 0, Q, i32([0, 20, 27]), None, 2, 9, 4096, 0.1, True, 0, O, None, ws)
    torch.cuda.synchronize()
    assert bool((O[9:20] == 7).all()) and not bool((O[:9] == 7).any()) and not bool((O[20:] == 7).any())
    out, lse = nv.kv_attention(c, 0, Q, i32([0, 20, 27]), max_kv=50, scale=0.1, causal=False)
    short = make_cache(nv, lens, 1, 128, 16, seed=41)
    short.pages.copy_(c.pages)
    short.lens[0] = 50
    check_attention(out, lse, attention(short, 0, Q, [0, 20, 27], [0, 1], 0.1, False, 0))


def test_same_inputs_same_bytes(nv):
    lens = [3000, 100, 900]
    c = make_cache(nv, lens, 2, 128, 16, seed=51)
    fill_cache(nv, c, lens, 51)
    for new in ([1, 1, 1], [7, 2, 5], [150, 100, 3]):
        cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
        Q = _q(sum(new), 8, 128, torch.bfloat16, 52)
        a = nv.kv_attention(c, 0, Q, cu)
        for _ in range(3):
            b = nv.kv_attention(c, 0, Q, cu)
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_beyond_32_bits(nv):
    """Pages whose records lie beyond 4 GiB of the cache."""
    H, D, P = 8, 256, 128                                     # 294,912 bytes a record
    n = (5 << 30) // nv.nvfp4_kv_page_bytes(H, D, P)
    S = torch.full((1, H), 0.01, device=DEV)
    c = nv.KVCache.empty(1, n, H, D, P, 2, 3, S, S)
    c.table[0] = i32([n - 1, 3, n - 7])
    c.table[1] = i32([n // 2, n - 2, 0])
    c.lens.copy_(i32([300, 257]))
    fill_cache(nv, c, [300, 257], 61)
    small = nv.KVCache.empty(1, 6, H, D, P, 2, 3, S, S)
    small.table[0], small.table[1] = i32([0, 1, 2]), i32([3, 4, 5])
    small.lens.copy_(c.lens)
    fill_cache(nv, small, [300, 257], 61)
    for new in ([1, 1], [150, 20]):
        Q = _q(sum(new), 16, D, torch.bfloat16, 62)
        cu = i32([0, new[0], sum(new)])
        for x, y in zip(nv.kv_attention(c, 0, Q, cu), nv.kv_attention(small, 0, Q, cu)):
            assert torch.equal(x, y)


def test_refusals(nv):
    c = make_cache(nv, [20], 2, 64, 16)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device=DEV)
    cu = i32([0, 1])
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(window=-1), dict(window=3, causal=False), dict(layer=1), dict(max_q=-1),
                dict(Q=torch.zeros((1, 3, 64), dtype=torch.bfloat16, device=DEV))):   # heads
        kw = dict(layer=0, Q=q, cu_tokens=cu)
        kw.update(bad)
        with pytest.raises(nv.Nvfp4Error):
            nv.kv_attention(c, **kw)
    for bad in (q.half(), q.cpu(), q.double()):
        with pytest.raises((TypeError, ValueError)):
            nv.kv_attention(c, 0, bad, cu)
    with pytest.raises(ValueError):
        nv.kv_attention(c, 0, q[..., :32], cu)
    with pytest.raises(nv.Nvfp4Error):                                                # rows of O overlap
        O = torch.zeros(64, dtype=torch.bfloat16, device=DEV).expand(1, 4, 64)
        nv.nvfp4_kv_attention(c, 0, q, cu, None, 1, 1, 20, 0.1, True, 0, O, None,
                              torch.empty(1 << 16, dtype=torch.uint8, device=DEV))
