"""Page calls of the paged key/value cache against the host model: tables, lengths, reference counts
and the pages' bytes, through random histories and at the refusals."""
import random

import pytest
import torch

from kv_helpers import DEV, Pool, i32

pytestmark = pytest.mark.gpu


def _new(nv, num_pages, page, slots, width, layers=2, heads=1, dim=64, stride=None):
    c = nv.KVCache.empty(layers, num_pages, heads, dim, page, slots, width, None, None)
    if stride:
        big = torch.empty((layers, num_pages, stride), dtype=torch.uint8, device=DEV)
        c = nv.KVCache(big, c.table, c.lens, c.refs, None, None, heads, dim, page)
    g = torch.Generator(device=DEV).manual_seed(num_pages)
    c.pages.copy_(torch.randint(0, 256, c.pages.shape, generator=g, device=DEV, dtype=torch.uint8))
    return c, Pool(num_pages, page, slots, width)


def _moved(before, copies, record):
    """The pages after copying records from -> to, all read before any is written."""
    after = before.clone()
    for a, b in copies:
        after[:, b, :record] = before[:, a, :record]
    return after


@pytest.mark.parametrize("seed,num_pages,page,slots,width,stride", [
    (1, 40, 16, 12, 9, None), (2, 300, 32, 40, 16, 2304 * 2 + 16), (3, 9000, 16, 700, 40, None),
    (4, 17, 16, 5, 17, None), (5, 20000, 16, 900, 40, None)])
def test_random_history(nv, seed, num_pages, page, slots, width, stride):
    r = random.Random(seed)
    c, pool = _new(nv, num_pages, page, slots, width, stride=stride)
    record = nv.nvfp4_kv_page_bytes(1, 64, page)
    seen = set()
    for step in range(60):
        before = c.pages.clone()
        kind = r.choice(("reserve", "reserve", "reserve", "fork", "free", "compact"))
        copies = []
        if kind == "reserve":
            k = r.randint(0, min(slots, 1500))
            s = r.sample(range(slots), k)
            n = [r.choice((0, 1, 1, r.randint(0, 4 * page))) for _ in s]
            got = nv.kv_reserve(c, i32(s), i32(n))
            want = pool.reserve(s, n)
        elif kind == "fork":
            empty = [i for i in range(slots) if not pool.lens[i]]
            kids = r.sample(empty, r.randint(0, len(empty)))
            rest = [i for i in range(slots) if i not in kids]
            dads = [r.choice(rest) for _ in kids] if rest else []
            kids = kids[:len(dads)]
            got = nv.kv_fork(c, i32(dads), i32(kids))
            want, copies = pool.fork(dads, kids)
        elif kind == "free":
            s = r.sample(range(slots), r.randint(0, slots // 2))
            got = nv.kv_free(c, i32(s))
            want = pool.free(s)
        else:
            got = nv.kv_compact(c)
            want, copies = pool.compact()
        torch.cuda.synchronize()
        assert got.item() == want, f"step {step} {kind}"
        seen.add((kind, want if kind != "compact" else bool(copies)))
        pool.check(c, f"step {step} {kind}")
        assert torch.equal(c.pages, _moved(before, copies, record)), f"step {step} {kind}: pages"
    assert ("reserve", 0) in seen and ("fork", 0) in seen and ("free", 0) in seen


@pytest.mark.parametrize("slots", [1, 17, 1025, 20000])
def test_many_slots_at_once(nv, slots):
    """Calls whose slots are shared out to several workgroups, one of them listed in two of their shares."""
    r = random.Random(slots)
    c, pool = _new(nv, 2 * slots + 3, 16, slots, 3, layers=1)
    every = r.sample(range(slots), slots)
    for counts in ([r.randint(0, 20) for _ in every], [1] * slots):
        assert nv.kv_reserve(c, i32(every), i32(counts)).item() == pool.reserve(every, counts)
        pool.check(c, f"reserve {slots}")
    twice = every + every[:1]
    assert nv.kv_free(c, i32(twice)).item() == pool.free(twice) == 1
    pool.check(c, f"refused {slots}")
    some = every[:slots - slots // 7]
    assert nv.kv_free(c, i32(some)).item() == pool.free(some) == 0
    pool.check(c, f"free {slots}")
    assert nv.kv_reserve(c, i32(some), i32([9] * len(some))).item() == pool.reserve(some, [9] * len(some)) == 0
    pool.check(c, f"again {slots}")


def test_refused_items_change_nothing(nv):
    c, pool = _new(nv, 20, 16, 6, 8)
    assert nv.kv_reserve(c, i32([0, 1, 2]), i32([40, 16, 1])).item() == pool.reserve([0, 1, 2], [40, 16, 1])
    pool.check(c)
    before = c.pages.clone()
    cases = [
        (nv.kv_reserve, [0, 0], [1, 1], nv.KV_BAD_SLOT), (nv.kv_reserve, [6], [1], nv.KV_BAD_SLOT),
        (nv.kv_reserve, [-1, 0], [1, 1], nv.KV_BAD_SLOT), (nv.kv_reserve, [0], [-1], nv.KV_BAD_LENGTH),
        (nv.kv_reserve, [0, 1], [1, 128 - 15], nv.KV_BAD_LENGTH),
        (nv.kv_reserve, [0], [0x7FFFFFFF], nv.KV_BAD_LENGTH),
        (nv.kv_reserve, [3, 4, 5], [128, 128, 1], nv.KV_NO_PAGES),
        (nv.kv_fork, [0, 1], [3, 3], nv.KV_BAD_SLOT), (nv.kv_fork, [0], [1], nv.KV_BAD_SLOT),
        (nv.kv_fork, [0, 3], [3, 4], nv.KV_BAD_SLOT), (nv.kv_fork, [9], [3], nv.KV_BAD_SLOT),
        (nv.kv_fork, [0], [-2], nv.KV_BAD_SLOT),
    ]
    for f, a, b, want in cases:
        assert f(c, i32(a), i32(b)).item() == want, (f.__name__, a, b)
        pool.check(c, f"{f.__name__} {a} {b}")
    for s, want in (([1, 1], nv.KV_BAD_SLOT), ([0, 6], nv.KV_BAD_SLOT), ([-1], nv.KV_BAD_SLOT)):
        assert nv.kv_free(c, i32(s)).item() == want
        pool.check(c, f"free {s}")
    # 15 pages left: a fork of a partly filled page needs one
    assert nv.kv_reserve(c, i32([3, 4]), i32([128, 112])).item() == pool.reserve([3, 4], [128, 112]) == 0
    assert sum(r == 0 for r in pool.refs) == 0
    assert nv.kv_fork(c, i32([0]), i32([5])).item() == nv.KV_NO_PAGES
    pool.check(c, "fork without a free page")
    assert nv.kv_fork(c, i32([1]), i32([5])).item() == pool.fork([1], [5])[0] == 0    # full pages only
    pool.check(c, "fork of full pages")
    assert torch.equal(c.pages, before)


def test_empty_calls(nv):
    """No items, no pages, nothing to move."""
    c, pool = _new(nv, 8, 16, 3, 2)
    e = i32([])
    assert nv.kv_reserve(c, e, e).item() == 0
    assert nv.kv_fork(c, e, e).item() == 0
    assert nv.kv_free(c, e).item() == 0
    assert nv.kv_compact(c).item() == 0
    assert nv.kv_fork(c, i32([0]), i32([1])).item() == 0              # an empty parent
    pool.check(c)
    z = nv.KVCache.empty(1, 0, 1, 64, 16, 2, 2, None, None)
    assert nv.kv_compact(z).item() == 0
    assert nv.kv_reserve(z, i32([0]), i32([1])).item() == nv.KV_NO_PAGES


def test_page_call_arguments(nv):
    c, _ = _new(nv, 8, 16, 3, 2)
    s = torch.empty(1, dtype=torch.int32, device=DEV)
    small = torch.empty(8, dtype=torch.uint8, device=DEV)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_kv_reserve(c, i32([0]), i32([1]), 1, s, small)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_kv_compact(c, s, small)
    with pytest.raises(TypeError):
        nv.kv_free(c, torch.zeros(1, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        nv.kv_reserve(c, i32([0, 1]), i32([1]))
    no_refs = nv.KVCache(c.pages, c.table, c.lens, None, None, None, 1, 64, 16)
    with pytest.raises(nv.Nvfp4Error):
        nv.kv_free(no_refs, i32([0]))
