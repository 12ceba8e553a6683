"""Rows of the key/value cache that hold what no other row may see: late maxima, infinities,
scales that are no number."""
import math

import pytest
import torch

from kv_helpers import DEV, attention, check_attention, i32, make_cache

pytestmark = pytest.mark.gpu

SHAPES = [([700], [1]), ([700], [6]), ([700], [40]), ([6000], [1]), ([6000], [5]), ([6000, 900], [200, 30])]


def _climbing(nv, lens, heads, dim, seed=0):
    """A cache whose keys' first 16 values are 0 in the first half of a slot and 30 behind it, the others small."""
    c = make_cache(nv, lens, heads, dim, 16, seed=seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    k = 0.5 * torch.randn((sum(lens), heads, dim), generator=g, device=DEV)
    v = torch.randn((sum(lens), heads, dim), generator=g, device=DEV)
    k[:, :, :16] = 0
    at = 0
    for n in lens:
        k[at + n // 2:at + n, :, :16] = 30
        at += n
    nv.kv_append(c, 0, k, v, i32([0] + torch.tensor(lens).cumsum(0).tolist()))
    return c


def _queries(new, heads, dim, dtype, seed=2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = 2 * torch.randn((sum(new), heads, dim), generator=g, device=DEV)
    q[:, :, :16] = 0
    return q.to(dtype), [0] + torch.tensor(new).cumsum(0).tolist()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,new", SHAPES)
def test_a_late_maximum_stays_in_its_row(nv, lens, new, dim, dtype):
    """A row whose logits rise by 2^50 and more halfway, and the same row as a NaN: every other row of its
    wave has the same bytes both times."""
    c = _climbing(nv, lens, 2, dim)
    Q, cu = _queries(new, 8, dim, dtype)
    bad = torch.zeros(Q.shape[:2], dtype=torch.bool)
    bad[cu[-1] - 1, 1] = bad[cu[-1] // 2, 6] = True
    Q[bad] = 1.0
    out, lse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    check_attention(out, lse, attention(c, 0, Q, cu, range(len(new)), dim ** -0.5, True, 0))
    Q[bad] = math.nan
    got, glse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    assert torch.isnan(got[bad]).all() and torch.isnan(glse[bad]).all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(glse[~bad], lse[~bad])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,new", SHAPES)
def test_infinite_queries_are_nan(nv, lens, new, dim, dtype):
    """A query row with an infinity that makes every logit -infinity (or +infinity) is NaN, as the softmax of
    such logits is; a row that sees nothing keeps its zeros; every other row keeps its bytes."""
    c = make_cache(nv, lens, 2, dim, 16)
    k = torch.randn((sum(lens), 2, dim), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    k[:, :, 3] = 4.0                                     # a code above 0 at every position
    nv.kv_append(c, 0, k, k, i32([0] + torch.tensor(lens).cumsum(0).tolist()))
    Q, cu = _queries(new, 8, dim, dtype)
    out, lse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    bad = torch.zeros(Q.shape[:2], dtype=torch.bool)
    for i, (t, h, x) in enumerate([(0, 1, -math.inf), (cu[-1] - 1, 6, math.inf), (cu[-1] // 2, 3, -math.inf)]):
        Q[t, h] *= 0.01                                  # beside it values that f16 holds after any scaling
        Q[t, h, 3 if i < 2 else 5] = x
        bad[t, h] = True
    got, glse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    assert torch.isnan(got[bad]).all() and torch.isnan(glse[bad]).all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(glse[~bad], lse[~bad])
    c.lens.zero_()
    got, glse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    assert bool((got == 0).all()) and bool((glse == -math.inf).all())


@pytest.mark.parametrize("bad_scale", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,new", SHAPES)
def test_a_scale_that_is_no_number(nv, lens, new, dim, dtype, bad_scale):
    """S_k of one head NaN or infinite: its query heads are NaN, the other head's keep their bytes, and rows
    that see nothing their zeros."""
    c = _climbing(nv, lens, 2, dim, 5)
    Q, cu = _queries(new, 8, dim, dtype)
    out, lse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    c.S_k[0, 1] = bad_scale
    got, glse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    assert torch.isnan(got[:, 4:]).all() and torch.isnan(glse[:, 4:]).all()
    assert torch.equal(got[:, :4], out[:, :4]) and torch.equal(glse[:, :4], lse[:, :4])
    c.lens.zero_()
    got, glse = nv.kv_attention(c, 0, Q, i32(cu), max_q=max(new))
    assert bool((got == 0).all()) and bool((glse == -math.inf).all())


READ = pytest.mark.parametrize("dtype,dim,bits", [(t, d, b) for t in (torch.bfloat16, torch.float32) for d in (64, 128, 256)
                               for b in (0x7FFFFFFF, -1, 0x7FC00000, 0x7F800001, 0x7F800000)])


def _read_before_and_after(nv, dtype, dim, bits):
    """What two slots read as, one with a page that the table does not name and one with more rows asked for than it
    is long, before and after the second head's S_k and S_v become the binary32 of `bits`; and which rows are
    cached."""
    c = make_cache(nv, [40, 8], 2, dim, 16)
    c.table[0, 1] = -1
    x = torch.randn((60, 2, dim), generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)
    cu = i32([0, 40, 60])
    nv.kv_append(c, 0, x, x, cu)
    want = nv.kv_read(c, 0, 60, cu, dtype=dtype)
    there = torch.ones(60, dtype=torch.bool, device=DEV)
    there[16:32] = there[40:52] = False
    for S in (c.S_k, c.S_v):
        S[0].view(torch.int32)[1] = bits
    return want, nv.kv_read(c, 0, 60, cu, dtype=dtype), there


@READ
def test_read_with_a_scale_that_is_no_number(nv, dtype, dim, bits):
    """Values of a head whose S is a NaN of any bits are NaN, of an infinite one NaN or infinite; the other
    head's values stay."""
    want, got, there = _read_before_and_after(nv, dtype, dim, bits)
    for x, ref in zip(got, want):
        assert torch.equal(x[:, 0], ref[:, 0])
        assert not torch.isfinite(x[there, 1]).any()
        assert bits == 0x7F800000 or torch.isnan(x[there, 1]).all()


@READ
def test_read_of_nothing_is_zero_at_any_scale(nv, dtype, dim, bits):
    """Positions that are not in the cache read as zeros where S is NaN or infinite, too."""
    want, got, there = _read_before_and_after(nv, dtype, dim, bits)
    for x in want + got:
        assert bool((x[~there] == 0).all())
