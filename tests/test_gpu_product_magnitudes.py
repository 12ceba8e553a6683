"""Rows whose values differ by many powers of two: a large value that meets weights of zero takes nothing from the small
ones beside it, however small they are."""
import pytest
import torch

from product_helpers import DEV, Weights, product, rows

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def same(got, want, what):
    assert torch.equal(got.cpu(), want.to(F32).to(got.dtype)), what


def inputs(T, out, inp, low, high):
    """Whole numbers times 2^low, all but the first row with a 2^high in every 1024 columns, where both matrices are
    zero. Of many columns few are not zero, so that sums are exact."""
    w, v = Weights(1, out, inp, inp, whole=True), Weights(1, out, inp, inp + 1, whole=True)
    at = torch.arange(6, inp, 1024)
    for one in (w, v):
        one.packed[..., at // 2] &= 0xF0
        one.values[..., at] = 0
    x = rows((T, inp), BF16, 1, whole=True).double()
    if inp > 2064:
        x[torch.rand(x.shape, generator=torch.Generator().manual_seed(2)) < 0.9] = 0
    x *= 2.0 ** low
    x[1:, at] = 2.0 ** high
    b = x.to(BF16)
    assert torch.equal(b.double(), x)
    return w, v, b


@pytest.mark.parametrize("inp", (64, 1040, 2064, 17408))
@pytest.mark.parametrize("low, high", [(0, 30), (0, 32), (0, 39), (0, 60), (-20, 40), (-110, 100), (-100, -40), (40, 120)])
@pytest.mark.parametrize("T", (1, 2, 4, 40, 140))
def test_small_values_beside_large_ones(nv, T, low, high, inp):
    w, v, x = inputs(T, 70, inp, low, high)
    z = product(x, w, [T])[0]
    same(nv.linear(w.matrix(nv), x.to(DEV)), z, "Y")
    _, g, u = nv.gated(w.matrix(nv), v.matrix(nv), x.to(DEV), with_pre=True)
    same(g, z, "G")
    same(u, product(x, v, [T])[0], "U")


@pytest.mark.parametrize("value", (float("inf"), float("nan"), -float("inf")))
def test_no_number_beside_small_values(nv, value):
    """Its row has no finite sum, the other rows of the wave are exact."""
    T, out, inp = 4, 70, 2064
    w, v, x = inputs(T, out, inp, -60, -10)
    z = product(x, w, [T])[0]
    bad = x.clone()
    bad[2, 1500] = value
    y = nv.linear(w.matrix(nv), bad.to(DEV))
    keep = torch.tensor([True, True, False, True])
    same(y[keep.to(DEV)], z[keep], "Y")
    assert not torch.isfinite(y[2]).any()


@pytest.mark.parametrize("inp", (1040, 17408))
def test_other_rows_keep_their_bits(nv, inp):
    """Random rows beside one that f16 does not hold, or that has a NaN, are the same to the last bit as beside others."""
    w = Weights(1, 70, inp, 3)
    x = rows((4, inp), BF16, 1, 0.3)
    y, m = None, w.matrix(nv)
    for value in (0.5, 2.0 ** 60, 2.0 ** -60, float("nan")):
        x[1, 7::1024] = value
        got = nv.linear(m, x.to(DEV))[[0, 2, 3]]
        y = got if y is None else y
        assert torch.equal(got, y), value
